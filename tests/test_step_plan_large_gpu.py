"""The plan of a step on the cluster and its slots kernel (many token rows or many
sequences): what is refused, skipped and reported must be what one CTA does, and agree
with a plain restatement."""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from test_step_plan_gpu import build, check, i32, lengths, plain

pytestmark = pytest.mark.gpu

ROWS = 9000  # token rows beyond what one CTA places


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def call(new, ctx, tables, ring, free, b, rows, nb):
    d = dict(new=i32(new), ctx=i32(ctx), ring=i32(ring), free=i32(free), tables=i32(tables))
    return api.plan_step(d["new"], d["ctx"], d["ring"], d["free"], d["tables"], b, rows, nb), d


@pytest.mark.parametrize("seqs,rows", [(4, ROWS), (2500, 1400), (2500, ROWS), (4, 8193), (2049, 1000)])
@pytest.mark.parametrize("what", ["blocks", "tokens", "ring", "head", "count"])
def test_a_step_that_does_not_fit_is_refused_whole(what, seqs, rows):
    b = 16
    new, ctx = [40, -1, 1, 0] + [0] * (seqs - 4), [0, 50, 32, 20] + [3] * (seqs - 4)
    if what == "tokens":
        new[0] = rows
    if what == "blocks":
        new[0] = 200
    tables, ring, head, count, total = build(new, ctx, b, 3, spare=0)
    free = [head, count]
    if what == "blocks":  # 14 are taken, 4 come back first: 9 free ones are one too few
        assert count == 14
        free = [head, 9]
    if what == "ring":
        ring, free = ring[:count + 3], [0, count]
    if what == "head":
        free = [len(ring), count]
    if what == "count":
        free = [head, -1]
    got, d = call(new, ctx, tables, ring, free, b, rows, total)
    assert api.get_device_error() == (-5, native.DEVERR_STEP)
    assert got.context_lens.tolist() == ctx and got.free_state.tolist() == free
    assert not got.query_start_loc.any()
    assert bool((got.slot_mapping == -1).all()) and bool((got.positions == -1).all())
    assert d["tables"].tolist() == tables and d["ring"].tolist() == ring


@pytest.mark.parametrize("seqs,rows", [(6, ROWS), (3000, 500), (3000, ROWS)])
def test_bad_lengths_leave_their_sequence_alone(seqs, rows):
    b, width = 16, 5
    some = min(seqs - 6, 20)
    new = [3, 5, -2, 1, 2 ** 31 - 1, 4] + [0] * (seqs - 6 - some) + [1] * some
    ctx = [10, -1, 20, 80, 30, 0] + [17] * (seqs - 6)
    tables = [[i * width + j for j in range(width)] for i in range(seqs)]
    ring = list(range(width * seqs, width * seqs + 10))
    got, d = call(new, ctx, tables, ring, [0, 10], b, rows, width * seqs + 10)
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    bad = [1, 2, 3, 4]
    want_new = [0 if s in bad else n for s, n in enumerate(new)]
    want_ctx = [0 if s in bad else c for s, c in enumerate(ctx)]
    want = plain(want_new, want_ctx, tables, ring, 0, 10, b, rows)  # updates its tables
    want[0][:] = [ctx[s] if s in bad else x for s, x in enumerate(want[0])]
    for name, x, y in zip(got._fields, got, want):
        assert x.tolist() == y, name
    assert d["tables"].tolist() == tables and d["ring"].tolist() == ring


@pytest.mark.parametrize("seqs,rows", [(3, ROWS), (2100, 2200)])
def test_bad_block_ids_are_reported(seqs, rows):
    """In a table (a block held) and in the ring (a block taken); one error each."""
    for table_id, ring_id, slots in ((-3, 5, [5 * 16, 35, -1]), (7, 50, [-1, 35, 7 * 16 + 5]), (7, 5, [5 * 16, 35, 7 * 16 + 5])):
        new, ctx = [1, 1, 1] + [0] * (seqs - 3), [16, 3, 5] + [0] * (seqs - 3)
        tables = [[1, -7], [2, -7], [table_id, -7]] + [[-7, -7]] * (seqs - 3)
        got, d = call(new, ctx, tables, [ring_id, 9], [0, 1], 16, rows, 50)
        assert api.get_device_error() == ((0, 0) if -1 not in slots else (-5, native.DEVERR_BLOCK_ID))
        assert got.slot_mapping.tolist() == slots + [-1] * (rows - 3)
        assert got.positions.tolist() == [16, 3, 5] + [-1] * (rows - 3)


@pytest.mark.parametrize("n", [2047, 2048, 2049, 4096, 4097, 8193])
def test_sequences_around_the_passes(n):
    for seed in range(2):
        new, ctx = lengths(n, 31 * n + seed, 3, 70)
        check(new, ctx, (16, 7)[seed], seed, pad=(0, 8300)[seed], in_place=bool(seed))


@pytest.mark.parametrize("rows", [8191, 8192, 8193])
def test_rows_around_the_change(rows):
    check([rows - 60, 1, -1, 30], [5, 16, 40, 0], 16, pad=29)


def test_no_rows():
    """Many sequences, and only finished and idle ones: nothing to place."""
    new = [-1 if s % 2 else 0 for s in range(3000)]
    check(new, [s % 40 for s in range(3000)], 16)
