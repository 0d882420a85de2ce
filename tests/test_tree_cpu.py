"""The calls of drafted trees without a GPU: argument errors are found on the host
before any CUDA call."""
import ctypes

import pytest

from paged_kv_cache_132_gb300 import build, native

FAKE = 0x10000  # aligned, never dereferenced: every case below fails validation first


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return native.load()


def _desc(nb=8, hkv=2, bs=16, d=64, dtype=native.PA_BF16):
    return native.CacheDesc(nb, hkv, bs, d, dtype)


def _plan(lib, **over):
    a = dict(parents=FAKE, qsl=FAKE, ctx=FAKE, seqs=2, tokens=5, pos=FAKE, mask=FAKE, words=1)
    a.update(over)
    return lib.pa_plan_tree(a["parents"], a["qsl"], a["ctx"], a["seqs"], a["tokens"], a["pos"], a["mask"], a["words"],
                            None)


@pytest.mark.parametrize("over,status", [
    (dict(seqs=-1), -1), (dict(tokens=-1), -1), (dict(words=0), -1), (dict(parents=0), -1), (dict(parents=FAKE + 2), -1),
    (dict(qsl=FAKE + 1), -1), (dict(qsl=0), -1), (dict(ctx=0), -1), (dict(pos=FAKE + 2), -1), (dict(mask=FAKE + 4), -1),
    (dict(words=17), -2), (dict(tokens=0, parents=0, pos=0, mask=0), 0),
])
def test_plan_tree(lib, over, status):
    assert _plan(lib, **over) == status


def _attend(lib, **over):
    a = dict(out=FAKE, q=FAKE, qs=256, qsl=FAKE, tokens=9, mask=FAKE, words=1, k=FAKE, v=FAKE, desc=_desc(), tables=FAKE,
             max_blocks=4, ctx=FAKE, seqs=2, heads=4, kv_heads=2, scale=0.125, ws=FAKE, ws_bytes=1 << 40)
    a.update(over)
    return lib.pa_tree_attention(a["out"], a["q"], a["qs"], a["qsl"], a["tokens"], a["mask"], a["words"], a["k"], a["v"],
                                 ctypes.byref(a["desc"]), a["tables"], a["max_blocks"], a["ctx"], a["seqs"], a["heads"],
                                 a["kv_heads"], a["scale"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,status", [
    (dict(desc=_desc(nb=0)), -1),
    (dict(desc=_desc(dtype=7)), -1),
    (dict(seqs=-1), -1),
    (dict(tokens=-1), -1),
    (dict(words=0), -1),
    (dict(heads=0), -1),
    (dict(heads=5), -1),                        # not a multiple of the KV heads
    (dict(kv_heads=4), -1),                     # differs from the pool
    (dict(max_blocks=0), -1),
    (dict(scale=0.0), -1),
    (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1),
    (dict(scale=3e38), -1),                     # in base-2 units infinite
    (dict(qs=255), -1),                         # shorter than a row
    (dict(qs=260), -1),                         # not a multiple of 16 bytes
    (dict(out=0), -1),
    (dict(out=FAKE + 16), -1),
    (dict(q=FAKE + 8), -1),
    (dict(k=0), -1),
    (dict(v=FAKE + 8), -1),
    (dict(mask=FAKE + 4), -1),
    (dict(tables=0), -1),
    (dict(ctx=FAKE + 2), -1),
    (dict(qsl=0), -1),
    (dict(desc=_desc(dtype=native.PA_F32)), -2),
    (dict(desc=_desc(d=96), qs=384), -2),
    (dict(desc=_desc(bs=64)), -2),
    (dict(desc=_desc(bs=4)), -2),
    (dict(desc=_desc(hkv=1), kv_heads=1, heads=129, qs=129 * 64), -2),
    (dict(words=17), -2),
    (dict(qs=1 << 39), -2),
    (dict(seqs=1 << 30, max_blocks=1 << 20), -2),  # a list of tiles beyond 32 bits
    (dict(ws=FAKE + 128), -3),
    (dict(ws_bytes=100), -3),
    (dict(ws=0), -3),
    (dict(seqs=0), 0),
    (dict(tokens=0), 0),
])
def test_tree_attention(lib, over, status):
    assert _attend(lib, **over) == status


def test_tree_attention_workspace_size(lib):
    ws = lib.pa_tree_attention_workspace_size
    assert ws(100, 1, 32, 8, 128) >= 2 * 152 * 256 * 128 * 4
    assert ws(8, 1, 32, 8, 128) < ws(100, 1, 32, 8, 128)   # few rows: smaller parts
    assert ws(8, 1, 32, 8, 128) >= 2 * 152 * 32 * 128 * 4
    assert ws(0, 1, 32, 8, 128) > 0
    for bad in ((-1, 1, 32, 8, 128), (8, 0, 32, 8, 128), (8, 17, 32, 8, 128), (8, 1, 0, 8, 128), (8, 1, 9, 8, 128),
                (8, 1, 32, 0, 128), (8, 1, 129, 1, 128), (8, 1, 32, 8, 0)):
        assert ws(*bad) == 0


def _verify(lib, **over):
    a = dict(ids=FAKE, parents=FAKE, qsl=FAKE, seqs=2, tokens=9, p=FAKE, ps=100, q=FAKE, qs=100, vocab=100,
             dtype=native.PA_F32, au=FAKE, su=FAKE, lens=FAKE, path=FAKE, next=FAKE)
    a.update(over)
    return lib.pa_verify_tree(a["ids"], a["parents"], a["qsl"], a["seqs"], a["tokens"], a["p"], a["ps"], a["q"], a["qs"],
                              a["vocab"], a["dtype"], a["au"], a["su"], a["lens"], a["path"], a["next"], None)


@pytest.mark.parametrize("over,status", [
    (dict(seqs=-1), -1), (dict(tokens=-1), -1), (dict(vocab=0), -1), (dict(dtype=5), -1), (dict(ps=99), -1),
    (dict(qs=99), -1), (dict(ids=0), -1), (dict(parents=FAKE + 2), -1), (dict(qsl=0), -1), (dict(p=0), -1),
    (dict(p=FAKE + 2), -1), (dict(q=FAKE + 2), -1), (dict(au=0), -1), (dict(su=FAKE + 1), -1), (dict(lens=0), -1),
    (dict(path=0), -1), (dict(next=FAKE + 2), -1), (dict(vocab=(1 << 20) + 1, ps=1 << 21, qs=1 << 21), -2),
    (dict(seqs=0), 0),
])
def test_verify_tree(lib, over, status):
    assert _verify(lib, **over) == status


def _commit(lib, **over):
    a = dict(k=[FAKE, FAKE], v=[FAKE, FAKE], layers=2, desc=_desc(), qsl=FAKE, seqs=2, tokens=9, path=FAKE, lens=FAKE,
             ctx=FAKE, ctx_out=FAKE, tables=FAKE, max_blocks=4, ring=FAKE, ring_size=8, free=FAKE, free_out=FAKE)
    a.update(over)
    k, v = ((ctypes.c_void_p * 2)(*a[x]) for x in "kv")
    return lib.pa_commit_tree(k, v, a["layers"], ctypes.byref(a["desc"]), a["qsl"], a["seqs"], a["tokens"], a["path"],
                              a["lens"], a["ctx"], a["ctx_out"], a["tables"], a["max_blocks"], a["ring"],
                              a["ring_size"], a["free"], a["free_out"], None)


@pytest.mark.parametrize("over,status", [
    (dict(desc=_desc(hkv=0)), -1), (dict(desc=_desc(d=60)), -1), (dict(layers=0), -1), (dict(layers=257), -1),
    (dict(seqs=-1), -1), (dict(tokens=-1), -1), (dict(max_blocks=0), -1), (dict(ring_size=0), -1), (dict(k=[FAKE, 0]), -1),
    (dict(v=[FAKE + 8, FAKE]), -1), (dict(qsl=0), -1), (dict(path=0), -1), (dict(lens=FAKE + 2), -1), (dict(ctx=0), -1),
    (dict(ctx_out=0), -1), (dict(tables=FAKE + 1), -1), (dict(ring=FAKE + 2), -1), (dict(free=0), -1),
    (dict(free_out=0), -1), (dict(seqs=16385), -2), (dict(ring_size=(1 << 30) - 1), -2),
])
def test_commit_tree(lib, over, status):
    assert _commit(lib, **over) == status


# Buffers apart, so that only the overlap that a case makes is one.
def _apart(*names):
    return {n: FAKE + (i + 1) * (1 << 24) for i, n in enumerate(names)}


def test_outputs_that_overlap_inputs(lib):
    a = _apart("parents", "qsl", "ctx", "pos", "mask")
    for over in (dict(pos=a["parents"]), dict(pos=a["parents"] + 16), dict(pos=a["parents"] - 16), dict(pos=a["qsl"] + 8),
                 dict(mask=a["ctx"]), dict(mask=a["parents"] - 32)):
        assert _plan(lib, **{**a, **over}) == -1, over
    a = _apart("out", "q", "qsl", "mask", "k", "v", "tables", "ctx", "ws")
    a.update(qs=512)                            # a slice of wider rows
    for at in (0, 9 * 512 - 32, 8 * 1024 + 480, -(9 * 512 - 32)):
        assert _attend(lib, **{**a, "out": a["q"] + at}) == -1, at
    a = _apart("ids", "parents", "qsl", "p", "q", "au", "su", "lens", "path", "next")
    for over in (dict(path=a["ids"]), dict(path=a["parents"] + 4), dict(lens=a["qsl"]), dict(next=a["qsl"] + 8),
                 dict(next=a["parents"] - 4)):
        assert _verify(lib, **{**a, **over}) == -1, over
    a = _apart("qsl", "path", "lens", "ctx", "ctx_out", "tables", "ring", "free", "free_out")
    for over in (dict(ctx_out=a["lens"]), dict(ctx_out=a["path"] + 32), dict(ctx_out=a["qsl"] + 8),
                 dict(ctx_out=a["ctx"] + 4)):
        assert _commit(lib, **{**a, **over}) == -1, over


def test_list_of_tiles_with_what_items_begin_with(lib):
    # 4e8 items of one tile: 2 half tiles each and up to 4 that an item begins with pass 2^31
    assert _attend(lib, seqs=200_000_000, max_blocks=8) == -2
