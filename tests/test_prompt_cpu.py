"""pa_prompt_attention without a GPU: argument errors are found on the host
before any CUDA call."""
import pytest

from paged_kv_cache_132_gb300 import build, native

FAKE = 0x10000  # aligned, never dereferenced: every case below fails validation first


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return native.load()


def _call(lib, **over):
    a = dict(out=FAKE, q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, qsl=FAKE, seqs=2, tokens=40, heads=4, kv_heads=2,
             d=64, dtype=native.PA_BF16, scale=0.125, ws=FAKE,
             ws_bytes=1 << 30, stream=None)
    a.update(over)
    return lib.pa_prompt_attention(a["out"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qsl"], a["seqs"],
                                   a["tokens"], a["heads"], a["kv_heads"], a["d"], a["dtype"], a["scale"],
                                   a["ws"], a["ws_bytes"], a["stream"])


@pytest.mark.parametrize("over,status", [
    (dict(dtype=9), -1),
    (dict(seqs=-1), -1),
    (dict(tokens=-1), -1),
    (dict(heads=0), -1),
    (dict(kv_heads=0), -1),
    (dict(heads=5), -1),                # not a multiple of num_kv_heads
    (dict(d=0), -1),
    (dict(scale=0.0), -1),
    (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1),
    (dict(scale=3e38), -1),             # in base-2 units infinite
    (dict(qs=192), -1),                 # shorter than a row
    (dict(ks=64), -1),
    (dict(vs=0), -1),
    (dict(qs=256 + 8), -1),             # not a multiple of head_dim
    (dict(ks=128 + 32), -1),
    (dict(out=0), -1),
    (dict(out=FAKE + 16), -1),          # 32 bytes
    (dict(q=0), -1),
    (dict(q=FAKE + 8), -1),             # misaligned
    (dict(k=FAKE + 2), -1),
    (dict(v=FAKE + 4), -1),
    (dict(qsl=FAKE + 2), -1),
    (dict(dtype=native.PA_F32), -2),    # tensor cores: 16-bit rows only
    (dict(d=96, qs=384, ks=192, vs=192), -2),
    (dict(d=32, qs=128, ks=64, vs=64), -2),
    (dict(heads=258, qs=258 * 64), -2),  # group 129
    (dict(qs=1 << 45), -2),             # beyond a tensor copy's strides
])
def test_rejects_on_host(lib, over, status):
    assert _call(lib, **over) == status


def test_nothing_to_do_is_noop(lib):
    assert _call(lib, seqs=0) == 0
    assert _call(lib, tokens=0, out=0) == 0


def test_workspace_size(lib):
    size = lib.pa_prompt_attention_workspace_size
    assert size(0, 0, 8, 8) > 0
    # at least an entry per pair of query tiles: 256 tokens of 1 head, 64 of a group of 4
    assert size(1, 25600, 8, 8) >= 100 * 16
    assert size(1, 6400, 32, 8) >= 100 * 16
    assert size(500, 500, 32, 8) >= 500 * 16
    for bad in ((-1, 5, 8, 8), (1, -5, 8, 8), (1, 5, 0, 8), (1, 5, 8, 0), (1, 5, 9, 8), (1, 5, 258, 2)):
        assert size(*bad) == 0
