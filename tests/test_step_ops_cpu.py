"""pa_rotary_and_cache and pa_plan_step without a GPU: argument errors are found
on the host before any CUDA call."""
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


def _rotary(lib, **over):
    a = dict(qo=FAKE, qos=256, ko=FAKE + 0x1000, kos=128, q=FAKE + 0x2000, qs=256, k=FAKE, ks=128, v=FAKE, vs=128,
             pos=FAKE, cs=FAKE, npos=100, rot=64, inter=0, kc=FAKE, vc=FAKE, slots=FAKE, tokens=3, heads=4,
             desc=_desc(), stream=None)
    a.update(over)
    return lib.pa_rotary_and_cache(a["qo"], a["qos"], a["ko"], a["kos"], a["q"], a["qs"], a["k"], a["ks"], a["v"],
                                   a["vs"], a["pos"], a["cs"], a["npos"], a["rot"], a["inter"], a["kc"], a["vc"],
                                   a["slots"], a["tokens"], a["heads"], ctypes.byref(a["desc"]), a["stream"])


@pytest.mark.parametrize("over,status", [
    (dict(desc=_desc(nb=0)), -1),
    (dict(desc=_desc(dtype=7)), -1),
    (dict(tokens=-1), -1),
    (dict(heads=0), -1),
    (dict(heads=5), -1),                 # not a multiple of the KV heads
    (dict(npos=0), -1),
    (dict(rot=0), -1),
    (dict(rot=33), -1),                  # pairs
    (dict(rot=66), -1),                  # more than the head
    (dict(inter=2), -1),
    (dict(qs=128), -1),                  # shorter than a row
    (dict(qos=128), -1),
    (dict(ks=64), -1),
    (dict(vs=64), -1),
    (dict(kos=64), -1),
    (dict(qs=260), -1),                  # not a multiple of 16 bytes
    (dict(vs=132), -1),
    (dict(q=FAKE + 8), -1),
    (dict(qo=0), -1),
    (dict(ko=FAKE + 4), -1),
    (dict(k=0), -1),
    (dict(v=FAKE + 2), -1),
    (dict(kc=0), -1),
    (dict(vc=FAKE + 8), -1),
    (dict(cs=FAKE + 4), -1),
    (dict(pos=FAKE + 2), -1),
    (dict(slots=FAKE + 4), -1),
    (dict(qo=FAKE, q=FAKE, qs=512), -1),  # in place with other strides
    (dict(ko=FAKE, k=FAKE, ks=256), -1),
    (dict(rot=8), -2),                   # 16 bytes: half a lane's pairs
    (dict(rot=24), -2),
    (dict(desc=_desc(dtype=native.PA_F32), rot=12), -2),
])
def test_rotary_rejects_on_host(lib, over, status):
    assert _rotary(lib, **over) == status


def test_rotary_without_tokens_is_noop(lib):
    assert _rotary(lib, tokens=0) == 0
    assert _rotary(lib, tokens=0, ko=None, kos=0) == 0


def _plan(lib, **over):
    a = dict(new=FAKE, ctx=FAKE, ctx_out=FAKE, seqs=3, ring=FAKE, ring_size=8, free=FAKE, free_out=FAKE, nb=8, bs=16,
             tables=FAKE, max_blocks=4, qsl=FAKE, slots=FAKE, pos=FAKE, tokens=10, stream=None)
    a.update(over)
    return lib.pa_plan_step(a["new"], a["ctx"], a["ctx_out"], a["seqs"], a["ring"], a["ring_size"], a["free"],
                            a["free_out"], a["nb"], a["bs"], a["tables"], a["max_blocks"], a["qsl"], a["slots"],
                            a["pos"], a["tokens"], a["stream"])


@pytest.mark.parametrize("over,status", [
    (dict(seqs=-1), -1),
    (dict(ring_size=0), -1),
    (dict(nb=0), -1),
    (dict(bs=0), -1),
    (dict(max_blocks=0), -1),
    (dict(tokens=-1), -1),
    (dict(new=0), -1),
    (dict(ctx=FAKE + 2), -1),
    (dict(ctx_out=0), -1),
    (dict(ring=0), -1),
    (dict(free=FAKE + 1), -1),
    (dict(free_out=0), -1),
    (dict(tables=0), -1),
    (dict(qsl=0), -1),
    (dict(slots=FAKE + 4), -1),
    (dict(pos=0), -1),
    (dict(seqs=16385), -2),
    (dict(tokens=(1 << 30) - 1), -2),
    (dict(ring_size=(1 << 30) - 1), -2),
])
def test_plan_rejects_on_host(lib, over, status):
    assert _plan(lib, **over) == status
