"""The calls of a step on memory beyond 2^31 elements and 2^32 bytes: pools, rows of a
wide stride, and slots of large block ids."""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from test_prompt_gpu import rows, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def test_rotary_into_a_large_pool():
    h, hkv, d, bs, t = 4, 2, 128, 16, 500
    nb = (1 << 31) // (hkv * bs * d) + 40  # 2^31 elements and some blocks
    q, k, v = rows(t, h, hkv, d, torch.bfloat16, 61)
    kc, vc = (torch.zeros(nb, hkv, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.cat([torch.arange(t - 250), nb * bs - 1 - torch.arange(250)]).cuda()
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    cs = torch.randn(t, d, device="cuda")
    ko = torch.empty_like(k)
    api.rotary_and_cache(q, k, v, pos, cs, slots, kc, vc, key_out=ko)
    assert api.get_device_error() == (0, 0)
    at, off = slots // bs, slots % bs
    assert torch.equal(kc[at, :, off], ko) and torch.equal(vc[at, :, off], v)
    kc[at, :, off] = 0
    vc[at, :, off] = 0
    assert not any(bool(part.any()) for pool in (kc, vc) for part in pool.chunk(64))


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
def test_rows_far_apart(d, dtype):
    """Strides of 2^17 elements, 20 000 tokens: the last rows begin beyond 2^31."""
    h, hkv, t, stride = 4, 2, 20000, 1 << 17
    q, k, v = rows(t, h, hkv, d, dtype, 62)
    wide = torch.zeros(t, stride, dtype=dtype, device="cuda")
    views = []
    for x, at in ((q, 0), (k, 4096), (v, 100 * d)):
        view = wide[:, at:at + x.shape[1] * d].unflatten(1, (-1, d))
        view.copy_(x)
        views.append(view)
    loc = starts([3, 700, 0, t - 1703, 900, 100])
    want = api.prompt_attention(q, k, v, loc, d ** -0.5)
    assert torch.equal(api.prompt_attention(*views, loc, d ** -0.5), want)
    v[t - 50, 0, 1] = views[2][t - 50, 0, 1] = float("inf")  # read again from memory
    want = api.prompt_attention(q, k, v, loc, d ** -0.5)
    assert not bool(want.isfinite().all()) and torch.equal(api.prompt_attention(*views, loc, d ** -0.5), want)

    pos = torch.arange(t, dtype=torch.int32, device="cuda") % 4096
    cs = torch.randn(4096, d, device="cuda")
    slots = torch.arange(t, device="cuda")
    pools = [torch.zeros(t // 16 + 1, hkv, 16, d, dtype=dtype, device="cuda") for _ in range(4)]
    want = api.rotary_and_cache(q, k, v, pos, cs, slots, *pools[:2])
    assert torch.equal(api.rotary_and_cache(*views, pos, cs, slots, *pools[2:]), want)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1].view(torch.int16), pools[3].view(torch.int16))
    api.rotary_and_cache(*views, pos, cs, slots, *pools[2:], query_out=views[0], key_out=views[1])
    assert torch.equal(views[0], want)
    assert api.get_device_error() == (0, 0)


@pytest.mark.parametrize("seqs,room", [(3, 60), (3, 9000), (2500, 2600)])
def test_slots_beyond_32_bits(seqs, room):
    """Block ids up to 2^31 - 1, 32 tokens each: slots up to 2^36."""
    b, top = 32, 2 ** 31 - 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    new, ctx = [40, 1, 1] + [0] * (seqs - 3), [0, 31, 32] + [0] * (seqs - 3)
    tables = i32([[0, 0], [top - 7, 0], [5, 0]] + [[0, 0]] * (seqs - 3))
    got = api.plan_step(i32(new), i32(ctx), i32([top - 1, 17, top, 9]), i32([2, 4]), tables, b, room, 2 ** 31)
    assert api.get_device_error() == (0, 0)
    ids = [top, 9, top - 1]  # from entry 2 on, around the ring's end
    want = [ids[p // b] * b + p % b for p in range(40)] + [(top - 7) * b + 31, ids[2] * b]
    assert got.slot_mapping.tolist() == want + [-1] * (room - 42)
    assert tables[:3].tolist() == [[top, 9], [top - 7, 0], [5, top - 1]]
