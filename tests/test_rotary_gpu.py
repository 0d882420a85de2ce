"""Rotary embedding fused with the cache write, against its definition in 64 bits.

Tolerance, per element, with u half a step of the type: u |y| for the rounding
of the result, and 3 * 2^-24 (|a cos| + |b sin|) for two products and a sum in
binary32 (f16 also half a subnormal step, 2^-25).  Values, and the elements from
rotary_dim on, are copied bit for bit.
"""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def table(n, rot):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def case(tokens, h, hkv, d, rot, dtype, bs=16, far=4096, fused=False, padding=0, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = tokens + padding
    x = torch.randn(total, (h + 2 * hkv) * d, generator=g, device="cuda").to(dtype)
    q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([h * d, hkv * d, hkv * d], dim=1))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    pos[:tokens] = torch.randint(far, (tokens,), generator=g, device="cuda").int()
    pos[0] = far - 1
    nb = -(-tokens // bs) + 3
    slots = torch.full((total,), -1, dtype=torch.int64, device="cuda")
    slots[:tokens] = torch.randperm(nb * bs, generator=g, device="cuda")[:tokens]
    pools = [torch.full((nb, hkv, bs, d), 9.0, dtype=dtype, device="cuda") for _ in range(2)]
    return q, k, v, pos, table(far, rot), slots, pools


def rotated(x, cs, rot, interleaved):
    """(y, tolerance) in float64; x [T][heads][d], cs [T][rot]."""
    x64 = x.double()
    c, s = (t.double()[:, None] for t in cs.split(rot // 2, dim=1))
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x64[..., ia], x64[..., ib]
    y, tol = x64.clone(), torch.zeros_like(x64)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    u = torch.finfo(x.dtype).eps / 2
    tol[..., ia] = 3 * 2.0 ** -24 * ((a * c).abs() + (b * s).abs())
    tol[..., ib] = 3 * 2.0 ** -24 * ((b * c).abs() + (a * s).abs())
    rotates = torch.zeros(x.shape[-1], dtype=torch.bool)
    rotates[:rot] = True
    tol[..., rotates] += u * y[..., rotates].abs() * (1 + 1e-6) + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
    return y, tol


def within(got, want):
    y, tol = want
    assert float(((got.double() - y).abs() - tol).max()) <= 0


def run_and_check(c, rot, interleaved, keep_key, tokens):
    q, k, v, pos, cs, slots, (kc, vc) = c
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    bs = kc.shape[2]
    qo = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    ko = torch.full(k.shape, 5.0, dtype=q.dtype, device="cuda") if keep_key else None
    out = api.rotary_and_cache(q, k, v, pos, cs, slots, kc, vc, interleaved=interleaved, query_out=qo, key_out=ko)
    assert out is qo and api.get_device_error() == (0, 0)
    assert torch.equal(q, q0) and torch.equal(k, k0) and torch.equal(v, v0)
    rows = cs[pos[:tokens].long()]
    wq, wk = rotated(q0[:tokens], rows, rot, interleaved), rotated(k0[:tokens], rows, rot, interleaved)
    within(qo[:tokens], wq)
    assert bool((qo[tokens:] == 5).all())
    blk, off = slots[:tokens] // bs, slots[:tokens] % bs
    within(kc[blk, :, off], wk)
    assert torch.equal(vc[blk, :, off], v0[:tokens])
    if keep_key:
        assert torch.equal(ko[:tokens], kc[blk, :, off]) and bool((ko[tokens:] == 5).all())
    free = torch.ones(kc.shape[0] * bs, dtype=torch.bool, device="cuda")
    free[slots[:tokens]] = False
    for pool in (kc, vc):
        assert bool((pool.transpose(1, 2).reshape(-1, *pool.shape[1::2])[free] == 9).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("h,hkv,d,rot", [(32, 8, 128, 128), (4, 4, 64, 32), (6, 2, 64, 16), (1, 1, 128, 64),
                                         (40, 40, 128, 128), (3, 1, 72, 32), (2, 1, 256, 256), (5, 5, 24, 16)])
def test_shapes(dtype, interleaved, h, hkv, d, rot):
    for tokens, keep, fused in ((1, False, False), (37, True, True)):
        c = case(tokens, h, hkv, d, rot, dtype, fused=fused, padding=5 if keep else 0, bs=8, seed=h + tokens)
        run_and_check(c, rot, interleaved, keep, tokens)


@pytest.mark.parametrize("bs", [1, 8, 16, 32, 48])
def test_block_sizes(bs):
    run_and_check(case(300, 8, 2, 128, 128, torch.bfloat16, bs=bs, far=131072), 128, False, True, 300)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(interleaved):
    """The outputs may be the inputs, slices of one projection included."""
    q, k, v, pos, cs, slots, (kc, vc) = case(70, 12, 4, 64, 64, torch.float16, fused=True, padding=3)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    want = api.rotary_and_cache(q0, k0, v0, pos, cs, slots, kc.clone(), vc.clone(), interleaved=interleaved)
    api.rotary_and_cache(q, k, v, pos, cs, slots, kc, vc, interleaved=interleaved, query_out=q, key_out=k)
    assert api.get_device_error() == (0, 0)
    assert torch.equal(q[:70], want[:70]) and torch.equal(q[70:], q0[70:]) and torch.equal(k[70:], k0[70:])
    assert torch.equal(v, v0)
    within(k[:70], rotated(k0[:70], cs[pos[:70].long()], 64, interleaved))
    assert torch.equal(kc[slots[:70] // 16, :, slots[:70] % 16], k[:70])


def test_uncached_and_bad_tokens():
    """A slot < 0 is rotated but not cached; a position or slot out of range is
    reported, and touches nothing."""
    q, k, v, pos, cs, slots, (kc, vc) = case(40, 4, 2, 64, 64, torch.bfloat16, far=100)
    clean = api.rotary_and_cache(q, k, v, pos, cs, slots, kc.clone(), vc.clone())
    slots[3] = -1
    slots[7] = kc.shape[0] * kc.shape[2]
    ko = torch.full_like(k, 5.0)
    out = torch.full_like(q, 5.0)
    k1, v1 = kc.clone(), vc.clone()
    api.rotary_and_cache(q, k, v, pos, cs, slots, k1, v1, query_out=out, key_out=ko)
    assert api.get_device_error() == (-5, native.DEVERR_SLOT)
    assert torch.equal(out, clean) and not bool((ko == 5).all(-1).any())
    written = (k1 != 9).any(-1).any(1).sum()
    assert int(written) == 38
    slots[7] = -1
    pos[11] = 100
    pos[12] = 2 ** 31 - 1
    pos[13] = -2 ** 31
    out.fill_(5.0)
    api.rotary_and_cache(q, k, v, pos, cs, slots, k1, v1, query_out=out)
    assert api.get_device_error() == (-5, native.DEVERR_POSITION)
    assert bool((out[11:14] == 5).all()) and torch.equal(out[14:], clean[14:]) and torch.equal(out[:11], clean[:11])


def test_checked_mode_reports_duplicate_slots():
    q, k, v, pos, cs, slots, (kc, vc) = case(40, 4, 2, 64, 64, torch.bfloat16)
    slots[5] = slots[9]
    with api.option("debug_checks"):
        api.rotary_and_cache(q, k, v, pos, cs, slots, kc, vc)
    assert api.get_device_error() == (-5, native.DEVERR_DUP_SLOT)


def test_captured_on_another_stream():
    q, k, v, pos, cs, slots, (kc, vc) = case(50, 8, 2, 128, 128, torch.bfloat16)
    out = torch.empty_like(q)
    api.rotary_and_cache(q, k, v, pos, cs, slots, kc, vc, query_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.rotary_and_cache(q, k, v, pos, cs, slots, kc, vc, query_out=out)
    q.neg_()
    pos.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    within(out, rotated(q, cs[pos.long()], 128, False))
    side = torch.cuda.Stream()
    got = api.rotary_and_cache(q, k, v, pos, cs, slots, kc, vc, stream=side)
    side.synchronize()
    assert torch.equal(got, out)


def test_refusals():
    q, k, v, pos, cs, slots, (kc, vc) = case(20, 4, 2, 64, 64, torch.float16)
    call = api.rotary_and_cache
    for bad in (dict(query=q.float()), dict(key=k[:19]), dict(value=v[:, :1]), dict(positions=pos.long()),
                dict(positions=pos[:19]), dict(slot_mapping=slots.int()), dict(cos_sin=cs.double()),
                dict(cos_sin=cs.t()), dict(query_out=torch.empty(20, 4, 64, device="cuda")), dict(key_out=k[:5]),
                dict(query=q.cpu()), dict(query=q.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(key_out=k[:1].expand(20, 2, 64)), dict(v_cache=vc[:1])):
        a = dict(query=q, key=k, value=v, positions=pos, cos_sin=cs, slot_mapping=slots, k_cache=kc, v_cache=vc)
        a.update(bad)
        with pytest.raises(ValueError):
            call(**a)
    with pytest.raises(native.PaError):
        call(q, k, v, pos, cs[:, :24].contiguous(), slots, kc, vc)
