"""Attention over whole packed prompts against its definition in 64 bits.

Tolerance, per element, with u half a step of the type (bf16 2^-8, f16 2^-11)
and A = sum_j p_j |v_j| the weighted sum of the values' magnitudes:
  u A       the weights' rounding to the type
  u |o|     the output's rounding
  2 delta A relative error of a weight, and of their sum, from the scores: a dot
            product in binary32 is off by at most d 2^-23 sum |q_e k_e| (each of
            d additions rounded or truncated), the exponent's argument by 2^-23
            of its magnitude, the hardware's 2^x by 2^-22
  n 2^-25 max|v|  f16 only: weights below 2^-14 of the row's reference are
            subnormal and off by up to 2^-25
"""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def starts(lens, first=0):
    return torch.tensor([first] + lens).cumsum(0).to(torch.int32).cuda()


def rows(tokens, h, hkv, d, dtype, seed, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, (h + 2 * hkv) * d, generator=g, device="cuda").to(dtype)
    q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([h * d, hkv * d, hkv * d], dim=1))
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def exact(q, k, v, scale):
    """(out, tolerance) of one sequence, float64."""
    n, h, d = q.shape
    g = h // k.shape[1]
    u = torch.finfo(q.dtype).eps / 2
    q64 = q.double().transpose(0, 1)
    k64 = k.double().transpose(0, 1).repeat_interleave(g, 0)
    v64 = v.double().transpose(0, 1).repeat_interleave(g, 0)
    z = q64 @ k64.transpose(1, 2) * scale
    zabs = q64.abs() @ k64.abs().transpose(1, 2) * scale
    future = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
    p = torch.softmax(z.masked_fill(future, float("-inf")), -1)
    out, a = p @ v64, p @ v64.abs()
    spread = z.masked_fill(future, 0).abs().amax(-1, keepdim=True)
    delta = (d * 2.0 ** -23 * zabs.masked_fill(future, 0)).amax(-1, keepdim=True) + 2.0 ** -22 + 3 * 2.0 ** -23 * spread
    tol = u * (a + out.abs()) * 1.01 + 2 * delta * a
    if q.dtype == torch.float16:
        tol = tol + n * 2.0 ** -25 * v64.abs().amax() + 2.0 ** -25
    return out.transpose(0, 1), tol.transpose(0, 1)


def check(q, k, v, lens, scale, out, first=0):
    at = first
    for n in lens:
        if n:
            ref, tol = exact(q[at:at + n], k[at:at + n], v[at:at + n], scale)
            off = (out[at:at + n].double() - ref).abs() - tol
            assert not torch.isnan(out[at:at + n]).any(), f"NaN in a sequence of {n}"
            assert float(off.max()) <= 0, f"sequence of {n}: {float(off.max())} over its tolerance"
        at += n


def run(lens, h, hkv, d, dtype, seed=1, fused=False, scale=None, extra=0, first=0):
    tokens = first + sum(lens) + extra
    q, k, v = rows(tokens, h, hkv, d, dtype, seed, fused)
    scale = d ** -0.5 if scale is None else scale
    out = torch.full((tokens, h, d), 7.0, dtype=dtype, device="cuda")
    got = api.prompt_attention(q, k, v, starts(lens, first), scale, out=out)
    assert got is out
    assert api.get_device_error() == (0, 0)
    check(q, k, v, lens, scale, out, first)
    end = first + sum(lens)
    assert bool((out[:first] == 7).all()) and bool((out[end:] == 7).all()), "rows outside the sequences were written"
    return q, k, v, out


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 257, 500])
@pytest.mark.parametrize("h,hkv,d,dtype", [(8, 2, 64, torch.bfloat16), (4, 4, 128, torch.float16)])
def test_one_sequence(n, h, hkv, d, dtype):
    run([n], h, hkv, d, dtype, seed=n)


@pytest.mark.parametrize("h,hkv", [(1, 1), (8, 8), (4, 2), (6, 2), (8, 2), (5, 1), (14, 2), (8, 1), (16, 1), (32, 1),
                                   (71, 1), (128, 1)])
@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
def test_groups(h, hkv, d, dtype):
    run([77, 0, 1, 300, 129, 64], h, hkv, d, dtype, seed=h, fused=True, extra=3, first=2)


def test_many_sequences_and_empty_ones():
    g = torch.Generator().manual_seed(5)
    lens = (torch.randint(0, 70, (300,), generator=g) * torch.randint(0, 2, (300,), generator=g)).tolist()
    run(lens, 16, 8, 64, torch.bfloat16, fused=True, extra=200)


def test_all_sequences_empty():
    run([0] * 40, 8, 2, 64, torch.bfloat16, extra=9)


@pytest.mark.parametrize("h,hkv,d,dtype", [(4, 1, 128, torch.bfloat16), (2, 2, 64, torch.float16)])
def test_long(h, hkv, d, dtype):
    run([2500, 4097], h, hkv, d, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_growing_scores(dtype):
    """Later keys score higher and higher: the running maximum grows in every tile."""
    n, h, d = 900, 4, 128
    q, k, v = rows(n, h, h, d, dtype, 3)
    ramp = torch.linspace(0.02, 6.0, n, device="cuda")[:, None, None]
    q, k = q.abs().to(dtype), (k.abs() * ramp).to(dtype)
    out = api.prompt_attention(q, k, v, starts([n]), d ** -0.5)
    assert api.get_device_error() == (0, 0)
    check(q, k, v, [n], d ** -0.5, out)


@pytest.mark.parametrize("what", ["nan", "inf", "lowest"])
@pytest.mark.parametrize("h,hkv,d,dtype", [(8, 2, 128, torch.bfloat16), (4, 4, 64, torch.float16),
                                           (6, 2, 64, torch.bfloat16)])
def test_unattended_rows_may_hold_anything(what, h, hkv, d, dtype):
    """Rows outside the sequences, and later tokens of a sequence, change nothing
    of what does not attend them, to the bit."""
    lens, first, extra = [70, 300, 5, 513], 7, 150
    tokens = first + sum(lens) + extra
    q, k, v = rows(tokens, h, hkv, d, dtype, 11)
    loc = starts(lens, first)
    clean = api.prompt_attention(q, k, v, loc, d ** -0.5)
    fill = {"nan": float("nan"), "inf": float("inf"), "lowest": torch.finfo(dtype).min}[what]
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    end = first + sum(lens)
    for x in (q2, k2, v2):
        x[:first] = fill
        x[end:] = fill
    poisoned = [(first + 70 + 211, 1), (first + 70 + 300 + 5 + 500, 0), (first + 69, 0)]  # (row, column)
    for row, col in poisoned:
        k2[row] = fill
        v2[row, :, col::3] = fill
    out = api.prompt_attention(q2, k2, v2, loc, d ** -0.5)
    assert api.get_device_error() == (0, 0)
    at = first
    for n in lens:
        bad = [r for r, _ in poisoned if at <= r < at + n]
        upto = min(bad) if bad else at + n
        assert torch.equal(out[at:upto], clean[at:upto])
        if bad and what != "lowest":
            assert not torch.isfinite(out[upto:at + n, :, :]).all(-1).any()  # each later row attends it
        at += n


def test_non_finite_values_reach_what_attends_them():
    """An infinite or NaN value decides its column of every row from its own on,
    and no other column."""
    n, h, hkv, d = 400, 4, 2, 128
    q, k, v = rows(n, h, hkv, d, torch.bfloat16, 12)
    loc = starts([n])
    clean = api.prompt_attention(q, k, v, loc, d ** -0.5)
    v2 = v.clone()
    v2[150, 0, 5] = float("inf")
    v2[390, 1, 100] = float("nan")
    v2[395, 0, 5] = float("-inf")
    v2[20, 1, 0] = float("-inf")
    out = api.prompt_attention(q, k, v2, loc, d ** -0.5)
    want = clean.clone()
    want[150:, :2, 5] = float("inf")
    want[395:, :2, 5] = float("nan")
    want[390:, 2:, 100] = float("nan")
    want[20:, 2:, 0] = float("-inf")
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out[~out.isnan()], want[~want.isnan()])


def test_bad_start_rows_are_reported():
    """Start rows out of range: the sequences they spoil are skipped, the others
    computed.  Out of order, so that sequences overlap: none is."""
    q, k, v = rows(300, 4, 2, 64, torch.float16, 13)
    loc = torch.tensor([0, 90, 90, 300, 301], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    api.prompt_attention(q, k, v, loc, 0.125, out=out)
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    check(q, k, v, [90, 210], 0.125, out)
    loc = torch.tensor([0, 90, 50, 300], dtype=torch.int32, device="cuda")
    out.fill_(7.0)
    api.prompt_attention(q, k, v, loc, 0.125, out=out)
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    assert bool((out == 7).all())
    loc = torch.tensor([-3, 100], dtype=torch.int32, device="cuda")
    out.fill_(7.0)
    api.prompt_attention(q, k, v, loc, 0.125, out=out)
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    assert bool((out == 7).all())


def test_captured_and_replayed_with_other_lengths():
    q, k, v = rows(400, 8, 2, 64, torch.bfloat16, 14)
    loc = starts([150, 250])
    out = torch.empty_like(q)
    api.prompt_attention(q, k, v, loc, 0.125, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.prompt_attention(q, k, v, loc, 0.125, out=out)
    for lens in ([150, 250], [399, 1], [0, 128]):
        loc.copy_(starts(lens))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(q, k, v, lens, 0.125, out)
        assert bool((out[sum(lens):] == 7).all())


def test_another_stream_and_two_calls_at_once():
    a = rows(600, 8, 2, 128, torch.bfloat16, 15)
    b = rows(600, 8, 8, 128, torch.bfloat16, 16)
    loc = starts([600])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(api.prompt_attention(*a, loc, 0.1, stream=s1), api.prompt_attention(*b, loc, 0.1, stream=s2))
            for _ in range(4)]
    torch.cuda.synchronize()
    assert api.get_device_error() == (0, 0)
    for x, y in outs:
        check(*a, [600], 0.1, x)
        check(*b, [600], 0.1, y)


def test_one_token_of_a_wider_array():
    """The stride of a single row does not matter."""
    wide = torch.randn(3, 4 * 64 + 8, device="cuda").half()[1:2, :256]
    q, k, v = wide.unflatten(1, (4, 64)), wide[:, :128].unflatten(1, (2, 64)), wide[:, 128:].unflatten(1, (2, 64))
    out = api.prompt_attention(q, k, v, starts([1]), 0.125)
    assert api.get_device_error() == (0, 0)
    assert torch.equal(out, v.repeat_interleave(2, 1))


def test_two_graphs_share_a_workspace():
    """Replayed one after the other: each call resets what it needs."""
    a, b = rows(700, 32, 8, 64, torch.bfloat16, 20), rows(900, 32, 8, 64, torch.bfloat16, 21)
    la, lb = starts([300, 400]), starts([50] * 18)
    size = max(api.prompt_attention_workspace_size(n, t, 32, 8) for n, t in ((2, 700), (18, 900)))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    oa, ob = torch.empty_like(a[0]), torch.empty_like(b[0])
    graphs = []
    for x, loc, o in ((a, la, oa), (b, lb, ob)):
        api.prompt_attention(*x, loc, 0.125, out=o, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.prompt_attention(*x, loc, 0.125, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        oa.zero_(), ob.zero_()
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        check(*a, [300, 400], 0.125, oa)
        check(*b, [50] * 18, 0.125, ob)
    assert api.get_device_error() == (0, 0)


def test_refusals():
    q, k, v = rows(20, 4, 2, 64, torch.float16, 17)
    loc = starts([20])
    with pytest.raises(ValueError):
        api.prompt_attention(q, k, v.bfloat16(), loc, 0.1)
    with pytest.raises(ValueError):
        api.prompt_attention(q, k[:19], v[:19], loc, 0.1)
    with pytest.raises(ValueError):
        api.prompt_attention(q, k, v, loc.long(), 0.1)
    with pytest.raises(ValueError):
        api.prompt_attention(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, loc, 0.1)  # heads outermost
    with pytest.raises(ValueError):
        api.prompt_attention(q, k[:1].expand(20, 2, 64), v, loc, 0.1)  # rows that overlap
    with pytest.raises(ValueError):
        api.prompt_attention(q, k, v, loc, 0.1, out=torch.empty(20, 4, 64, device="cuda"))
    with pytest.raises(ValueError):
        api.prompt_attention(q.cpu(), k.cpu(), v.cpu(), loc.cpu(), 0.1)
    with pytest.raises(native.PaError):
        api.prompt_attention(q.float(), k.float(), v.float(), loc, 0.1)
    with pytest.raises(native.PaError):
        api.prompt_attention(q, k, v, loc, 0.0)
    with pytest.raises(native.PaError):
        api.prompt_attention(q, k, v, loc, 0.1, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("h,hkv", [(8, 1), (8, 8)])
def test_overlapping_start_rows_stay_inside_the_workspace(h, hkv):
    """Start rows that go back and forth claim more work than the rows hold: the
    call reports it, and writes nothing outside its buffers."""
    n = 4000
    q, k, v = rows(n, h, hkv, 64, torch.float16, 18)
    loc = torch.tensor([0, n] * 20, dtype=torch.int32, device="cuda")
    need = api.prompt_attention_workspace_size(39, n, h, hkv)
    room = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0)
    api.prompt_attention(q, k, v, loc, 0.1, workspace=room[:need], out=out)
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    assert bool((room[need:] == 0x5a).all()) and bool((out == 7).all())


def test_scores_of_minus_infinity_have_no_weight():
    """A whole tile of keys whose scores overflow to -inf: weight 0, whatever comes later."""
    n, d = 300, 64
    q, k, v = rows(n, 2, 2, d, torch.bfloat16, 19)
    q = q.abs() + 1
    k2 = k.clone()
    k2[:140] = -3e38
    out = api.prompt_attention(q, k2, v, starts([n]), d ** -0.5)
    assert api.get_device_error() == (0, 0)
    ref, tol = exact(q[140:], k[140:], v[140:], d ** -0.5)
    assert bool(out[:140].isnan().all())  # nothing but such scores
    assert float(((out[140:].double() - ref).abs() - tol).max()) <= 0
