"""Guard regions around every buffer that the calls of a step write: each output
is a view into a larger allocation whose margins must still hold their pattern
afterwards, and the results equal those on plain buffers bit for bit."""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from test_guards_gpu import Guarded, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


@pytest.mark.parametrize("lens", [[1], [17, 0, 300], [129] * 40])
@pytest.mark.parametrize("h,hkv,d", [(8, 2, 128), (6, 2, 64), (5, 5, 64)])
def test_prompt_attention(lens, h, hkv, d):
    t = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(t + h)
    q, k, v = (torch.randn(t, n, d, generator=g, device="cuda").half() for n in (h, hkv, hkv))
    loc = torch.tensor([0] + lens).cumsum(0).int().cuda()
    want = api.prompt_attention(q, k, v, loc, 0.1)
    out = Guarded((t, h, d), torch.float16)
    ws = Guarded((api.prompt_attention_workspace_size(len(lens), t, h, hkv),), torch.uint8)
    ins = [Guarded(x.shape, x.dtype, init=x) for x in (q, k, v)]
    api.prompt_attention(*(x.t for x in ins), loc, 0.1, out=out.t, workspace=ws.t)
    assert api.get_device_error() == (0, 0)
    assert out.intact() and ws.intact() and all(x.intact() for x in ins)
    assert same_bits(out.t, want) and all(same_bits(x.t, y) for x, y in zip(ins, (q, k, v)))


@pytest.mark.parametrize("dtype,d,rot,tokens", [(torch.bfloat16, 128, 128, 77), (torch.float32, 72, 32, 5),
                                                (torch.float16, 24, 16, 2000)])
def test_rotary_and_cache(dtype, d, rot, tokens):
    h, hkv, bs = 6, 2, 16
    g = torch.Generator(device="cuda").manual_seed(tokens)
    q, k, v = (torch.randn(tokens, n, d, generator=g, device="cuda").to(dtype) for n in (h, hkv, hkv))
    nb = -(-tokens // bs)
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:tokens]
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    cs = torch.randn(tokens, rot, generator=g, device="cuda")
    plain = [torch.zeros(nb, hkv, bs, d, dtype=dtype, device="cuda") for _ in range(2)]
    ko = torch.empty_like(k)
    want = api.rotary_and_cache(q, k, v, pos, cs, slots, *plain, key_out=ko)
    pools = [Guarded(x.shape, dtype, init=torch.zeros_like(x)) for x in plain]
    qo, kg = Guarded(q.shape, dtype), Guarded(k.shape, dtype)
    api.rotary_and_cache(q, k, v, pos, cs, slots, *(x.t for x in pools), query_out=qo.t, key_out=kg.t)
    assert api.get_device_error() == (0, 0)
    assert qo.intact() and kg.intact() and all(x.intact() for x in pools)
    assert same_bits(qo.t, want) and same_bits(kg.t, ko) and all(same_bits(x.t, y) for x, y in zip(pools, plain))


@pytest.mark.parametrize("seqs,tokens", [(1, 5), (70, 41), (3000, 3), (40, 700)])
def test_plan_step(seqs, tokens):
    b = 16
    g = torch.Generator().manual_seed(seqs)
    ctx = torch.randint(0, 50, (seqs,), generator=g)
    new = torch.where(torch.arange(seqs) % 3 == 1, -1, torch.randint(0, tokens + 1, (seqs,), generator=g))
    after = (ctx + new.clamp(min=0) + b - 1) // b
    total, width = int(after.sum()) + 3, int(after.max())
    held = (ctx + b - 1) // b
    order = torch.randperm(total, generator=g).int()
    tables = torch.zeros(seqs, width, dtype=torch.int32)
    tables[torch.arange(width) < held[:, None]] = order[:int(held.sum())]
    ring = torch.cat([order[int(held.sum()):], torch.zeros(int(held.sum()), dtype=torch.int32)])
    free = torch.tensor([0, total - int(held.sum())], dtype=torch.int32)
    rows = int(new.clamp(min=0).sum())
    args = (new.int().cuda(), ctx.int().cuda(), ring.cuda(), free.cuda(), tables.cuda())
    want = api.plan_step(*args, b, rows, total)
    boxes = [Guarded(x.shape, x.dtype, init=y.cuda()) for x, y in zip(args, (new.int(), ctx.int(), ring, free, tables))]
    outs = [Guarded(x.shape, x.dtype) for x in want]
    api.plan_step(*(x.t for x in boxes), b, rows, total, out=api.StepPlan(*(x.t for x in outs)))
    assert api.get_device_error() == (0, 0)
    assert all(x.intact() for x in boxes + outs)
    assert all(same_bits(x.t, y) for x, y in zip(outs, want))
    assert same_bits(boxes[2].t, args[2]) and same_bits(boxes[4].t, args[4])
