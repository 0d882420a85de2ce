"""Calls of a step that follow one another on a stream without a wait of the host
between them: each must see what the ones before it wrote, and leave alone what
they still use, however early its kernels are launched.  The same calls with the
GPU waited for after each one are the reference, bit for bit."""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


H, HKV, D, B = 8, 2, 128, 16


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def randn(*shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("seqs,room", [(5, 5), (300, 300), (300, 9000), (2100, 2100)])
def test_a_captured_step_of_plan_rotary_and_decode(seqs, room):
    """The plan advances the lengths in place; the decode that follows reads them.
    Contexts cross blocks and partitions; one CTA, the cluster, and its slots kernel."""
    captured_steps(seqs, room, ("plan", "rotary", "decode"))


@pytest.mark.parametrize("seqs,room", [(300, 300), (300, 9000), (2100, 2100)])
@pytest.mark.parametrize("order", [("plan", "decode"), ("plan", "prefill"), ("plan", "rotary", "prefill", "decode"),
                                   ("plan", "rotary", "prompt"), ("plan", "write", "decode", "rotary", "decode")])
def test_other_orders(order, seqs, room):
    captured_steps(seqs, room, order)


def captured_steps(seqs, room, order):
    steps, width = 12, 44
    g = torch.Generator().manual_seed(seqs)
    ctx0 = torch.randint(240, 640, (seqs,), generator=g).int()
    nb = seqs * width
    table0 = torch.randperm(nb, generator=g).int().view(seqs, width)
    held = (ctx0 + B - 1) // B
    spare = table0[torch.arange(width) >= held[:, None]]
    ring0, state0 = spare.cuda(), torch.tensor([0, spare.numel()], dtype=torch.int32).cuda()
    kc, vc = randn(nb, HKV, B, D, seed=1), randn(nb, HKV, B, D, seed=2)
    rows = randn(room, (H + 2 * HKV) * D, seed=3)
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split([H * D, HKV * D, HKV * D], 1))
    kr, vr = k.contiguous(), v.contiguous()
    angles = torch.arange(width * B, dtype=torch.float64)[:, None] * 0.7 ** torch.arange(D // 2)
    cs = torch.cat([angles.cos(), angles.sin()], 1).float().cuda()
    new = torch.ones(seqs, dtype=torch.int32, device="cuda")

    class Run:
        def __init__(self):
            self.ctx, self.state, self.ring, self.tables = ctx0.cuda(), state0.clone(), ring0.clone(), table0.cuda()
            self.k, self.v = kc.clone(), vc.clone()
            i32 = dict(dtype=torch.int32, device="cuda")
            self.plan = api.StepPlan(self.ctx, self.state, torch.empty(seqs + 1, **i32),
                                     torch.empty(room, dtype=torch.int64, device="cuda"), torch.empty(room, **i32))
            self.q = q.contiguous()  # what decode and prefill read where no call rotates it
            self.out = torch.zeros(seqs, H, D, device="cuda")
            self.rows = torch.zeros(room, H, D, dtype=q.dtype, device="cuda")
            need = max(api.decode_workspace_size(seqs, H, width * B, 0, D),
                       api.prompt_attention_workspace_size(seqs, room, H, HKV))
            self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def calls(self):
            p = self.plan
            made = dict(
                plan=lambda: api.plan_step(new, self.ctx, self.ring, self.state, self.tables, B, room, nb, out=p),
                rotary=lambda: api.rotary_and_cache(q, k, v, p.positions, cs, p.slot_mapping, self.k, self.v,
                                                    query_out=self.q),
                write=lambda: api.reshape_and_cache(kr, vr, self.k, self.v, p.slot_mapping),
                decode=lambda: api.decode(self.q[:seqs], self.k, self.v, self.tables, self.ctx, D ** -0.5, out=self.out,
                                          workspace=self.ws),
                prefill=lambda: api.prefill(self.q, p.query_start_loc, self.k, self.v, self.tables, self.ctx, D ** -0.5,
                                            1, out=self.rows),
                prompt=lambda: api.prompt_attention(self.q, k, v, p.query_start_loc, D ** -0.5, out=self.rows,
                                                    workspace=self.ws))
            return [made[x] for x in order]

    waited, graphed = Run(), Run()
    for call in graphed.calls():  # not captured: what the first call of each sets up
        call()
        torch.cuda.synchronize()
    graphed = Run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for call in graphed.calls():
            call()
    for _ in range(steps):
        for call in waited.calls():
            call()
            torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert api.get_device_error() == (0, 0)
        assert torch.equal(waited.ctx, graphed.ctx) and torch.equal(waited.tables, graphed.tables)
        assert torch.equal(waited.plan.slot_mapping, graphed.plan.slot_mapping)
        assert same(waited.k, graphed.k) and same(waited.v, graphed.v)
        assert same(waited.out, graphed.out) and same(waited.rows, graphed.rows)
    assert torch.equal(waited.ctx.cpu(), ctx0 + steps)


@pytest.mark.parametrize("before", ["rotary", "cache_write", "prompt", "decode"])
def test_a_workspace_in_memory_that_the_call_before_reads(before):
    """Inputs of a call may be freed once it returns, and an allocator of the stream
    gives them out again: here the decode's workspace is the rows that the call
    before reads."""
    seqs, width, tokens = 64, 64, 4000
    g = torch.Generator(device="cuda").manual_seed(9)
    nb = seqs * width
    tables = torch.randperm(nb, generator=g, device="cuda").int().view(seqs, width)
    ctx = torch.randint(1, width * B + 1, (seqs,), generator=g, device="cuda").int()
    kc, vc = randn(nb, HKV, B, D, seed=4), randn(nb, HKV, B, D, seed=5)
    dq = randn(seqs, H, D, seed=6)
    rows = randn(tokens, (H + 2 * HKV) * D, seed=7)
    slots = torch.randperm(nb * B, generator=g, device="cuda")[:tokens]
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda") % 512
    cs = torch.randn(512, D, generator=g, device="cuda")
    loc = torch.tensor([0, tokens // 2, tokens], dtype=torch.int32, device="cuda")
    need = api.decode_workspace_size(seqs, H, width * B, 0, D)
    short_ctx = ctx.clamp(max=250)  # one partition: no planning kernel, no merge

    def first(mem, k, v):
        q, key, val = (x.unflatten(1, (-1, D)) for x in mem.split([H * D, HKV * D, HKV * D], 1))
        if before == "rotary":
            return api.rotary_and_cache(q, key, val, pos, cs, slots, k, v)
        if before == "prompt":
            return api.prompt_attention(q, key, val, loc, D ** -0.5)
        if before == "decode":  # its queries are the rows
            return api.decode(mem.view(-1)[:seqs * H * D].view(seqs, H, D), k, v, tables, short_ctx, D ** -0.5,
                              max_context_len=250)
        flat = mem.view(-1)[:2 * tokens * HKV * D].view(2, tokens, HKV, D)
        return api.reshape_and_cache(flat[0], flat[1], k, v, slots)

    results = []
    for waited in (True, False):
        mem = torch.empty(max(need, rows.numel() * 2), dtype=torch.uint8, device="cuda")
        for _ in range(1 if waited else 5):
            k, v = kc.clone(), vc.clone()
            out = torch.empty(seqs, H, D, device="cuda")
            at = mem[:rows.numel() * 2].view(torch.bfloat16).view(rows.shape)
            at.copy_(rows)
            torch.cuda.synchronize()
            made = first(at, k, v)
            if waited:
                torch.cuda.synchronize()
            api.decode(dq, k, v, tables, ctx, D ** -0.5, out=out, workspace=mem)
            assert api.get_device_error() == (0, 0)
            results.append((made, k, v, out))
    for got in results[1:]:
        for x, y in zip(got, results[0]):
            assert (x is None and y is None) or same(x, y)
