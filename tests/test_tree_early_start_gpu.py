"""The calls of drafted trees behind a caller's kernel that lets its dependents start before it
has written what they read (programmatic dependent launch): old lengths, rows and masks must not
be seen.  The kernel signals, waits 100 microseconds by the clock and then copies the new values."""
import ctypes
import os
import subprocess

import pytest
import torch

from paged_kv_cache_132_gb300 import api, build, native
from test_tree_verify_gpu import Case
from trees import Cache, i32, random_trees, starts

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <cuda_runtime.h>
__global__ void late(int* dst, const int* src, int n, unsigned long long ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (int i = 0; i < (1 << 20); ++i) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 > ns) break;
    }
    for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}
extern "C" int write_late(int* dst, const int* src, int n, unsigned long long ns, void* stream) {
    late<<<1, 256, 0, (cudaStream_t)stream>>>(dst, src, n, ns);
    return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def write_late(tmp_path_factory):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()
    folder = tmp_path_factory.mktemp("late")
    source, lib = str(folder / "late.cu"), str(folder / "late.so")
    with open(source, "w") as f:
        f.write(SOURCE)
    subprocess.run([os.path.join(build.cuda_home(), "bin", "nvcc"), *build.ARCH, "-O2", "-shared", "-cudart", "shared",
                    "-Xcompiler", "-fPIC", source, "-o", lib], check=True, capture_output=True, text=True)
    fn = ctypes.CDLL(lib).write_late
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_ulonglong, ctypes.c_void_p]

    def call(dst, src):
        assert dst.dtype == src.dtype and dst.is_contiguous() and src.is_contiguous() and dst.shape == src.shape
        words = dst.numel() * dst.element_size() // 4
        assert fn(dst.data_ptr(), src.data_ptr(), words, 100_000, torch.cuda.current_stream().cuda_stream) == 0

    return call


OLD = ([3, 1, 0, 20], [5, 300, 0, 40])          # nodes, tokens before them
NEW = ([40, 9, 30, 2], [2900, 700, 1800, 3000])


class Step:
    def __init__(self, d, dtype):
        g = torch.Generator(device="cuda").manual_seed(d)
        h, hkv = 16, 4
        nodes, before = NEW
        ctx = [b + n for b, n in zip(before, nodes)]
        c = Cache(ctx, hkv, d, 16, dtype, 1, stale=0.0)
        self.k, self.v, self.tables = c.k, c.v, c.tables.clamp(min=0)
        self.start, self.ctx = starts(nodes), i32(ctx)
        self.old_start, self.old_ctx = starts(OLD[0]), i32([a + b for a, b in zip(*OLD)])
        self.parents = i32([p for t in random_trees(nodes, 3, 5) for p in t])
        self.q = torch.randn(sum(nodes), h, d, generator=g, device="cuda").to(dtype)
        self.scale = d ** -0.5

    def plan(self, start, ctx):
        return api.plan_tree(self.parents, start, ctx, 64)


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])
def test_lengths_written_late(write_late, d, dtype):
    s = Step(d, dtype)
    tree = s.plan(s.start, s.ctx)
    want = api.tree_attention(s.q, s.start, tree.tree_mask, s.k, s.v, s.tables, s.ctx, s.scale)
    torch.cuda.synchronize()
    assert api.get_device_error() == (0, 0)
    for late in ("ctx", "start", "mask", "tables"):
        start = (s.old_start if late == "start" else s.start).clone()
        ctx = (s.old_ctx if late == "ctx" else s.ctx).clone()
        mask = torch.zeros_like(tree.tree_mask) if late == "mask" else tree.tree_mask
        tables = s.tables.flip(0).contiguous() if late == "tables" else s.tables
        # the call's workspace and output exist, and its code is loaded: nothing comes between
        out = torch.zeros_like(s.q)
        size = api.tree_attention_workspace_size(s.q.shape[0], 1, 16, 4, d)
        work = torch.empty(size, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        src, dst = {"ctx": (s.ctx, ctx), "start": (s.start, start), "mask": (tree.tree_mask, mask),
                    "tables": (s.tables, tables)}[late]
        write_late(dst, src)
        api.tree_attention(s.q, start, mask, s.k, s.v, tables, ctx, s.scale, out=out, workspace=work)
        torch.cuda.synchronize()
        assert api.get_device_error() == (0, 0)
        assert torch.equal(out, want), late


def test_plans_of_lengths_written_late(write_late):
    s = Step(64, torch.bfloat16)
    want = s.plan(s.start, s.ctx)
    out = api.TreePlan(*(torch.zeros_like(x) for x in want))
    start, ctx = s.start.clone(), s.old_ctx.clone()
    torch.cuda.synchronize()
    write_late(ctx, s.ctx)
    api.plan_tree(s.parents, start, ctx, 64, out=out)
    torch.cuda.synchronize()
    assert api.get_device_error() == (0, 0) and all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("drafted", [True, False])
def test_probabilities_written_late(write_late, drafted):
    """The rows and the nodes of a verification, which a call on the same SMs has just read."""
    c, other = Case([6] * 40, 3000, drafted=drafted), Case([6] * 40, 3000, drafted=drafted, seed=2)
    want = [x.clone() for x in other.call()]
    out = c.call()
    names = ["p", "ids", "up", "accept", "sample"] + (["q"] if drafted else [])
    own = {n: getattr(c, n) for n in names}
    for name in names:
        for n in names:
            buffer = getattr(other, n).contiguous() if n != name else own[n].contiguous()
            setattr(c, n, buffer.clone())
        torch.cuda.synchronize()
        c.call(out=out)
        write_late(getattr(c, name), getattr(other, name).contiguous())
        c.call(out=out)
        torch.cuda.synchronize()
        assert api.get_device_error() == (0, 0)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), name
