"""Drafted trees for the tests: random shapes, caches whose stale slots are NaN, and
the operators' definitions on the CPU or in 64 bits."""
from __future__ import annotations

import random

import torch


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def starts(lens, first=0):
    return torch.tensor([first] + list(lens)).cumsum(0).to(torch.int32).cuda()


def parents_of(n, width, r):
    """A tree of n nodes; width 1 is a chain."""
    return [-1] + [r.randrange(max(0, i - width), i) for i in range(1, n)] if n else []


def ancestors(parents):
    out = []
    for i, p in enumerate(parents):
        out.append(([] if p < 0 else out[p]) + [i])
    return out


def words(rows, count):
    """Rows of node numbers -> int64 [rows][count]."""
    out = []
    for nodes in rows:
        bits = sum(1 << j for j in nodes)
        row = [(bits >> (64 * w)) & (2 ** 64 - 1) for w in range(count)]
        out.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in row])
    return torch.tensor(out, dtype=torch.int64).reshape(len(rows), count)


class Cache:
    """Pools and tables of sequences of `ctx` tokens; slots of no token hold `stale`."""

    def __init__(self, ctx, hkv, d, block, dtype, seed, spare=3, stale=float("nan")):
        g = torch.Generator(device="cuda").manual_seed(seed)
        held = [-(-c // block) for c in ctx]
        total = sum(held) + spare
        order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
        self.block, self.num_blocks = block, total
        self.tables = torch.full((len(ctx), max(held + [1]) + 1), -1, dtype=torch.int32)
        self.k = torch.full((total, hkv, block, d), stale, dtype=dtype, device="cuda")
        self.v = self.k.clone()
        self.left = order[sum(held):]
        at = 0
        for s, (c, n) in enumerate(zip(ctx, held)):
            self.tables[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
            slots = self.slots(s, c)
            for pool in (self.k, self.v):
                pool[slots // block, :, slots % block] = torch.randn(c, hkv, d, generator=g, device="cuda").to(dtype)
        self.tables = self.tables.cuda()

    def slots(self, s, tokens):
        p = torch.arange(tokens, device="cuda")
        return self.tables[s].to("cuda").long()[p // self.block] * self.block + p % self.block

    def rows(self, s, tokens):
        """k, v [tokens][Hkv][d] of a sequence."""
        at = self.slots(s, tokens)
        return self.k[at // self.block, :, at % self.block], self.v[at // self.block, :, at % self.block]


def attention(q, k, v, base, attends, scale):
    """(out, tolerance) [n][H][d] in 64 bits of one sequence: `attends` bool [n][n], its
    nodes from position `base` on.  Tolerance, per element, with u half a step of the type
    (bf16 2^-8, f16 2^-11) and A = sum_j p_j |v_j|:
      u A             the weights' rounding to the type
      u |o|           the output's rounding
      2 delta A       relative error of a weight, and of their sum, from the scores: a dot
                      product in binary32 is off by at most d 2^-23 sum |q_e k_e| (each of d
                      additions rounded or truncated), the exponent's argument by 2^-23 of
                      its magnitude, the hardware's 2^x by 2^-22; joined parts have two
                      powers more
      (L + 64) 2^-23 A  the sums over L positions, rounded or truncated one by one
      L 2^-25 max|v|  f16 only: small weights are subnormal and off by up to 2^-25 (of
                      weights 2^7 larger: a bound with room)."""
    n, h, d = q.shape
    g, size = h // k.shape[1], k.shape[0]
    u = torch.finfo(q.dtype).eps / 2
    hidden = torch.cat([torch.zeros(n, base, dtype=torch.bool, device="cuda"), ~attends.cuda()], 1)
    seen = ~hidden.all(0)
    q64 = q.double().transpose(0, 1)
    k64 = torch.where(seen[:, None, None], k.double(), 0.0).transpose(0, 1).repeat_interleave(g, 0)
    v64 = torch.where(seen[:, None, None], v.double(), 0.0).transpose(0, 1).repeat_interleave(g, 0)
    z = (q64 @ k64.transpose(1, 2) * scale).masked_fill(hidden, float("-inf"))
    zabs = (q64.abs() @ k64.abs().transpose(1, 2) * scale).masked_fill(hidden, 0)
    p = torch.softmax(z, -1)
    p = torch.where(hidden.all(1)[:, None], 0.0, p)
    out, a = p @ v64, p @ v64.abs()
    spread = z.masked_fill(hidden, 0).abs().amax(-1, keepdim=True)
    delta = (d * 2.0 ** -23 * zabs).amax(-1, keepdim=True) + 3 * 2.0 ** -22 + 9 * 2.0 ** -23 * spread
    tol = u * (a + out.abs()) * 1.01 + 2 * delta * a + (size + 64) * 2.0 ** -23 * a
    if q.dtype == torch.float16:
        tol = tol + size * 2.0 ** -25 * v64.abs().amax() + 2.0 ** -25
    return out.transpose(0, 1), tol.transpose(0, 1)


def random_trees(lens, width, seed):
    r = random.Random(seed)
    return [parents_of(n, width, r) for n in lens]
