"""The weights p - c q of a verification: how near their sums come to the exact ones.  Per weight:
2^-57 for the first difference (c = 1), 2^-46 for any c."""
from fractions import Fraction

import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from trees import i32, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


# ---------------------------------------------------------------------------
# the sums after refusals, measured by a child's acceptance
# ---------------------------------------------------------------------------
# Children of one node: k with p = 0, refused for certain, then X with u = 0, accepted if
# p(X) > c q(X), c = 1 + s_1 + ... + s_(k-1) with the sums of the refusals before the last.  So p(X) / q(X), next to c, tells on which side of it the
# call's c lies.  p(X) and q(X) are below 2^-76: X adds less than 2^-76 to a sum.
def near(c, gap):
    """Binary32 pairs (p, q) below 2^-76 with p / q beyond c - gap and c + gap, as near as a search
    of continued fractions finds."""
    out = []
    for side in (-1, 1):
        for k in (2, 3, 4, 6, 8, 16, 32):
            f = (c + side * k * gap).limit_denominator(int((2 ** 24 - 2) / (c + 32 * gap)))
            if side * (f - c) > gap and f.numerator < 2 ** 24:
                out.append((f.numerator * 2.0 ** -100, f.denominator * 2.0 ** -100))
                break
    assert len(out) == 2
    return out


def measured(p, q, c, gap, refusals):
    """Rows p, q [n][V] (binary32 in binary64); whether X is accepted, for the pair below c and the
    one above, [n][2].  Two entries are added to each row: Z, which is refused, and X."""
    n, v = p.shape
    nodes = refusals + 2
    rows_p = torch.zeros(n, 2, nodes, v + 2, dtype=torch.float64)
    rows_q = torch.zeros_like(rows_p)
    rows_p[..., :v], rows_q[..., :v] = p[:, None, None], q[:, None, None]
    rows_q[..., v] = 0.25
    for s in range(n):
        for k, (a, b) in enumerate(near(c[s], gap)):
            rows_p[s, k, :, v + 1], rows_q[s, k, :, v + 1] = a, b
    total = n * 2 * nodes
    rows_p, rows_q = rows_p.view(total, v + 2).float().cuda(), rows_q.view(total, v + 2).float().cuda()
    ids = i32(([0] + [v] * refusals + [v + 1]) * (2 * n))
    up = i32(([-1] + [0] * (nodes - 1)) * (2 * n))
    got = api.verify_tree(ids, up, starts([nodes] * (2 * n)), rows_p, rows_q, torch.zeros(total, device="cuda"),
                          torch.zeros(2 * n, device="cuda"))
    assert api.get_device_error() == (0, 0)
    return (got.accepted_lens == 2).view(n, 2).cpu()


def f32(x):
    return x.float().double()


def test_sums_of_differences():
    """c = 1: every weight p - q is within half a unit, 2^-57 (and 2^-69 for the sum of what is below
    a unit's step of the difference and of its rounding error), a row of 1024 within 2^-46; 1 + s in
    binary64 is off by 2^-53.  Rows of one pair repeated, so that errors add up."""
    g = torch.Generator().manual_seed(11)
    n, v = 400, 1024
    one = f32(2.0 ** (-10 - 2 * torch.rand(n, 1, generator=g, dtype=torch.float64)))
    other = f32(one * 2.0 ** (-28 * torch.rand(n, 1, generator=g, dtype=torch.float64)))
    c = [1 + v * max(Fraction(a) - Fraction(b), 0) for a, b in zip(one[:, 0].tolist(), other[:, 0].tolist())]
    got = measured(one.expand(n, v), other.expand(n, v), c, Fraction(1, 2 ** 43), 2)
    assert not got[:, 0].any() and got[:, 1].all()


def test_sums_after_a_second_refusal():
    """Any c, where the weight is positive and so c q < 1: c is split into two binary32 (2^-48 c q),
    and what the product and the difference leave, up to 2^-24 and 2^-23, is rounded (2^-48 each):
    less than 2^-46.  Nine of them and the sums in binary64: less than 16 x 2^-46.  First entries
    with p next to c q, where the difference cancels, and behind them small ones."""
    g = torch.Generator().manual_seed(12)
    n, v = 3000, 9
    rand = lambda *shape: torch.rand(*shape, generator=g, dtype=torch.float64)  # noqa: E731
    p = rand(n, v) * 2.0 ** (-4 - 6 * rand(n, v))
    p[:, 0] = 0.5 + 0.5 * rand(n)
    e = 2.0 ** (-1 - 23 * rand(n, 1))
    p[:, 1:] *= 1 - p[:, :1]
    p = f32(p)
    q = f32(p / (1 + e * (0.25 + 0.75 * rand(n, v))))
    q[:, 0] = f32(p[:, 0] / (1 + e[:, 0]))
    c, lost = [], 0
    for a, b in zip(p.tolist(), q.tolist()):
        a, b = [Fraction(x) for x in a], [Fraction(x) for x in b]
        c2 = Fraction(1.0 + float(sum(max(x - y, 0) for x, y in zip(a, b))))
        w = [max(x - c2 * y, 0) for x, y in zip(a, b)]
        lost += w[0] > 0 and a[0] < c2 * b[0] + Fraction(1, 2 ** 25)
        c.append(c2 + sum(w))
    assert lost > 50   # rows that the cancellation is about
    got = measured(p, q, c, Fraction(16, 2 ** 46), 3)
    assert not got[:, 0].any() and got[:, 1].all(), (got[:, 0].sum(), (~got[:, 1]).sum())
