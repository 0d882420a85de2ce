"""The weights p - c q of a verification.  They count in units of 2^-56, each entry by itself, so
that a row's sum, a segment's, a vector's and an entry's agree.  A weight is within 2^-57 for the
row itself and the first difference (c = 0 and 1), within 2^-46 for any c."""
from fractions import Fraction

import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from trees import i32, starts

pytestmark = pytest.mark.gpu

UNIT = 2 ** 56


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def units(x):
    """A weight in units, rounded to nearest, ties to even."""
    return round(Fraction(x) * UNIT)


def place(values, dtype, skew):
    """Rows [n][V] that begin `skew` entries behind a 16-byte boundary, NaN around them."""
    n, v = values.shape
    wide = torch.full((n, -(-(v + skew) // 16) * 16), float("nan"), dtype=dtype, device="cuda")
    wide[:, skew:skew + v] = values.to(dtype)
    return wide[:, skew:skew + v]


def token_of(row, u):
    """The lowest t whose cumulative units exceed u times their sum, which stays below 2^64."""
    w = [units(x) for x in row]
    left = int(Fraction(u) * min(sum(w), 2 ** 64 - 1))
    for t, x in enumerate(w):
        if x > left:
            return t
        left -= x
    return -1


# ---------------------------------------------------------------------------
# weights of a unit and less: every level of the sums counts them alike
# ---------------------------------------------------------------------------
SMALL = [2.0 ** -60, 0.3 * 2.0 ** -56, 0.5 * 2.0 ** -56, 0.6 * 2.0 ** -56, 1.4 * 2.0 ** -56]


@pytest.mark.parametrize("small", SMALL)
@pytest.mark.parametrize("skew", [0, 1, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [5, 512, 1024, 6000])
def test_first_token_behind_small_weights(vocab, dtype, skew, small):
    rows = torch.full((2, vocab), small, dtype=torch.float64)
    rows[:, -1] = 1.0
    p = place(rows, dtype, skew)
    u = torch.tensor([0.0, 2.0 ** -40], device="cuda")
    got = api.verify_tree(i32([0, 0]), i32([-1, -1]), starts([1, 1]), p, None, torch.zeros(2, device="cuda"), u)
    assert api.get_device_error() == (0, 0)
    assert got.next_tokens.tolist() == [token_of(r, x) for r, x in zip(p.double().tolist(), u.tolist())]


@pytest.mark.parametrize("skew", [0, 1, 2])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_rows_of_small_weights(dtype, skew):
    """Nothing but weights around a unit (16-bit floats of 5 exponent bits: their smallest, 2^-24)."""
    g = torch.Generator().manual_seed(3 + skew)
    n, vocab = 96, 1201
    low = 2.0 ** -24 if dtype is torch.float16 else 2.0 ** -60
    rows = low * 2.0 ** (8 * torch.rand(n, vocab, generator=g, dtype=torch.float64))
    rows[torch.rand(n, vocab, generator=g) < 0.4] = 0.0
    p = place(rows, dtype, skew)
    u = torch.rand(n, generator=g).cuda()
    u[:8] = 0.0
    got = api.verify_tree(i32([0] * n), i32([-1] * n), starts([1] * n), p, None, torch.zeros(n, device="cuda"), u)
    assert api.get_device_error() == (0, 0)
    assert got.next_tokens.tolist() == [token_of(r, x) for r, x in zip(p.double().tolist(), u.tolist())]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_refused_token_beside_small_weights(dtype):
    """Token 0 is refused and out of the row; what is left of its vector is below half a unit."""
    rows = torch.full((2, 700), 0.3 / UNIT, dtype=torch.float64)
    rows[:, 0], rows[:, 600] = 0.25, 0.5
    p = place(rows, dtype, 1)
    got = api.verify_tree(i32([0, 0]), i32([-1, 0]), starts([2]), p, None, torch.full((2,), 0.9, device="cuda"),
                          torch.zeros(1, device="cuda"))
    assert api.get_device_error() == (0, 0)
    assert got.accepted_lens.tolist() == [1] and got.next_tokens.tolist() == [600]


def test_a_row_below_half_a_unit_has_no_weight():
    p = place(torch.full((1, 900), 0.49 / UNIT, dtype=torch.float64), torch.float32, 0)
    got = api.verify_tree(i32([0]), i32([-1]), starts([1]), p, None, torch.zeros(1, device="cuda"),
                          torch.zeros(1, device="cuda"))
    assert api.get_device_error() == (-5, native.DEVERR_PROBS)
    assert got.next_tokens.tolist() == [-1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [239, 240, 241, 245, 255, 256, 257, 500, 40000])
def test_rows_of_ones(vocab, dtype):
    """No probabilities: sums around 2^64 units and beyond."""
    p = place(torch.ones(7, vocab, dtype=torch.float64), dtype, 1)
    u = torch.tensor([0.0, 0.3, 0.9375, 0.95, 0.98, 0.997, 0.99999994], device="cuda")
    got = api.verify_tree(i32([0] * 7), i32([-1] * 7), starts([1] * 7), p, None, torch.zeros(7, device="cuda"), u)
    assert got.next_tokens.tolist() == [token_of([1.0] * vocab, x) for x in u.tolist()]


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
