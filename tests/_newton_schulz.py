"""The orthogonalisation in 64 bits, exactly and with the roundings that the kernels are written to make.

The kernels round X, P and Q to fp16 at stated points and keep X's remainder and what rounding takes from P's and Q's
diagonals; ``rounded`` does that with exact sums. They differ from it by fp32 sums alone: a sum off
by about 2^-20 of its value lands on the other side of a rounding of 2^-10 once in 2^10, which moves the
rounded matrix by 2^-15 of its norm; the 15 roundings of five steps, each passed on with a factor of at most 1.6, give
less than 2^-12.3 in quadrature. ``bound`` allows a tenth of the simulation's own error and 2^-13 beside it. An output's own
rounding is spread evenly over a step: u / sqrt(3) of the norm; no element is further off than 16 times the whole share of
the result's rms."""

import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
MUON = (3.4445, -4.7750, 2.0315)


def product(a, b):
    return torch.mm(a, b.contiguous())


def exact(x, steps=5, co=MUON, eps=1e-7):
    """newton_schulz of a matrix from its definition, on x's device."""
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x
    x = x / (torch.linalg.vector_norm(x) + eps)
    a, b, c = co
    for _ in range(steps):
        p = product(x, x.t())
        x = a * x + product(b * p + c * product(p, p), x)
    return x.t() if tall else x


def f16(v):
    return v.half().double()


def rounded(x, steps=5, co=MUON, eps=1e-7, diagonals=True, remainder=True):
    """The same with X, P and Q rounded to fp16 at their powers of two, X's remainder kept (in fp16 too) for all but the last two
    steps where it exists, and what rounding takes from P's and Q's diagonals. Sums are exact. Without ``diagonals``
    or ``remainder`` that part is left out."""
    a, b, c = co
    fine = x.dtype == torch.float32
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x
    rows, cols = x.shape
    kx = 1.0
    while kx * kx * 2 < rows * cols and kx < 8192:
        kx *= 2
    norm = float(torch.linalg.vector_norm(x)) + eps
    k = math.floor(math.log2(kx)) - (math.frexp(norm)[1] - 1)
    scaled = math.ldexp(norm, k)
    x = x * 2.0 ** k
    kp, most = 16384.0, 1.5 * abs(b) + 2.25 * abs(c)
    kq = 4096.0 if most * 4096 <= 60000 else 2.0 ** math.floor(math.log2(60000 / most))
    hi = f16(x)
    lo = f16(x - hi) if fine and remainder else torch.zeros_like(x)
    for i in range(steps):
        fp, fx = (kp / scaled ** 2, kx / scaled) if i == 0 else (kp / kx ** 2, 1.0)
        whole = fp * product(hi, hi.t())
        p = f16(whole)
        d = (whole - p).diagonal().clone() if diagonals else torch.zeros(rows, dtype=x.dtype, device=x.device)
        q = kq * b / kp * (p + torch.diag(d)) + kq * c / kp ** 2 * (product(p, p) + p * (d[:, None] + d[None, :]))
        whole = q
        q = f16(whole)
        e = (whole - q).diagonal().clone() if diagonals else torch.zeros_like(d)
        x = fx * (a * (hi + lo) + (product(q, hi) + e[:, None] * hi) / kq)
        hi = f16(x)
        lo = f16(x - hi) if i < steps - 3 and remainder else torch.zeros_like(x)
    x = x / kx
    return x.t() if tall else x


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def bound(x):
    return 1.1 * off(rounded(x), exact(x)) + 2.0 ** -13


def normal(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, cols, generator=g).to(dtype).cuda()


def strong(rows, cols, dtype, seed=0):
    """A few strong directions above noise."""
    g = torch.Generator().manual_seed(seed)
    few = max(1, min(rows, cols) // 16)
    x = torch.randn(rows, cols, generator=g) + 3 / few ** 0.5 * torch.randn(rows, few, generator=g) @ torch.randn(few, cols, generator=g)
    return (x * 1e-3).to(dtype).cuda()


def check(got, x, want=None, most=None):
    want = exact(x) if want is None else want
    most = (bound(x) if most is None else most) + U[got.dtype] / 3 ** 0.5
    assert got.shape == x.shape
    err = off(got, want)
    assert err <= most, (err, most)
    worst = float((got.double() - want).abs().max() / want.square().mean().sqrt())
    assert worst <= 16 * most, (worst, most)
