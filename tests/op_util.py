"""Plain 64-bit forms of the operators around the AllReduce, and bounds on what 32-bit kernels may be off.

u = 2^-24 is half a step of float32 and h(T) = finfo(T).eps / 2 half a step of an element type T.  A sum of n
terms whose longest chain of additions is k long is off by at most about k u times the sum of the terms'
sizes; the kernels keep several partial sums per row, so k = n / 32 + 32 covers every row width used here."""
import torch

U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}   # half a subnormal step

TYPES = [(torch.float32, torch.float32), (torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
         (torch.float16, torch.float32), (torch.bfloat16, torch.float32)]


def half(t):
    return torch.finfo(t).eps / 2


def chain(n):
    return n / 32 + 32


def rows_of(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std + mean).to(dtype)


def ln_forward(x, gamma, beta, eps):
    """(y, mean, rstd) in float64 and a bound for each, elementwise, before rounding to x's type."""
    d, c = x.double(), x.shape[-1]
    k = chain(c)
    mean = d.mean(1, keepdim=True)
    e = d - mean
    v = (e * e).mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(v + eps)
    g = gamma.double() if gamma is not None else torch.ones(c, dtype=torch.float64)
    b = beta.double() if beta is not None else torch.zeros(c, dtype=torch.float64)
    y = e * rstd * g + b
    dm = (k + 2) * U * d.abs().mean(1, keepdim=True)
    # each deviation is off by dm and one rounding; their squares add up with k more roundings
    dv = (k + 6) * U * v + 2 * dm * e.abs().mean(1, keepdim=True) + dm * dm
    rel = dv / (2 * (v + eps)) + 4 * U
    dy = (rstd * g).abs() * (dm + U * e.abs()) * (1 + rel) + (e * rstd * g).abs() * (rel + 3 * U) + U * (y.abs() + b.abs())
    return y, mean[:, 0], rstd[:, 0], dy, dm[:, 0], (rel * rstd)[:, 0]


def ln_backward(dy, x, mean, rstd, gamma):
    """(dx, bound of dx, dy * h, dy) in float64 from the given float statistics."""
    c = x.shape[-1]
    k = chain(c)
    d, m, r = dy.double(), mean.double()[:, None], rstd.double()[:, None]
    h = (x.double() - m) * r
    q = d * (gamma.double() if gamma is not None else 1.0)
    s = q.mean(1, keepdim=True)
    t = (q * h).mean(1, keepdim=True)
    dx = r * (q - s - h * t)
    ds = (k + 3) * U * q.abs().mean(1, keepdim=True)
    dt = (k + 6) * U * (q * h).abs().mean(1, keepdim=True)
    bound = r.abs() * (ds + h.abs() * dt + 6 * U * (q.abs() + s.abs() + (h * t).abs()))
    return dx, bound, d * h, d


def within(got, want, bound, dtype, what):
    """got (of type dtype) is want up to bound and one rounding to dtype; NaN and infinities agree."""
    g = got.detach().cpu().double()
    assert g.shape == want.shape, what
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(g), torch.isnan(want)), what + ": NaN elsewhere"
    assert torch.equal(g[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what + ": infinities"
    off = (g - want).abs()[fine]
    may = (bound + half(dtype) * (want.abs() + bound) + TINY[dtype])[fine]
    if off.numel():
        worst = (off / may).max().item()
        assert worst <= 1.0, "%s: off by %.3g of the bound" % (what, worst)
