"""Plain 64-bit forms of dropout, token log-probabilities and the policy loss, and bounds on what kernels that work
in 32 bits may be off (U = 2^-24 is half a step of float32)."""
import math

import numpy as np
import torch
from op_util import U

MASK = np.uint64(0xFFFFFFFF)


def philox(c, key):
    """Philox4x32-10: c is four arrays of 32-bit words (as uint64), key two integers."""
    c = [np.asarray(w, dtype=np.uint64) for w in c]
    k0, k1 = key
    for _ in range(10):
        p, q = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), q & MASK, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p & MASK]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def drawn(rows, first, cols, seed, offset, start=0):
    """The 16-bit numbers of rows first .. first + rows - 1, columns start (a multiple of 8) and following."""
    groups = (cols + 7) // 8
    offset %= 1 << 64
    g, r = np.meshgrid(np.arange(start // 8, start // 8 + groups, dtype=np.uint64), np.arange(first, first + rows, dtype=np.uint64))
    words = philox([g, r, np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, offset >> 32)],
                   (seed & 0xFFFFFFFF, seed >> 32))
    out = np.stack([(w >> np.uint64(16 * h)) & np.uint64(0xFFFF) for w in words for h in (0, 1)], axis=2)
    return torch.from_numpy(out.reshape(rows, groups * 8)[:, :cols].astype(np.int64))


def scale_of(p):
    t = threshold(p)
    return 0.0 if t == 65536 else 65536.0 / (65536 - t)


def dropout(x, bias, residual, kept, p):
    """(y, bound) in float64."""
    v = x.double() + (bias.double() if bias is not None else 0.0)
    z = residual.double() if residual is not None else torch.zeros_like(v)
    y = torch.where(kept, z + v * scale_of(p), z)
    # the sum, the scale, the fused product
    return y, torch.where(kept, U * (2.01 * scale_of(p) * v.abs() + y.abs()), 0.0)


def logprob(x, targets, scale, ranks=1):
    """(logp, top, logSum, bound of logp, bound of logSum) in float64 from a row's whole logits."""
    d, n = x.double(), x.shape[1]
    top = d.amax(1, keepdim=True)
    t = (d - top) * scale
    e = torch.exp(t)
    s = e.sum(1, keepdim=True)
    far = (torch.where(e > 0, e * -t, 0.0)).sum(1, keepdim=True) / s
    # an exponential: its difference, factor and product 3 U of its size, itself 2 U; it is carried on by at most
    # `hops` more of them and added up in as many sums
    hops = n / 1024 + 2 * ranks + 32
    ds = U * (4 * hops + 3 * far) + 2.0 ** -126 * n
    log_sum = torch.log(s)
    at = t.gather(1, targets.clamp(min=0, max=n - 1)[:, None])
    logp = at - log_sum
    d_sum = ds * 1.01 + 3 * U * log_sum.abs() + U * U
    d_logp = d_sum + 3 * U * at.abs() + U * logp.abs()
    logp = torch.where(logp.abs() >= 2.0 ** 128 * (1 - 2.0 ** -25), logp * float("inf"), logp)   # rounds to an infinity
    live = (targets >= 0)
    out = [torch.where(live, v[:, 0], 0.0) for v in (logp, top, log_sum, d_logp, d_sum)]
    return out


def logprob_backward(dlogp, x, targets, scale, top, log_sum):
    """(dlogits, bound) in float64 from the float statistics."""
    d, n = x.double(), x.shape[1]
    g = torch.where(targets >= 0, dlogp.double() * scale, 0.0)[:, None]
    t = (d - top.double()[:, None]) * scale
    arg = t - log_sum.double()[:, None]
    p = torch.exp(arg)
    hot = torch.zeros_like(d)
    hot.scatter_(1, targets.clamp(min=0, max=n - 1)[:, None], 1.0)
    out = torch.where(g == 0.0, 0.0, g * (hot - p))
    far = torch.where(p > 0, 3 * t.abs() + 2 * log_sum.double().abs()[:, None] + arg.abs() + 3, 0.0)
    bound = g.abs() * (U * 1.01 * p * far + 4 * U * (hot - p).abs() + 2.0 ** -126)
    return out, bound


def policy(logps, olds, refs, advantages, weights, low, high, kl_coef, denominator=0.0, grad_scale=1.0):
    """(stats, dlogps) in float64, of lists of one tensor a rank."""
    logp, old, adv = (torch.cat(v).double() for v in (logps, olds, advantages))
    w = torch.cat(weights).double() if weights is not None else torch.ones_like(logp)
    ratio = torch.exp(logp - old)
    loss = torch.maximum(-adv * ratio, -adv * ratio.clamp(1 - low, 1 + high))
    clipped = ((adv > 0) & (ratio > 1 + high)) | ((adv < 0) & (ratio < 1 - low))
    g = torch.where(clipped, 0.0, -adv * ratio)
    kl = torch.zeros_like(loss)
    if refs is not None:
        d = torch.cat(refs).double() - logp
        kl = torch.expm1(d) - d
        g = g - kl_coef * torch.expm1(d)
    zero = w == 0
    total = w.sum()
    over = denominator if denominator > 0 else total.item()
    part = 1.0 / over if over != 0 else 0.0

    def mean(v):
        return torch.where(zero, 0.0, w * v).sum() * part

    # What 32 bits are off.  The ratio: its logarithm's rounding, the product with log2(e) and that factor's own (2.5 U of
    # the logarithm), the exponential (2 U, nothing below 2^-126), the product with A.
    change = (logp - old).abs()
    d_pg = U * (2.5 * change + 4) * (adv * ratio).abs() + 2.0 ** -126 * adv.abs()
    d_loss = torch.where(clipped, 2 * U * loss.abs(), d_pg)
    d_kl = torch.zeros_like(loss)
    d_grad = torch.where(clipped, 0.0, d_pg)
    if refs is not None:
        # the difference's rounding moves kl by |d (exp(d) - 1)| U and exp(d) - 1 by |d| exp(d) U; the series' factors
        # and products 8 U of kl; past 1 the exponential as the ratio's, the differences' roundings
        e, less, far = torch.exp(d), torch.expm1(d).abs(), d.abs() >= 1
        d_kl = U * (d.abs() * less + 8 * kl + torch.where(far, (2 + 1.5 * d.abs()) * e + less + 2.0 ** -100, 0.0))
        d_less = d_kl + U * (d.abs() * e + less + 2 * d.abs())
        d_grad = d_grad + kl_coef * (d_less + 3 * U * less)
    d_grad = (d_grad + 3 * U * g.abs()) * (grad_scale * part * w).abs()
    stats = torch.stack((mean(loss) + kl_coef * mean(kl), mean(loss), mean(kl), mean(clipped.double()), total))
    # sums in 64 bits of n terms: n 2^-53 of the terms' sizes
    n = loss.numel() + 64

    def off(v, dv):
        return mean(dv) + n * 2.0 ** -53 * mean(v.abs())

    bounds = torch.stack((off(loss, d_loss) + kl_coef * off(kl, d_kl) + 2.0 ** -53 * 8 * mean(loss.abs()), off(loss, d_loss), off(kl, d_kl),
                          n * 2.0 ** -53 * mean(clipped.double()), n * 2.0 ** -53 * w.abs().sum()))
    widths = [len(t) for t in logps]
    grads = torch.where(zero, 0.0, grad_scale * part * w * g)
    return stats, bounds, list(grads.split(widths)), list(torch.where(zero, 0.0, d_grad + n * 2.0 ** -53 * grads.abs()).split(widths))
