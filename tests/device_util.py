"""What tests of large calls need on the device itself, where 64-bit forms of hundreds of MB take milliseconds."""
import op_util as ou
import step_util as su
import torch

MASK = 0xFFFFFFFF


def drawn(rows, first, cols, seed, offset, device):
    """step_util.drawn on any device: 64-bit products wrap, their halves do not."""
    groups = (cols + 7) // 8
    offset %= 1 << 64
    words = [torch.arange(groups, device=device).expand(rows, groups),
             (torch.arange(rows, device=device) + first)[:, None].expand(rows, groups)]
    words += [torch.full((rows, groups), w, dtype=torch.int64, device=device) for w in (offset & MASK, offset >> 32)]
    k0, k1 = seed & MASK, seed >> 32
    for _ in range(10):
        p, q = words[0] * 0xD2511F53, words[2] * 0xCD9E8D57
        words = [(q >> 32 & MASK) ^ words[1] ^ k0, q & MASK, (p >> 32 & MASK) ^ words[3] ^ k1, p & MASK]
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    out = torch.stack([w >> 16 * h & 0xFFFF for w in words for h in (0, 1)], dim=2)
    return out.reshape(rows, groups * 8)[:, :cols]


def masks(rows, cols, p, seed, offset, device):
    return [drawn(k, sum(rows[:r]), cols, seed, offset, device) >= su.threshold(p) for r, k in enumerate(rows)]


def padded(t, pad, offs=0):
    """t in rows `pad` elements longer than its own, from element `offs` of a buffer on; what is around it is 77."""
    rows, cols = t.shape
    flat = torch.full((rows * (cols + pad) + offs,), 77.0, dtype=t.dtype, device=t.device)
    view = flat[offs:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def within(got, want, bound, what):
    """op_util.within where all is finite and on the device."""
    g = got.double()
    assert g.shape == want.shape, what
    assert torch.isfinite(g).all(), what + ": not finite"
    may = bound + ou.half(got.dtype) * (want.abs() + bound) + ou.TINY[got.dtype]
    worst = ((g - want).abs() / may).max().item()
    assert worst <= 1.0, "%s: off by %.3g of the bound" % (what, worst)


def around(view):
    """What lies between the rows of a padded view, without the last row's."""
    rows, cols = view.shape
    gap = view.stride(0) - cols
    return view.as_strided((rows - 1, gap), view.stride(), view.storage_offset() + cols) if rows > 1 and gap else view[:0]
