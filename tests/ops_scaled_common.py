"""The 8-bit format of packed arrays, written out for the tests: a table of e4m3, the
nearest code with ties to even, and the scale of a block, all in 64 bits."""
import torch

BLOCK = 128
E4M3 = torch.tensor([(k & 7) * 2.0 ** -9 if k < 8 else (1 + (k & 7) / 8) * 2.0 ** ((k >> 3) - 7) for k in range(127)], dtype=torch.float64)


def blocks_of(x, square):
    """Largest finite |x| of every block, spread over its elements, and by block."""
    rows, width = x.shape
    a = torch.where(torch.isfinite(x), x.abs(), 0.0)
    by = torch.nn.functional.pad(a, (0, -width % BLOCK, 0, -rows % BLOCK if square else 0))
    if square:
        m = by.view(by.shape[0] // BLOCK, BLOCK, -1, BLOCK).amax((1, 3))
    else:
        m = by.view(rows, -1, BLOCK).amax(2)
    return spread(m, rows, width, square), m


def spread(m, rows, width, square):
    if square:
        m = m.repeat_interleave(BLOCK, 0)[:rows]
    return m.repeat_interleave(BLOCK, 1)[:, :width]


def scale_byte(big):
    """E for a largest value: the least with big <= 448 * 2^(E - 127), 27 at least."""
    frac, e = torch.frexp(big)
    return torch.where(big > 0, e - 9 + (frac > 0.875), -100).clamp_min(-100) + 127


def codes(y):
    """Bytes of the numbers nearest to y (64 bits, already divided by its scale)."""
    table = E4M3.to(y.device)
    mids = (table[1:] + table[:-1]) / 2
    a = y.abs()
    i = torch.searchsorted(mids, a)
    tie = (i < 126) & (mids[i.clamp_max(125)] == a)
    i = i + (tie & (i % 2 == 1))
    i = torch.where(torch.isfinite(y), i, 127)
    return i + 128 * ((y < 0) | ((y == 0) & (torch.signbit(y))))


def values(codes, exps, square):
    """What codes and exps stand for, in 64 bits."""
    c = codes.view(torch.uint8).long()
    table = torch.cat([E4M3, torch.tensor([float("nan")], dtype=torch.float64)]).to(c.device)
    v = table[c & 127]
    v = torch.where(c > 127, -v, v)
    scale = torch.exp2(exps.double() - 127)
    scale = torch.where(exps == 255, float("nan"), scale)
    return v * spread(scale, *codes.shape, square)
