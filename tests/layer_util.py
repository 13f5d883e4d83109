"""The layer operators' formulas in 64 bits, on torch tensors, without the package's code."""
import math

import torch

BLOCK = 128
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# half a step of a code next to its value, and half the smallest step, next to the scale
HALF = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
LEAST = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}
ACTS = ("none", "relu", "silu", "gelu")


def blocks(n):
    return -(-n // BLOCK)


def half_step(dtype):
    """Rounding to nearest is off by at most this, relative to the value."""
    return torch.finfo(dtype).eps / 2


def pack(x, fmt):
    """(codes [rows, whole blocks] as uint8, E8M0 bytes [rows, blocks]) of a float tensor, with the rules of
    the scale read off the 32-bit amax's bits."""
    r, c = x.shape
    nb = blocks(c)
    full = torch.zeros(r, nb * BLOCK, dtype=torch.float32, device=x.device)
    full[:, :c] = x
    v = full.view(r, nb, BLOCK)
    bits = (v.abs().view(torch.int32)).amax(2)
    e, man = bits >> 23, bits & 0x7FFFFF
    k = e - 126 - (9 if fmt == "e4m3" else 16) + (man > 0x600000).int()
    k = torch.where(e == 0, torch.full_like(k, -126), k).clamp(-126, 126)
    k = torch.where((bits == 0) | (e == 255), torch.zeros_like(k), k)
    s = ((k + 127) << 23).view(torch.float32)
    q = (v.double() / s.double()[:, :, None]).float()  # exact: a power of two (or rounded where the code is 0 anyway)
    codes = q.clamp(-FMAX[fmt], FMAX[fmt]).to(FP8[fmt]).view(torch.uint8)
    codes = torch.where(q.isnan(), torch.full_like(codes, 0x7F) | (codes & 0x80), codes)
    return codes.view(r, -1), (k + 127).to(torch.uint8)


def decode(codes, scales, cols, fmt):
    """Values in 64 bits; scales as bytes or fp32."""
    s = scales.double() if scales.dtype == torch.float32 else torch.exp2(scales.double() - 127).float().double()
    s = s[:, :blocks(cols)].repeat_interleave(BLOCK, 1)[:, :cols]
    return codes.view(torch.uint8).view(FP8[fmt])[:, :cols].double() * s


def values(p):
    """A Packed8's values in 64 bits."""
    return decode(p.codes, p.scales, p.cols, p.fmt)


def act(z, kind):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    return z


def slope(z, kind):
    if kind == "relu":
        return (z > 0).double()
    if kind == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def randn(shape, seed, device="cuda", dtype=torch.float32, spread=0.0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    x = torch.randn(shape, generator=g, device=device)
    if spread:
        x = x * torch.exp(torch.randn((*shape[:-1], 1), generator=g, device=device) * spread)
    return x.to(dtype)


def strided(t, pad, off=0):
    """t's values as rows that lie `pad` elements further apart than they are long, `off` elements into a buffer
    whose other places hold NaN."""
    r, c = t.shape
    room = torch.full((r * (c + pad) + off + 8,), float("nan"), dtype=t.dtype, device=t.device)
    v = room[off:off + r * (c + pad)].view(r, c + pad)[:, :c]
    v.copy_(t)
    return v


def sum_bound(terms, count):
    """How far a sum of `count` terms in 32 bits may be off, in any order and with cut as well as rounded
    additions: each of the count additions by at most 2^-23 of a partial sum, none of which exceeds the
    sum of the terms' sizes `terms` (the 1.01 covers the errors' own growth)."""
    return 1.01 * count * 2.0 ** -23 * terms


def eights_bound(x, w):
    """How far the FP8 matrix instruction's sums of eight consecutive products may be off: seven products
    (the largest keeps its bits) are cut at 2^-13 of the largest's power of two, at most."""
    k = x.shape[1]
    x, w = (torch.nn.functional.pad(v.abs().float(), (0, -k % 8)) for v in (x, w))
    total = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[1], 8):
        big = x[:, c, None] * w[None, :, c]
        for j in range(c + 1, c + 8):
            torch.maximum(big, x[:, j, None] * w[None, :, j], out=big)
        total += big
    return 1.001 * 7 * 2.0 ** -13 * total
