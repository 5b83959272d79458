"""The cache in 4 bits in plain evaluations: rows of exact fractions for single vectors, of 64-bit
arithmetic for whole tensors, and the values that rows stand for."""
import math
from fractions import Fraction

import torch

D, ROW = 128, 144


def bf16_of(x: Fraction) -> Fraction:
    """x rounded to bf16 (8 significant bits, exponents from -126, ties to even); beyond the largest: not handled."""
    if x == 0:
        return Fraction(0)
    e = math.floor(math.log2(abs(x.numerator)) - math.log2(x.denominator))
    while Fraction(2) ** e > abs(x):
        e -= 1
    while Fraction(2) ** (e + 1) <= abs(x):
        e += 1
    step = Fraction(2) ** (max(e, -126) - 7)
    return round(x / step) * step          # (round of a Fraction: ties to even)


def fractions_of(x):
    """(codes, scale, zero) of 64 bf16 numbers in exact arithmetic."""
    v = [Fraction(float(a)) for a in x]
    zero, scale = min(v), bf16_of((max(v) - min(v)) / 15)
    return [min(round((a - zero) / scale), 15) if scale else 0 for a in v], scale, zero


def codes_of(x):
    """(codes [.., 128], scale [.., 2], zero [.., 2]) in 64 bits."""
    g = x.double().unflatten(-1, (2, D // 2))
    zero = g.amin(-1)
    scale = ((g.amax(-1) - zero) / 15).float().bfloat16()
    s = torch.where(scale > 0, scale, 1.0).double()
    codes = ((g - zero[..., None]) / s[..., None]).round().clamp(0, 15) * (scale > 0)[..., None]
    return codes.flatten(-2).to(torch.uint8), scale, zero.bfloat16() + 0.0


def rows_of(k, v):
    parts, numbers = [], []
    for x in (k, v):
        codes, scale, zero = codes_of(x)
        parts.append(codes[..., 0::2] | codes[..., 1::2] << 4)
        numbers += [scale[..., 0], zero[..., 0], scale[..., 1], zero[..., 1]]
    return torch.cat([*parts, torch.stack(numbers, -1).contiguous().view(torch.uint8)], -1)


def values_of(rows):
    """Keys and values in 64 bits."""
    numbers = rows[..., 128:].contiguous().view(torch.bfloat16).double()
    out = []
    for i in range(2):
        b = rows[..., 64 * i:64 * i + 64]
        codes = torch.stack([b & 15, b >> 4], -1).flatten(-2).double()
        scale, zero = (numbers[..., [4 * i + j, 4 * i + 2 + j]].repeat_interleave(D // 2, -1) for j in (0, 1))
        out.append(codes * scale + zero)
    return out


def empty_cache(n, room, hk, order="heads", fill=255, device="cuda"):
    """[n, room, hk, 144] bytes in one of three orders in memory; rows of 255 stand for NaN."""
    if order == "heads":
        return torch.full((n, hk, room, ROW), fill, dtype=torch.uint8, device=device).transpose(1, 2)
    if order == "rows":
        return torch.full((n, room, hk, ROW), fill, dtype=torch.uint8, device=device)
    wide = torch.full((n, hk + 1, room + 3, ROW + 16), fill, dtype=torch.uint8, device=device)   # "padded": gaps everywhere
    return wide[:, :hk, :room, :ROW].transpose(1, 2)
