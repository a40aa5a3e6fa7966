"""Angles of far positions on the host, in whole numbers: pos * f (f a 64-bit float) modulo 2 pi without rounding."""
import math

import torch

BITS = 160
# pi to 60 decimal places
PI = 3141592653589793238462643383279502884197169399375105820974944 * (1 << BITS) // 10 ** 60


def angle(pos: int, f: float) -> float:
    """pos * f modulo 2 pi, in [-pi, pi]."""
    num, den = f.as_integer_ratio()
    a = ((pos * num << BITS) // den) % (2 * PI)
    return (a - 2 * PI if a > PI else a) / (1 << BITS)


def turns(pos: int, f: float) -> float:
    """The same in half turns, in [-1, 1]."""
    num, den = f.as_integer_ratio()
    a = ((pos * num << BITS) // den) % (2 * PI)
    return (((a - 2 * PI if a > PI else a) << 64) // PI) / (1 << 64)


def angles(pos, f):
    """pos [tokens] int64 and f [pairs] float64 tensors -> float64 [tokens, pairs]."""
    fs = f.tolist()
    return torch.tensor([[angle(p, x) for x in fs] for p in pos.tolist()], dtype=torch.float64).view(len(pos), len(fs))


def rotate(x, pos, f, offset=0, interleaved=False, mscale=1.0, inverse=False):
    """x [tokens, channels] float64 rotated at pos [tokens]."""
    n, t = f.numel(), angles(pos, f)
    c, s = torch.cos(t) * mscale, torch.sin(t) * mscale * (-1 if inverse else 1)
    ia = offset + (2 * torch.arange(n) if interleaved else torch.arange(n))
    ib = ia + (1 if interleaved else n)
    y = x.clone()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


assert abs(PI / (1 << BITS) - math.pi) < 1e-15
