"""Plain 64-bit forms of the operators around the core (include/csa2_layer.h), on the host, for the
tests: rotation, norm, the codecs on real values, FP8 products and attention over given keys."""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def nearest(x, table):
    """Codes of |x| in `table` (ascending from 0): nearest, ties to the even code, saturating."""
    mid = (table[1:] + table[:-1]) / 2
    a = x.abs().contiguous()
    at = torch.bucketize(a, mid)
    tie = (at < mid.numel()) & (a == mid[at.clamp(max=mid.numel() - 1)]) & (at % 2 == 1)
    return at + tie


def rotate(x, pos, f, offset=0, interleaved=False, mscale=1.0, inverse=False):
    """x [tokens, heads, d] (any type) -> float64; also the sum |a| + |b| of each channel's pair."""
    x = x.detach().cpu().double()
    f = f.detach().cpu().double()
    n = f.numel()
    y, size = x.clone(), x.abs().clone()
    t = pos.detach().cpu().double()[:, None, None] * f
    c, s = torch.cos(t) * mscale, torch.sin(t) * mscale * (-1 if inverse else 1)
    ia = offset + (2 * torch.arange(n) if interleaved else torch.arange(n))
    ib = ia + (1 if interleaved else n)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * abs(mscale)
    return y, size


def norm(x, w, eps):
    x = x.detach().cpu().double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.detach().cpu().double()


def e2m1_rows(y):
    """y [.., ch] float64 -> (code bytes [.., ch / 2], E4M3 scale bytes [.., ch / 16]): the rule of csa2.h."""
    b = y.unflatten(-1, (-1, 16))
    sb = nearest(b.abs().amax(-1) / 6.0, E4M3)
    s = E4M3[sb][..., None]
    code = nearest(torch.where(s > 0, b / s, 0.0), E2M1) + 8 * (torch.signbit(b) & (s > 0))
    code = code.flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), sb.to(torch.uint8)


def mx_rows(y):
    """MXFP4: (code bytes, E8M0 bytes [.., ch / 32])."""
    b = y.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    e = torch.frexp(top).exponent.long() - 1  # floor(log2)
    sb = torch.where(top > 0, (e - 2 + 127).clamp(0, 254), 0)
    x = torch.exp2((sb - 127).double())[..., None]
    code = nearest(b / x, E2M1) + 8 * torch.signbit(b)
    code = torch.where(top[..., None] > 0, code, 0).flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), sb.to(torch.uint8)


def e4m3_rows(y):
    return (nearest(y, E4M3) + 128 * torch.signbit(y)).to(torch.uint8)


def e2m1_values(data, scale):
    """Code bytes [.., ch / 2] and E4M3 bytes [.., ch / 16] -> float64 values."""
    data = data.detach().cpu().long()
    v = torch.stack([data & 15, data >> 4], -1).flatten(-2)
    v = torch.where(v >= 8, -E2M1[v & 7], E2M1[v & 7])
    return v * scale.detach().cpu().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def mx_values(data, scale):
    data = data.detach().cpu().long()
    v = torch.stack([data & 15, data >> 4], -1).flatten(-2)
    v = torch.where(v >= 8, -E2M1[v & 7], E2M1[v & 7])
    return v * torch.exp2(scale.detach().cpu().double() - 127).repeat_interleave(32, -1)


def fp8_values(data, row_scale=None, block_scale=None):
    """E4M3 bytes [rows, k] with the scales of csa2_fp8_quantize ([kb, rows]) or _weight ([rb, kb]), float64."""
    rows, k = data.shape
    v = data.detach().cpu().view(torch.float8_e4m3fn).double()
    if row_scale is not None:
        s = row_scale.detach().cpu().double().T.repeat_interleave(128, 1)[:, :k]
    else:
        s = block_scale.detach().cpu().double().repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :k]
    return v * s


def attend(q, keys, scale):
    """q [heads, ch], keys [n, ch] float64 -> (out, lse); no key: zeros and -inf."""
    if keys.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    logits = q @ keys.T * scale
    return torch.softmax(logits, -1) @ keys, torch.logsumexp(logits, -1)
