"""csa2_rope and csa2_norm_rope on the GPU against the formulas in 64 bits.

Tolerance. cos and sin: the angle is reduced in 64 bits to half turns in [-1, 1] and rounded to fp32
(2^-25 half turns, 2^-23.3 radians), sincospif is good to 2 ulp: less than 2^-21.5 together. The rotation
adds two products and a sum (3 * 2^-24). The norm: at most 37 fp32 additions of positive squares
(32 in a lane, 5 across the warp), 37 * 2^-24 of the sum, half of that in its root, and 4 further
roundings: less than 2^-19. Together below 2^-18 of |a| + |b| (the pair of channels), and then half a
step of the output type.
"""
import pytest
import torch

import _layer_ref as R
import compressed_sparse_attention_append_b200 as csa

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def _tol(y, size, dtype):
    return y.abs() * (torch.finfo(dtype).eps / 2) + size * 2.0 ** -18


def _rand(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _rope(rot, offset, interleaved, inverse=False, scaling="yarn", base=10000.0):
    r = csa.Rope.for_context(rot, base, scaling, 16.0, 4096, offset=offset, interleaved=interleaved)
    return r.transposed() if inverse else r


def _pos(seed, t, hi=1 << 20):
    return torch.randint(0, hi, (t,), generator=torch.Generator().manual_seed(seed)).to(DEV)


def _check(got, want, size):
    y = got.detach().cpu().double()
    assert bool(((y - want).abs() <= _tol(want, size, got.dtype)).all()), float((y - want).abs().max())


CASES = [  # tokens, heads, d, rot, offset
    (1, 1, 64, 64, 0), (1, 16, 128, 128, 0), (5, 64, 512, 64, 448), (300, 1, 512, 64, 448), (129, 3, 192, 96, 96),
    (64, 32, 128, 64, 64), (700, 40, 64, 32, 0), (2, 1, 1024, 1024, 0), (3, 2, 1024, 8, 1016),
    (33, 5, 80, 20, 60),     # rot / 2 = 10: no vectors in halves; interleaved in 8-byte ones
    (17, 2, 36, 12, 4),      # 4-element rows (bf16: 8-byte vectors)
    (9, 3, 7, 6, 1),         # odd width and offset
    (4, 2, 130, 2, 127), (2, 2, 1, 0, 0), (6, 4, 96, 0, 0),
    (2500, 16, 64, 64, 0),   # several rows per group of lanes
    (20000, 1, 512, 512, 0),  # many tokens of one head, rotated whole: the largest tables
    (700, 60, 512, 64, 448), (9000, 2, 256, 256, 0),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,h,d,rot,offset", CASES)
def test_rope_matches_the_formula(t, h, d, rot, offset, dtype, interleaved):
    x, pos = _rand(t + d, t, h, d, dtype=dtype), _pos(t, t)
    for inverse in (False, True):
        r = _rope(rot, offset, interleaved, inverse)
        out = torch.full_like(x, float("nan"))
        csa.csa2_rope(r, pos, x, out)
        want, size = R.rotate(x, pos, r.inv_freq, offset, interleaved, r.mscale, inverse)
        _check(out, want, size)
        same = x.clone()
        csa.csa2_rope(r, pos, same, same)  # in place: the same bits
        assert torch.equal(same, out)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,h,d,rot,offset", CASES)
def test_norm_rope_matches_the_formula(t, h, d, rot, offset, dtype, interleaved):
    hk = 1 + t % 3
    fused = _rand(3 * t + d, t, (h + hk) * d, dtype=dtype)  # queries and keys out of one projection
    q, k = fused[:, :h * d].view(t, h, d), fused[:, h * d:].view(t, hk, d)
    wq, wk = (1.0 + 0.2 * _rand(s, d, dtype=dtype) for s in (1, 2))
    pos, r = _pos(t + 1, t), _rope(rot, offset, interleaved)
    qo = torch.full((t, h, d), float("nan"), device=DEV, dtype=dtype)
    ko = torch.full((t, hk, d), float("nan"), device=DEV, dtype=dtype)
    csa.csa2_norm_rope(r, pos, EPS, q, wq, qo, k, wk, ko)
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        _check(y, *R.rotate(R.norm(x, w, EPS), pos, r.inv_freq, offset, interleaved, r.mscale))
    only = torch.empty_like(qo)
    csa.csa2_norm_rope(None, None, EPS, q, None, only)  # the norm alone, without weights, q alone
    want = R.norm(q, None, EPS)
    _check(only, want, want.abs())
    csa.csa2_norm_rope(r, pos, EPS, q, wq, q, k, wk, k)  # in place, in the fused rows
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_strided_rows_and_padding_are_left_as_they_were():
    t, h, d = 20, 4, 64
    big = _rand(5, t + 3, h + 2, d + 16)
    x = big[1:t + 1, 1:h + 1, 8:8 + d]
    pos = _pos(6, t)
    pos[[3, 19]] = -1
    r = _rope(32, 16, True)
    frame = torch.full((t, 2 * h, d + 8), 7.0, device=DEV, dtype=torch.bfloat16)
    out = frame[:, ::2, :d]
    csa.csa2_rope(r, pos, x, out)
    want, size = R.rotate(x, pos.clamp_min(0), r.inv_freq, 16, True, r.mscale)
    live = (pos >= 0).cpu()
    _check(out[live.to(DEV)], want[live], size[live])
    assert bool((out[[3, 19]] == 7).all()) and bool((frame[:, 1::2] == 7).all()) and bool((frame[..., d:] == 7).all())
    # an odd element offset: narrow accesses, the same values
    odd = torch.empty(t * h * d + 1, device=DEV, dtype=torch.bfloat16)[1:].view(t, h, d)
    odd.copy_(x)
    csa.csa2_rope(r, pos, odd, odd)
    _check(odd[live.to(DEV)], want[live], size[live])
    w = torch.ones(d, device=DEV, dtype=torch.bfloat16)
    before = big.clone()
    csa.csa2_norm_rope(r, pos, EPS, x, w, x)
    changed = big != before
    assert not bool(changed[4].any()) and not bool(changed[20].any())  # the padded tokens
    assert not bool(changed[:, :, :8].any()) and not bool(changed[:, 0].any()) and not bool(changed[0].any())


def test_far_positions_zero_rows_and_values_that_are_not_finite():
    d = 128
    r = _rope(d, 0, False, scaling="plain")
    pos = torch.tensor([0, 1, (1 << 31) - 1, 1 << 30], device=DEV)
    x = _rand(8, 4, 2, d, dtype=torch.float32)
    out = torch.empty_like(x)
    csa.csa2_rope(r, pos, x, out)
    _check(out, *R.rotate(x, pos, r.inv_freq, 0, False))
    assert torch.equal(out[0], x[0])  # position 0 turns nothing
    back = torch.empty_like(x)
    csa.csa2_rope(r.transposed(), pos, out, back)  # there and back
    assert float((back - x).abs().max()) < 2.0 ** -17 * float(x.abs().max())
    z = torch.zeros(4, 2, d, device=DEV, dtype=torch.bfloat16)
    z[1, 1, 5] = float("inf")
    z[2, 0, 3] = float("nan")
    w, o = torch.ones(d, device=DEV, dtype=torch.bfloat16), torch.empty_like(z)
    csa.csa2_norm_rope(r, pos, EPS, z, w, o)
    bad = ~torch.isfinite(o).all(-1)
    assert bad.cpu().tolist() == [[False, False], [False, True], [True, False], [False, False]]
    assert not bool(o[0].any()) and not bool(o[3].any())  # a row of zeros stays zero


def test_the_transpose_is_the_gradient():
    """<R x, g> = <x, R^T g>, and R^T g is what a difference quotient of <R x, g> gives."""
    t, h, d = 3, 2, 64
    r = _rope(32, 8, True)
    pos = _pos(11, t)
    x, g = (_rand(s, t, h, d, dtype=torch.float32) for s in (12, 13))
    y, gx = torch.empty_like(x), torch.empty_like(x)
    csa.csa2_rope(r, pos, x, y)
    csa.csa2_rope(r.transposed(), pos, g, gx)
    a, b = float((y.double() * g.double()).sum()), float((x.double() * gx.double()).sum())
    assert abs(a - b) < 1e-4
    for at in ((0, 0, 9), (2, 1, 40), (1, 0, 0)):
        up, yu = x.clone(), torch.empty_like(x)
        up[at] += 1.0
        csa.csa2_rope(r, pos, up, yu)
        # linear: the difference of step 1 is the derivative, to the rounding of two fp32 rows
        assert abs(float(((yu.double() - y.double()) * g.double()).sum()) - float(gx[at])) < 1e-4


def test_streams_and_graphs():
    t, h, d = 64, 16, 128
    x, pos, r = _rand(21, t, h, d), _pos(22, t), _rope(64, 64, True)
    w = _rand(23, d)
    want, other, got = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    csa.csa2_norm_rope(r, pos, EPS, x, w, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    csa.csa2_norm_rope(r, pos, EPS, x, w, other, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa.csa2_norm_rope(r, pos, EPS, x, w, got)
        csa.csa2_rope(r.transposed(), pos, got, got)
    for seed in (31, 32):
        x.copy_(_rand(seed, t, h, d))
        g.replay()
        csa.csa2_norm_rope(r, pos, EPS, x, w, want)
        csa.csa2_rope(r.transposed(), pos, want, want)
        assert torch.equal(got, want)
