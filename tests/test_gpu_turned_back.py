"""A stretched context's rotation scales what it turns (mscale 1.277 for a factor of 16), and with K = V the cached values
with it: the inverse rotation has to give the values back, alone and at the end of a layer step."""
import pytest
import torch

import _layer_ref as R
import compressed_sparse_attention_append_b200 as csa

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def _rope(rot, offset, interleaved):
    return csa.Rope.for_context(rot, 10000.0, "yarn", 16.0, 4096, offset=offset, interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,offset", [(512, 64, 448), (128, 128, 0), (80, 20, 60)])
def test_there_and_back(d, rot, offset, interleaved):
    """Each way is off by 2^-18 of the pair's |a| + |b| at its scale (as in test_gpu_rope.py), the way there counted twice by
    the way back, whose own pair is up to twice as large: 4 * 2^-18, and 2^-23 for 1 / mscale in fp32."""
    r = _rope(rot, offset, interleaved)
    assert r.mscale > 1.2
    g = torch.Generator().manual_seed(d)
    x = torch.randn(50, 3, d, generator=g).to(DEV)
    pos = torch.randint(0, 1 << 20, (50,), generator=g).to(DEV)
    y, z = torch.empty_like(x), torch.empty_like(x)
    csa.csa2_rope(r, pos, x, y)
    csa.csa2_rope(r.inverted(), pos, y, z)
    size = R.rotate(x, pos, r.inv_freq, offset, interleaved)[1]
    assert bool(((z - x).abs().cpu().double() <= size * (2.0 ** -16 + 2.0 ** -22)).all())


@pytest.mark.parametrize("B", [3, 100])  # a row's tiles over a cluster; a CTA per row
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_row_that_attends_to_itself_alone_comes_back_as_its_latent(B, interleaved):
    """Tolerances. An entry: a code is off by 1 scale at most (between 4 and 6; the scale is amax / 6 to 2^-4, so nothing
    is cut by more than 0.4). A window row: E4M3 is off by 2^-4, or 2^-10 below its normal numbers. The way back
    mixes the errors of a pair and divides them by mscale. Two roundings to bf16 (2^-8 each) and the attention's fp32 terms
    add 2^-6.9 of |a| + |b| with their errors."""
    page, rot = 16, 64
    r = _rope(rot, 512 - rot, interleaved)
    g = torch.Generator().manual_seed(B)
    lat, swa = (torch.randn(B, 1, 512, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    w = (1.0 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16).to(DEV)
    pos = torch.randint(0, 64, (B,), generator=g).to(DEV)
    rpos = torch.randint(0, 1 << 20, (B, 1), generator=g).to(DEV)
    c = csa.PagedCache(4 * B, page, B, 4, page_table=torch.randperm(4 * B, generator=g).to(torch.int32).view(B, 4).to(DEV),
                       indexer=False)
    csa.csa2_paged_append(c, B, 1, pos, lat, swa=swa, rope=r, w_latent=w, w_swa=w, eps=EPS, rpos=rpos)
    q = torch.randn(B, 64, 512, generator=g).to(torch.bfloat16).to(DEV)
    out = torch.empty(B, 64, 512, device=DEV, dtype=torch.bfloat16)
    eps = float(torch.tensor(EPS, dtype=torch.float32))
    for source, idx, win in ((lat, pos.to(torch.int32)[:, None].contiguous(), 0), (swa, None, 1)):
        csa.csa2_paged_attend(c, B, 1, pos, q, idx, 0 if idx is None else 1, out, win=win)
        csa.csa2_rope(r.inverted(), rpos[:, 0].contiguous(), out, out)
        want = R.norm(source[:, 0], w, eps)
        _, size = R.rotate(want[:, None], rpos[:, 0], r.inv_freq, r.offset, interleaved)
        size = size[:, 0]  # |a| + |b| on turned channels, |y| on the others
        if win == 0:
            page_of = c.table[torch.arange(B, device=DEV), pos // page].long()
            s = c.l_scale[page_of, pos % page].cpu().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
            if interleaved:
                other = s
            else:  # the pair's other channel lies half a range away
                other = torch.cat([s[:, :448], s[:, 480:], s[:, 448:480]], 1)
            tol = torch.where(torch.arange(512) >= 448, (s + other) / r.mscale, s)
        else:
            tol = torch.where(torch.arange(512) >= 448, size * 2.0 ** -3 + 2.0 ** -9, size * 2.0 ** -4 + 2.0 ** -10)
        tol = tol * (1 + 2.0 ** -6) + size * 2.0 ** -6.9
        err = (out.cpu().double() - want[:, None]).abs()
        assert bool((err <= tol[:, None]).all()), float((err / tol[:, None]).max())
        # and a scale of 1.63 on the turned channels would show: they have the size of the others
        ratio = out[:, 0, 448:].cpu().double().norm() / want[:, 448:].norm()
        assert 0.9 < float(ratio) < 1.1
