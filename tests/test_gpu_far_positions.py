"""Rotations at positions near 2^31, against angles formed in whole numbers."""
import pytest
import torch

import _angles
import _layer_ref as R
import compressed_sparse_attention_append_b200 as csa

pytestmark = pytest.mark.gpu
DEV = "cuda"
FAR = (1 << 31) - 1


def test_sines_and_cosines():
    """(1, 0) turned gives (cos, sin). The half turns round to fp32 (2^-25, 2^-23.3 radians); sincospif is off by 2 ulp,
    2^-23; the products with 0 and 1 are exact: 2^-22.1 together."""
    f, _ = csa.csa2_rope_frequencies(64)
    rope = csa.Rope(f.to(DEV))
    pos = torch.tensor([0, 1, 131071, 1 << 30] + [FAR - 7919 * i for i in range(60)])
    x = torch.zeros(len(pos), 1, 64, device=DEV)
    x[..., :32] = 1.0
    out = torch.empty_like(x)
    csa.csa2_rope(rope, pos.to(DEV), x, out)
    t = _angles.angles(pos, f)
    want = torch.cat([torch.cos(t), torch.sin(t)], 1)
    assert float((out[:, 0].cpu().double() - want).abs().max()) <= 2.0 ** -22


@pytest.mark.parametrize("normed", [False, True])
def test_codes_of_an_append(normed):
    """Codes and scales are those of the rotated row in 64 bits: half a million rotated channels a plane."""
    t, g = 1024, torch.Generator().manual_seed(17)
    rows = [torch.randn(1, t, n, generator=g).to(torch.bfloat16) for n in (512, 128, 512)]
    w = [(1.0 + 0.1 * torch.randn(x.shape[-1], generator=g)).to(torch.bfloat16) if normed else None for x in rows]
    rpos = FAR - torch.randperm(1 << 20, generator=g)[:t]
    freqs = [10000.0 ** (-torch.arange(n // 2, dtype=torch.float64) / n) for n in (512, 128)]  # (1 .. 0.01: fast ones)
    ropes = [csa.Rope(f.to(DEV), interleaved=True) for f in freqs]
    table = torch.arange(t // 64, dtype=torch.int32, device=DEV).view(1, -1)
    c = csa.PagedCache(t // 64, 64, 1, t // 64, t, page_table=table)
    dev = lambda x: None if x is None else x.to(DEV)
    csa.csa2_paged_append(c, 1, t, torch.zeros(1, dtype=torch.int64, device=DEV), *map(dev, rows), rope=ropes[0], idx_rope=ropes[1],
                          w_latent=dev(w[0]), w_idx_k=dev(w[1]), w_swa=dev(w[2]), eps=0.0, rpos=rpos[None].to(DEV))
    y = [_angles.rotate(x[0].double() if v is None else R.norm(x[0], v, 0.0), rpos, freqs[x.shape[-1] == 128], interleaved=True)
         for x, v in zip(rows, w)]
    flat = lambda plane: plane.flatten(0, 1).cpu()
    data, scale = R.e2m1_rows(y[0])
    assert torch.equal(flat(c.l_scale), scale) and torch.equal(flat(c.l_data), data)
    data, scale = R.mx_rows(y[1])
    assert torch.equal(flat(c.k_scale), scale) and torch.equal(flat(c.k_data), data)
    assert torch.equal(c.swa[0].cpu(), R.e4m3_rows(y[2]))
