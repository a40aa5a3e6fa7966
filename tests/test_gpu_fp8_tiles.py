"""csa2_fp8_gemm by the way it is split: contractions over a cluster's CTAs. Held to the exact product of the values that
codes and scales stand for; tolerance as in test_gpu_fp8.py: a block's sum in fp32 (2^-16 of the terms' absolute sum),
(blocks + 2) 2^-24 for scales and additions, half a step of the output type."""
import pytest
import torch

import _layer_ref as R
import compressed_sparse_attention_append_b200 as csa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _operands(m, n, k, seed=0):
    """E4M3 codes and scales of random rows and weights."""
    g = torch.Generator(device=DEV).manual_seed(seed + m + 3 * n + 7 * k)
    x = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
    w = (0.05 * torch.randn(n, k, generator=g, device=DEV)).to(torch.bfloat16)
    nb = -(-k // 128)
    xq, xs = torch.empty(m, k, device=DEV, dtype=torch.float8_e4m3fn), torch.empty(nb, m, device=DEV)
    wq, ws = torch.empty(n, k, device=DEV, dtype=torch.float8_e4m3fn), torch.empty(-(-n // 128), nb, device=DEV)
    csa.csa2_fp8_quantize(x, xq, xs)
    csa.csa2_fp8_quantize_weight(w, wq, ws)
    return xq, xs, wq, ws


def _check(out, xq, xs, wq, ws):
    a, b = R.fp8_values(xq, row_scale=xs).to(DEV), R.fp8_values(wq, block_scale=ws).to(DEV)
    want, size = a @ b.T, a.abs() @ b.abs().T
    nb = -(-xq.shape[1] // 128)
    tol = want.abs() * (torch.finfo(out.dtype).eps / 2) + size * (2.0 ** -16 + (nb + 2) * 2.0 ** -24)
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err / tol).max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 1, 8192), (5, 131, 8192), (16, 1031, 4096), (33, 257, 4112), (64, 129, 2048), (17, 640, 1040)])
def test_joins_of_few_tiles_that_end_inside(m, n, k, dtype):
    ops = _operands(m, n, k)
    frame = torch.full((m + 2, n + 5), 7.0, device=DEV, dtype=dtype)
    out = frame[1:m + 1, 2:n + 2]
    csa.csa2_fp8_gemm(*ops, out)
    _check(out, *ops)
    out.fill_(7.0)
    assert bool((frame == 7.0).all())
