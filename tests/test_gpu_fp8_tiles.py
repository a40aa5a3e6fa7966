"""csa2_fp8_gemm by the way it is split: contractions over a cluster's CTAs, and the persistent kernel's CTAs with several
tiles each (test_fp8_plan.py checks that these sizes reach it). Held to the exact product of the values that
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


JOINS = [(1, 1, 8192), (5, 131, 8192), (16, 1031, 4096), (33, 257, 4112), (64, 129, 2048), (17, 640, 1040), (50, 8000, 2064),
         (60, 16000, 512)]
# more tiles (128 x 256) than SMs: odd and even numbers of blocks, contractions that end inside one
MANY = [(2100, 6001, 656), (1300, 4000, 128), (2500, 5200, 1152), (3000, 3333, 400), (700, 20000, 272), (4099, 2600, 16)]
FRAME, NOT_FINITE, STREAMS = (2051, 3001, 656), (2100, 3000, 384), (1500, 4100, 1040)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", MANY)
def test_ctas_with_several_tiles(m, n, k, dtype):
    ops = _operands(m, n, k)
    out = torch.full((m, n), float("nan"), device=DEV, dtype=dtype)
    csa.csa2_fp8_gemm(*ops, out)
    _check(out, *ops)
    again = torch.full_like(out, float("nan"))
    csa.csa2_fp8_gemm(*ops, again)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("left,right", [(1, 2), (2, 5), (8, 23)])  # odd rows, odd strides, rows on 16 bytes
def test_tiles_write_their_rows_and_columns_alone(left, right, dtype):
    m, n, k = FRAME
    ops = _operands(m, n, k)
    frame = torch.full((m + 2, n + left + right), 7.0, device=DEV, dtype=dtype)
    out = frame[1:m + 1, left:n + left]
    csa.csa2_fp8_gemm(*ops, out)
    _check(out, *ops)
    out.fill_(7.0)
    assert bool((frame == 7.0).all())


def test_tiles_keep_values_that_are_not_finite_in_their_rows():
    m, n, k = NOT_FINITE
    xq, xs, wq, ws = _operands(m, n, k)
    want = torch.empty(m, n, device=DEV)
    csa.csa2_fp8_gemm(xq, xs, wq, ws, want)
    xs[1, 7], xs[2, 1900] = float("nan"), float("inf")
    ws[5, 0], ws[-1, 2] = float("nan"), float("inf")
    xq.view(torch.uint8)[1000, 300] = 0x7F  # a code that is NaN
    out = torch.empty_like(want)
    csa.csa2_fp8_gemm(xq, xs, wq, ws, out)
    bad = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    bad[[7, 1900, 1000]] = True
    bad[:, 640:768] = True
    bad[:, (n - 1) // 128 * 128:] = True
    assert not bool(torch.isfinite(out[bad]).any())
    assert torch.equal(out[~bad], want[~bad])


def test_two_calls_at_once_and_a_captured_one():
    m, n, k = STREAMS
    ops = _operands(m, n, k)
    want = torch.empty(m, n, device=DEV, dtype=torch.bfloat16)
    outs = [torch.empty_like(want) for _ in range(3)]
    csa.csa2_fp8_gemm(*ops, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, o in zip(streams, outs):
            csa.csa2_fp8_gemm(*ops, o, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.csa2_fp8_gemm(*ops, outs[2])
        csa.csa2_fp8_gemm(*ops, outs[2])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", JOINS)
def test_joins_of_few_tiles_that_end_inside(m, n, k, dtype):
    ops = _operands(m, n, k)
    frame = torch.full((m + 2, n + 5), 7.0, device=DEV, dtype=dtype)
    out = frame[1:m + 1, 2:n + 2]
    csa.csa2_fp8_gemm(*ops, out)
    _check(out, *ops)
    out.fill_(7.0)
    assert bool((frame == 7.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(40, 300, 512), (2100, 6001, 656)])
@pytest.mark.parametrize("up", [1.0, -1.0])
def test_scales_of_opposite_extremes(m, n, k, dtype, up):
    """Scales far outside each other's size whose product is an ordinary number (powers of two: the same result but for
    them, bit for bit)."""
    xq, xs, wq, ws = _operands(m, n, k)
    want, out = torch.empty(m, n, device=DEV, dtype=dtype), torch.empty(m, n, device=DEV, dtype=dtype)
    csa.csa2_fp8_gemm(xq, xs, wq, ws, want)
    csa.csa2_fp8_gemm(xq, xs * 2.0 ** (100 * up), wq, ws * 2.0 ** (-100 * up), out)
    assert torch.equal(out, want)
