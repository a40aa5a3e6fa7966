"""csa2_fp8_quantize, csa2_fp8_quantize_weight and csa2_fp8_gemm on the GPU.

The quantisers are held to the bytes of their rule (fp32 quotients, E4M3 to nearest even). The product is
held to the exact product of the values that codes and scales stand for. Tolerance: E4M3 products are
exact; a block's 128 terms are added in fp32, each addition off by at most 2^-23 (a truncated sum) of the
terms' absolute sum: 2^-16; scale product and the additions of nb blocks add (nb + 2) 2^-24; then half a
step of the output type.
"""
import pytest
import torch

import _layer_ref as R
import compressed_sparse_attention_append_b200 as csa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(seed, *shape, sigma=1.0):
    return (sigma * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).to(DEV)


def _quantized(x):
    rows, k = x.shape
    q = torch.empty(rows, k, device=DEV, dtype=torch.float8_e4m3fn)
    s = torch.empty(-(-k // 128), rows, device=DEV)
    csa.csa2_fp8_quantize(x, q, s)
    return q, s


def _weights(w):
    n, k = w.shape
    q = torch.empty(n, k, device=DEV, dtype=torch.float8_e4m3fn)
    s = torch.empty(-(-n // 128), -(-k // 128), device=DEV)
    csa.csa2_fp8_quantize_weight(w, q, s)
    return q, s


def _rule(blocks):
    """Codes and scales of [.., block] fp32 values on the host."""
    s = blocks.abs().amax(-1, keepdim=True) / torch.tensor(448.0)
    return torch.where(s > 0, blocks / s, 0.0).to(torch.float8_e4m3fn).view(torch.uint8), s[..., 0]


@pytest.mark.parametrize("rows,k", [(1, 16), (3, 128), (17, 144), (130, 4096), (1000, 272), (257, 2064), (4096, 2048)])
def test_row_quantiser_bytes(rows, k):
    x = _rand(rows + k, rows, k, sigma=3.0)
    x[rows // 2, :min(k, 128)] = 0.0
    wide = torch.cat([x, x[:, :8]], 1)[:, :k]  # another row stride
    for src in (x, wide):
        q, s = _quantized(src)
        pad = torch.nn.functional.pad(x.cpu().float(), (0, -k % 128)).unflatten(1, (-1, 128))
        codes, scale = _rule(pad)
        assert torch.equal(s.cpu().T, scale)
        assert torch.equal(q.view(torch.uint8).cpu(), codes.flatten(1)[:, :k])


@pytest.mark.parametrize("n,k", [(1, 16), (128, 128), (129, 144), (1000, 2064), (640, 4096)])
def test_weight_quantiser_bytes(n, k):
    w = _rand(n + k, n, k, sigma=0.02)
    q, s = _weights(w)
    pad = torch.nn.functional.pad(w.cpu().float(), (0, -k % 128, 0, -n % 128))
    blocks = pad.view(-(-n // 128), 128, -1, 128).transpose(1, 2)
    codes, scale = _rule(blocks.flatten(2))
    codes = codes.view(blocks.shape).transpose(1, 2).reshape(pad.shape)
    assert torch.equal(s.cpu(), scale)
    assert torch.equal(q.view(torch.uint8).cpu(), codes[:n, :k])


def test_quantiser_extremes():
    """The largest value of a block is code 448 whatever its size; an infinity or NaN stays in its block."""
    x = torch.zeros(4, 256, device=DEV, dtype=torch.bfloat16)
    x[0, 0], x[0, 1] = 3.0e38, -3.0e38
    x[1, 5], x[1, 200] = 1e-38, 1.0
    x[2, 7], x[2, 130] = float("inf"), 2.0
    x[3, 9], x[3, 131] = float("nan"), 2.0
    q, s = _quantized(x)
    v = q.float().cpu()
    assert v[0, 0] == 448 and v[0, 1] == -448 and v[1, 200] == 448 and v[2, 130] == 448 and v[3, 131] == 448
    assert torch.isnan(v[2, 7]) and torch.isnan(v[3, 9]) and not v[0, 2:].any()
    assert torch.isnan(s[0, 3]) and torch.isinf(s[0, 2]) and torch.isnan(v[3, :128]).all()


def _check(out, x, xs, w, ws):
    a, b = R.fp8_values(x, row_scale=xs).to(DEV), R.fp8_values(w, block_scale=ws).to(DEV)
    want, size = a @ b.T, a.abs() @ b.abs().T
    nb = -(-x.shape[1] // 128)
    tol = want.abs() * (torch.finfo(out.dtype).eps / 2) + size * (2.0 ** -16 + (nb + 2) * 2.0 ** -24)
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err / tol).max()))


SIZES = [  # m, n, k
    (1, 1, 16), (1, 128, 128), (1, 1536, 1024), (2, 130, 144), (16, 257, 4096), (17, 128, 272), (32, 4099, 512),
    (33, 640, 2064), (64, 2048, 1024), (65, 129, 400), (100, 8192, 256), (128, 1000, 4096), (129, 384, 1040),
    (200, 2500, 768), (256, 256, 128), (257, 4100, 640), (300, 127, 8192), (777, 1031, 1296), (1024, 2048, 512),
    (2100, 1300, 384),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm_matches_the_exact_product(m, n, k, dtype):
    x, xs = _quantized(_rand(m + k, m, k))
    w, ws = _weights(_rand(n + k, n, k, sigma=0.05))
    out = torch.full((m, n), float("nan"), device=DEV, dtype=dtype)
    csa.csa2_fp8_gemm(x, xs, w, ws, out)
    _check(out, x, xs, w, ws)
    again = torch.empty_like(out)
    csa.csa2_fp8_gemm(x, xs, w, ws, again)
    assert torch.equal(again, out)  # no order of additions depends on timing


@pytest.mark.parametrize("m,n,k", [(5, 200, 256), (150, 300, 640), (600, 900, 256)])
def test_gemm_writes_its_rows_and_columns_alone(m, n, k):
    """A strided output: columns and rows around it stay; scales of very different sizes; a zero block."""
    xb = _rand(1, m, k)
    xb[:, :128] *= 1e4
    xb[m // 2] = 0.0
    x, xs = _quantized(xb)
    wb = _rand(2, n, k)
    wb[:128, 128:256] = 0.0
    wb[128:] *= 1e-3
    w, ws = _weights(wb)
    for dtype in (torch.bfloat16, torch.float32):
        frame = torch.full((m + 2, n + 3), 7.0, device=DEV, dtype=dtype)
        out = frame[1:m + 1, 1:n + 1]  # (rows at odd elements)
        csa.csa2_fp8_gemm(x, xs, w, ws, out)
        _check(out, x, xs, w, ws)
        assert not bool(out[m // 2].any())
        frame[1:m + 1, 1:n + 1] = 7.0
        assert bool((frame == 7.0).all())


def test_gemm_keeps_values_that_are_not_finite_in_their_rows():
    x, xs = _quantized(_rand(3, 40, 512))
    w, ws = _weights(_rand(4, 300, 512))
    xs[1, 7] = float("nan")
    ws[2, 3] = float("inf")
    out = torch.empty(40, 300, device=DEV)
    csa.csa2_fp8_gemm(x, xs, w, ws, out)
    fine = torch.isfinite(out)
    assert not bool(fine[7].any()) and not bool(fine[:, 256:].any())
    keep = [i for i in range(40) if i != 7]
    assert bool(fine[keep][:, :256].all())


def test_two_streams_and_a_graph():
    x, xs = _quantized(_rand(5, 96, 1024))
    w, ws = _weights(_rand(6, 2048, 1024))
    a, b, c = (torch.empty(96, 2048, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    csa.csa2_fp8_gemm(x, xs, w, ws, a)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):  # two calls at once share nothing
        csa.csa2_fp8_gemm(x, xs, w, ws, b, stream=s1)
        csa.csa2_fp8_gemm(x, xs, w, ws, c, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    src = _rand(7, 96, 1024)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa.csa2_fp8_quantize(src, x, xs)
        csa.csa2_fp8_gemm(x, xs, w, ws, b)
    src.copy_(_rand(8, 96, 1024))
    g.replay()
    x2, xs2 = _quantized(src)
    csa.csa2_fp8_gemm(x2, xs2, w, ws, c)
    assert torch.equal(b, c)
