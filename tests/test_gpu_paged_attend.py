"""csa2_paged_attend where rows are few (a row's tiles over a cluster) and many (one CTA a row): values that are not
finite, and every size of cluster. Against the formula in 64 bits, tolerance as in test_gpu_paged.py: probabilities in
fp16 (2^-11) and fp32 terms (2^-12) of the largest key value; lse 2^-12."""
import math

import pytest
import torch

import _layer_ref as R
import compressed_sparse_attention_append_b200 as csa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(B, n, seed, page=16):
    """A cache of n entries and a full window ring per sequence; queries at token n - 1."""
    g = torch.Generator().manual_seed(seed)
    pages = -(-n // page)
    table = torch.randperm(B * pages + 1, generator=g)[:B * pages].to(torch.int32).view(B, pages)
    c = csa.PagedCache(B * pages + 1, page, B, pages, indexer=False, page_table=table.to(DEV))
    c.l_data.copy_(torch.randint(0, 256, c.l_data.shape, generator=g, dtype=torch.uint8))
    c.l_scale.copy_(torch.randint(0x20, 0x39, c.l_scale.shape, generator=g, dtype=torch.uint8))
    c.swa.copy_(torch.randn(c.swa.shape, generator=g).to(torch.float8_e4m3fn).view(torch.uint8))
    q = torch.randn(B, 64, 512, generator=g).to(torch.bfloat16).to(DEV)
    return c, q, torch.full((B,), n - 1, device=DEV)


def _attend(c, qp, q, idx, k, **kw):
    B = q.shape[0]
    out = torch.full((B, 64, 512), 7.0, device=DEV, dtype=torch.bfloat16)
    of, lse = torch.full((B, 64, 512), 7.0, device=DEV), torch.full((B, 64), 7.0, device=DEV)
    csa.csa2_paged_attend(c, B, 1, qp, q, idx, k, out, out_f32=of, lse=lse, **kw)
    return out, of, lse


def _select(B, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.stack([torch.randperm(n, generator=g)[:k].sort().values for _ in range(B)]).to(torch.int32).to(DEV)


@pytest.mark.parametrize("B", [1, 3, 20, 60, 80])  # clusters of 5, 5, 5, 2 and no split
def test_queries_that_are_not_finite_give_nan_in_their_heads_alone(B):
    n, k = 600, 512
    c, q, qp = _case(B, n, seed=B)
    idx = _select(B, n, k, seed=B + 1)
    if B > 1:
        idx[1], qp[1] = -1, -1  # no key: zeros, whatever its query is
    clean = _attend(c, qp, q, idx, k)
    bad = q.clone()
    bad[0, 3, 7], bad[0, 4, 500], bad[0, 5, 0], bad[B // 2, 63, 64] = math.nan, math.inf, -math.inf, math.nan
    if B > 1:
        bad[1, 8, 8] = math.nan
    hit = torch.zeros(B, 64, dtype=torch.bool, device=DEV)
    hit[0, 3:6], hit[B // 2, 63] = True, True
    if B > 1:
        hit[1] = False
    got = _attend(c, qp, bad, idx, k)
    for a, b in zip(got, clean):
        assert bool(torch.isnan(a[hit]).all())
        assert torch.equal(a[~hit], b[~hit])
    if B > 1:
        assert not bool(got[0][1].any()) and bool((got[2][1] == -math.inf).all())


@pytest.mark.parametrize("B", [1, 20, 80])
def test_nan_in_a_key_that_counts_reaches_its_row_alone(B):
    n, k = 600, 500
    for where in ("entry", "window"):
        c, q, qp = _case(B, n, seed=B + 5)
        idx = _select(B, n, k, seed=B + 6)
        idx[:, 100:230] = -1
        clean = _attend(c, qp, q, idx, k)
        taken = set(idx[0].tolist())
        free = next(i for i in range(n) if i not in taken)
        cell = lambda i: (int(c.table[0, i // c.page]), i % c.page)
        # places that do not count: an entry that is not selected, window rows before swa_begin
        c.l_scale[cell(free)] = 0x7F
        c.swa[0, (n - 128) % 128] = 0x7F
        begin = torch.full((B,), n - 127, device=DEV)
        masked = _attend(c, qp, q, idx, k, swa_begin=begin)
        assert all(bool(torch.isfinite(x).all()) for x in masked)
        assert all(torch.equal(a[1:], b[1:]) for a, b in zip(_attend(c, qp, q, idx, k), clean))
        c.swa[0, (n - 128) % 128] = 0
        if where == "entry":
            at = cell(int(idx[0, 400]))
            c.l_scale[at[0], at[1], 9] = 0x7F
        else:
            c.swa[0, (n - 5) % 128, 77] = 0x7F
        got = _attend(c, qp, q, idx, k, swa_begin=begin)
        assert all(bool(torch.isnan(x[0]).all()) for x in got)
        assert all(torch.equal(a[1:], b[1:]) for a, b in zip(got, masked))


# rows, selected entries, window: clusters of 2 .. 16 CTAs on a whole B200 (test_attend_plan.py), one tile a CTA and several
CLUSTERS = [(1, 128 * t - t % 3, 0) for t in range(1, 17)] + [(2, 2048, 0), (7, 2048, 0), (6, 1793, 128), (1, 2048, 128),
            (8, 2048, 0), (20, 1000, 128), (24, 600, 0), (30, 500, 100), (42, 300, 128), (70, 640, 64), (76, 256, 128)]


@pytest.mark.parametrize("B,k,win", CLUSTERS)
def test_every_size_of_cluster(B, k, win):
    n = 2500
    c, q, qp = _case(B, n, seed=k + B)
    idx = _select(B, n, k, seed=k)
    idx[B // 2, k // 3:k // 2] = -1  # a gap
    if B > 1:
        idx[1, 128:] = -1            # CTAs without a key
    got = _attend(c, qp, q, idx, k, win=win)
    for r in range(B) if B < 9 else (0, 1, B // 2, B - 1):
        e = idx[r][idx[r] >= 0].long()
        page = c.table[r, e // c.page].long()
        keys = R.e2m1_values(c.l_data[page, e % c.page], c.l_scale[page, e % c.page])
        w = torch.arange(n - win, n, device=DEV)
        keys = torch.cat([keys, c.swa[r, w % 128].cpu().view(torch.float8_e4m3fn).double()])
        want, lse = R.attend(q[r].cpu().double(), keys, 512 ** -0.5)
        tol = float(keys.abs().max()) * (2.0 ** -11 + 2.0 ** -12)
        assert float((got[1][r].cpu().double() - want).abs().max()) <= tol
        assert float((got[2][r].cpu().double() - lse).abs().max()) <= 2.0 ** -12 * max(1.0, float(lse.abs().max()))
        assert torch.equal(got[0][r], got[1][r].to(torch.bfloat16))
    again = _attend(c, qp, q, idx, k, win=win)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
