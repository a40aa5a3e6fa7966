"""The paged latent cache on the GPU: csa2_paged_append (norm, rotation and codecs in one pass),
csa2_paged_gather, csa2_paged_attend and csa2_paged_index_topk.

Codes and scales are held byte for byte to the rule in 64 bits (they are decided there, so only a value
within 2^-50 of a rounding border could differ). Attention: q and the dequantised keys are exact in fp16,
logits and sums are fp32 and probabilities are rounded to fp16 (at most 2^-11 each), so an output is
off by at most 2^-11 times the largest key value plus fp32 terms; lse has no rounded probabilities.
"""
import math

import numpy as np
import pytest
import torch

import _layer_ref as R
import compressed_sparse_attention_append_b200 as csa

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


class Status:
    def __init__(self):
        self.buf = torch.zeros(256, dtype=torch.uint8, device=DEV)

    ptr = property(lambda self: self.buf.data_ptr())
    nbytes = 256

    def read(self):
        return csa.csa2_get_device_status(self)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(seed, *shape, sigma=1.0):
    return (sigma * torch.randn(*shape, generator=_gen(seed))).to(torch.bfloat16).to(DEV)


def _cache(B, pages, page, swa_cap=128, spare=3, seed=0, **kw):
    n = B * pages + spare
    table = torch.randperm(n, generator=_gen(seed))[:B * pages].to(torch.int32).view(B, pages).to(DEV)
    return csa.PagedCache(n, page, B, pages, swa_cap, page_table=table, **kw)


def _logical(cache, plane, b, n):
    """Rows of entries 0 .. n - 1 of sequence b, through the page table."""
    p = torch.arange(n, device=DEV)
    page = cache.table[b, p // cache.page].long()
    return plane[page, p % cache.page]


def _ropes(interleaved, rot=64):
    main = csa.Rope.for_context(rot, 10000.0, "yarn", 16.0, 4096, offset=512 - rot, interleaved=interleaved)
    return main, csa.Rope.for_context(64, 10000.0, offset=64, interleaved=interleaved)


def _want(x, w, rope, at, eps=EPS):
    """The 64-bit values of rows x [n, ch] at rotation positions at [n]."""
    y = x.detach().cpu().double() if w is None else R.norm(x, w, eps)
    if rope is None:
        return y
    return R.rotate(y[:, None], at, rope.inv_freq, rope.offset, rope.interleaved, rope.mscale)[0][:, 0]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,t,page,start,normed,rot", [
    (1, 1, 8, 0, True, 64), (3, 5, 16, 13, True, 64), (2, 300, 64, 1000, True, 64), (4, 129, 32, 7, False, 128),
    (2, 40, 64, 131071, True, 512), (2, 33, 8, 100000, True, 2), (1, 2000, 128, 3, True, 64),
])
def test_append_bytes(B, t, page, start, normed, rot, interleaved):
    main, krope = _ropes(interleaved, rot)
    pages = (start + t + 50) // page + 1
    c = _cache(B, pages, page, seed=t)
    lat, key, swa = _rand(1, B, t, 512, sigma=2.0), _rand(2, B, t, 128), _rand(3, B, t, 512)
    lat[0, 0, :16] = 0.0
    lat[-1, -1] *= 1e-6
    key[0, -1, 32:64] = 0.0
    w = [1.0 + 0.2 * _rand(s, n) if normed else None for s, n in ((4, 512), (5, 128), (6, 512))]
    pos = start + torch.randint(0, 40, (B,), generator=_gen(t)).to(DEV)
    ws = Status()
    csa.csa2_paged_append(c, B, t, pos, lat, key, swa, rope=main, idx_rope=krope, w_latent=w[0], w_idx_k=w[1],
                          w_swa=w[2], eps=EPS, ws=ws)
    assert ws.read() == 0
    touched = torch.zeros(c.n_pages, page, dtype=torch.bool)
    for b in range(B):
        p0 = int(pos[b])
        at = torch.arange(p0, p0 + t)
        rows = lambda plane: _logical(c, plane, b, p0 + t)[p0:].cpu()
        data, scale = R.e2m1_rows(_want(lat[b], w[0], main, at))
        assert torch.equal(rows(c.l_scale), scale) and torch.equal(rows(c.l_data), data)
        data, scale = R.mx_rows(_want(key[b], w[1], krope, at))
        assert torch.equal(rows(c.k_scale), scale) and torch.equal(rows(c.k_data), data)
        ring = torch.zeros(128, 512, dtype=torch.uint8)
        ring[at[-128:] % 128] = R.e4m3_rows(_want(swa[b], w[2], main, at))[-128:]
        assert torch.equal(c.swa[b].cpu(), ring)
        touched[c.table[b].cpu().long()[at // page], at % page] = True
    for plane in (c.l_data, c.l_scale, c.k_data, c.k_scale):  # nothing but the appended entries
        assert not bool(plane.cpu()[~touched].any())


def test_append_without_norm_and_rotation_is_the_contiguous_append():
    """Bytes of csa2_latent_append on the same rows (bf16 values next to every border, subnormals, extremes)."""
    B, t = 2, 96
    lat, key, swa = (_rand(s, B, t, n, sigma=3.0) for s, n in ((1, 512), (2, 128), (3, 512)))
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    every = every[torch.isfinite(every)]
    lat[0, :32] = every[:32 * 512].view(32, 512).to(DEV)
    lat[1, :32] = every[-32 * 512:].view(32, 512).to(DEV)
    lat[0, 40] = (torch.arange(512) % 13).to(torch.bfloat16).to(DEV) * 0.25  # ties
    key[0, 40] = (torch.arange(128) % 13).to(torch.bfloat16).to(DEV) * 0.25
    flat = csa.LatentCache(B, 128)
    pos = torch.tensor([3, 32], device=DEV)
    csa.csa2_latent_append(flat, B, t, pos, lat, key, swa)
    c = _cache(B, 16, 8)
    csa.csa2_paged_append(c, B, t, pos, lat, key, swa)
    for b in range(B):
        for a, f in ((c.l_data, flat.l_data), (c.l_scale, flat.l_scale), (c.k_data, flat.k_data),
                     (c.k_scale, flat.k_scale)):
            assert torch.equal(_logical(c, a, b, 128), f[b])
        assert torch.equal(c.swa[b], flat.swa[b])


def test_append_of_extreme_rows():
    """Rows whose squares leave fp32, rows of tiny and of mixed sizes, weights of any size: the 64-bit codes."""
    t = 12
    main, krope = _ropes(True)
    g = _gen(12)
    mag = torch.tensor([1.0, 3e19, 1e30, 3e38, 1e-18, 1e-25, 1e-38, 1e-40, 0.0, 1e4, 1.0, 1.0])[:, None]
    lat = (torch.randn(1, t, 512, generator=g) * mag).clamp(-3e38, 3e38).to(torch.bfloat16)
    key = (torch.randn(1, t, 128, generator=g) * mag).clamp(-3e38, 3e38).to(torch.bfloat16)
    lat[0, 10, ::2] = -0.0
    key[0, 10, ::2] = -0.0
    lat[0, 11, ::3] *= 1e6
    key[0, 11, ::3] *= 1e-6
    w = (torch.randn(512, generator=g) * torch.exp2(torch.randint(-40, 40, (512,), generator=g).float())).to(torch.bfloat16)
    w[7], w[300] = 0.0, 1e-39
    for eps in (0.0, 1e-30, 1e-5):
        for wl in (w, torch.ones(512, dtype=torch.bfloat16)):
            c = _cache(1, 2, 8)
            pos = torch.zeros(1, dtype=torch.int64, device=DEV)
            csa.csa2_paged_append(c, 1, t, pos, lat.to(DEV), key.to(DEV), lat.to(DEV), rope=main, idx_rope=krope,
                                  w_latent=wl.to(DEV), w_idx_k=wl[:128].to(DEV), w_swa=wl.to(DEV), eps=eps)
            at = torch.arange(t)
            ok = torch.ones(t, dtype=torch.bool)
            if eps == 0.0:
                ok[8] = False  # 0 / 0
            eps32 = float(torch.tensor(eps, dtype=torch.float32))
            y = _want(lat[0], wl, main, at, eps32)
            data, scale = R.e2m1_rows(y)
            rows = lambda plane: _logical(c, plane, 0, t).cpu()[ok]
            assert torch.equal(rows(c.l_scale), scale[ok]) and torch.equal(rows(c.l_data), data[ok])
            assert torch.equal(c.swa[0, :t].cpu()[ok], R.e4m3_rows(y)[ok])
            y = _want(key[0], wl[:128], krope, at, eps32)
            data, scale = R.mx_rows(y)
            ok &= y.abs().amax(-1) < 2.0 ** 126
            assert torch.equal(rows(c.k_scale), scale[ok]) and torch.equal(rows(c.k_data), data[ok])


def test_append_of_padded_batches_strides_and_own_rotation_positions():
    B, t, page = 5, 24, 8
    main, krope = _ropes(True)
    big = _rand(7, t, B, 512 + 128 + 512)  # token major, one projection
    lat, key, swa = big[..., :512].transpose(0, 1), big[..., 512:640].transpose(0, 1), big[..., 640:].transpose(0, 1)
    pos = torch.tensor([0, 5, 100, 9, -7], device=DEV)
    ln = torch.tensor([0, 24, 7, 1, 0], dtype=torch.int32, device=DEV)
    rpos = torch.randint(0, 1 << 20, (B, t), generator=_gen(8)).to(DEV)
    w = 1.0 + 0.1 * _rand(9, 512)
    slot = torch.tensor([6, 2, 4, 0, 1], dtype=torch.int32, device=DEV)
    c = _cache(B, 16, page, n_slots=7, swa_slot=slot)
    ws = Status()
    csa.csa2_paged_append(c, B, t, pos, lat, key, swa, rope=main, idx_rope=krope, w_latent=w, length=ln, rpos=rpos,
                          eps=EPS, ws=ws)
    assert ws.read() == 0  # an empty sequence at a negative position is padding
    for b in (1, 2, 3):
        n, p0 = int(ln[b]), int(pos[b])
        data, scale = R.e2m1_rows(_want(lat[b, :n], w, main, rpos[b, :n]))
        assert torch.equal(_logical(c, c.l_data, b, p0 + n)[p0:].cpu(), data)
        data, scale = R.mx_rows(_want(key[b, :n], None, krope, rpos[b, :n]))
        assert torch.equal(_logical(c, c.k_data, b, p0 + n)[p0:].cpu(), data)
        ring = R.e4m3_rows(_want(swa[b, :n], None, main, rpos[b, :n]))
        assert torch.equal(c.swa[int(slot[b]), torch.arange(p0, p0 + n) % 128].cpu(), ring)
    assert int((c.swa.view(7, -1) != 0).any(1).sum()) == 3
    assert int((c.l_data != 0).any(-1).sum()) == 24 + 7 + 1


@pytest.mark.parametrize("normed", [False, True])
def test_append_of_more_tokens_than_the_ring_holds(normed):
    """Window rows only: the latest swa_cap of each sequence land, whatever its length; a bad length is reported once."""
    B, t, cap = 7, 77, 16
    main, _ = _ropes(False)
    x = _rand(21, B, t, 512)
    w = 1.0 + 0.1 * _rand(22, 512) if normed else None
    pos = torch.tensor([0, 3, 1000, 15, 16, 2, 9], device=DEV)
    ln = torch.tensor([77, 16, 17, 1, 0, 78, 31], dtype=torch.int32, device=DEV)
    rpos = torch.randint(0, 1 << 20, (B, t), generator=_gen(23)).to(DEV)
    for length, turned in ((ln, None), (ln, rpos), (None, None)):
        c = _cache(B, 200, 8, swa_cap=cap)
        c.swa.fill_(0x55)
        ws = Status()
        csa.csa2_paged_append(c, B, t, pos, swa=x, rope=main, w_swa=w, length=length, rpos=turned, eps=EPS, ws=ws)
        assert ws.read() == (0 if length is None else csa.CSA2_DEV_BAD_POS)
        for b in range(B):
            n, p0 = t if length is None else int(ln[b]), int(pos[b])
            want = torch.full((cap, 512), 0x55, dtype=torch.uint8)
            if n <= t:
                i = torch.arange(max(n - cap, 0), n)
                at = (p0 + i) if turned is None else rpos[b, i.to(DEV)].cpu()
                want[(p0 + i) % cap] = R.e4m3_rows(_want(x[b, i.to(DEV)], w, main, at))
            assert torch.equal(c.swa[b].cpu(), want)


def test_append_reports_and_skips_what_does_not_fit():
    B, t, page, pages = 6, 4, 8, 4
    c = _cache(B, pages, page, swa_slot=torch.tensor([0, 1, 2, 3, 9, 5], dtype=torch.int32, device=DEV))
    c.table[2, 1] = -1
    c.table[3, 0] = c.n_pages
    x = _rand(1, B, t, 512)
    pos = torch.tensor([30, -1, 6, 0, 0, 0], device=DEV)
    ln = torch.tensor([4, 4, 4, 4, 4, 5], dtype=torch.int32, device=DEV)
    ws = Status()
    csa.csa2_paged_append(c, B, t, pos, latent=x, length=ln, ws=ws)
    assert ws.read() == csa.CSA2_DEV_BAD_POS | csa.CSA2_DEV_BAD_PAGE
    got = (c.l_data != 0).any(-1)
    assert int(got.sum()) == 2 + 4  # sequence 2's two tokens before the missing page, sequence 4's four
    csa.csa2_paged_append(c, B, t, pos.clamp_min(0), swa=x, ws=ws)  # ring of sequence 4 is not there
    assert ws.read() == csa.CSA2_DEV_BAD_PAGE
    assert (c.swa != 0).any(-1).sum(1).tolist() == [4, 4, 4, 4, 0, 4]
    csa.csa2_paged_append(c, B, t, pos, latent=x, length=ln)  # without a workspace: skipped all the same


def test_gather_gives_the_values():
    B, n, page = 3, 70, 16
    c = _cache(B, 5, page)
    g = _gen(3)
    c.l_data.copy_(torch.randint(0, 256, c.l_data.shape, generator=g, dtype=torch.uint8))
    c.l_scale.copy_(torch.randint(0, 0x7f, c.l_scale.shape, generator=g, dtype=torch.uint8))
    c.k_data.copy_(torch.randint(0, 256, c.k_data.shape, generator=g, dtype=torch.uint8))
    c.k_scale.copy_(torch.randint(0, 252, c.k_scale.shape, generator=g, dtype=torch.uint8))
    idx = torch.randint(0, 80, (B, n), generator=g, dtype=torch.int32)
    idx[0, 0], idx[1, 1], idx[2, 2] = -1, 80, -2
    idx[2, 3] = 64
    c.table[2, 4] = -1
    lat = torch.full((B, n, 512), 7.0, device=DEV, dtype=torch.bfloat16)
    key = torch.full((B, n, 128), 7.0, device=DEV, dtype=torch.bfloat16)
    ws = Status()
    csa.csa2_paged_gather(c, B, idx.to(DEV), lat, key, ws=ws)
    assert ws.read() == csa.CSA2_DEV_BAD_INDEX | csa.CSA2_DEV_BAD_PAGE
    for b in range(B):
        ok = (idx[b] >= 0) & (idx[b] < (64 if b == 2 else 80))
        at = idx[b][ok].long()
        for out, d, s, f in ((lat, c.l_data, c.l_scale, R.e2m1_values), (key, c.k_data, c.k_scale, R.mx_values)):
            want = f(_logical(c, d, b, 80)[at.to(DEV)], _logical(c, s, b, 80)[at.to(DEV)])
            assert torch.equal(out[b].cpu()[ok].double(), want)  # exact in bf16
            assert not bool(out[b].cpu()[~ok].any())
    only = torch.empty_like(key)
    csa.csa2_paged_gather(c, B, idx.to(DEV), key=only)
    assert torch.equal(only, key)


def _filled(B, n, page, swa_cap, seed, sigma=1.0):
    """A paged and a contiguous cache with the same entries and window rows."""
    cap = -(-n // page) * page
    flat = csa.LatentCache(B, cap, swa_cap)
    g = _gen(seed)
    lat, key, swa = (_rand(seed + s, B, n, ch, sigma=sigma) for s, ch in ((1, 512), (2, 128), (3, 512)))
    zero = torch.zeros(B, dtype=torch.int64, device=DEV)
    csa.csa2_latent_append(flat, B, n, zero, lat, key, swa)
    slot = torch.randperm(B + 2, generator=g)[:B].to(torch.int32).to(DEV)
    c = _cache(B, cap // page, page, swa_cap, seed=seed, n_slots=B + 2, swa_slot=slot)
    csa.csa2_paged_append(c, B, n, zero, lat, key, swa)
    return c, flat


def _select(rows, vis, k, seed):
    idx = torch.full((rows, k), -1, dtype=torch.int32)
    for r in range(rows):
        m = min(k, max(vis[r], 0))
        m = m if r % 2 == 0 else m - m // 3  # odd rows: gaps
        place = torch.randperm(k, generator=_gen(seed + r))[:m]
        idx[r, place] = torch.randperm(max(vis[r], 1), generator=_gen(seed + 50 + r))[:m].to(torch.int32)
    return idx.to(DEV)


def _attend(call, c, B, tq, qp, q, idx, k, **kw):
    rows = B * tq
    out = torch.full((rows, 64, 512), float("nan"), device=DEV, dtype=torch.bfloat16)
    of = torch.full((rows, 64, 512), float("nan"), device=DEV)
    lse = torch.full((rows, 64), float("nan"), device=DEV)
    ws = Status()
    call(c, B, tq, qp, q, idx, k, out, out_f32=of, lse=lse, ws=ws, **kw)
    return out, of, lse, ws.read()


def _reference(c, b, qpos, q, idx, win, ratio, begin, scale):
    vis = min((qpos + 1) // ratio, c.max_pages * c.page)
    at = [int(i) for i in idx if 0 <= int(i) < vis and 0 <= int(c.table[b, int(i) // c.page]) < c.n_pages]
    at = torch.tensor(at, dtype=torch.int64, device=DEV)
    page = c.table[b, at // c.page].long()
    keys = R.e2m1_values(c.l_data[page, at % c.page], c.l_scale[page, at % c.page])
    slot = int(c.swa_slot[b]) if c.swa_slot is not None else b
    w = torch.arange(max(begin, qpos - win + 1, 0), qpos + 1) if win and 0 <= slot < c.n_slots else torch.arange(0)
    window = c.swa[slot, (w % c.swa_cap).to(DEV)].cpu().view(torch.float8_e4m3fn).double() if w.numel() else torch.zeros(0, 512, dtype=torch.float64)
    keys = torch.cat([keys, window])
    return (*R.attend(q.cpu().double(), keys, scale), float(keys.abs().max()) if keys.numel() else 1.0)


def _close(out, of, lse, want, want_lse, largest):
    assert torch.equal(out, of.to(torch.bfloat16))
    y = of.cpu().double()
    # fp16 probabilities 2^-11, exponentials and fp32 sums of up to 2176 logits below 2^-12 together
    assert float((y - want).abs().max()) <= largest * (2.0 ** -11 + 2.0 ** -12)
    g = lse.cpu().double()
    fin = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(g), fin) and bool((g[~fin] == -math.inf).all())
    assert not fin.any() or float((g[fin] - want_lse[fin]).abs().max()) <= 2.0 ** -12 * max(1.0, float(want_lse[fin].abs().max()))


@pytest.mark.parametrize("B,tq,n,k,page,win,ratio", [
    (1, 1, 1, 1, 8, 128, 1), (1, 1, 40, 17, 8, 16, 1), (3, 1, 700, 512, 64, 128, 1), (1, 1, 3000, 2048, 16, 128, 1),
    (2, 1, 1500, 300, 128, 0, 1), (2, 3, 900, 129, 32, 100, 2), (1, 1, 300, 0, 64, 128, 1), (1, 5, 1200, 640, 64, 128, 1),
    (9, 1, 500, 384, 64, 77, 1), (40, 2, 400, 100, 16, 128, 1),
])
def test_attend_over_pages(B, tq, n, k, page, win, ratio):
    c, flat = _filled(B, n, page, 256, seed=n + k)
    rows = B * tq
    qpos = [max(0, n - 1 - 2 * (r // tq) - (tq - 1 - r % tq)) for r in range(rows)]
    qp = torch.tensor(qpos, device=DEV)
    q = _rand(9, rows, 64, 512)
    idx = _select(rows, [(p + 1) // ratio for p in qpos], k, seed=n) if k else None
    out, of, lse, st = _attend(csa.csa2_paged_attend, c, B, tq, qp, q, idx, k, win=win, ratio=ratio)
    assert st == 0
    for r in range(rows):
        want = _reference(c, r // tq, qpos[r], q[r], idx[r] if k else [], win, ratio, 0, 512 ** -0.5)
        _close(out[r], of[r], lse[r], *want)
    again = _attend(csa.csa2_paged_attend, c, B, tq, qp, q, idx, k, win=win, ratio=ratio)
    assert torch.equal(again[0], out) and torch.equal(again[2], lse)
    if k:  # the contiguous cache with the same contents
        o2, f2, l2, _ = _attend(csa.csa2_latent_attend, flat, B, tq, qp, q, idx, k, win=win, ratio=ratio)
        assert float((f2 - of).abs().max()) <= 2.0 ** -8 and float((l2 - lse).abs().max()) <= 2.0 ** -10


def test_attend_rows_without_keys_bad_entries_and_missing_pages():
    B, n, k, page = 6, 600, 200, 32
    c, _ = _filled(B, n, page, 128, seed=4)
    qpos = [n - 1, -1, n - 1, n - 1, 300, n - 1]
    qp = torch.tensor(qpos, device=DEV)
    begin = torch.tensor([n, 0, 0, n, 0, n - 50], device=DEV)
    idx = _select(B, [600, 1, 600, 600, 301, 600], k, seed=3)
    idx[0] = -1                      # row 0: nothing at all
    idx[2, 7], idx[2, 8] = n + 5000, -3
    idx[4, 3] = 301                  # not visible yet
    c.table[3, 2:9] = -1             # pages that are not there
    c.table[5] = c.n_pages + 3       # none of this row's pages: the window alone
    q = _rand(10, B, 64, 512)
    out, of, lse, st = _attend(csa.csa2_paged_attend, c, B, 1, qp, q, idx, k, swa_begin=begin)
    assert st == csa.CSA2_DEV_BAD_INDEX | csa.CSA2_DEV_BAD_PAGE
    for r in (0, 1):
        assert not bool(out[r].any()) and not bool(of[r].any()) and bool((lse[r] == -math.inf).all())
    for r in (2, 3, 4, 5):
        _close(out[r], of[r], lse[r], *_reference(c, r, qpos[r], q[r], idx[r], 128, 1, int(begin[r]), 512 ** -0.5))
    c.swa_slot[2] = 99               # the ring is not there: the selected entries alone
    out, of, lse, st = _attend(csa.csa2_paged_attend, c, B, 1, qp, q, idx, k, swa_begin=begin)
    assert st & csa.CSA2_DEV_BAD_PAGE
    _close(out[2], of[2], lse[2], *_reference(c, 2, qpos[2], q[2], idx[2], 128, 1, 0, 512 ** -0.5))


def test_the_window_alone_and_tokens_past_the_table():
    """k = 0 needs no page: the window counts wherever the token is. Entries past the table are refused one by one."""
    c, _ = _filled(1, 300, 8, 512, seed=9)
    few = csa.PagedCache(c.n_pages, 8, 1, 2, 512, n_slots=c.n_slots, swa_slot=c.swa_slot, page_table=c.table[:, :2].contiguous(),
                         l_data=c.l_data, l_scale=c.l_scale, k_data=c.k_data, k_scale=c.k_scale, swa=c.swa)
    none = csa.PagedCache(0, 8, 1, 0, 512, n_slots=c.n_slots, swa_slot=c.swa_slot, swa=c.swa, latent=False, indexer=False,
                          page_table=torch.empty(1, 0, dtype=torch.int32, device=DEV))
    q, qp = _rand(3, 1, 64, 512), torch.tensor([299], device=DEV)
    want = _reference(c, 0, 299, q[0], [], 128, 1, 0, 512 ** -0.5)
    for cache in (c, few, none):
        out, of, lse, st = _attend(csa.csa2_paged_attend, cache, 1, 1, qp, q, None, 0)
        assert st == 0
        _close(out[0], of[0], lse[0], *want)
    idx = torch.tensor([[3, 15, 16, 3]], dtype=torch.int32, device=DEV)  # (an entry twice counts twice)
    out, of, lse, st = _attend(csa.csa2_paged_attend, few, 1, 1, qp, q, idx, 4)
    assert st == csa.CSA2_DEV_BAD_INDEX
    _close(out[0], of[0], lse[0], *_reference(few, 0, 299, q[0], idx[0], 128, 1, 0, 512 ** -0.5))


def test_pages_shared_by_sequences_and_two_calls_at_once():
    """Sequences with a common prefix read the same pages; calls on two streams share nothing but the cache."""
    c, _ = _filled(3, 256, 16, 128, seed=11)
    c.table[1, :8] = c.table[0, :8]
    c.table[2, :16] = c.table[0, :16]
    q, qp = _rand(4, 3, 64, 512), torch.tensor([255, 200, 255], device=DEV)
    idx = _select(3, [256, 201, 256], 100, seed=5)
    out, of, lse, st = _attend(csa.csa2_paged_attend, c, 3, 1, qp, q, idx, 100)
    assert st == 0
    for r in range(3):
        _close(out[r], of[r], lse[r], *_reference(c, r, int(qp[r]), q[r], idx[r], 128, 1, 0, 512 ** -0.5))
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(out) for _ in range(2)]
    for _ in range(10):
        for s, o in zip(streams, outs):
            csa.csa2_paged_attend(c, 3, 1, qp, q, idx, 100, o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)


@pytest.mark.parametrize("B,tq,n,hi,k,page,flags", [(2, 1, 700, 32, 64, 16, 1), (1, 3, 2500, 4, 512, 64, 0), (3, 1, 20, 8, 64, 8, 1)])
def test_index_over_pages_is_the_contiguous_selection(B, tq, n, hi, k, page, flags):
    c, flat = _filled(B, n, page, 128, seed=n + hi)
    rows = B * tq
    qp = torch.tensor([n - 1 - (tq - 1 - r % tq) for r in range(rows)], device=DEV)
    iq = _rand(11, rows, hi, 128)
    ws = csa.LatentIndexWorkspace(rows, hi, flat.cap)
    a, b = (torch.empty(rows, k, dtype=torch.int32, device=DEV) for _ in range(2))
    csa.csa2_latent_index_topk(flat, B, tq, qp, iq, k, a, ws, flags=flags)
    csa.csa2_paged_index_topk(c, B, tq, qp, iq, k, b, ws, flags=flags)
    assert csa.csa2_get_device_status(ws) == 0
    assert torch.equal(a, b)
    c.table[0, 1] = -1  # entries of a missing page are taken last
    csa.csa2_paged_index_topk(c, B, tq, qp, iq, k, b, ws, flags=flags)
    assert csa.csa2_get_device_status(ws) == csa.CSA2_DEV_BAD_PAGE
    if n - page > k:
        assert not bool(((b[:tq] >= page) & (b[:tq] < 2 * page)).any())


def test_large_cache_offsets_pass_32_bits():
    """A pool of 20 GB of latent rows: entries in its last pages, written and read back."""
    page, pages = 65536, 2
    n_pages = (1 << 31) // 256 // page * 9  # 75 million rows: l_data past 2^34 bytes
    c = csa.PagedCache(n_pages, page, 1, pages, 128, indexer=False,
                       page_table=torch.tensor([[n_pages - 1, 0]], dtype=torch.int32, device=DEV))
    lat = _rand(1, 1, 3, 512)
    csa.csa2_paged_append(c, 1, 3, torch.tensor([page - 2], device=DEV), latent=lat)
    data, scale = R.e2m1_rows(lat[0].cpu().double())
    assert torch.equal(c.l_data[n_pages - 1, -2:].cpu(), data[:2]) and torch.equal(c.l_data[0, 0].cpu(), data[2])
    out = torch.empty(1, 3, 512, device=DEV, dtype=torch.bfloat16)
    idx = torch.tensor([[page - 2, page - 1, page]], dtype=torch.int32, device=DEV)
    csa.csa2_paged_gather(c, 1, idx, out)
    assert torch.equal(out[0].cpu().double(), R.e2m1_values(data, scale))
    q = _rand(2, 1, 64, 512)
    o, of, lse, st = _attend(csa.csa2_paged_attend, c, 1, 1, torch.tensor([page], device=DEV), q, idx[0, :3].view(1, 3), 3, win=0)
    want, want_lse = R.attend(q[0].cpu().double(), R.e2m1_values(data, scale), 512 ** -0.5)
    assert st == 0
    _close(o[0], of[0], lse[0], want, want_lse, float(out.abs().max()))
    del c
    torch.cuda.empty_cache()


def test_capture_and_streams():
    B, t, page = 4, 2, 16
    main, krope = _ropes(True)
    w = 1.0 + 0.1 * _rand(1, 512)
    c, ref = (_cache(B, 8, page, seed=1) for _ in range(2))
    pos = torch.arange(B, device=DEV) * 5
    lat, key, swa = _rand(2, B, t, 512), _rand(3, B, t, 128), _rand(4, B, t, 512)
    q, idx = _rand(5, B, 64, 512), torch.arange(8, dtype=torch.int32, device=DEV).expand(B, 8).contiguous()
    out, want = (torch.empty(B, 64, 512, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa.csa2_paged_append(c, B, t, pos, lat, key, swa, rope=main, idx_rope=krope, w_latent=w)
        csa.csa2_paged_attend(c, B, 1, pos + 1, q, idx, 8, out)
    side = torch.cuda.Stream()
    for seed in (7, 8):
        lat.copy_(_rand(seed, B, t, 512))
        g.replay()
        side.wait_stream(torch.cuda.current_stream())
        csa.csa2_paged_append(ref, B, t, pos, lat, key, swa, rope=main, idx_rope=krope, w_latent=w, stream=side)
        with torch.cuda.stream(side):
            csa.csa2_paged_attend(ref, B, 1, pos + 1, q, idx, 8, want)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(c.l_data, ref.l_data) and torch.equal(c.swa, ref.swa) and torch.equal(out, want)
