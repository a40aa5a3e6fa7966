"""The operators around the core run together, as a layer of the pages' own shape is served: FP8 projections,
norms and rotations, the paged append, the selection, the attention, the output turned back and the
output projection; a prompt, then single tokens of several sequences, eagerly and as a captured graph.

Each step is held to its formula on the inputs it had (tolerances: those of the operators' own tests), so
that a wrong layout, stride, position or order between two of them shows.
"""
import pytest
import torch

import _layer_ref as R
import compressed_sparse_attention_append_b200 as csa

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
HIDDEN, HQ, D, HI, K, PAGE = 1024, 64, 512, 32, 128, 16
PARTS = (("q", HQ * D), ("latent", D), ("idx_q", HI * 128), ("idx_k", 128), ("swa", D))


def _rand(seed, *shape, sigma=1.0):
    return (sigma * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).to(DEV)


class Layer:
    """One layer's weights and cache, and a step of it, in the calls that a user's program makes."""

    def __init__(self, batch, pages, seed=0):
        n = sum(w for _, w in PARTS)
        self.w_in, self.s_in = self._weights(_rand(seed, n, HIDDEN, sigma=HIDDEN ** -0.5))
        self.w_out, self.s_out = self._weights(_rand(seed + 1, HIDDEN, HQ * D, sigma=(HQ * D) ** -0.5))
        self.norm = {k: 1.0 + 0.1 * _rand(seed + 2 + i, w) for i, (k, w) in
                     enumerate((("q", D), ("latent", D), ("idx_q", 128), ("idx_k", 128), ("swa", D)))}
        self.rope = csa.Rope.for_context(64, 10000.0, "yarn", 16.0, 4096, offset=D - 64, interleaved=True)
        self.idx_rope = csa.Rope.for_context(64, 10000.0, offset=64, interleaved=True)
        self.back = self.rope.transposed()
        table = torch.randperm(batch * pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.cache = csa.PagedCache(batch * pages, PAGE, batch, pages, 256, page_table=table.view(batch, pages).to(DEV))
        self.batch, self.ctx = batch, pages * PAGE

    @staticmethod
    def _weights(w):
        n, k = w.shape
        q = torch.empty(n, k, device=DEV, dtype=torch.float8_e4m3fn)
        s = torch.empty(-(-n // 128), -(-k // 128), device=DEV)
        csa.csa2_fp8_quantize_weight(w, q, s)
        return q, s

    def buffers(self, t):
        rows = self.batch * t
        e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, device=DEV, dtype=dtype)
        return {"hq": e(rows, HIDDEN, dtype=torch.float8_e4m3fn), "hs": e(HIDDEN // 128, rows, dtype=torch.float32),
                "proj": e(rows, sum(w for _, w in PARTS)), "qr": e(rows, HQ, D), "iq": e(rows, HI, 128),
                "idx": e(rows, K, dtype=torch.int32), "att": e(rows, HQ, D), "back": e(rows, HQ, D),
                "oq": e(rows, HQ * D, dtype=torch.float8_e4m3fn), "os": e(HQ * D // 128, rows, dtype=torch.float32),
                "out": e(rows, HIDDEN), "ws": csa.LatentIndexWorkspace(rows, HI, self.ctx)}

    def step(self, b, hidden, pos, t):
        """hidden [batch * t, HIDDEN] at tokens pos [batch] .. pos + t - 1."""
        rows = self.batch * t
        at = (pos[:, None] + torch.arange(t, device=DEV)).flatten()
        csa.csa2_fp8_quantize(hidden, b["hq"], b["hs"])
        csa.csa2_fp8_gemm(b["hq"], b["hs"], self.w_in, self.s_in, b["proj"])
        part, off = {}, 0
        for name, w in PARTS:
            part[name] = b["proj"][:, off:off + w]
            off += w
        csa.csa2_norm_rope(self.rope, at, EPS, part["q"].view(rows, HQ, D), self.norm["q"], b["qr"])
        csa.csa2_norm_rope(self.idx_rope, at, EPS, part["idx_q"].view(rows, HI, 128), self.norm["idx_q"], b["iq"])
        seq = lambda x: x.view(self.batch, t, -1)
        csa.csa2_paged_append(self.cache, self.batch, t, pos, seq(part["latent"]), seq(part["idx_k"]), seq(part["swa"]),
                              rope=self.rope, idx_rope=self.idx_rope, w_latent=self.norm["latent"],
                              w_idx_k=self.norm["idx_k"], w_swa=self.norm["swa"], eps=EPS, ws=b["ws"])
        csa.csa2_paged_index_topk(self.cache, self.batch, t, at, b["iq"], K, b["idx"], b["ws"], flags=csa.CSA2_SCORE_RELU)
        csa.csa2_paged_attend(self.cache, self.batch, t, at, b["qr"], b["idx"], K, b["att"], ws=b["ws"])
        csa.csa2_rope(self.back, at, b["att"], b["back"])
        csa.csa2_fp8_quantize(b["back"].view(rows, -1), b["oq"], b["os"])
        csa.csa2_fp8_gemm(b["oq"], b["os"], self.w_out, self.s_out, b["out"], status=b["ws"])
        return part, at


def _near(got, want, tol):
    err = (got.detach().cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def _product(x, xs, w, ws, out):
    a, b = R.fp8_values(x, row_scale=xs).to(DEV), R.fp8_values(w, block_scale=ws).to(DEV)
    want, size = a @ b.T, a.abs() @ b.abs().T
    _near(out, want.cpu(), (want.abs() * 2.0 ** -8 + size * 2.0 ** -15).cpu())


def _check(L, b, part, at, pos, t):
    rows = L.batch * t
    assert csa.csa2_get_device_status(b["ws"]) == 0
    _product(b["hq"], b["hs"], L.w_in, L.s_in, b["proj"])
    for name, heads, d, got, rope in (("q", HQ, D, b["qr"], L.rope), ("idx_q", HI, 128, b["iq"], L.idx_rope)):
        want, size = R.rotate(R.norm(part[name].reshape(rows, heads, d), L.norm[name], EPS), at, rope.inv_freq, rope.offset,
                              True, rope.mscale)
        _near(got, want, want.abs() * 2.0 ** -8 + size * 2.0 ** -18)
    c = L.cache
    for r in range(rows):
        s, p = r // t, int(at[r])
        page, slot = c.table[s, p // PAGE].long(), p % PAGE
        eps = float(torch.tensor(EPS, dtype=torch.float32))
        one = lambda name, rope: R.rotate(R.norm(part[name][r:r + 1], L.norm[name], eps)[:, None], at[r:r + 1], rope.inv_freq,
                                          rope.offset, True, rope.mscale)[0][:, 0]
        data, scale = R.e2m1_rows(one("latent", L.rope))
        assert torch.equal(c.l_data[page, slot].cpu(), data[0]) and torch.equal(c.l_scale[page, slot].cpu(), scale[0])
        data, scale = R.mx_rows(one("idx_k", L.idx_rope))
        assert torch.equal(c.k_data[page, slot].cpu(), data[0]) and torch.equal(c.k_scale[page, slot].cpu(), scale[0])
        assert torch.equal(c.swa[s, p % 256].cpu(), R.e4m3_rows(one("swa", L.rope))[0])
    # the selection: that of the contiguous indexer over the same keys
    flat = csa.LatentCache(L.batch, L.ctx, 128, latent=False)
    flat.k_data.copy_(c.k_data[c.table.long()].view(L.batch, L.ctx, 64))
    flat.k_scale.copy_(c.k_scale[c.table.long()].view(L.batch, L.ctx, 4))
    idx = torch.empty_like(b["idx"])
    csa.csa2_latent_index_topk(flat, L.batch, t, at, b["iq"], K, idx, csa.LatentIndexWorkspace(rows, HI, L.ctx),
                               flags=csa.CSA2_SCORE_RELU)
    assert torch.equal(b["idx"], idx)
    for r in sorted({0, 1, rows // 2, rows - 1}):
        s, p = r // t, int(at[r])
        e = idx[r][idx[r] >= 0].long()
        assert e.numel() == min(K, p + 1)
        page = c.table[s, e // PAGE].long()
        keys = R.e2m1_values(c.l_data[page, e % PAGE], c.l_scale[page, e % PAGE])
        w = torch.arange(max(0, p - 127), p + 1)
        keys = torch.cat([keys, c.swa[s, (w % 256).to(DEV)].cpu().view(torch.float8_e4m3fn).double()])
        want, _ = R.attend(b["qr"][r].cpu().double(), keys, D ** -0.5)
        _near(b["att"][r], want, want.abs() * 2.0 ** -8 + float(keys.abs().max()) * (2.0 ** -11 + 2.0 ** -12))
    want, size = R.rotate(b["att"], at, L.back.inv_freq, D - 64, True, L.back.mscale, True)
    _near(b["back"], want, want.abs() * 2.0 ** -8 + size * 2.0 ** -18)
    _product(b["oq"], b["os"], L.w_out, L.s_out, b["out"])


def test_a_layer_serves_a_prompt_and_single_tokens():
    batch, t = 3, 40
    L = Layer(batch, 16)
    pos = torch.tensor([0, 0, 0], device=DEV)
    b = L.buffers(t)
    part, at = L.step(b, _rand(50, batch * t, HIDDEN), pos, t)
    _check(L, b, part, at, pos, t)
    pos = pos + t
    one = L.buffers(1)
    hidden = _rand(51, batch, HIDDEN)
    part, at = L.step(one, hidden, pos, 1)
    _check(L, one, part, at, pos, 1)
    # the same step captured: replayed on other tokens it gives what the eager calls give
    graph, hidden_in, pos_in, got = torch.cuda.CUDAGraph(), torch.empty_like(hidden), torch.empty_like(pos), L.buffers(1)
    hidden_in.copy_(hidden)
    pos_in.copy_(pos)
    with torch.cuda.graph(graph):
        L.step(got, hidden_in, pos_in, 1)
    for n in range(1, 4):
        hidden_in.copy_(_rand(60 + n, batch, HIDDEN))
        pos_in.copy_(pos + n)
        graph.replay()
        L.step(one, hidden_in, pos_in, 1)
        for k in ("idx", "att", "out"):
            assert torch.equal(got[k], one[k]), k
    part, at = L.step(one, hidden_in, pos_in, 1)
    _check(L, one, part, at, pos_in, 1)
