// layer_abi.cu -- the extern "C" entry points declared in include/csa2_layer.h: argument checks and
// launches; the work is done by the kernels of rope.cu, fp8.cu, paged.cu, latent.cu and latent_index.cu.
#include <math.h>

#include "csa2_internal.cuh"
#include "csa2_layer.cuh"

using namespace csa2;

namespace {

bool al(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool al16(const void* p) { return al(p, 16); }
csa2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }

#define CSA2_TRY(x)                          \
    do {                                     \
        csa2_status _s = (x);                \
        if (_s != CSA2_OK) return _s;        \
    } while (0)

csa2_status check_rope(const csa2_rope_spec* r, int d) {
    if (r->rot < 0 || (r->rot & 1) || r->offset < 0 || r->rot > d || r->offset > d - r->rot) return CSA2_ERR_INVALID_ARG;
    if (r->layout != CSA2_ROPE_HALF && r->layout != CSA2_ROPE_INTERLEAVED) return CSA2_ERR_INVALID_ARG;
    if (r->transposed != 0 && r->transposed != 1) return CSA2_ERR_INVALID_ARG;
    if (!isfinite(r->mscale) || (r->rot > 0 && (!r->inv_freq || !al(r->inv_freq, 8)))) return CSA2_ERR_INVALID_ARG;
    return CSA2_OK;
}

csa2_status check_heads(const csa2_heads* h, int size, int64_t tokens) {
    if (h->heads < 0 || h->x_token < 0 || h->x_head < 0 || h->out_token < 0 || h->out_head < 0)
        return CSA2_ERR_INVALID_ARG;
    if (h->heads == 0 || tokens == 0) return CSA2_OK;
    if (!h->x || !h->out || !al(h->x, size) || !al(h->out, size) || !al(h->weight, size)) return CSA2_ERR_INVALID_ARG;
    if (h->x == h->out && (h->x_token != h->out_token || h->x_head != h->out_head)) return CSA2_ERR_INVALID_ARG;
    return CSA2_OK;
}

// the checks of csa2_rope and csa2_norm_rope, then their launch
csa2_status do_rotate(const csa2_rope_spec* rope, int dtype, int64_t tokens, int d, const int64_t* pos, float eps,
                      const csa2_heads* q, const csa2_heads* k, bool norm, void* stream) {
    if (dtype != CSA2_BF16 && dtype != CSA2_F32) return CSA2_ERR_INVALID_ARG;
    if (tokens < 0 || !q) return CSA2_ERR_INVALID_ARG;
    if (d < 1 || d > 1024) return CSA2_ERR_UNSUPPORTED_SHAPE;
    if (!(eps >= 0.f) || isinf(eps)) return CSA2_ERR_INVALID_ARG;
    const int size = dtype == CSA2_BF16 ? 2 : 4;
    if (rope) CSA2_TRY(check_rope(rope, d));
    CSA2_TRY(check_heads(q, size, tokens));
    if (k) CSA2_TRY(check_heads(k, size, tokens));
    const int hk = k ? k->heads : 0;
    if ((int64_t)q->heads + hk > 65536) return CSA2_ERR_UNSUPPORTED_SHAPE;
    if (tokens == 0 || q->heads + hk == 0) return CSA2_OK;
    if (rope && rope->rot > 0 && !pos) return CSA2_ERR_INVALID_ARG;
    RotateArgs a{};
    a.q = *q;
    if (k) a.k = *k;
    a.pos = pos;
    a.tokens = tokens;
    a.heads = q->heads + hk;
    a.d = d;
    if (rope) {
        a.inv_freq = rope->inv_freq;
        a.rot = rope->rot;
        a.offset = rope->offset;
        a.layout = rope->layout;
        a.transposed = rope->transposed;
        a.mscale = rope->mscale == 0.f ? 1.f : rope->mscale;
    }
    a.eps = eps;
    a.inv_d = 1.f / (float)d;
    a.in_place = !norm && q->x == q->out;
    return from_cuda(launch_rotate(a, dtype, norm, (cudaStream_t)stream));
}

// planes: 1 = latent, 2 = indexer key, 4 = window
csa2_status check_paged(const csa2_paged_cache* c, int planes, PageMap* pg) {
    if (!c || c->page < 8 || c->page > 65536 || (c->page & (c->page - 1))) return CSA2_ERR_INVALID_ARG;
    if (c->n_pages < 0 || c->max_pages < 0) return CSA2_ERR_INVALID_ARG;
    if (c->n_pages > 0x7FFFFFFFll / c->page || c->max_pages > (1ll << 30) / c->page) return CSA2_ERR_CAPACITY;
    *pg = PageMap{c->table, c->swa_slot, c->n_pages, c->max_pages, c->n_slots, 0};
    while ((1 << pg->shift) < c->page) ++pg->shift;
    if ((planes & 3) && (!c->table || !al(c->table, 4))) return CSA2_ERR_INVALID_ARG;
    if ((planes & 1) && (!c->l_data || !c->l_scale || !al16(c->l_data) || !al16(c->l_scale))) return CSA2_ERR_INVALID_ARG;
    if ((planes & 2) && (!c->k_data || !c->k_scale || !al16(c->k_data) || !al16(c->k_scale))) return CSA2_ERR_INVALID_ARG;
    if (planes & 4) {
        if (!c->swa || !al16(c->swa) || c->n_slots < 0 || !al(c->swa_slot, 4)) return CSA2_ERR_INVALID_ARG;
        if (c->swa_cap <= 0 || (c->swa_cap & (c->swa_cap - 1))) return CSA2_ERR_INVALID_ARG;
        if (c->swa_cap > (1ll << 30)) return CSA2_ERR_CAPACITY;
    }
    return CSA2_OK;
}

csa2_latent_cache planes_of(const csa2_paged_cache* c) {
    return csa2_latent_cache{c->l_data, c->l_scale, c->k_data, c->k_scale, c->swa, c->max_pages * c->page, c->swa_cap};
}

csa2_status append_row(const csa2_append_row* r, int channels, AppendRow* out) {
    if (!r || !r->x) return CSA2_OK;  // not appended
    if (!al16(r->x) || !al16(r->weight) || r->x_batch < 0 || r->x_token < 0 || r->x_batch % 8 || r->x_token % 8)
        return CSA2_ERR_INVALID_ARG;
    out->x = r->x;
    out->x_batch = r->x_batch;
    out->x_token = r->x_token;
    out->weight = r->weight;
    if (r->rope) {
        CSA2_TRY(check_rope(r->rope, channels));
        if (r->rope->transposed) return CSA2_ERR_INVALID_ARG;
        out->inv_freq = r->rope->rot > 0 ? r->rope->inv_freq : nullptr;
        out->rot = r->rope->rot;
        out->offset = r->rope->offset;
        out->layout = r->rope->layout;
        out->mscale = r->rope->mscale == 0.f ? 1.0 : (double)r->rope->mscale;
    }
    return CSA2_OK;
}

}  // namespace

extern "C" {

csa2_status csa2_rope_frequencies(int rot, double base, int kind, double factor, int64_t orig_ctx, double beta_fast,
                                  double beta_slow, double* inv_freq, float* mscale) {
    if (rot < 0 || (rot & 1) || !(base > 1.0) || !isfinite(base) || !(factor >= 1.0) || !isfinite(factor) || !mscale ||
        (rot > 0 && !inv_freq))
        return CSA2_ERR_INVALID_ARG;
    if (kind < CSA2_ROPE_PLAIN || kind > CSA2_ROPE_YARN) return CSA2_ERR_INVALID_ARG;
    *mscale = 1.f;
    double lo = 0.0, hi = 0.0;
    if (kind == CSA2_ROPE_NTK) {
        if (rot == 2 && factor != 1.0) return CSA2_ERR_INVALID_ARG;  // one pair: the rule has no exponent
        if (rot > 2) base *= pow(factor, (double)rot / (rot - 2));
    } else if (kind == CSA2_ROPE_YARN) {
        if (orig_ctx < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast))
            return CSA2_ERR_INVALID_ARG;
        // the channel pair that turns `beta` times in orig_ctx positions
        const double k = rot / (2.0 * log(base)), two_pi = 6.283185307179586477;
        lo = floor(k * log(orig_ctx / (beta_fast * two_pi)));
        hi = ceil(k * log(orig_ctx / (beta_slow * two_pi)));
        lo = lo > 0.0 ? lo : 0.0;
        hi = hi < rot - 1 ? hi : rot - 1;
        if (hi <= lo) hi = lo + 0.001;
        *mscale = (float)(0.1 * log(factor) + 1.0);
    }
    for (int j = 0; j < rot / 2; ++j) {
        double f = pow(base, -2.0 * j / rot);
        if (kind == CSA2_ROPE_LINEAR) f /= factor;
        if (kind == CSA2_ROPE_YARN) {
            double slow = (j - lo) / (hi - lo);
            slow = slow < 0.0 ? 0.0 : (slow > 1.0 ? 1.0 : slow);
            f = f / factor * slow + f * (1.0 - slow);
        }
        inv_freq[j] = f;
    }
    return CSA2_OK;
}

csa2_status csa2_rope(const csa2_rope_spec* rope, int dtype, int64_t tokens, int d, const int64_t* pos,
                      const csa2_heads* h, void* stream) {
    if (!rope || !h || h->weight) return CSA2_ERR_INVALID_ARG;
    return do_rotate(rope, dtype, tokens, d, pos, 0.f, h, nullptr, false, stream);
}

csa2_status csa2_norm_rope(const csa2_rope_spec* rope, int dtype, int64_t tokens, int d, const int64_t* pos, float eps,
                           const csa2_heads* q, const csa2_heads* k, void* stream) {
    return do_rotate(rope, dtype, tokens, d, pos, eps, q, k, true, stream);
}

csa2_status csa2_fp8_quantize(int64_t rows, int k, const uint16_t* x, int64_t x_stride, uint8_t* data, float* scale,
                              void* stream) {
    if (rows < 0 || k <= 0 || k % 16 || x_stride < 0 || x_stride % 8) return CSA2_ERR_INVALID_ARG;
    if (rows == 0) return CSA2_OK;
    if (!x || !data || !scale || !al16(x) || !al16(data) || !al(scale, 4)) return CSA2_ERR_INVALID_ARG;
    if (rows > 0x7FFFFFFF || k > (1 << 23)) return CSA2_ERR_UNSUPPORTED_SHAPE;
    return from_cuda(launch_fp8_rows(rows, k, x, x_stride, data, scale, (cudaStream_t)stream));
}

csa2_status csa2_fp8_quantize_weight(int64_t n, int k, const uint16_t* w, uint8_t* data, float* scale, void* stream) {
    if (n < 0 || k <= 0 || k % 16) return CSA2_ERR_INVALID_ARG;
    if (n == 0) return CSA2_OK;
    if (!w || !data || !scale || !al16(w) || !al16(data) || !al(scale, 4)) return CSA2_ERR_INVALID_ARG;
    if (n > 65535ll * 128 || k > (1 << 23)) return CSA2_ERR_UNSUPPORTED_SHAPE;
    return from_cuda(launch_fp8_weight(n, k, w, data, scale, (cudaStream_t)stream));
}

csa2_status csa2_fp8_gemm(int64_t m, int64_t n, int k, const uint8_t* x, const float* xs, const uint8_t* w,
                          const float* ws, int out_dtype, void* out, int64_t out_stride, void* status,
                          size_t status_bytes, void* stream) {
    if (m < 0 || n < 0 || k <= 0 || k % 16 || out_stride < n) return CSA2_ERR_INVALID_ARG;
    if (out_dtype != CSA2_BF16 && out_dtype != CSA2_F32) return CSA2_ERR_INVALID_ARG;
    if (m > 0x7FFFFFFF || n > 0x7FFFFFFF || k > (1 << 23)) return CSA2_ERR_UNSUPPORTED_SHAPE;
    if (status && status_bytes < 256) return CSA2_ERR_WORKSPACE;
    if (m == 0 || n == 0) return CSA2_OK;
    if (!x || !xs || !w || !ws || !out || !al16(x) || !al16(w) || !al(xs, 4) || !al(ws, 4) ||
        !al(out, out_dtype == CSA2_BF16 ? 2 : 4))
        return CSA2_ERR_INVALID_ARG;
    Fp8GemmArgs a{};
    a.m = m;
    a.n = n;
    a.k = k;
    a.x = x;
    a.xs = xs;
    a.w = w;
    a.ws = ws;
    a.out = out;
    a.out_stride = out_stride;
    a.out_f32 = out_dtype == CSA2_F32;
    a.status = reinterpret_cast<uint32_t*>(status);
    return from_cuda(launch_fp8_gemm(a, (cudaStream_t)stream));
}

csa2_status csa2_paged_append(const csa2_paged_cache* cache, int batch, int t, const int64_t* pos, const int32_t* len,
                              const int64_t* rpos, float eps, const csa2_append_row* latent,
                              const csa2_append_row* idx_k, const csa2_append_row* swa, void* ws, size_t ws_bytes,
                              void* stream) {
    if (batch < 0 || t < 0 || !(eps >= 0.f) || isinf(eps)) return CSA2_ERR_INVALID_ARG;
    PagedAppendArgs a{};
    CSA2_TRY(append_row(latent, kLatD, &a.row[0]));
    CSA2_TRY(append_row(idx_k, 128, &a.row[1]));
    CSA2_TRY(append_row(swa, kLatD, &a.row[2]));
    CSA2_TRY(check_paged(cache, (a.row[0].x ? 1 : 0) | (a.row[1].x ? 2 : 0) | (a.row[2].x ? 4 : 0), &a.pg));
    if (ws && ws_bytes < 256) return CSA2_ERR_WORKSPACE;
    if (batch == 0 || t == 0 || (!a.row[0].x && !a.row[1].x && !a.row[2].x)) return CSA2_OK;
    if (!pos || !al(pos, 8) || !al(len, 4) || !al(rpos, 8)) return CSA2_ERR_INVALID_ARG;
    a.c = *cache;
    a.batch = batch;
    a.t = t;
    a.pos = pos;
    a.len = len;
    a.rpos = rpos;
    a.eps = (double)eps;
    a.status = reinterpret_cast<uint32_t*>(ws);
    for (int i = 0; i < 3; ++i)
        if (a.row[i].x) a.kind[a.kinds++] = i;
    return from_cuda(launch_paged_append(a, (cudaStream_t)stream));
}

csa2_status csa2_paged_gather(const csa2_paged_cache* cache, int batch, int n, const int32_t* idx, uint16_t* latent,
                              uint16_t* key, void* ws, size_t ws_bytes, void* stream) {
    if (batch < 0 || n < 0) return CSA2_ERR_INVALID_ARG;
    PagedGatherArgs a{};
    CSA2_TRY(check_paged(cache, (latent ? 1 : 0) | (key ? 2 : 0), &a.pg));
    if (!al16(latent) || !al16(key)) return CSA2_ERR_INVALID_ARG;
    if (ws && ws_bytes < 256) return CSA2_ERR_WORKSPACE;
    if (batch == 0 || n == 0 || (!latent && !key)) return CSA2_OK;
    if (!idx || !al(idx, 4)) return CSA2_ERR_INVALID_ARG;
    a.c = *cache;
    a.rows = (int64_t)batch * n;
    a.n = n;
    a.idx = idx;
    a.latent = latent;
    a.key = key;
    a.status = reinterpret_cast<uint32_t*>(ws);
    return from_cuda(launch_paged_gather(a, (cudaStream_t)stream));
}

csa2_status csa2_paged_attend(const csa2_paged_cache* cache, int batch, int tq, const int64_t* qpos, const uint16_t* q,
                              const int32_t* idx, int k, const int64_t* swa_begin, int win, int ratio, float sm_scale,
                              uint16_t* out, float* out_f32, float* lse, void* ws, size_t ws_bytes, void* stream) {
    if (batch < 0 || tq < 1 || k < 0 || k > kMaxK) return CSA2_ERR_INVALID_ARG;
    if (win < 0 || win > 128 || (ratio != 1 && ratio != 2)) return CSA2_ERR_UNSUPPORTED_SHAPE;
    if (!(sm_scale >= 0.f) || isinf(sm_scale)) return CSA2_ERR_INVALID_ARG;
    LatentAttendArgs a{};
    CSA2_TRY(check_paged(cache, (k > 0 ? 1 : 0) | (win > 0 ? 4 : 0), &a.pg));
    if (win > 0 && cache->swa_cap < win) return CSA2_ERR_CAPACITY;  // the ring must hold the window
    if (ws && ws_bytes < 256) return CSA2_ERR_WORKSPACE;
    if ((long long)batch * tq > (1ll << 31) - 1) return CSA2_ERR_INVALID_ARG;
    if (batch == 0) return CSA2_OK;
    if (!qpos || !q || !out || (k > 0 && !idx) || !al16(q) || !al16(out) || !al16(out_f32) || !al(lse, 4) ||
        !al(qpos, 8) || !al(idx, 4) || !al(swa_begin, 8))
        return CSA2_ERR_INVALID_ARG;
    a.c = planes_of(cache);
    a.rows = batch * tq;
    a.tq = tq;
    a.k = k;
    a.win = win;
    a.ratio = ratio;
    a.qpos = qpos;
    a.swa_begin = swa_begin;
    a.q = q;
    a.idx = idx;
    a.sm_scale = sm_scale == 0.f ? 1.0f / sqrtf((float)kLatD) : sm_scale;
    a.out = out;
    a.out_f32 = out_f32;
    a.lse = lse;
    a.status = reinterpret_cast<uint32_t*>(ws);
    return from_cuda(launch_paged_attend(a, (cudaStream_t)stream));
}

csa2_status csa2_paged_index_topk(const csa2_paged_cache* cache, int batch, int tq, const int64_t* qpos,
                                  const uint16_t* idx_q, int hi, int k, int ratio, int64_t max_ctx, uint32_t flags,
                                  int32_t* out_idx, void* ws, size_t ws_bytes, void* stream) {
    if (batch < 0 || tq < 1 || hi < 1 || hi > kLatMaxHI || k < 1 || k > kMaxK || max_ctx < 1) return CSA2_ERR_INVALID_ARG;
    if (ratio != 1 && ratio != 2) return CSA2_ERR_UNSUPPORTED_SHAPE;
    if ((long long)batch * tq > 65535 || (flags & ~CSA2_SCORE_RELU)) return CSA2_ERR_INVALID_ARG;
    LatIndexArgs a{};
    CSA2_TRY(check_paged(cache, 2, &a.pg));
    const int rows = batch * tq;
    if (rows == 0) return CSA2_OK;
    if (!qpos || !idx_q || !out_idx || !al16(idx_q) || !al(qpos, 8) || !al(out_idx, 4)) return CSA2_ERR_INVALID_ARG;
    if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < latent_index_ws_bytes(rows, hi, max_ctx)) return CSA2_ERR_WORKSPACE;
    a.c = planes_of(cache);
    a.rows = rows;
    a.tq = tq;
    a.hi = hi;
    a.k = k;
    a.ratio = ratio;
    a.max_ctx = max_ctx;
    a.qpos = qpos;
    a.flags = flags;
    a.out_idx = out_idx;
    return from_cuda(launch_latent_index(a, true, idx_q, reinterpret_cast<unsigned char*>(ws), (cudaStream_t)stream));
}

}  // extern "C"
