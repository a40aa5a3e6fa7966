// rope.cu -- rotary positions, alone and after the norm of each head (csa2_rope, csa2_norm_rope).
//
// y = R_pos(x * w / sqrt(mean(x^2) + eps)): pair j of the rotated channels turns by t = pos * f_j,
//   (a, b) -> m (a cos t - b sin t, b cos t + a sin t).
// The angle is a 64-bit product (a far position times a frequency loses whole radians in 32 bits),
// reduced to half turns in 64 bits and handed to sincospif, whose argument then lies in [-1, 1].
// Everything else is fp32, rounded once when it is stored.
//
// Both calls move each row once and compute little, so device memory bounds them. Split: a block
// takes a few rows (a row: one head of one token), each row on 1 .. 32 lanes with 1 .. 8 vectors of
// 16 (or 8) bytes per lane, all loads of the block's rows in flight before the sines and cosines
// are formed; these are shared by the block's heads of a token through shared memory. A channel whose
// partner sits in another vector (CSA2_ROPE_HALF) reads that vector too: it is in L1, since
// the row's own lanes have just asked for it.
#include "csa2_internal.cuh"
#include "csa2_layer.cuh"

namespace csa2 {

namespace {

constexpr int kThr = 256;
constexpr double kInvPi = 0.31830988618379067154;

// cos and sin of pos * f (radians)
__device__ __forceinline__ float2 turn(int64_t pos, double f, float mscale, int transposed) {
    double h = ((double)pos * f) * kInvPi;  // half turns
    h -= 2.0 * rint(0.5 * h);
    float s, c;
    sincospif((float)h, &s, &c);
    return make_float2(c * mscale, (transposed ? -s : s) * mscale);
}

template <int VB>
struct alignas(VB) Vec {
    uint32_t w[VB / 4];
};

template <typename T, int VB>
__device__ __forceinline__ void unpack(const Vec<VB>& v, float* f) {
#pragma unroll
    for (int i = 0; i < VB / 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            f[2 * i] = __uint_as_float(v.w[i] << 16);
            f[2 * i + 1] = __uint_as_float(v.w[i] & 0xFFFF0000u);
        } else {
            f[i] = __uint_as_float(v.w[i]);
        }
    }
}
template <typename T, int VB>
__device__ __forceinline__ Vec<VB> pack(const float* f) {
    Vec<VB> v;
#pragma unroll
    for (int i = 0; i < VB / 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            v.w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            v.w[i] = __float_as_uint(f[i]);
        }
    }
    return v;
}

// One row per group of a.lanes lanes, CPL vectors per lane, ITER rows per group.
template <typename T, int VB, int CPL, int ITER, bool NORM>
__global__ void __launch_bounds__(kThr) rotate_kernel(RotateArgs a) {
    constexpr int E = VB / (int)sizeof(T);
    using V = Vec<VB>;
    extern __shared__ float2 cs[];  // [tokens of the block][rot / 2]
    const int tid = threadIdx.x, lanes = a.lanes, per = kThr / lanes;
    const int gl = tid & (lanes - 1), gr = tid / lanes;
    const int64_t tok0 = (int64_t)(blockIdx.x / (unsigned)a.hblocks) * a.tb;
    const int head0 = (int)(blockIdx.x % (unsigned)a.hblocks) * a.hb;
    const int ntok = (int)(a.tokens - tok0 < a.tb ? a.tokens - tok0 : a.tb);
    const int nh = a.heads - head0 < a.hb ? a.heads - head0 : a.hb;
    const int nrows = ntok * nh, half = a.rot >> 1, nc = a.d / E;
    wait_prior_grid();

    V x[ITER][CPL], p[ITER][CPL];
    int tl[ITER];
    T* out[ITER];
    const T* wt[ITER];
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
        const int row = it * per + gr;
        out[it] = nullptr;
        tl[it] = 0;
        wt[it] = nullptr;
        if (row >= nrows) continue;
        tl[it] = row / nh;
        const int hh = head0 + row % nh;
        const int64_t tok = tok0 + tl[it];
        if (a.pos && a.pos[tok] < 0) continue;  // padding: nothing written
        const bool isq = hh < a.q.heads;
        const csa2_heads& H = isq ? a.q : a.k;
        const int64_t h = isq ? hh : hh - a.q.heads;
        const T* src = reinterpret_cast<const T*>(H.x) + tok * H.x_token + h * H.x_head;
        out[it] = reinterpret_cast<T*>(H.out) + tok * H.out_token + h * H.out_head;
        wt[it] = reinterpret_cast<const T*>(H.weight);
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const int ch = gl + c * lanes, r = ch * E - a.offset;  // first channel, within the rotated range
            const bool turned = r >= 0 && r < a.rot;
            if (ch < nc && (turned || !a.in_place)) x[it][c] = *reinterpret_cast<const V*>(src + ch * E);
            if (ch < nc && turned && a.layout == CSA2_ROPE_HALF)
                p[it][c] = *reinterpret_cast<const V*>(src + ch * E + (r < half ? half : -half));
        }
    }
    for (int i = tid; i < ntok * half; i += kThr)
        cs[i] = turn(a.pos[tok0 + i / half], a.inv_freq[i % half], a.mscale, a.transposed);
    __syncthreads();  // the table; also: every row of the block is loaded before one is stored (out == x)

#pragma unroll
    for (int it = 0; it < ITER; ++it) {
        float r = 1.f;
        if constexpr (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                if (out[it] && gl + c * lanes < nc) {
                    float f[E];
                    unpack<T, VB>(x[it][c], f);
#pragma unroll
                    for (int e = 0; e < E; ++e) ss = fmaf(f[e], f[e], ss);
                }
            }
            for (int o = lanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = rsqrtf(ss * a.inv_d + a.eps);
        }
        if (!out[it]) continue;
        const float2* t = cs + tl[it] * half;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const int ch = gl + c * lanes, k = ch * E - a.offset;
            const bool turned = k >= 0 && k < a.rot;
            if (ch >= nc || (!turned && a.in_place)) continue;
            float f[E];
            unpack<T, VB>(x[it][c], f);
            auto weigh = [&](float* v, int at) {
                if constexpr (NORM) {
                    if (wt[it]) {
                        float w[E];
                        unpack<T, VB>(*reinterpret_cast<const V*>(wt[it] + at), w);
#pragma unroll
                        for (int e = 0; e < E; ++e) v[e] *= r * w[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < E; ++e) v[e] *= r;
                    }
                }
            };
            weigh(f, ch * E);
            if (turned) {
                if (a.layout == CSA2_ROPE_HALF) {
                    float g[E];
                    unpack<T, VB>(p[it][c], g);
                    const bool first = k < half;
                    weigh(g, ch * E + (first ? half : -half));
                    const float2* u = t + (first ? k : k - half);
#pragma unroll
                    for (int e = 0; e < E; ++e) f[e] = fmaf(f[e], u[e].x, first ? -g[e] * u[e].y : g[e] * u[e].y);
                } else {
                    const float2* u = t + (k >> 1);
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float2 v = u[e >> 1];
                        const float y0 = fmaf(f[e], v.x, -f[e + 1] * v.y);
                        f[e + 1] = fmaf(f[e + 1], v.x, f[e] * v.y);
                        f[e] = y0;
                    }
                }
            }
            *reinterpret_cast<V*>(out[it] + ch * E) = pack<T, VB>(f);
        }
    }
}

__device__ __forceinline__ float ld(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ void st(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ void st(float* p, float v) { *p = v; }

// Rows that allow no vectors: a warp per row, one element (or pair) per lane and step.
template <typename T, bool NORM>
__global__ void __launch_bounds__(kThr) rotate_scalar_kernel(RotateArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (kThr / 32) + (threadIdx.x >> 5);
    wait_prior_grid();
    if (row >= a.tokens * a.heads) return;
    const int64_t tok = row / a.heads;
    const int hh = (int)(row % a.heads);
    const int64_t pos = a.pos ? a.pos[tok] : 0;
    if (pos < 0) return;
    const bool isq = hh < a.q.heads;
    const csa2_heads& H = isq ? a.q : a.k;
    const int64_t h = isq ? hh : hh - a.q.heads;
    const T* src = reinterpret_cast<const T*>(H.x) + tok * H.x_token + h * H.x_head;
    T* out = reinterpret_cast<T*>(H.out) + tok * H.out_token + h * H.out_head;
    const T* wt = reinterpret_cast<const T*>(H.weight);
    float r = 1.f;
    if constexpr (NORM) {
        float ss = 0.f;
        for (int i = lane; i < a.d; i += 32) ss = fmaf(ld(src + i), ld(src + i), ss);
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = rsqrtf(ss * a.inv_d + a.eps);
        __syncwarp();  // the row is read whole before any of it is written (out == x)
    }
    auto value = [&](int i) { return NORM ? ld(src + i) * (wt ? r * ld(wt + i) : r) : ld(src + i); };
    // every element belongs to one lane and is read by it alone before it is written
    const int half = a.rot >> 1;
    for (int j = lane; j < half; j += 32) {
        const int ia = a.offset + (a.layout == CSA2_ROPE_HALF ? j : 2 * j);
        const int ib = ia + (a.layout == CSA2_ROPE_HALF ? half : 1);
        const float2 t = turn(pos, a.inv_freq[j], a.mscale, a.transposed);
        const float u = value(ia), v = value(ib);
        st(out + ia, fmaf(u, t.x, -v * t.y));
        st(out + ib, fmaf(v, t.x, u * t.y));
    }
    if (a.in_place) return;
    for (int i = lane; i < a.d; i += 32)
        if (i < a.offset || i >= a.offset + a.rot) st(out + i, value(i));
}

int ceil_pow2(int x) {
    int p = 1;
    while (p < x) p <<= 1;
    return p;
}

template <typename T, int VB, int CPL, int ITER, bool NORM>
cudaError_t launch_vec(RotateArgs a, cudaStream_t s) {
    const int rows = kThr / a.lanes * ITER;  // per block
    if (a.heads >= rows) {
        a.tb = 1;
        a.hb = rows;
    } else {
        a.tb = rows / a.heads;
        a.hb = a.heads;
    }
    a.hblocks = (a.heads + a.hb - 1) / a.hb;
    const int64_t grid = (a.tokens + a.tb - 1) / a.tb * a.hblocks;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    // at most 32 KB: tb * rot / 2 <= rows * d / 2 <= 256 / lanes * ITER * lanes * CPL * E / 2 pairs,
    // ITER * CPL * E <= 32
    const size_t smem = (size_t)a.tb * (a.rot / 2) * sizeof(float2);
    return launch_after_prior(rotate_kernel<T, VB, CPL, ITER, NORM>, dim3((unsigned)grid), dim3(kThr), smem, s, a);
}

template <typename T, int VB, bool NORM>
cudaError_t launch_rows(RotateArgs a, cudaStream_t s) {
    const int nc = a.d / (VB / (int)sizeof(T));
    a.lanes = nc < 32 ? ceil_pow2(nc) : 32;
    // several rows per group where the blocks still fill the GPU (about eight of 256 threads an SM);
    // below that a block does less, for latency
    const bool many = a.tokens * a.heads >= (int64_t)148 * 8 * (kThr / a.lanes) * 2;
    if (nc <= 32) return many ? launch_vec<T, VB, 1, 4, NORM>(a, s) : launch_vec<T, VB, 1, 1, NORM>(a, s);
    if (nc <= 64) return many ? launch_vec<T, VB, 2, 2, NORM>(a, s) : launch_vec<T, VB, 2, 1, NORM>(a, s);
    if (nc <= 128) return launch_vec<T, VB, 4, 1, NORM>(a, s);
    return launch_vec<T, VB, 8, 1, NORM>(a, s);
}

template <typename T, bool NORM>
cudaError_t launch_typed(const RotateArgs& a, cudaStream_t s) {
    // the widest vectors that every row, and both channels of every pair, allow
    auto fits = [&](int vb) {
        const int e = vb / (int)sizeof(T);
        const int run = a.rot == 0 ? 0 : (a.layout == CSA2_ROPE_HALF ? a.rot / 2 : a.rot);
        if (a.d % e || (a.d / e) > 256 || (run && (run % e || a.offset % e))) return false;
        for (const csa2_heads* h : {&a.q, &a.k}) {
            if (!h->heads) continue;
            for (const void* p : {h->x, (const void*)h->out, h->weight})
                if ((uintptr_t)p % vb) return false;
            for (int64_t st : {h->x_token, h->x_head, h->out_token, h->out_head})
                if (st % e) return false;
        }
        return true;
    };
    if (fits(16)) return launch_rows<T, 16, NORM>(a, s);
    if (fits(8)) return launch_rows<T, 8, NORM>(a, s);
    const int64_t grid = (a.tokens * a.heads + kThr / 32 - 1) / (kThr / 32);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_after_prior(rotate_scalar_kernel<T, NORM>, dim3((unsigned)grid), dim3(kThr), 0, s, a);
}

}  // namespace

cudaError_t launch_rotate(const RotateArgs& a, int dtype, bool norm, cudaStream_t s) {
    if (dtype == CSA2_BF16) return norm ? launch_typed<uint16_t, true>(a, s) : launch_typed<uint16_t, false>(a, s);
    return norm ? launch_typed<float, true>(a, s) : launch_typed<float, false>(a, s);
}

}  // namespace csa2
