// rope.cu -- rotary positions, alone and after the norm of each head (csa2_rope, csa2_norm_rope).
//
// y = R_pos(x * w / sqrt(mean(x^2) + eps)): pair j of the rotated channels turns by t = pos * f_j,
//   (a, b) -> m (a cos t - b sin t, b cos t + a sin t).
// The angle (a far position times a frequency loses whole radians in 32 bits) is formed and reduced to half
// turns in 64 bits, their rounding errors carried along (angle.cuh), and handed to sincospif, whose argument
// then lies in [-1, 1].
// Everything else is fp32, rounded once when it is stored.
//
// Both calls move each row once and compute little, so device memory bounds them. Split: a block
// takes a few rows (a row: one head of one token), each row on 1 .. 32 lanes with 1 .. 8 vectors of
// 16 (or 8) bytes per lane, all loads of the block's rows in flight before the sines and cosines
// are formed; these are shared by the block's heads of a token through shared memory. The rows of a
// block run on from one token to the next, so no head count leaves a block half empty. With
// CSA2_ROPE_HALF a lane takes vectors in pairs, rot / 2 channels apart where they turn, so that both
// channels of every rotated pair are its own.
#include "angle.cuh"
#include "csa2_internal.cuh"
#include "csa2_layer.cuh"

namespace csa2 {

namespace {

constexpr int kThr = 256;

// cos and sin of pos * f (radians)
__device__ __forceinline__ float2 turn(int64_t pos, double f, float mscale, int transposed) {
    float s, c;
    sincospif((float)half_turns(pos, f), &s, &c);
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

// The cosines and sines of pairs j, j + 1, ..: read at once where there is no norm (whose kernels have no
// registers to spare for them), one by one where there is.
template <int N, bool WIDE>
struct Turns {
    float c[WIDE ? N : 1], s[WIDE ? N : 1];
    const float *cp, *sp;
    __device__ __forceinline__ Turns(const float* cosines, const float* sines) : cp(cosines), sp(sines) {
        if constexpr (WIDE) {
            ld(cp, c);
            ld(sp, s);
        }
    }
    __device__ __forceinline__ float cosine(int i) const { return WIDE ? c[WIDE ? i : 0] : cp[i]; }
    __device__ __forceinline__ float sine(int i) const { return WIDE ? s[WIDE ? i : 0] : sp[i]; }
    static __device__ __forceinline__ void ld(const float* p, float (&v)[WIDE ? N : 1]) {
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(p + i);
                v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
            }
        } else if constexpr (N == 2) {
            const float2 f = *reinterpret_cast<const float2*>(p);
            v[0] = f.x, v[1] = f.y;
        } else {
            v[0] = *p;
        }
    }
};

// One row per group of a.lanes lanes, CPL vectors per lane; ITER rows of a group are in flight, and with a
// norm a group takes a.rounds * ITER rows in turn. Measured for 4096 tokens x 64 heads x 512, bf16: the
// rotation alone is fastest with four rows in flight, three blocks an SM and one round (83 us, 6.4 TB/s; two rows 88,
// two blocks an SM 99); the norm, whose instructions
// weigh as much as its bytes, with one row, eight rounds and five blocks an SM (99 us,
// 5.5 TB/s; one round 108, two rows 118). Rows of 128 channels: 16384 tokens x 33 heads 81 us (3.4 TB/s), in
// halves over the whole head 16384 x 20 heads 46 us (3.7 TB/s): shorter rows, more instructions per byte.
template <typename T, int VB, int CPL, int ITER, bool NORM, bool HALF>
__global__ void __launch_bounds__(kThr, NORM && CPL <= 2 ? (HALF ? 4 : 5) : ITER == 4 && CPL == 2 ? 3 : 1) rotate_kernel(RotateArgs a) {
    constexpr int E = VB / (int)sizeof(T);
    using V = Vec<VB>;
    extern __shared__ __align__(16) float table[];  // [tokens of the block][rot / 2] cosines, then the sines
    // where a row is always a warp's, its number, and all that follows from it, is the same in every lane
    constexpr bool WARP = CPL > (HALF ? 2 : 1);
    const int tid = threadIdx.x, lanes = WARP ? 32 : a.lanes, per = kThr / lanes;
    const int gl = tid & (lanes - 1);
    const int gr = WARP || lanes == 32 ? __shfl_sync(0xffffffffu, tid >> 5, 0) : tid / lanes;
    const int rounds = NORM ? a.rounds : 1;
    // the block's rows, in the order token, head: row0 .. row0 + nrows - 1, of tokens tok0 .. tok0 + ntok - 1
    const int most = per * ITER * rounds;
    const int64_t row0 = (int64_t)blockIdx.x * most, left = a.tokens * a.heads - row0;
    const int nrows = left < most ? (int)left : most;
    // (a 64-bit division costs as much as a row's arithmetic)
    const int64_t tok0 = a.tokens * a.heads <= 0x7FFFFFFF ? (int64_t)((uint32_t)row0 / (uint32_t)a.heads) : row0 / a.heads;
    const int head0 = (int)(row0 - tok0 * a.heads), ntok = (head0 + nrows - 1) / a.heads + 1;
    const int half = a.rot >> 1;
    // this lane's vectors: first element, whether it is there, whether it turns
    int at[CPL];
    bool there[CPL], turned[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        if constexpr (HALF) {
            // pairs of vectors: the rp pairs that turn, rp vectors apart, then the others (np pairs, np apart)
            const int nc = a.d / E, rp = half / E, np = (nc - 2 * rp + 1) / 2, pi = gl + (c >> 1) * lanes, q = pi - rp;
            const int o = q + (c & 1) * np, i = o < a.offset / E ? o : o + 2 * rp;
            turned[c] = q < 0;
            at[c] = turned[c] ? a.offset + (pi + (c & 1) * rp) * E : i * E;
            there[c] = turned[c] || (q < np && o < nc - 2 * rp && !a.in_place);
        } else {
            at[c] = (gl + c * lanes) * E;
            const int k = at[c] - a.offset;
            turned[c] = at[c] < a.d && k >= 0 && k < a.rot;
            there[c] = at[c] < a.d && (turned[c] || !a.in_place);
        }
    }
    wait_prior_grid();

    V x[ITER][CPL];
    int tl[ITER];
    T* out[ITER];
    bool isq[ITER];
    float w[NORM ? CPL : 1][E];  // the weights of the rows so far (queries first)
    bool have = false, have_q = false;
    auto load = [&](int it, int row) {  // row `row` of the block into slot it
        out[it] = nullptr;
        if (row >= nrows) return;
        tl[it] = (int)(((float)(head0 + row) + 0.5f) * a.inv_heads);  // the quotient by heads: below 2^17, exact
        const int hh = head0 + row - tl[it] * a.heads;
        const int64_t tok = tok0 + tl[it];
        if (a.pos && a.pos[tok] < 0) return;  // padding: nothing written
        isq[it] = hh < a.q.heads;
        const csa2_heads& H = isq[it] ? a.q : a.k;
        const int64_t h = isq[it] ? hh : hh - a.q.heads;
        const T* src = reinterpret_cast<const T*>(H.x) + tok * H.x_token + h * H.x_head;
        out[it] = reinterpret_cast<T*>(H.out) + tok * H.out_token + h * H.out_head;
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            if (there[c]) x[it][c] = *reinterpret_cast<const V*>(src + at[c]);
    };
#pragma unroll
    for (int it = 0; it < ITER; ++it) load(it, it * per + gr);
    float* const sines = table + ntok * half;
    for (int i = tid; i < ntok * half; i += kThr) {
        const int t = (int)(((float)i + 0.5f) * a.inv_half);  // the quotient by half: below 2^14, exact
        const float2 v = turn(a.pos[tok0 + t], a.inv_freq[i - t * half], a.mscale, a.transposed);
        table[i] = v.x;
        sines[i] = v.y;
    }
    __syncthreads();

    for (int round = 0; round < rounds; ++round) {
#pragma unroll
        for (int it = 0; it < ITER; ++it) {
            float r = 1.f;
            if constexpr (NORM) {
                float ss = 0.f;
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    if (out[it] && there[c]) {
                        float f[E];
                        unpack<T, VB>(x[it][c], f);
#pragma unroll
                        for (int e = 0; e < E; ++e) ss = fmaf(f[e], f[e], ss);
                    }
                }
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    if (o < lanes) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                r = rsqrtf(ss * a.inv_d + a.eps);
                if (out[it] && (!have || have_q != isq[it])) {  // (a block's rows are mostly of one kind)
                    const T* wt = reinterpret_cast<const T*>(isq[it] ? a.q.weight : a.k.weight);
                    have = true;
                    have_q = isq[it];
#pragma unroll
                    for (int c = 0; c < CPL; ++c) {
                        if (wt && there[c])
                            unpack<T, VB>(*reinterpret_cast<const V*>(wt + at[c]), w[c]);
                        else
#pragma unroll
                            for (int e = 0; e < E; ++e) w[c][e] = 1.f;
                    }
                }
            }
            if (out[it]) {
                const float *cosines = table + tl[it] * half, *sn = sines + tl[it] * half;
                constexpr int G = HALF ? 2 : 1;  // vectors that turn together
#pragma unroll
                for (int c = 0; c < CPL; c += G) {
                    float f[G][E];
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        if (!there[c + g]) continue;
                        unpack<T, VB>(x[it][c + g], f[g]);
                        if constexpr (NORM) {
#pragma unroll
                            for (int e = 0; e < E; ++e) f[g][e] *= r * w[c + g][e];
                        }
                    }
                    if (turned[c]) {
                        if constexpr (HALF) {
                            const int j = at[c] - a.offset;
                            const Turns<E, !NORM> t(cosines + j, sn + j);
#pragma unroll
                            for (int e = 0; e < E; ++e) {
                                const float cv = t.cosine(e), sv = t.sine(e), y0 = fmaf(f[0][e], cv, -f[1][e] * sv);
                                f[1][e] = fmaf(f[1][e], cv, f[0][e] * sv);
                                f[0][e] = y0;
                            }
                        } else {
                            const int j = (at[c] - a.offset) >> 1;
                            const Turns<E / 2, !NORM> t(cosines + j, sn + j);
#pragma unroll
                            for (int e = 0; e < E; e += 2) {
                                const float cv = t.cosine(e / 2), sv = t.sine(e / 2);
                                const float y0 = fmaf(f[0][e], cv, -f[0][e + 1] * sv);
                                f[0][e + 1] = fmaf(f[0][e + 1], cv, f[0][e] * sv);
                                f[0][e] = y0;
                            }
                        }
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        if (there[c + g]) *reinterpret_cast<V*>(out[it] + at[c + g]) = pack<T, VB>(f[g]);
                }
            }
            if (round + 1 < rounds) load(it, ((round + 1) * ITER + it) * per + gr);
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

template <typename T, int VB, int CPL, int ITER, bool NORM, bool HALF>
cudaError_t launch_vec(RotateArgs a, cudaStream_t s) {
    const int rows = kThr / a.lanes * ITER;  // per block and round
    const int64_t all = a.tokens * a.heads;
    // the table of a block of n rows: the tokens of n rows in a run
    auto table = [&](int64_t n) {
        const int64_t toks = (n - 1) / a.heads + 2;
        return (size_t)(toks < n ? toks : n) * (a.rot / 2) * sizeof(float2);
    };
    // Rounds: the index arithmetic, the table and the weights are once per block, so with a norm a block takes
    // up to eight rounds of rows while six blocks an SM remain and the table stays small. (One round's table
    // is at most 36 KB: rows * rot / 2 <= 256 / lanes * ITER * lanes * CPL * E / 2 pairs with
    // ITER * CPL * E <= 32 but for the case of four rows, and one token more of up to 512 pairs.)
    a.rounds = 1;
    while (NORM && a.rounds < 8 && all >= (int64_t)148 * 6 * rows * a.rounds * 2 && table((int64_t)rows * a.rounds * 2) <= 16384)
        a.rounds *= 2;
    const int64_t most = (int64_t)rows * a.rounds, grid = (all + most - 1) / most;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    a.inv_heads = 1.f / (float)a.heads;
    a.inv_half = a.rot ? 2.f / (float)a.rot : 0.f;
    const size_t smem = table(most);
    return launch_after_prior(rotate_kernel<T, VB, CPL, ITER, NORM, HALF>, dim3((unsigned)grid), dim3(kThr), smem, s, a);
}

template <typename T, int VB, bool NORM, bool HALF>
cudaError_t launch_rows(RotateArgs a, cudaStream_t s) {
    constexpr int G = HALF ? 2 : 1;  // vectors that a lane takes together
    const int nc = a.d / (VB / (int)sizeof(T)), need = (nc + G - 1) / G;
    a.lanes = need < 32 ? ceil_pow2(need) : 32;
    // several rows per group where the blocks still fill the GPU (about eight of 256 threads an SM);
    // below that a block does less, for latency
    const bool many = a.tokens * a.heads >= (int64_t)148 * 8 * (kThr / a.lanes) * 2;
    if (need <= 32)
        return many ? launch_vec<T, VB, G, NORM ? 1 : 4 / G, NORM, HALF>(a, s) : launch_vec<T, VB, G, 1, NORM, HALF>(a, s);
    if (need <= 64) {
        if constexpr (!NORM && !HALF) {
            // four rows in flight where the table of 32 rows is small (few heads rotated whole: 64 KB)
            if (many && (31 / a.heads + 2) * (a.rot / 2) * (int)sizeof(float2) <= 32768)
                return launch_vec<T, VB, 2, 4, NORM, HALF>(a, s);
        }
        return launch_vec<T, VB, 2 * G, 1, NORM, HALF>(a, s);
    }
    if (need <= 128) return launch_vec<T, VB, 4 * G, 1, NORM, HALF>(a, s);
    if constexpr (!HALF) return launch_vec<T, VB, 8, 1, NORM, HALF>(a, s);  // (256 vectors at most)
    return cudaErrorInvalidValue;
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
    const bool half = a.layout == CSA2_ROPE_HALF;
    if (fits(16)) return half ? launch_rows<T, 16, NORM, true>(a, s) : launch_rows<T, 16, NORM, false>(a, s);
    if (fits(8)) return half ? launch_rows<T, 8, NORM, true>(a, s) : launch_rows<T, 8, NORM, false>(a, s);
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
