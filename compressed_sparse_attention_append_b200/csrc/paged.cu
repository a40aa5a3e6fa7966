// paged.cu -- the paged latent cache: append with norm and rotation on the way (csa2_paged_append) and
// entries read back as values (csa2_paged_gather).
//
// [C] "DeepSeek-V4.1-Flash: Pushing KV Cache Compression to 890 Bytes per Token", sec. XI: cached
// values are quantised after the rotation. Here one kernel does
//   y = R_pos(x * w / sqrt(mean(x^2) + eps)),  then the codecs of csa2.h on y,
// with nothing rounded in between, and every code and scale is the one that y has. A value next to a
// rounding border of a 4-bit code falls on the wrong side in fp32, so:
//   - y is formed in fp32 with a bound e on its error, and both y - e and y + e are converted: where the two
//     conversions agree (codes and scales are monotone in y) the code is y's;
//   - a row in which any two differ (one in several hundred) is formed again in 64 bits, norm, rotation
//     and quotients, and reaches the conversion instructions by rounding to odd. Rows without a norm,
//     whose bf16 values lie on borders often, are always formed so.
// The error of fp32: the sum of squares is off by 4 roundings (a lane's 16 as a tree, the lanes' sums in 64 bits),
// its root by half of that and 2^-23.4, the product by 2^-24, the quotient by 2^-23 more: below 2^-21.3. Cosine
// and sine are off by 2^-21.4 at any position below 2^31 (angle.cuh). So e = 2^-21 |y|, and 2^-20 m (|a| + |b|) for
// the channels of a rotated pair (a, b), cover y and its quotient.
//
// Work split: 16 channels per lane (one scale block of the latent, half an MXFP4 block), so a warp takes one
// latent or window row, or the indexer keys of four tokens. A row's rotated pairs are turned by its
// lanes in turn, through shared memory. A row is a chain of loads and some 690 instructions (170 of them the
// rotation's; a row of padding 106, the keys of four tokens 980), which bound it (issue slots 77 % busy): 16
// sequences of 2048 tokens at most, 853 on average, take 24 us.
#include "angle.cuh"
#include "csa2_internal.cuh"
#include "csa2_layer.cuh"

namespace csa2 {

namespace {

constexpr int kWarps = 4;    // per block
// Blocks per SM (registers): a row is a chain of loads, so many rows at once, though at 48 registers the rare 64-bit
// calls spill 96 bytes. 16 sequences of 2048 tokens with their read-back: 42 us at 6 blocks (79 registers, no spill), 40.2
// at 8, 39.3 at 10, 38.5 at 12 (284 bytes spilled), each to 1.5 us; single tokens are the same at all.
constexpr int kBlocks = 10;

// Rounding to odd: the fp32 value next to v towards zero, its last bit set unless it is v. A further
// rounding to a format of at most 22 bits then decides as it would for v.
__device__ __forceinline__ float to_odd(double v) {
    const float f = __double2float_rz(v);
    return (double)f == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// A warp's shared memory: 8 bytes per rotated channel of the widest rotation (channel k of the rotated range).
struct WarpMem {
    unsigned char* p;
    int rot;
    __device__ __forceinline__ float* y() const { return reinterpret_cast<float*>(p); }             // values
    __device__ __forceinline__ float* err() const { return reinterpret_cast<float*>(p) + rot; }     // and their errors
    __device__ __forceinline__ double* wide() const { return reinterpret_cast<double*>(p); }        // values in 64 bits
};

// this lane's N channels of a row of 32 N
template <int N>
__device__ __forceinline__ void load_row(const uint16_t* src, int lane, float (&x)[N]) {
    if constexpr (N == 16) {
        load16_bf16(src + lane * 16, x);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src + lane * 4);
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
}
// the channels of pair j within the rotated range
__device__ __forceinline__ int2 pair_of(const AppendRow& R, int j) {
    const bool inter = R.layout == CSA2_ROPE_INTERLEAVED;
    return make_int2(inter ? 2 * j : j, inter ? 2 * j + 1 : j + (R.rot >> 1));
}

// ---- rows in 64 bits -----------------------------------------------------------------------------------

// N channels of this lane, normed and rotated; CH = 32 N channels in the row.
template <int N>
__device__ __forceinline__ void exact_row(const AppendRow& R, const uint16_t* src, int64_t rpos, double eps,
                                          const WarpMem& sm, int lane, double (&y)[N]) {
    constexpr int CH = 32 * N;
    float x[N];
    load_row<N>(src, lane, x);
    double r = 1.0;
    if (R.weight) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fma((double)x[i], (double)x[i], ss);
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = 1.0 / sqrt(ss / CH + eps);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)  // (exact: two bf16 factors)
        y[i] = R.weight ? (double)x[i] * (double)bf16_bits_to_f32(R.weight[lane * N + i]) : (double)x[i];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] *= r;
    if (R.inv_freq) {
        const int k0 = lane * N - R.offset;
        double* const ys = sm.wide();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (k0 + i >= 0 && k0 + i < R.rot) ys[k0 + i] = y[i];
        __syncwarp();
        for (int j = lane; j < (R.rot >> 1); j += 32) {
            double sn, cs;
            sincospi(half_turns(rpos, R.inv_freq[j]), &sn, &cs);
            const int2 p = pair_of(R, j);
            const double u = ys[p.x] * R.mscale, v = ys[p.y] * R.mscale;
            ys[p.x] = u * cs - v * sn;
            ys[p.y] = v * cs + u * sn;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (k0 + i >= 0 && k0 + i < R.rot) y[i] = ys[k0 + i];
    }
}

// eight fp32 -> eight E2M1 codes, RNE, saturating
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// a row's 16-channel E2M1 block, 4 MXFP4 channels or 16 window channels of this lane
struct Coded {
    uint4 codes;
    uint32_t scale;
};

__device__ __noinline__ Coded exact_latent(const AppendRow& R, const uint16_t* src, int64_t rpos, double eps, const WarpMem& sm,
                                           int lane) {
    double y[16], top = 0.0;
    exact_row<16>(R, src, rpos, eps, sm, lane, y);
#pragma unroll
    for (int j = 0; j < 16; ++j) top = fmax(top, fabs(y[j]));
    Coded c{};
    c.scale = f32x2_to_e4m3x2(to_odd(top / 6.0), 0.f) & 0xFFu;
    const float s = e4m3_to_f32((uint8_t)c.scale);
    if (s != 0.f) {
        const double inv = 1.0 / (double)s;
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j >> 2] |= f32x2_to_e2m1x2(to_odd(y[2 * j] * inv), to_odd(y[2 * j + 1] * inv)) << (8 * (j & 3));
        c.codes.x = w[0];
        c.codes.y = w[1];
    }
    return c;
}

__device__ __noinline__ Coded exact_key(const AppendRow& R, const uint16_t* src, int64_t rpos, double eps, const WarpMem& sm,
                                        int lane) {
    double y[4];
    exact_row<4>(R, src, rpos, eps, sm, lane, y);
    double top = fmax(fmax(fabs(y[0]), fabs(y[1])), fmax(fabs(y[2]), fabs(y[3])));
    for (int o = 4; o; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));  // the block's 8 lanes
    Coded c{};
    if (top > 0.0) {
        const int sb = ilogb(top) - 2 + 127;
        c.scale = (uint32_t)(sb < 0 ? 0 : (sb > 254 ? 254 : sb));
        const double inv = ldexp(1.0, 127 - (int)c.scale);
        c.codes.x = f32x2_to_e2m1x2(to_odd(y[0] * inv), to_odd(y[1] * inv)) |
                    (f32x2_to_e2m1x2(to_odd(y[2] * inv), to_odd(y[3] * inv)) << 8);
    }
    return c;
}

__device__ __noinline__ Coded exact_window(const AppendRow& R, const uint16_t* src, int64_t rpos, double eps, const WarpMem& sm,
                                           int lane) {
    double y[16];
    exact_row<16>(R, src, rpos, eps, sm, lane, y);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = f32x2_to_e4m3x2(to_odd(y[4 * j]), to_odd(y[4 * j + 1])) |
               (f32x2_to_e4m3x2(to_odd(y[4 * j + 2]), to_odd(y[4 * j + 3])) << 16);
    return Coded{make_uint4(w[0], w[1], w[2], w[3]), 0u};
}

// ---- rows in 32 bits, with the bound of each value's error --------------------------------------------------

constexpr float kErr = 1.f / 2097152.f, kErrTurn = 1.f / 1048576.f;  // 2^-21, 2^-20

// y, and L: a value y[i] is within |y[i]| kErr + L of the row's (L: the largest bound of this lane's rotated
// channels). False where fp32 cannot hold the row's norm (squares past its range): no bound is valid then.
// The row lies on LANES lanes, `lane` of them this one; a row that is not live is read as zeros.
template <int LANES>
__device__ __forceinline__ bool quick_row(const AppendRow& R, bool live, const uint16_t* src, int64_t rpos, float eps,
                                          const WarpMem& sm, int lane, float (&y)[16], float& L) {
    constexpr int N = 16;
    float w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = 0.f;
    if (live) load16_bf16(src + lane * N, y);
    load16_bf16(R.weight + lane * N, w);
    // sine and cosine of this lane's first pair are formed while the row is on its way
    const int half = R.inv_freq ? R.rot >> 1 : 0;
    float c0 = 0.f, s0 = 0.f;
    if (lane < half) sincospif((float)half_turns(rpos, R.inv_freq[lane]), &s0, &c0);
    // the lane's squares (exact) as a tree, the lanes' sums in 64 bits
    float t[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) t[i] = fmaf(y[2 * i + 1], y[2 * i + 1], y[2 * i] * y[2 * i]);
#pragma unroll
    for (int o = N / 4; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) t[i] += t[i + o];
    double ss = (double)t[0];
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // 1 / sqrt with one step of Newton's iteration, the product's rounding carried along
    const float mean = (float)fma(ss, 1.0 / (LANES * N), (double)eps), r0 = rsqrtf(mean), h = mean * r0;
    const float r = fmaf(0.5f * r0, fmaf(-h, r0, 1.f) - fmaf(mean, r0, -h) * r0, r0);
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = (y[i] * w[i]) * r;  // (two bf16 factors: exact)
    L = 0.f;
    if (half) {
        const int k0 = lane * N - R.offset;  // this lane's first channel within the rotated range
        const bool mine = k0 < R.rot && k0 + N > 0;
        // all of its channels turn, at a place that allows vectors
        const bool whole = k0 >= 0 && k0 + N <= R.rot && !((k0 | R.rot) & 3);
        float *const ys = sm.y(), *const es = sm.err();
        __syncwarp();  // the row before is done with the shared memory
        if (whole) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4*>(ys + k0 + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
        } else if (mine) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (k0 + i >= 0 && k0 + i < R.rot) ys[k0 + i] = y[i];
        }
        __syncwarp();
        const float m = (float)R.mscale, me = fabsf(m) * kErrTurn;
        for (int j = lane; j < half; j += LANES) {
            if (j != lane) sincospif((float)half_turns(rpos, R.inv_freq[j]), &s0, &c0);
            const int2 p = pair_of(R, j);
            const float a = ys[p.x], b = ys[p.y], err = (fabsf(a) + fabsf(b)) * me;
            ys[p.x] = m * fmaf(a, c0, -b * s0);
            ys[p.y] = m * fmaf(b, c0, a * s0);
            es[p.x] = es[p.y] = err;
        }
        __syncwarp();
        if (whole) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(ys + k0 + i), e = *reinterpret_cast<const float4*>(es + k0 + i);
                y[i] = v.x, y[i + 1] = v.y, y[i + 2] = v.z, y[i + 3] = v.w;
                L = fmaxf(L, fmaxf(fmaxf(e.x, e.y), fmaxf(e.z, e.w)));
            }
        } else if (mine) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (k0 + i >= 0 && k0 + i < R.rot) {
                    y[i] = ys[k0 + i];
                    L = fmaxf(L, es[k0 + i]);
                }
            }
        }
    }
    return mean >= 1e-25f && mean <= 1e34f;
}

// Each returns whether every code (and scale) of the warp's row is certain.
__device__ __forceinline__ bool quick_latent(const float (&y)[16], float L, Coded& c) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(y[i]));
    const float err = fmaf(top, kErr, L);
    const uint32_t sc = f32x2_to_e4m3x2((top - err) * (1.f / 6.f), (top + err) * (1.f / 6.f));
    c.scale = sc & 0xFFu;
    const float s = e4m3_to_f32((uint8_t)c.scale), inv = s != 0.f ? 1.f / s : 0.f, d = L * inv;
    uint32_t lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float l[8], u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = y[8 * h + j] * inv, da = fmaf(fabsf(a), kErr, d);
            l[j] = a - da;
            u[j] = a + da;
        }
        lo[h] = e2m1x8(l);
        hi[h] = e2m1x8(u);
    }
    const bool none = s == 0.f;  // a scale of 0: codes +0
    c.codes.x = none ? 0u : lo[0];
    c.codes.y = none ? 0u : lo[1];
    return __all_sync(0xffffffffu, c.scale == (sc >> 8) && (none || (lo[0] == hi[0] && lo[1] == hi[1])));
}

// half an MXFP4 block; certain of this lane's channels alone
__device__ __forceinline__ bool quick_key(const float (&y)[16], float L, Coded& c) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(y[i]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));  // the block's other lane
    const float most = fmaxf(L, __shfl_xor_sync(0xffffffffu, L, 1)), err = fmaf(top, kErr, most), hi = top + err;
    // the exponents of both ends: all zeros, or far above the smallest normal number (w / sqrt(mean) is then
    // normal wherever it matters)
    const int xl = (int)(__float_as_uint(fmaxf(top - err, 0.f)) >> 23), xh = (int)(__float_as_uint(hi) >> 23);
    const bool none = hi == 0.f;
    c.scale = none ? 0u : (uint32_t)(xl - 2);
    const float inv = none ? 0.f : __uint_as_float((uint32_t)(254 - (xl - 2)) << 23);  // 2^(127 - scale)
    const float d = L * inv;
    uint32_t lo[2], up[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float l[8], u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = y[8 * h + j] * inv, da = fmaf(fabsf(a), kErr, d);
            l[j] = a - da;
            u[j] = a + da;
        }
        lo[h] = e2m1x8(l);
        up[h] = e2m1x8(u);
    }
    c.codes.x = none ? 0u : lo[0];
    c.codes.y = none ? 0u : lo[1];
    return none || (xl == xh && xl > 64 && xl < 255 && lo[0] == up[0] && lo[1] == up[1]);
}

__device__ __forceinline__ bool quick_window(const float (&y)[16], float L, Coded& c) {
    uint32_t lo[4] = {}, hi[4] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = y[2 * j], b = y[2 * j + 1], da = fmaf(fabsf(a), kErr, L), db = fmaf(fabsf(b), kErr, L);
        lo[j >> 1] |= f32x2_to_e4m3x2(a - da, b - db) << (16 * (j & 1));
        hi[j >> 1] |= f32x2_to_e4m3x2(a + da, b + db) << (16 * (j & 1));
    }
    c.codes = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    return __all_sync(0xffffffffu, lo[0] == hi[0] && lo[1] == hi[1] && lo[2] == hi[2] && lo[3] == hi[3]);
}

// Where token `tok` of one kind of row is read and written.
struct Token {
    bool live;            // to be written
    const uint16_t* src;
    int64_t rpos;         // its position for the rotation
    int64_t row;          // plane row (latent, key) or ring row (window)
};
// Rows that a sequence may have of one kind: the ring keeps the latest swa_cap tokens (an older one of the call would
// share its slot with a newer one), so no warp is started for the others.
__host__ __device__ __forceinline__ int rows_of(const PagedAppendArgs& a, int kind) {
    return kind == 2 && a.c.swa_cap < a.t ? (int)a.c.swa_cap : a.t;
}
// Row `id` of a kind. `first`: one lane of those that work on it, which reports what is wrong with it
__device__ __forceinline__ Token locate(const PagedAppendArgs& a, int kind, int64_t id, bool first) {
    Token k{};
    const int t = rows_of(a, kind);
    const int64_t ids = (int64_t)a.batch * t;
    if (id >= ids) return k;
    // (in 32 bits where they suffice: a 64-bit division costs a fifth of a row's arithmetic)
    const int b = ids <= 0x7FFFFFFF ? (int)((uint32_t)id / (uint32_t)t) : (int)(id / t);
    int i = (int)(id - (int64_t)b * t);
    const int n = a.len ? a.len[b] : a.t;
    const int64_t p0 = a.pos[b];
    const int64_t cap = a.pg.max_pages << a.pg.shift;
    if (n < 0 || n > a.t || (n > 0 && (p0 < 0 || (kind < 2 && (p0 > cap || p0 + n > cap))))) {
        if (i == 0 && first) set_status(a.status, CSA2_DEV_BAD_POS);
        return k;
    }
    if (n > t) i += n - t;
    if (i >= n) return k;  // padding
    const int64_t p = p0 + i;
    if (kind == 2) {
        const int64_t slot = paged_slot(a.pg, b);
        k.live = slot >= 0;
        k.row = slot * a.c.swa_cap + (p & (a.c.swa_cap - 1));
    } else {
        k.row = paged_row(a.pg, b, p);
        k.live = k.row >= 0;
    }
    if (!k.live && first) set_status(a.status, CSA2_DEV_BAD_PAGE);
    const AppendRow& R = a.row[kind];
    k.src = R.x + (int64_t)b * R.x_batch + (int64_t)i * R.x_token;
    k.rpos = a.rpos ? a.rpos[(int64_t)b * a.t + i] : p;
    return k;
}

// (the arguments stay in constant memory: the 64-bit functions take references into them)
__global__ void __launch_bounds__(32 * kWarps, kBlocks) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    wait_prior_grid();  // the rows come from, and the slots may still be read by, earlier work
    // a kind's rows lie together (their work is alike): blocks first[i] .. first[i + 1] - 1 are kind[i]'s
    int at = 0;
    while (at + 1 < a.kinds && blockIdx.x >= a.first[at + 1]) ++at;
    const int kind = a.kind[at];
    const AppendRow& R = a.row[kind];
    const int64_t wid = (int64_t)(blockIdx.x - a.first[at]) * kWarps + warp;
    unsigned char* const mem = smem + (size_t)a.warp_bytes * warp;
    const WarpMem sm{mem, a.warp_bytes / 8};
    const float eps = (float)a.eps;
    Coded c{};
    float y[16], L;
    if (kind == 1) {
        // the keys of four tokens, 8 lanes each
        const int g = lane >> 3, gl = lane & 7, rot = (R.rot + 3) & ~3;
        const Token k = locate(a, 1, wid * 4 + g, gl == 0);
        if (!__any_sync(0xffffffffu, k.live)) return;
        bool sure = false;
        if (R.weight) {
            const bool held = quick_row<8>(R, k.live, k.src, k.rpos, eps, WarpMem{mem + 8 * rot * g, rot}, gl, y, L);
            sure = quick_key(y, L, c) && held;
        }
        sure = ((__ballot_sync(0xffffffffu, sure) >> (8 * g)) & 0xFFu) == 0xFFu;
        if (k.live && sure) {
            *reinterpret_cast<uint2*>(a.c.k_data + k.row * kLatKBytes + gl * 8) = make_uint2(c.codes.x, c.codes.y);
            if (!(gl & 1)) a.c.k_scale[k.row * kLatKScales + (gl >> 1)] = (uint8_t)c.scale;
        }
        unsigned todo = __ballot_sync(0xffffffffu, gl == 0 && k.live && !sure);
        for (; todo; todo &= todo - 1) {  // the others by the whole warp, one after the other
            const int from = __ffs(todo) - 1;
            const int64_t row = __shfl_sync(0xffffffffu, k.row, from), rpos = __shfl_sync(0xffffffffu, k.rpos, from);
            const uint16_t* src = reinterpret_cast<const uint16_t*>(
                __shfl_sync(0xffffffffu, (unsigned long long)(uintptr_t)k.src, from));
            c = exact_key(R, src, rpos, a.eps, sm, lane);
            *reinterpret_cast<uint16_t*>(a.c.k_data + row * kLatKBytes + lane * 2) = (uint16_t)c.codes.x;
            if (!(lane & 7)) a.c.k_scale[row * kLatKScales + (lane >> 3)] = (uint8_t)c.scale;
        }
        return;
    }
    const Token k = locate(a, kind, wid, lane == 0);
    if (!k.live) return;
    bool sure = false;
    if (R.weight) {
        sure = quick_row<32>(R, true, k.src, k.rpos, eps, sm, lane, y, L);
        sure = (kind == 0 ? quick_latent(y, L, c) : quick_window(y, L, c)) && sure;
    }
    if (kind == 0) {
        if (!sure) c = exact_latent(R, k.src, k.rpos, a.eps, sm, lane);
        *reinterpret_cast<uint2*>(a.c.l_data + k.row * kLatBytes + lane * 8) = make_uint2(c.codes.x, c.codes.y);
        a.c.l_scale[k.row * kLatScales + lane] = (uint8_t)c.scale;
    } else {
        if (!sure) c = exact_window(R, k.src, k.rpos, a.eps, sm, lane);
        *reinterpret_cast<uint4*>(a.c.swa + k.row * kLatSwa + lane * 16) = c.codes;
    }
}

// Entries as bf16 values: a warp per entry, 16 latent channels (one scale block) a lane and 8 key channels
// a lane of the first half.
__global__ void __launch_bounds__(256) paged_gather_kernel(PagedGatherArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    wait_prior_grid();
    if (id >= a.rows) return;
    const int b = a.rows <= 0x7FFFFFFF ? (int)((uint32_t)id / (uint32_t)a.n) : (int)(id / a.n);
    const int64_t p = a.idx[id];
    int64_t row = -1;
    if (p >= 0 && p < (a.pg.max_pages << a.pg.shift)) {
        row = paged_row(a.pg, b, p);
        if (row < 0 && lane == 0) set_status(a.status, CSA2_DEV_BAD_PAGE);
    } else if (p != -1 && lane == 0) {
        set_status(a.status, CSA2_DEV_BAD_INDEX);
    }
    if (a.latent) {
        uint32_t o[8] = {};
        if (row >= 0) {
            const uint2 v = *reinterpret_cast<const uint2*>(a.c.l_data + row * kLatBytes + lane * 8);
            const float s = e4m3_to_f32(a.c.l_scale[row * kLatScales + lane]);
            uint32_t h[8];
            e2m1x8_to_h2x4(v.x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
            e2m1x8_to_h2x4(v.y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = h2_to_f2(h[j]);
                const __nv_bfloat162 w = __floats2bfloat162_rn(f.x * s, f.y * s);  // exact
                o[j] = *reinterpret_cast<const uint32_t*>(&w);
            }
        }
        uint4* dst = reinterpret_cast<uint4*>(a.latent + id * kLatD + lane * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    if (a.key && lane < 16) {
        uint32_t o[4] = {};
        if (row >= 0) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(a.c.k_data + row * kLatKBytes + lane * 4);
            const float s = ldexpf(1.f, (int)a.c.k_scale[row * kLatKScales + (lane >> 2)] - 127);
            uint32_t h[4];
            e2m1x8_to_h2x4(v, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = h2_to_f2(h[j]);
                const __nv_bfloat162 w = __floats2bfloat162_rn(f.x * s, f.y * s);  // exact
                o[j] = *reinterpret_cast<const uint32_t*>(&w);
            }
        }
        *reinterpret_cast<uint4*>(a.key + id * 128 + lane * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

cudaError_t launch_paged_append(PagedAppendArgs a, cudaStream_t s) {
    int64_t blocks = 0;
    for (int i = 0; i < a.kinds; ++i) {
        const int per = kWarps * (a.kind[i] == 1 ? 4 : 1);  // rows of a block
        a.first[i] = (unsigned)blocks;
        blocks += ((int64_t)a.batch * rows_of(a, a.kind[i]) + per - 1) / per;
        if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
        // 8 bytes per rotated channel of the rows that a warp holds
        const int rot = a.row[a.kind[i]].inv_freq ? (a.row[a.kind[i]].rot + 3) / 4 * 4 : 0;
        const int bytes = 8 * rot * (a.kind[i] == 1 ? 4 : 1);
        if (bytes > a.warp_bytes) a.warp_bytes = bytes;
    }
    return launch_after_prior(paged_append_kernel, dim3((unsigned)blocks), dim3(32 * kWarps), (size_t)a.warp_bytes * kWarps,
                              s, a);
}

cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t s) {
    const int64_t grid = (a.rows + 7) / 8;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_after_prior(paged_gather_kernel, dim3((unsigned)grid), dim3(256), 0, s, a);
}

}  // namespace csa2
