// paged.cu -- the paged latent cache: append with norm and rotation on the way (csa2_paged_append) and
// entries read back as values (csa2_paged_gather).
//
// [C] "DeepSeek-V4.1-Flash: Pushing KV Cache Compression to 890 Bytes per Token", sec. XI: cached
// values are quantised after the rotation. Here one kernel does
//   y = R_pos(x * w / sqrt(mean(x^2) + eps)),  then the codecs of csa2.h on y,
// with nothing rounded in between, and every code and scale is the one that y has: a value next to a
// rounding border of a 4-bit code falls on the wrong side in fp32, so norm, rotation and quotients
// are formed in 64 bits and reach the conversion instructions by rounding to odd.
//
// Work split: one warp per row (a token's latent, indexer key or window row), 16 channels per lane
// (one scale block of the latent) or 4 (an eighth of an MXFP4 block).
#include "csa2_internal.cuh"
#include "csa2_layer.cuh"

namespace csa2 {

namespace {

constexpr int kWarps = 4;  // per block
constexpr double kInvPi = 0.31830988618379067154;

// Rounding to odd: the fp32 value next to v towards zero, its last bit set unless it is v. A further
// rounding to a format of at most 22 bits then decides as it would for v.
__device__ __forceinline__ float to_odd(double v) {
    const float f = __double2float_rz(v);
    return (double)f == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

struct WarpMem {
    double2 cs[256];   // cos, sin of the row's pairs
    float xw[kLatD];   // x * w, exact in fp32 (two bf16 factors)
};

// N channels of this lane, normed and rotated (64 bits); CH = 32 N channels in the row.
template <int N>
__device__ __forceinline__ void normed_row(const AppendRow& R, const uint16_t* src, int64_t rpos, double eps,
                                           WarpMem& sm, int lane, double (&y)[N]) {
    constexpr int CH = 32 * N;
    float x[N];
    if constexpr (N == 16) {
        load16_bf16(src + lane * 16, x);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src + lane * 4);
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    double r = 1.0;
    if (R.weight) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < N; ++i) ss += (double)(x[i] * x[i]);  // (exact products)
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = 1.0 / sqrt(ss / CH + eps);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= bf16_bits_to_f32(R.weight[lane * N + i]);
    }
    __syncwarp();  // the row before is done with the shared memory
    if (R.inv_freq) {
        const int half = R.rot >> 1;
#pragma unroll
        for (int i = 0; i < N; ++i) sm.xw[lane * N + i] = x[i];
        for (int j = lane; j < half; j += 32) {
            double h = ((double)rpos * R.inv_freq[j]) * kInvPi, s, c;
            h -= 2.0 * rint(0.5 * h);
            sincospi(h, &s, &c);
            sm.cs[j] = make_double2(c * R.mscale, s * R.mscale);
        }
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int ch = lane * N + i, k = ch - R.offset;
        y[i] = (double)x[i] * r;
        if (R.inv_freq && k >= 0 && k < R.rot) {
            const int half = R.rot >> 1;
            const bool inter = R.layout == CSA2_ROPE_INTERLEAVED;
            const int j = inter ? k >> 1 : (k < half ? k : k - half);
            const bool first = inter ? !(k & 1) : k < half;
            const int other = inter ? (first ? ch + 1 : ch - 1) : (first ? ch + half : ch - half);
            const double2 t = sm.cs[j];
            const double z = (double)sm.xw[other] * r;
            y[i] = y[i] * t.x + (first ? -z * t.y : z * t.y);
        }
    }
}

__global__ void __launch_bounds__(32 * kWarps) paged_append_kernel(PagedAppendArgs a) {
    __shared__ WarpMem mem[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    WarpMem& sm = mem[warp];
    const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
    wait_prior_grid();  // the rows come from, and the slots may still be read by, earlier work
    if (id >= (int64_t)a.batch * a.t * 3) return;
    const int kind = (int)(id % 3);
    const int64_t tok = id / 3;
    const int b = (int)(tok / a.t), i = (int)(tok % a.t);
    const AppendRow& R = a.row[kind];
    if (!R.x) return;
    const int64_t p0 = a.pos[b], p = p0 + i;
    const int n = a.len ? a.len[b] : a.t;
    const bool tell = i == 0 && lane == 0;
    const int64_t cap = a.pg.max_pages << a.pg.shift;
    if (n < 0 || n > a.t || (n > 0 && (p0 < 0 || (kind < 2 && (p0 > cap || p0 + n > cap))))) {
        if (tell) set_status(a.status, CSA2_DEV_BAD_POS);
        return;
    }
    if (i >= n) return;  // padding
    const uint16_t* src = R.x + (int64_t)b * R.x_batch + (int64_t)i * R.x_token;
    const int64_t rpos = a.rpos ? a.rpos[tok] : p;
    if (kind == 2) {
        // the ring keeps the latest swa_cap tokens: an older one of this call shares its slot with a newer one
        if ((int64_t)i < (int64_t)n - a.c.swa_cap) return;
        const int64_t slot = paged_slot(a.pg, b);
        if (slot < 0) {
            if (lane == 0) set_status(a.status, CSA2_DEV_BAD_PAGE);
            return;
        }
        double y[16];
        normed_row<16>(R, src, rpos, a.eps, sm, lane, y);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = f32x2_to_e4m3x2(to_odd(y[4 * j]), to_odd(y[4 * j + 1])) |
                   (f32x2_to_e4m3x2(to_odd(y[4 * j + 2]), to_odd(y[4 * j + 3])) << 16);
        uint8_t* dst = a.c.swa + (slot * a.c.swa_cap + (p & (a.c.swa_cap - 1))) * kLatSwa + lane * 16;
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
    const int64_t row = paged_row(a.pg, b, p);
    if (row < 0) {
        if (lane == 0) set_status(a.status, CSA2_DEV_BAD_PAGE);
        return;
    }
    if (kind == 0) {
        double y[16];
        normed_row<16>(R, src, rpos, a.eps, sm, lane, y);
        double top = 0.0;
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmax(top, fabs(y[j]));
        const uint8_t sc = (uint8_t)f32x2_to_e4m3x2(to_odd(top / 6.0), 0.f);
        const float s = e4m3_to_f32(sc);
        uint32_t c[2] = {0u, 0u};
        if (s != 0.f) {
            const double inv = 1.0 / (double)s;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                c[j >> 2] |= f32x2_to_e2m1x2(to_odd(y[2 * j] * inv), to_odd(y[2 * j + 1] * inv)) << (8 * (j & 3));
        }
        *reinterpret_cast<uint2*>(a.c.l_data + row * kLatBytes + lane * 8) = make_uint2(c[0], c[1]);
        a.c.l_scale[row * kLatScales + lane] = sc;
    } else {
        double y[4];
        normed_row<4>(R, src, rpos, a.eps, sm, lane, y);
        double top = fmax(fmax(fabs(y[0]), fabs(y[1])), fmax(fabs(y[2]), fabs(y[3])));
        for (int o = 4; o; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));  // the block's 8 lanes
        int sb = 0;
        uint32_t c = 0;
        if (top > 0.0) {
            sb = ilogb(top) - 2 + 127;
            sb = sb < 0 ? 0 : (sb > 254 ? 254 : sb);
            const double inv = ldexp(1.0, 127 - sb);
            c = f32x2_to_e2m1x2(to_odd(y[0] * inv), to_odd(y[1] * inv)) |
                (f32x2_to_e2m1x2(to_odd(y[2] * inv), to_odd(y[3] * inv)) << 8);
        }
        *reinterpret_cast<uint16_t*>(a.c.k_data + row * kLatKBytes + lane * 2) = (uint16_t)c;
        if (!(lane & 7)) a.c.k_scale[row * kLatKScales + (lane >> 3)] = (uint8_t)sb;
    }
}

// Entries as bf16 values: a warp per entry, 16 latent channels (one scale block) a lane and 8 key channels
// a lane of the first half.
__global__ void __launch_bounds__(256) paged_gather_kernel(PagedGatherArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    wait_prior_grid();
    if (id >= a.rows) return;
    const int b = (int)(id / a.n);
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

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
    const int64_t warps = (int64_t)a.batch * a.t * 3;
    const int64_t grid = (warps + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_after_prior(paged_append_kernel, dim3((unsigned)grid), dim3(32 * kWarps), 0, s, a);
}

cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t s) {
    const int64_t grid = (a.rows + 7) / 8;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_after_prior(paged_gather_kernel, dim3((unsigned)grid), dim3(256), 0, s, a);
}

}  // namespace csa2
