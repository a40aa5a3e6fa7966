// fp8.cu -- products in E4M3 with one scale per 128 channels of a row and per 128 x 128 block of the
// weights, and the two quantisers that write those formats (csa2_fp8_quantize,
// csa2_fp8_quantize_weight, csa2_fp8_gemm).
//
//   out[i][j] = sum_b xs[b][i] ws[j / 128][b] sum_{c in block b} x[i][c] w[j][c]
//
// A block's sum (128 exact products) comes from tcgen05 (kind::f8f6f4) in fp32 tensor memory; the
// scales differ per row and block, so each block's sum is read back, scaled and added to the tile's
// sums in fp32 registers while the tensor cores form the next block's.
#include <mutex>

#include "csa2_internal.cuh"
#include "csa2_layer.cuh"
#include "fp8_plan.h"
#include "tc.cuh"

namespace csa2 {

namespace {

using namespace tc;

constexpr float kE4M3Max = 448.f;

// ---- quantisers --------------------------------------------------------------------------------------

__device__ __forceinline__ void load8_bf16(const uint16_t* p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
// the larger one, NaN when either is (a NaN is not lost in a block's maximum)
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float amax8(const float (&x)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
    return m;
}
// the codes of x / s (fp32 quotients; s == 0: +0)
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s) {
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    if (s != 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// 16 lanes per (row, block of 128), 16 rows per CTA, U blocks per lane group: all loads first.
template <int U>
__global__ void __launch_bounds__(256) fp8_rows_kernel(int64_t rows, int k, const uint16_t* x, int64_t x_stride,
                                                       uint8_t* data, float* scale) {
    const int l = threadIdx.x & 15, nb = (k + 127) / 128, b0 = blockIdx.y * U;
    const int64_t r = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    start_next_grid();  // the product's barriers and tensor memory are set up meanwhile
    wait_prior_grid();
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (b0 + u) * 128 + l * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
        if (r < rows && c < k) load8_bf16(x + r * x_stride + c, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float m = amax8(v[u]);
        for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = __fdiv_rn(m, kE4M3Max);
        const int c = (b0 + u) * 128 + l * 8;
        if (r < rows && c < k) *reinterpret_cast<uint2*>(data + r * k + c) = codes8(v[u], s);
        if (r < rows && l == 0 && b0 + u < nb) scale[(int64_t)(b0 + u) * rows + r] = s;
    }
}

// One CTA per 128 x 128 block: 16 rows of 16 lanes at a time, eight times.
__global__ void __launch_bounds__(256) fp8_weight_kernel(int64_t n, int k, const uint16_t* w, uint8_t* data,
                                                         float* scale) {
    __shared__ float red[8];
    const int c = blockIdx.x * 128 + (threadIdx.x & 15) * 8;
    const int64_t r0 = (int64_t)blockIdx.y * 128 + (threadIdx.x >> 4);
    wait_prior_grid();
    float v[8][8], m = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int64_t r = r0 + 16 * u;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
        if (r < n && c < k) load8_bf16(w + r * k + c, v[u]);
        m = max_nan(m, amax8(v[u]));
    }
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!(threadIdx.x & 31)) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, red[i]);
    const float s = __fdiv_rn(m, kE4M3Max);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int64_t r = r0 + 16 * u;
        if (r < n && c < k) *reinterpret_cast<uint2*>(data + r * k + c) = codes8(v[u], s);
    }
    if (threadIdx.x == 0) scale[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// Waits for this thread's tensor-memory loads; v passes through, so that no use of it moves ahead.
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t (&v)[N]) {
    static_assert(N == 16 || N == 32, "registers of one load");
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; i += 16)
        asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]),
                          "+r"(v[i + 6]), "+r"(v[i + 7]), "+r"(v[i + 8]), "+r"(v[i + 9]), "+r"(v[i + 10]), "+r"(v[i + 11]),
                          "+r"(v[i + 12]), "+r"(v[i + 13]), "+r"(v[i + 14]), "+r"(v[i + 15]));
}

// ---- the product ---------------------------------------------------------------------------------------

constexpr uint64_t kWaitNs = 200000000ull;

// D[tmem] (+)= A B^T, E4M3 x E4M3 -> fp32, both K-major; K = 32 per instruction. Issued by one thread.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__host__ __device__ constexpr uint32_t f8_idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void store_out(const Fp8GemmArgs& a, int64_t i, int64_t j, float v) {
    if (a.out_f32)
        reinterpret_cast<float*>(a.out)[i * a.out_stride + j] = v;
    else
        reinterpret_cast<uint16_t*>(a.out)[i * a.out_stride + j] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// two fp32 as the 64-bit operand of the packed instructions, and back
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
// acc (two fp32) += v * s, element by element
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t v0, uint32_t v1, uint64_t s) {
    asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}" : "+l"(acc) : "r"(v0), "r"(v1), "l"(s));
}

// Tiles of 128 weight rows (the MMA's M: a lane of tensor memory per output column) x NT rows of x.
// The weights' scale of a block is then one number per tile, the rows' scales are along the
// registers of a thread. Warp 0 copies, warp 1 issues the MMAs, the others scale and add: four of them (one
// per quarter of tensor memory's lanes), or eight for 64 columns (half the columns each). The
// blocks of the contraction are split over a cluster's CTAs; their sums meet in shared memory and
// are added in rank order.
template <int NT>
struct Cols {
    static constexpr int kParts = NT >= 64 ? 2 : 1;               // warps per quarter of the lanes
    static constexpr int kCols = NT / kParts;                     // columns (and fp32 sums) of a thread
    static constexpr int kReaders = 128 * kParts;
    static constexpr int kThreads = 64 + kReaders;
    static constexpr int kStage = 128 * 128 + NT * 128;
    static constexpr int kStages = NT <= 32 ? 5 : 4;
    static constexpr uint32_t kTmem = 2 * NT < 32 ? 32 : 2 * NT;  // two accumulators
    static constexpr int kJoin = NT * 128 * 4;                    // this CTA's sums for the join
    static constexpr int kData = kStages * kStage > kJoin ? kStages * kStage : kJoin;
    static constexpr int kSmem = kData + 2 * NT * 4 + (2 * kStages + 4) * 8 + 16 + 1024;
};

template <int NT>
__global__ void __launch_bounds__(Cols<NT>::kThreads, 2)
fp8_cols_kernel(Fp8GemmArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, int split) {
    using G = Cols<NT>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* sc = reinterpret_cast<float*>(sm + G::kData);  // [2][NT]: the rows' scales of a block
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + G::kData + 2 * NT * 4);
    uint64_t* empty = full + G::kStages;
    uint64_t* tfull = empty + G::kStages;
    uint64_t* tempty = tfull + 2;
    uint32_t* slot = reinterpret_cast<uint32_t*>(tempty + 2);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    const int64_t tile = blockIdx.x / (unsigned)split, mt = (a.m + NT - 1) / NT;
    const int64_t m0 = tile % mt * NT, n0 = tile / mt * 128;
    const int nb = (a.k + 127) / 128;
    const int b0 = (int)((int64_t)nb * rank / split), b1 = (int)((int64_t)nb * (rank + 1) / split);

    if (tid == 0) {
        for (int i = 0; i < G::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], G::kReaders / 32);
        }
        mbar_fence_init();
        prefetch_tmap(&wmap);
        prefetch_tmap(&xmap);
    }
    if (warp == 1) tmem_alloc(slot, G::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *slot;
    wait_prior_grid();
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !mbar_wait(bar, parity, kWaitNs)) {
            ok = false;
            set_status(a.status, CSA2_DEV_TIMEOUT);
        }
        return ok;
    };

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int b = b0, i = 0; b < b1; ++b, ++i) {
                const int st = i % G::kStages;
                if (i >= G::kStages && !wait(&empty[st], ((i / G::kStages) - 1) & 1)) break;
                unsigned char* d = sm + st * G::kStage;
                mbar_expect_tx(&full[st], G::kStage);
                tma_2d_g2s(d, &wmap, b * 128, (int)n0, &full[st]);
                tma_2d_g2s(d + 128 * 128, &xmap, b * 128, (int)m0, &full[st]);
                issued = i + 1;
            }
            // no copy is in flight when the CTA ends, even when a wait ran out (bounded again)
            for (int i = issued > G::kStages ? issued - G::kStages : 0; i < issued; ++i)
                mbar_wait(&full[i % G::kStages], (i / G::kStages) & 1, kWaitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            for (int b = b0, i = 0; b < b1; ++b, ++i) {
                const int st = i % G::kStages, buf = i & 1;
                if (i >= 2 && !wait(&tempty[buf], ((i >> 1) - 1) & 1)) break;
                if (!wait(&full[st], (i / G::kStages) & 1)) break;
                tc_fence_after();
                const uint32_t ad = smem_u32(sm + st * G::kStage), bd = ad + 128 * 128;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    mma_f8(tb + buf * NT, sw128_desc(ad + 32 * q), sw128_desc(bd + 32 * q), f8_idesc(128, NT), q > 0);
                mma_commit(&tfull[buf]);
                mma_commit(&empty[st]);
            }
        }
        __syncwarp();
    } else {
        const int et = tid - 64;          // 0 .. kReaders - 1
        const int quad = warp & 3;        // the tensor-memory lanes this warp may read
        const int col0 = G::kParts == 2 ? (warp - 2) / 4 * G::kCols : 0;
        // this thread's row of x, whose scales it fetches (two blocks ahead: nothing waits for them)
        const bool mine = et < NT && m0 + et < a.m;
        const float* xs = a.xs + (int64_t)b0 * a.m + (mine ? m0 + et : 0);
        const float* ws = a.ws + (n0 >> 7) * nb;
        uint64_t acc[G::kCols / 2];
#pragma unroll
        for (int i = 0; i < G::kCols / 2; ++i) acc[i] = 0ull;
        float x0 = __ldg(xs), w0 = __ldg(ws + b0), x1 = 0.f, w1 = 0.f;
        if (b0 + 1 < b1) {
            x1 = __ldg(xs += a.m);
            w1 = __ldg(ws + b0 + 1);
        }
        for (int b = b0, i = 0; b < b1; ++b, ++i) {
            const int buf = i & 1;
            float x2 = 0.f, w2 = 0.f;
            if (b + 2 < b1) {
                x2 = __ldg(xs += a.m);
                w2 = __ldg(ws + b + 2);
            }
            if (et < NT) sc[buf * NT + et] = mine ? x0 * w0 : 0.f;
            x0 = x1, w0 = w1, x1 = x2, w1 = w2;
            asm volatile("bar.sync 1, %0;" ::"n"(G::kReaders) : "memory");  // the scales of block b (and b - 1 is read)
            wait(&tfull[buf], (i >> 1) & 1);
            tc_fence_after();
            constexpr int W = G::kCols < 32 ? 16 : 32;
            const uint32_t at = tb + ((uint32_t)(32 * quad) << 16) + buf * NT + col0;
            const float* s = sc + buf * NT + col0;
#pragma unroll
            for (int c = 0; c < G::kCols; c += W) {
                uint32_t v[W];
                if constexpr (W == 32) tmem_ld32(at + c, v); else tmem_ld16(at + c, v);
                tmem_ld_done(v);
                if (c + W == G::kCols) {  // the last part is in registers: the accumulator may be written again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tempty[buf]);
                }
#pragma unroll
                for (int j = 0; j < W; j += 4) {
                    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(s + c + j);
                    fma2(acc[(c + j) / 2], v[j], v[j + 1], f.x);
                    fma2(acc[(c + j) / 2 + 1], v[j + 2], v[j + 3], f.y);
                }
            }
        }
        const int n = 32 * quad + lane;
        // every copy of this CTA has landed and been read: with a split the stages become the sums [NT][128]
        float* part = reinterpret_cast<float*>(sm);
#pragma unroll
        for (int i = 0; i < G::kCols; ++i) {
            const float2 x = unpack2(acc[i / 2]);
            const float v = i & 1 ? x.y : x.x;
            if (split > 1)
                part[(col0 + i) * 128 + n] = v;
            else if (n0 + n < a.n && m0 + col0 + i < a.m)
                store_out(a, m0 + col0 + i, n0 + n, v);
        }
    }
    if (split > 1) {
        cluster_sync();
        const int i0 = NT * rank / split, i1 = NT * (rank + 1) / split;
        for (int e = tid + i0 * 128; e < i1 * 128; e += G::kThreads) {
            const int i = e >> 7, n = e & 127;
            if (m0 + i >= a.m || n0 + n >= a.n) continue;
            float v = 0.f;
            for (int r = 0; r < split; ++r) v += ld_cluster(smem_u32(sm) + 4u * e, r);
            store_out(a, m0 + i, n0 + n, v);
        }
        cluster_sync();  // the peers have read this CTA's sums
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tb, G::kTmem);
}

// ---- large products: rows of x on the lanes --------------------------------------------------------------
//
// Tiles of 128 rows of x x 256 weight rows. A lane of tensor memory is a row of x: the row's scale of a
// block is one number per thread. Persistent: each CTA takes tiles in turn, rows fastest, so that those at
// work share weight rows in L2.
// Warp 0 copies, warp 1 issues the MMAs, warps 4 .. 11 scale and add (two per quarter of the lanes, 128
// columns and 128 fp32 sums a thread). Two accumulators of 256 columns alternate block by block: while the
// tensor cores write one, the other is read. The reading bounds it: without the products of the scales the
// rest of the kernel takes 420 us where the whole takes 565 (4096 x 4096 x 32768, 1.95 PFLOP/s). Tried and
// slower there: 16 reading warps (700 us), four accumulators of 128 columns (917), pairs of CTAs sharing
// the weights (cta_group::2: 571, and 45 against 28 for 128 rows), the two column halves on barriers of their
// own (710). Tiles of 224 columns would give 128 x 32768 all SMs, but a part of theirs has two scales: 38 us
// against 29. Asking L2 for the first weights while the kernel before runs: no gain.
// The tile leaves through shared memory, so that a warp's stores are whole lines of a row at any alignment.
constexpr int kRowsThreads = 384;
// registers at launch: 168 x 384; the copying warpgroup gives up 112, the two others take 56 each
constexpr uint32_t kRegsFew = 56, kRegsMany = 224;
constexpr int kRowsStage = 128 * 128 + 256 * 128, kRowsStages = 4;
constexpr int kRowsOut = 8 * 32 * 33 * 4;  // per reading warp: 32 rows of 32 words, rows one bank apart
constexpr int kRowsSmem = kRowsStages * kRowsStage + kRowsOut + (2 * kRowsStages + 4) * 8 + 16 + 1024;

// The warp's 32 rows (row0 + lane), 32 words each in its buffer (row r at 33 r; a word one fp32 or two bf16
// columns from col on), to out. wide: every row starts on 16 bytes.
__device__ __forceinline__ void store_words(const Fp8GemmArgs& a, const uint32_t* b, int64_t row0, int64_t col, bool wide,
                                            int lane) {
    __syncwarp();
    const int per = a.out_f32 ? 1 : 2;  // columns of a word
    const int rows = a.m - row0 < 32 ? (int)(a.m - row0) : 32;
    if (wide && col + 32 * per <= a.n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), c = 4 * (lane & 7);
            const uint4 v = make_uint4(b[r * 33 + c], b[r * 33 + c + 1], b[r * 33 + c + 2], b[r * 33 + c + 3]);
            if (r < rows)
                *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(a.out) +
                                          ((row0 + r) * a.out_stride + col + per * c) * (4 / per)) = v;
        }
    } else if (a.out_f32) {
        for (int r = 0; r < rows; ++r)
            if (col + lane < a.n)
                reinterpret_cast<uint32_t*>(a.out)[(row0 + r) * a.out_stride + col + lane] = b[r * 33 + lane];
    } else {
        for (int r = 0; r < rows; ++r) {
            const uint32_t v = b[r * 33 + lane];
            uint16_t* d = reinterpret_cast<uint16_t*>(a.out) + (row0 + r) * a.out_stride + col + 2 * lane;
            if (col + 2 * lane < a.n) d[0] = (uint16_t)v;
            if (col + 2 * lane + 1 < a.n) d[1] = (uint16_t)(v >> 16);
        }
    }
}

__global__ void __launch_bounds__(kRowsThreads, 1)
fp8_rows_gemm_kernel(Fp8GemmArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                     int mt, int tiles) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* outs = reinterpret_cast<float*>(sm + kRowsStages * kRowsStage);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + kRowsStages * kRowsStage + kRowsOut);
    uint64_t* empty = full + kRowsStages;
    uint64_t* tfull = empty + kRowsStages;
    uint64_t* tempty = tfull + 2;
    uint32_t* slot = reinterpret_cast<uint32_t*>(tempty + 2);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int step = (int)gridDim.x, first = (int)blockIdx.x;
    const int nb = (a.k + 127) / 128;

    if (tid == 0) {
        for (int i = 0; i < kRowsStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 8);
        }
        mbar_fence_init();
        prefetch_tmap(&wmap);
        prefetch_tmap(&xmap);
    }
    if (warp == 1) tmem_alloc(slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *slot;
    wait_prior_grid();
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !mbar_wait(bar, parity, kWaitNs)) {
            ok = false;
            set_status(a.status, CSA2_DEV_TIMEOUT);
        }
        return ok;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
        int st = 0;
        uint32_t ph = 0;  // the stage in turn and how often (parity) the ring has gone round
        auto next = [&]() {
            if (++st == kRowsStages) {
                st = 0;
                ph ^= 1u;
            }
        };
        if (warp == 0 && lane == 0) {
            for (int t = first; t < tiles && ok; t += step) {
                const int m0 = (int)(t % mt * 128), n0 = (int)(t / mt * 256);
                for (int b = 0; b < nb; ++b) {
                    if (!wait(&empty[st], ph ^ 1u)) break;  // (passes at once in the first round)
                    unsigned char* d = sm + st * kRowsStage;
                    mbar_expect_tx(&full[st], kRowsStage);
                    tma_2d_g2s(d, &xmap, b * 128, m0, &full[st]);
                    tma_2d_g2s(d + 128 * 128, &wmap, b * 128, n0, &full[st]);
                    tma_2d_g2s(d + 2 * 128 * 128, &wmap, b * 128, n0 + 128, &full[st]);
                    next();
                }
            }
            // every stage is read (its last commit has arrived) before this CTA may end
            for (int j = 0; j < kRowsStages; ++j) {
                mbar_wait(&empty[st], ph ^ 1u, kWaitNs);
                next();
            }
        } else if (warp == 1 && lane == 0) {
            uint32_t i = 0;  // accumulators written so far
            for (int t = first; t < tiles && ok; t += step) {
                for (int b = 0; b < nb && ok; ++b, ++i) {
                    const uint32_t buf = i & 1u;
                    if (!wait(&full[st], ph) || !wait(&tempty[buf], ((i >> 1) & 1u) ^ 1u)) break;
                    tc_fence_after();
                    const uint32_t ad = smem_u32(sm + st * kRowsStage), bd = ad + 128 * 128;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mma_f8(tb + buf * 256, sw128_desc(ad + 32 * q), sw128_desc(bd + 32 * q), f8_idesc(128, 256), q > 0);
                    mma_commit(&tfull[buf]);
                    mma_commit(&empty[st]);
                    next();
                }
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
        const int quad = warp & 3, part = (warp - 4) >> 2;
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        uint32_t i = 0;
        for (int t = first; t < tiles; t += step) {
            const int row0 = t % mt * 128 + 32 * quad, row = row0 + lane;
            const int col = t / mt * 256 + 128 * part;  // (below 2^31: the padded sizes are checked at launch)
            // the next block's scales are on their way (their product is formed when they are used, so that
            // nothing waits for them before)
            const bool live = row < a.m && col < a.n;
            const float* xs = a.xs + (live ? row : 0);
            const float* ws = a.ws + (live ? (col >> 7) * nb : 0);
            uint64_t acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = 0ull;
            float x0 = __ldg(xs), w0 = __ldg(ws);
            for (int b = 0; b < nb; ++b, ++i) {
                const float f = x0 * w0;
                const uint64_t s = pack2(f, f);
                if (b + 1 < nb) {
                    x0 = __ldg(xs += a.m);
                    w0 = __ldg(ws + b + 1);
                }
                const uint32_t buf = i & 1u;
                wait(&tfull[buf], (i >> 1) & 1u);
                tc_fence_after();
                const uint32_t at = tb + lanes + buf * 256 + 128 * part;
                uint32_t v[2][32];
                tmem_ld32(at, v[0]);
                tmem_ld_done(v[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c < 3) tmem_ld32(at + 32 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
                    for (int j = 0; j < 16; ++j) fma2(acc[16 * c + j], v[c & 1][2 * j], v[c & 1][2 * j + 1], s);
                    if (c < 3) tmem_ld_done(v[(c + 1) & 1]);
                    if (c == 2) {  // the last part is in registers: the accumulator may be written again
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tempty[buf]);
                    }
                }
            }
            if (row0 < a.m && col < a.n) {
                // (the words leave the registers one by one: no copy of them is live beside the sums)
                uint32_t* buffer = reinterpret_cast<uint32_t*>(outs) + (warp - 4) * 32 * 33;
                // 16-byte stores where every row starts on 16 bytes
                const bool wide = ((uintptr_t)a.out & 15) == 0 && a.out_stride % (a.out_f32 ? 4 : 8) == 0;
                if (a.out_f32) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        __syncwarp();  // the words before are read
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 x = unpack2(acc[16 * c + j]);
                            buffer[lane * 33 + 2 * j] = __float_as_uint(x.x);
                            buffer[lane * 33 + 2 * j + 1] = __float_as_uint(x.y);
                        }
                        store_words(a, buffer, row0, col + 32 * c, wide, lane);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float2 x = unpack2(acc[32 * c + j]);
                            const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
                            buffer[lane * 33 + j] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                        store_words(a, buffer, row0, col + 64 * c, wide, lane);
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tb, 512);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// rows x k bytes, boxes of box_rows x 128 in the 128-byte swizzle; past the edges zeros are read
cudaError_t make_map(CUtensorMap* map, const uint8_t* p, int64_t rows, int k, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dim[2] = {(cuuint64_t)k, (cuuint64_t)rows}, str[1] = {(cuuint64_t)k};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dim, str, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess : cudaErrorInvalidValue;
}

template <int NT>
cudaError_t launch_cols(const Fp8GemmArgs& a, cudaStream_t s) {
    using G = Cols<NT>;
    auto k = fp8_cols_kernel<NT>;
    CUtensorMap wmap, xmap;
    cudaError_t e = make_map(&wmap, a.w, a.n, a.k, 128);
    if (e == cudaSuccess) e = make_map(&xmap, a.x, a.m, a.k, NT);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((a.n + 127) / 128) * ((a.m + NT - 1) / NT);
    const int nb = (a.k + 127) / 128;
    const int split = fp8_cols_split(tiles, nb);
    if (tiles * split > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_cluster(k, dim3((unsigned)(tiles * split)), dim3(G::kThreads), split, G::kSmem, s, a, wmap, xmap, split);
}

cudaError_t launch_rows_gemm(const Fp8GemmArgs& a, cudaStream_t s) {
    CUtensorMap wmap, xmap;
    cudaError_t e = make_map(&wmap, a.w, a.n, a.k, 128);
    if (e == cudaSuccess) e = make_map(&xmap, a.x, a.m, a.k, 128);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fp8_rows_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t mt = (a.m + 127) / 128, tiles = mt * ((a.n + 255) / 256);
    if (tiles > 0x3FFFFFFF || a.m > 0x7FFFFE00 || a.n > 0x7FFFFE00) return cudaErrorInvalidConfiguration;
    return launch_after_prior(fp8_rows_gemm_kernel, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(kRowsThreads),
                              kRowsSmem, s, a, wmap, xmap, (int)mt, (int)tiles);
}

}  // namespace

cudaError_t launch_fp8_rows(int64_t rows, int k, const uint16_t* x, int64_t x_stride, uint8_t* data, float* scale,
                            cudaStream_t s) {
    const int nb = (k + 127) / 128;
    const int64_t gx = (rows + 15) / 16;
    if (gx > 0x7FFFFFFF || nb > 65535) return cudaErrorInvalidConfiguration;
    // several blocks per lane group once they fill the GPU (eight CTAs an SM)
    if (gx * nb >= 148 * 8 * 4)
        return launch_after_prior(fp8_rows_kernel<4>, dim3((unsigned)gx, (unsigned)((nb + 3) / 4)), dim3(256), 0, s,
                                  rows, k, x, x_stride, data, scale);
    return launch_after_prior(fp8_rows_kernel<1>, dim3((unsigned)gx, (unsigned)nb), dim3(256), 0, s, rows, k, x,
                              x_stride, data, scale);
}

cudaError_t launch_fp8_weight(int64_t n, int k, const uint16_t* w, uint8_t* data, float* scale, cudaStream_t s) {
    const int64_t gy = (n + 127) / 128;
    if (gy > 65535) return cudaErrorInvalidConfiguration;
    return launch_after_prior(fp8_weight_kernel, dim3((unsigned)((k + 127) / 128), (unsigned)gy), dim3(256), 0, s, n, k,
                              w, data, scale);
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t s) {
    if (a.m <= 16) return launch_cols<16>(a, s);
    if (a.m <= 32) return launch_cols<32>(a, s);
    if (a.m <= 64) return launch_cols<64>(a, s);
    return fp8_by_columns(a.m, a.n, a.k) ? launch_cols<64>(a, s) : launch_rows_gemm(a, s);
}

}  // namespace csa2
