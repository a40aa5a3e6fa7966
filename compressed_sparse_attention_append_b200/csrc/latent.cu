// latent.cu -- sparse attention in the pages' own shape on the tensor cores: 64 query heads of 512
// channels over a 512-channel latent that is both key and value.
//
// [C] "DeepSeek-V4.1-Flash: Pushing KV Cache Compression to 890 Bytes per Token":
//   sec. VII: the main KV is one 512-channel latent per entry (288 B: E2M1 codes and an E4M3 scale
//   per 16 channels); the configuration list: 64 query heads of dimension 512;
//   sec. VI: the query attends to its selected entries plus its own recent window;
//   sec. XI: cached values are dequantised before attention (E2M1 x E4M3 products and E4M3 window
//   values are exact in fp16);
//   sec. XII: a query at token i sees window tokens [max(s, i - win + 1), i].
// Reading taken here: one softmax over selected and window entries, the latent serving as K and
// V (no separate value projection), default scale 1/sqrt(512).
//
// One CTA per query row, 16 worker warps and one that issues the MMAs. The row's keys come in tiles of 128: ceil(k / 128) tiles of
// selected entries (-1 or invalid entries are zero rows, masked), then one tile of up to 128 window
// rows. Per tile:
//   1. the tile's raw rows (loaded into registers while the previous tile was being processed) are
//      dequantised ONCE into a 128 x 512 fp16 tile L in shared memory (K-major rows of 128-byte
//      swizzled 64-channel blocks);
//   2. S^T = L Q^T on tcgen05 (kind::f16, M = 128 keys, N = 64 heads, K = 512), fp32 in tensor
//      memory;
//   3. softmax: each thread has one key's logits for 16 heads; the tile's per-head maxima are
//      reduced across the CTA (a warp reduction per head, then the four lane quarters through
//      shared memory); the running maximum m of a head moves only when the tile exceeds it
//      by more than 8 (in log2 units), and then the head's accumulated O and l are rescaled (in
//      tensor memory), so P = exp2(logit - m) <= 2^8 stays well inside fp16; P is rounded to fp16
//      into shared memory, [key][head] (MN-major). Every warp moves the maxima of its own heads, so
//      a tile has one barrier;
//   4. O^T += L^T P^T on tcgen05 (M = 128 channels, four M tiles, N = 64 heads, K = 128 keys): the
//      same shared-memory bytes of L, read MN-major (channels contiguous), so the latent is
//      dequantised once for both products.
// The two channel halves of L (64-channel blocks 0..3 and 4..7) are dequantised one after the other,
// each as soon as the O^T MMAs of the previous tile that read it have completed, and the
// S^T k-steps of a half are issued as soon as that half is in place (mbarriers between the workers
// and the MMA warp), so dequantisation overlaps the tensor pipe. An MMA is issued only once the pipe has
// room for it: 32 of them hold their thread for as long as they run (2,300 to 3,200 cycles), which is why
// they have a warp of their own. With it 96 registers a thread are left, so the softmax reads its logits
// twice instead of keeping them. Five tiles at 128 rows: 29.7 us a call, against 37.2 with the MMAs on a
// worker and two barriers more per tile (channel quarters in place of halves 30.9; 20 warps with
// setmaxnreg spill).
// Four lanes take a key, 16 bytes each of every 64 of its row: a warp's load touches 8 lines, not 32; a key's
// scales are read once, 8 a lane, and passed between its lanes. The row's indices are checked
// and staged in shared memory once, so no tile waits on a dependent index load. Q arrives by one bulk copy.
// Tensor memory: S^T in columns 0..63, O^T in columns 64..319 (channels on the lanes).
// The result is normalised by the per-head sum of P at the end: out = O / l, lse = m ln 2 + ln l. A row without a
// key has l = 0 exactly; with one, l is about 1 or more, or NaN (a logit that is not finite), which goes into out and lse.
// Every wait on the tensor cores is bounded; one that runs out sets CSA2_DEV_TIMEOUT.
#include <atomic>

#include "attend_plan.h"
#include "csa2_internal.cuh"
#include "tc.cuh"

namespace csa2 {

namespace {

using namespace tc;

constexpr int kT = 512;                       // workers; loads: key tid >> 2, a quarter of its chunks each
constexpr int kThreads = kT + 32;             // and a warp one thread of which issues the MMAs
constexpr int kTile = 128;                    // keys per tile (MMA M of S^T)
constexpr int kBlk = kTile * 128;             // 16384: one 64-channel block of the L tile
constexpr int kLTile = 8 * kBlk;              // 131072: the fp16 L tile
constexpr int kQBlk = kLatHQ * 128;           // 8192: one 64-channel block of Q (64 heads)
constexpr int kQBytes = 8 * kQBlk;            // 65536
constexpr int kPBytes = kTile * 128;          // 16384: P, 128 keys x 64 heads fp16
constexpr uint32_t kCols = 512;               // tensor memory allocated (power of two >= 320)
constexpr uint32_t kSCol = 0, kOCol = 64;
constexpr float kLazy = 8.f;
constexpr uint64_t kWaitNs = 200000000ull;
// f16 x f16 -> f32, M 128, N 64; S^T: both operands K-major; O^T: both MN-major (bits 15, 16)
constexpr uint32_t kIdescS = (1u << 4) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescO = kIdescS | (1u << 15) | (1u << 16);
constexpr size_t kOffQ = kLTile, kOffP = kOffQ + kQBytes, kOffIdx = kOffP + kPBytes;
constexpr size_t kOffRed = kOffIdx + 4 * kMaxK;
constexpr size_t kOffM = kOffRed + 4 * 64 * 4, kOffAl = kOffM + 64 * 4, kOffL = kOffAl + 64 * 4;
constexpr size_t kOffW = kOffL + 64 * 4, kOffBar = kOffW + (kT / 32) * 32 * 4, kOffSlot = kOffBar + 8 * 8;
constexpr size_t kUsed = kOffSlot + 16;
// the whole 227 KB: one CTA per SM (tensor memory and the L tile allow no second one)
constexpr size_t kSmem = 232448;
static_assert(kUsed + 1024 <= kSmem, "shared memory plan");
// mbarriers: S^T done; O^T of channel half 0 / 1 done; channel half 0 / 1 of L dequantised; Q as it is in place;
// P in place
enum { kBarS = 0, kBarO0 = 1, kBarO1 = 2, kBarH0 = 3, kBarH1 = 4, kBarQ = 5, kBarP = 6 };

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

// MN-major operand in the 128-byte swizzle pattern: 64-element groups of the M (or N) dimension
// `lbo` bytes apart, 8-row groups of K 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t addr, uint32_t lbo) {
    return sw128_desc(addr) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16);
}

// byte offset of 16-byte chunk c of row r in a 128-byte-swizzled block (8-row groups of 1024 bytes)
__device__ __forceinline__ uint32_t sw(int r, int c) { return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t scale_h2(uint32_t s) { return e4m3x2_to_h2((uint16_t)(s | (s << 8))); }

// the largest value of v over the warp, in every lane (sm_100a warp reduction)
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// 2^x (the hardware approximation: relative error about 2^-22; results below 2^-126 flush to 0)
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 8 columns of this warp's lanes of tensor memory
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// a barrier of the worker warps alone
__device__ __forceinline__ void workers_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kT) : "memory"); }

// 16 lanes' worth of sums reduced across the warp: lane L < 16 ends with the sum over all 32 lanes
// of element L (the transposing butterfly: each step halves the elements a lane keeps).
__device__ __forceinline__ float warp_sum16(float (&v)[16], int lane) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float keep = up ? v[i + w] : v[i], send = up ? v[i] : v[i + w];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
        }
    }
    return v[0];
}

// PAGED: the entries and window rings are those of a paged cache (a.pg); the row's indices are
// translated to plane rows while they are staged, once per row. There a row's tiles may be split over the
// a.split CTAs of a cluster (few rows leave most of the GPU idle): each runs its tiles as a row of its
// own, and the partial results meet in shared memory: the CTAs' maxima and sums give each its factor
// 2^(m_r - m) / l, each writes its scaled O over its L tile, and each adds up its share of the heads in
// rank order.
template <bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) latent_attend_kernel(LatentAttendArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* Lt = sm;
    unsigned char* Qs = sm + kOffQ;
    unsigned char* Ps = sm + kOffP;
    int* sidx = reinterpret_cast<int*>(sm + kOffIdx);       // the row's selected entries, -1 if unusable
    float* red = reinterpret_cast<float*>(sm + kOffRed);   // [4 lane quarters][64 heads]
    float* s_m = reinterpret_cast<float*>(sm + kOffM);     // final maximum per head (log2 units)
    float* s_al = reinterpret_cast<float*>(sm + kOffAl);   // final factor per head
    float* s_l = reinterpret_cast<float*>(sm + kOffL);     // final sum per head
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + kOffSlot);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lkey = tid >> 2, qq = tid & 3;       // load / dequantise: key of the tile, 16-byte chunks 4 c + qq of its row
    const int key = tid & 127;                     // softmax: key (tensor-memory lane 32 quad + lane)
    const int quad = warp & 3, cg = warp >> 2;     // softmax / epilogue: lanes 32 quad .., heads 16 cg ..
    const int split = PAGED ? a.split : 1;
    const int rank = PAGED && split > 1 ? (int)cluster_rank() : 0;
    const int row = PAGED ? (int)(blockIdx.x / (unsigned)split) : (int)blockIdx.x, K = a.k;
    const bool issuer = warp == kT / 32;
    if (tid == kT) {
        mbar_init(&bars[kBarS], 1);
        mbar_init(&bars[kBarP], kT / 32);
        mbar_init(&bars[kBarO0], 1);
        mbar_init(&bars[kBarO1], 1);
        mbar_init(&bars[kBarH0], kT / 32);
        mbar_init(&bars[kBarH1], kT / 32);
        mbar_init(&bars[kBarQ], 1);
        mbar_fence_init();
    }
    start_next_grid();  // (0.5 us less in a run of calls: the next launch is set up beside this one)
    wait_prior_grid();  // indices, cache and queries come from earlier work on the stream
    // Q goes to the L tile's place as it is, past the registers and the load path, while the row's indices are
    // staged and tile 0's rows requested; it is converted there before the first dequantisation.
    if (tid == kT) {
        mbar_expect_tx(&bars[kBarQ], kQBytes);
        bulk_g2s(Lt, a.q + (size_t)row * kLatHQ * kLatD, kQBytes, &bars[kBarQ]);
    }
    __syncwarp();
    // (takes some 3500 cycles: under way while the workers fetch the row's position and indices)
    if (issuer) tmem_alloc(tslot, kCols);

    // the row's tiles, of which this CTA has t0 .. t0 + nt - 1
    const int b = row / a.tq;
    const int ft = (K + kTile - 1) / kTile, all = ft + (a.win > 0 ? 1 : 0);
    const int t0 = PAGED ? all * rank / split : 0, t1 = PAGED ? all * (rank + 1) / split : all;
    const int i0 = t0 * kTile, i1 = t1 * kTile < K ? t1 * kTile : K;
    // (the loads that wait for nothing are all under way before the first of them is used)
    const int first = !issuer && i0 + tid < i1 ? __ldg(a.idx + (size_t)row * K + i0 + tid) : -1;
    const int64_t qpos = __ldg(a.qpos + row);
    const int64_t sb = __ldg(a.swa_begin ? a.swa_begin + b : a.qpos + row);  // (no branch: it would keep the next load back)
    int64_t ring = b;  // the window ring of this row
    if constexpr (PAGED) ring = a.win > 0 ? paged_slot(a.pg, b) : -1;
    const int64_t qlast = ((qpos + 1) >> (a.ratio - 1)) - 1;  // the last visible entry (below 0 for qpos < 0)
    // (a page table bounds its own entries, each index is checked against it: the window needs none of them)
    const bool row_ok = qpos >= 0 && (PAGED || qlast < a.c.cap);
    int64_t lo = qpos - a.win + 1;
    if (a.swa_begin && lo < sb) lo = sb;
    if (lo < 0) lo = 0;
    if (PAGED && ring < 0 && a.win > 0 && tid == 0) set_status(a.status, CSA2_DEV_BAD_PAGE);
    const int nwin = (row_ok && qpos >= lo && (!PAGED || ring >= 0)) ? (int)(qpos - lo + 1) : 0;
    int nt = row_ok ? t1 - t0 : 0;
    if (nt > 0 && t1 > ft && nwin == 0) --nt;
    const float scale2 = a.sm_scale * 1.4426950408889634f;  // logits in log2 units
    uint32_t* status = a.status;

    // the row's indices, checked once (an entry that is -1, not visible or out of range becomes -1)
    for (int i = i0 + tid; i < (row_ok && !issuer ? i1 : 0); i += kT) {
        const int v = i == i0 + tid ? first : __ldg(a.idx + (size_t)row * K + i);
        const bool ok = v >= 0 && (int64_t)v <= qlast && (int64_t)v < a.c.cap;
        if (!ok && v != -1) set_status(status, CSA2_DEV_BAD_INDEX);
        if constexpr (PAGED) {
            const int64_t at = ok ? paged_row(a.pg, b, v) : -1;  // a plane row (below 2^31)
            if (ok && at < 0) set_status(status, CSA2_DEV_BAD_PAGE);
            sidx[i] = (int)at;
        } else {
            sidx[i] = ok ? v : -1;
        }
    }

    const size_t seq_row0 = PAGED ? 0 : (size_t)b * a.c.cap;
    const size_t swa_row0 = (size_t)(PAGED ? ring : (int64_t)b) * a.c.swa_cap;
    bool ok_all = true;
    auto wait_bar = [&](int i, uint32_t parity) {
        if (!mbar_wait(&bars[i], parity, kWaitNs)) {
            if (ok_all) set_status(status, CSA2_DEV_TIMEOUT);
            ok_all = false;
        }
    };

    // this thread's chunks of its window row (16 channels: 16 qq .. of 64-channel block i in chunk 4 i)
    auto win_src = [&]() {
        const int64_t p = lo + lkey;
        return reinterpret_cast<const uint4*>(a.c.swa + (swa_row0 + (size_t)(p & (a.c.swa_cap - 1))) * kLatSwa) + qq;
    };
    // ---- raw rows of tile j into registers (this thread: key lkey, of each 128 channels c the 32 from 32 qq on) ----
    // (of a window row only the first channel half: the other is loaded while it is dequantised, so that no
    // more than 18 registers of raw data stay live across the softmax of the tile before)
    uint4 raw[4];
    uint2 rsc;  // eight scales: those of channels 128 qq .. (the four lanes of a key hold each other's)
    auto load_tile = [&](int j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = make_uint4(0, 0, 0, 0);
        rsc = make_uint2(0, 0);
        if (j < nt && t0 + j < ft) {  // (the indices of this CTA's tiles are staged, no others)
            const int i = (t0 + j) * kTile + lkey;
            const int v = i < K ? sidx[i] : -1;
            if (v >= 0) {
                const uint4* src = reinterpret_cast<const uint4*>(a.c.l_data + (seq_row0 + (size_t)v) * kLatBytes) + qq;
                const uint2* sc = reinterpret_cast<const uint2*>(a.c.l_scale + (seq_row0 + (size_t)v) * kLatScales) + qq;
#pragma unroll
                for (int c = 0; c < 4; ++c) raw[c] = __ldg(src + 4 * c);
                rsc = __ldg(sc);
            }
        } else if (j < nt && lkey < nwin) {
#pragma unroll
            for (int c = 0; c < 4; ++c) raw[c] = __ldg(win_src() + 4 * c);
        }
    };
    // whether this thread's softmax key counts in tile j
    auto key_valid = [&](int j) {
        const int i = (t0 + j) * kTile + key;
        return t0 + j < ft ? i < K && sidx[i] >= 0 : key < nwin;
    };
    // channel half hh of the registers into the L tile (8-channel chunks of row lkey in its 64-channel blocks)
    auto dequant = [&](int hh, bool fp4, bool more) {
        if (fp4) {
#pragma unroll
            for (int c = 2 * hh; c < 2 * hh + 2; ++c) {
                // lanes 2 and 3 of a key, which write the next 64-channel block (the same banks), begin with their
                // second two chunks: the stores of 8 lanes then fall on different banks
                const bool far = qq >= 2;
                const uint32_t w[4] = {far ? raw[c].z : raw[c].x, far ? raw[c].w : raw[c].y, far ? raw[c].x : raw[c].z,
                                       far ? raw[c].y : raw[c].w};
                // this lane's two scales are bytes 2 qq, 2 qq + 1 of those that the key's lane c holds
                const uint32_t lo4 = __shfl_sync(0xffffffffu, rsc.x, c, 4), hi4 = __shfl_sync(0xffffffffu, rsc.y, c, 4);
                const uint32_t s16 = (far ? hi4 : lo4) >> (16 * (qq & 1));
                const uint32_t first = (far ? s16 >> 8 : s16) & 0xFFu, second = (far ? s16 : s16 >> 8) & 0xFFu;
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // 8 channels; two code words share a scale
                    const uint32_t s2 = scale_h2(i < 2 ? first : second);
                    uint32_t h[4];
                    e2m1x8_to_h2x4(w[i], h);
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = hmul2(h[k], s2);
                    *reinterpret_cast<uint4*>(Lt + (2 * c + (qq >> 1)) * kBlk + sw(lkey, 4 * (qq & 1) + (far ? i ^ 2 : i))) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
        } else {
            if (hh == 1) {
#pragma unroll
                for (int c = 0; c < 4; ++c) raw[c] = more ? __ldg(win_src() + 16 + 4 * c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // 16 window channels: two chunks of 64-channel block 4 hh + c
                const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint4*>(Lt + (4 * hh + c) * kBlk + sw(lkey, 2 * qq + i)) =
                        make_uint4(e4m3x2_to_h2((uint16_t)(w[2 * i] & 0xFFFFu)), e4m3x2_to_h2((uint16_t)(w[2 * i] >> 16)),
                                   e4m3x2_to_h2((uint16_t)(w[2 * i + 1] & 0xFFFFu)), e4m3x2_to_h2((uint16_t)(w[2 * i + 1] >> 16)));
            }
        }
    };

    __syncthreads();  // barriers, indices
    if (!issuer) {
        load_tile(0);
        wait_bar(kBarQ, 0);
        // Q -> fp16 (B operand of S^T, K-major: row = head, 64-channel blocks)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int g = tid + kT * c, h = g >> 6, ch = g & 63;  // head, 8-channel chunk
            const uint4 qv = reinterpret_cast<const uint4*>(Lt)[g];
            const uint32_t w[4] = {qv.x, qv.y, qv.z, qv.w};
            uint32_t hv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) hv[i] = pack_h2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            *reinterpret_cast<uint4*>(Qs + (ch >> 3) * kQBlk + sw(h, ch & 7)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();  // Q, tensor memory address
    tc_fence_after();
    const uint32_t tb = *tslot;
    const uint32_t lane_base = (uint32_t)(32 * quad) << 16;

    float lsum[16];  // this thread's key slot: sum of P per head 16 cg + i over the tiles so far
#pragma unroll
    for (int i = 0; i < 16; ++i) lsum[i] = 0.f;

    // Per tile j: each channel half of L is dequantised as soon as the O^T MMAs of tile j - 1 that read it
    // have completed (O^T m-tiles 0, 1 read half 0, m-tiles 2, 3 half 1), and the S^T k-steps of a half are
    // issued as soon as the half is in shared memory, so that dequantisation overlaps the tensor pipe.
    // The softmax then runs on the 16 worker warps.
    if (tid == kT) {  // the MMAs
        // (operand addresses are in the descriptors' low bits, in units of 16 bytes)
        const uint64_t sl = sw128_desc(smem_u32(Lt)), sq = sw128_desc(smem_u32(Qs)), sp = sw128_desc_mn(smem_u32(Ps), 0);
        constexpr uint64_t lbo = (uint64_t)(kBlk >> 4) << 16;
        for (int j = 0; j < nt; ++j) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                wait_bar(hh ? kBarH1 : kBarH0, (uint32_t)j & 1u);
                tc_fence_after();
#pragma unroll
                for (int kk = 16 * hh; kk < 16 * hh + 16; ++kk)
                    mma_f16(tb + kSCol, sl + ((kk >> 2) * kBlk + 32 * (kk & 3)) / 16, sq + ((kk >> 2) * kQBlk + 32 * (kk & 3)) / 16,
                            kIdescS, kk > 0);
            }
            mma_commit(&bars[kBarS]);
            wait_bar(kBarP, (uint32_t)j & 1u);
            tc_fence_after();
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                // A = L^T: channels 128 mt .. (blocks 2 mt, 2 mt + 1, kBlk apart), keys 16 kk ..;
                // B = P: heads 0..63 (one 64-element group), keys 16 kk ..
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_f16(tb + kOCol + 64 * mt, sl + lbo + (2 * mt * kBlk >> 4) + 128 * kk, sp + 128 * kk, kIdescO, j > 0 || kk > 0);
                if (mt == 1) mma_commit(&bars[kBarO0]);  // channel half 0 of L is free again
            }
            mma_commit(&bars[kBarO1]);
        }
    }
    __syncwarp();
    float m_run = -INFINITY;  // running maximum of head 16 cg + (lane & 15) (log2 units)
    float* wm = reinterpret_cast<float*>(sm + kOffW) + 32 * warp;  // this warp's maxima and rescale factors
    for (int j = 0; j < (issuer ? 0 : nt); ++j) {
        const bool fp4 = t0 + j < ft;  // CTA-uniform
        const bool more = lkey < nwin;
        const bool valid = key_valid(j);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            if (j > 0) wait_bar(hh ? kBarO1 : kBarO0, (uint32_t)(j - 1) & 1u);
            dequant(hh, fp4, more);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[hh ? kBarH1 : kBarH0]);
        }
        if (j + 1 < nt) load_tile(j + 1);  // in flight during this tile's MMAs and softmax
        wait_bar(kBarS, (uint32_t)j & 1u);  // also every earlier MMA (the O^T of tile j - 1)
        tc_fence_after();

        // ---- softmax of the tile: this thread's key 32 quad + lane (= key), heads 16 cg .. +15 ----
        {  // (raw logits q . l: the scale is applied inside the exponent)
            uint32_t v[16];
            tmem_ld16(tb + lane_base + kSCol + 16 * cg, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                float r[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)  // (any sign of the scale)
                    r[k] = warp_max(valid ? __uint_as_float(v[i + k]) * scale2 : -INFINITY);
                if (lane == 0) *reinterpret_cast<float4*>(red + quad * 64 + 16 * cg + i) = make_float4(r[0], r[1], r[2], r[3]);
            }
        }
        workers_sync();
        // every warp moves the maxima of its heads itself (the same in the four warps that have them)
        {
            const float* rd = red + 16 * cg + (lane & 15);
            const float tmax = fmaxf(fmaxf(rd[0], rd[64]), fmaxf(rd[128], rd[192]));
            float al = 1.f;
            bool moved = false;
            if (tmax > m_run + kLazy) {  // also the first finite maximum (m_run = -inf: nothing is summed yet)
                moved = m_run != -INFINITY;
                if (moved) al = exp2f(m_run - tmax);
                m_run = tmax;
            }
            wm[lane] = lane < 16 ? m_run : al;
            const bool resc = __any_sync(0xffffffffu, moved);
            __syncwarp();
            if (resc) {
                // every O^T MMA so far has completed (the S^T commit tracks them): scale in place
#pragma unroll
                for (int o = 0; o < 16; o += 8) {
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) {
                        uint32_t v[8];
                        const uint32_t addr = tb + lane_base + kOCol + 64 * mt + 16 * cg + o;
                        tmem_ld8(addr, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * wm[16 + o + i]);
                        tmem_st8(addr, v);
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) lsum[i] *= wm[16 + i];
                tmem_st_wait();
            }
        }
        // a valid key makes every head's maximum finite, so p needs no test of m for -inf
        // (the logits are read again: registers to keep them are not there)
#pragma unroll
        for (int o = 0; o < 16; o += 8) {
            uint32_t v[8], ph[4];
            tmem_ld8(tb + lane_base + kSCol + 16 * cg + o, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float p0 = valid ? ex2(fmaf(__uint_as_float(v[i]), scale2, -wm[o + i])) : 0.f;
                const float p1 = valid ? ex2(fmaf(__uint_as_float(v[i + 1]), scale2, -wm[o + i + 1])) : 0.f;
                lsum[o + i] += p0;
                lsum[o + i + 1] += p1;
                ph[i >> 1] = pack_h2(p0, p1);
            }
            // P [key][head]: heads 16 cg .. +7 -> chunk 2 cg, 16 cg + 8 .. -> chunk 2 cg + 1
            *reinterpret_cast<uint4*>(Ps + sw(key, 2 * cg + o / 8)) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarP]);
    }
    if (nt > 0) {
        wait_bar(kBarO1, (uint32_t)(nt - 1) & 1u);  // the last MMAs (in issue order)
        tc_fence_after();
    }

    // ---- epilogue: l per head, then out = O / l (warp: channels 128 mt + 32 quad + lane, heads 16 cg ..) ----
    if (!issuer) {
        const float r = warp_sum16(lsum, lane);
        if (lane < 16) red[quad * 64 + 16 * cg + lane] = r;
        if (quad == 0 && lane < 16) s_m[16 * cg + lane] = m_run;
    }
    __syncthreads();
    if (PAGED && split > 1) {
        // this CTA's l and m per head, then the row's: its factor is 2^(m_r - m) / l (0 without a key)
        if (tid < 64) s_l[tid] = nt > 0 ? (red[tid] + red[64 + tid]) + (red[128 + tid] + red[192 + tid]) : 0.f;
        __syncthreads();
        cluster_sync();
        if (tid < 64) {
            float m = -INFINITY, l = 0.f;
            for (int r = 0; r < split; ++r) m = fmaxf(m, ld_cluster(smem_u32(&s_m[tid]), r));
            for (int r = 0; r < split; ++r) {
                const float mr = ld_cluster(smem_u32(&s_m[tid]), r), lr = ld_cluster(smem_u32(&s_l[tid]), r);
                if (lr != 0.f) l = fmaf(lr, exp2f(mr - m), l);
            }
            const bool em = l == 0.f;
            s_al[tid] = s_l[tid] == 0.f ? 0.f : exp2f(s_m[tid] - m) / l;
            if (a.lse && rank == 0) a.lse[(size_t)row * kLatHQ + tid] = em ? -INFINITY : m * 0.6931471805599453f + logf(l);
        }
        __syncthreads();
        // every MMA that reads L has completed: O goes there as fp32 [head][512]
        float* part = reinterpret_cast<float*>(Lt);
#pragma unroll
        for (int mt = 0; mt < (issuer ? 0 : 4); ++mt) {
            uint32_t v[16] = {};
            if (nt > 0) {
                tmem_ld16(tb + lane_base + kOCol + 64 * mt + 16 * cg, v);
                tmem_ld_wait();
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float f = s_al[16 * cg + i];
                part[(16 * cg + i) * kLatD + 128 * mt + 32 * quad + lane] = f != 0.f ? __uint_as_float(v[i]) * f : 0.f;
            }
        }
        __syncthreads();
        cluster_sync();
        const int e0 = kLatHQ * rank / split * kLatD, e1 = kLatHQ * (rank + 1) / split * kLatD;
        for (int e = e0 + 4 * tid; e < (issuer ? 0 : e1); e += 4 * kT) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < split; ++r) {
                const float4 x = ld_cluster4(smem_u32(part + e), r);
                o = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
            }
            const size_t ob = (size_t)row * kLatHQ * kLatD + e;
            const __nv_bfloat162 h0 = __floats2bfloat162_rn(o.x, o.y), h1 = __floats2bfloat162_rn(o.z, o.w);
            *reinterpret_cast<uint2*>(a.out + ob) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
            if (a.out_f32) *reinterpret_cast<float4*>(a.out_f32 + ob) = o;
        }
        cluster_sync();  // the others have read this CTA's part
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (issuer) tmem_dealloc(tb, kCols);
        return;
    }
    if (tid < 64) {
        const float l = (red[tid] + red[64 + tid]) + (red[128 + tid] + red[192 + tid]);
        s_l[tid] = l;
        const bool em = nt == 0 || l == 0.f;
        s_al[tid] = em ? 0.f : 1.f / l;  // 1 / l per head (0 for a row with no key: O is 0 there)
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < (issuer ? 0 : 4); ++mt) {
        uint32_t v[16] = {};
        if (nt > 0) {
            tmem_ld16(tb + lane_base + kOCol + 64 * mt + 16 * cg, v);
            tmem_ld_wait();
        }
        // lanes 2 i and 2 i + 1 exchange halves of their heads: a lane ends with a pair of channels of every second
        // head (half the stores; 28.8 us at 128 rows against 29.3, four channels a lane 29.6)
        const int d = 128 * mt + 32 * quad + (lane & 30), odd = lane & 1;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float x0 = __uint_as_float(v[i]) * s_al[16 * cg + i], x1 = __uint_as_float(v[i + 1]) * s_al[16 * cg + i + 1];
            const float got = __shfl_xor_sync(0xffffffffu, odd ? x0 : x1, 1);
            const float2 o = odd ? make_float2(got, x1) : make_float2(x0, got);
            const size_t ob = ((size_t)row * kLatHQ + 16 * cg + i + odd) * kLatD + d;
            const __nv_bfloat162 h = __floats2bfloat162_rn(o.x, o.y);
            *reinterpret_cast<__nv_bfloat162*>(a.out + ob) = h;
            if (a.out_f32) *reinterpret_cast<float2*>(a.out_f32 + ob) = o;
        }
    }
    if (a.lse && tid < 64) {
        const bool e = nt == 0 || s_l[tid] == 0.f;
        a.lse[(size_t)row * kLatHQ + tid] = e ? -INFINITY : (s_m[tid] * 0.6931471805599453f + logf(s_l[tid]));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (issuer) tmem_dealloc(tb, kCols);
}

}  // namespace

size_t latent_attend_smem_bytes() { return kSmem; }

cudaError_t launch_latent_attend(const LatentAttendArgs& a, cudaStream_t s) {
    auto k = latent_attend_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    if (a.rows == 0) return cudaSuccess;
    return launch_after_prior(k, dim3((unsigned)a.rows), dim3(kThreads), kSmem, s, a);
}

// Clusters of `size` CTAs of the paged kernel that the current device (number dev) holds at once; asked once a device and
// size. Which sizes there are and how many fit is a matter of the SMs per GPC: 7 of 16, 15 of 8, 74 of 2 on a whole
// B200, fewer on a part of one.
static int clusters_at_once(int dev, int size) {
    constexpr int kDevices = 64, kSizes = 17;
    static std::atomic<int> known[kDevices][kSizes];  // 1 more than the number; 0: not asked yet
    if (dev >= 0 && dev < kDevices)
        if (const int n = known[dev][size].load(std::memory_order_relaxed)) return n - 1;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, latent_attend_kernel<true>, &cfg) != cudaSuccess) {
        cudaGetLastError();  // (a size that the device does not take)
        n = 0;
    }
    if (dev >= 0 && dev < kDevices) known[dev][size].store(n + 1, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_paged_attend(LatentAttendArgs a, cudaStream_t s) {
    auto k = latent_attend_kernel<true>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    const int tiles = (a.k + kTile - 1) / kTile + (a.win > 0 ? 1 : 0);
    a.split = paged_attend_split(a.rows, tiles, [&](int size) { return clusters_at_once(dev, size); });
    if (a.split == 1) return launch_after_prior(k, dim3((unsigned)a.rows), dim3(kThreads), kSmem, s, a);
    return launch_cluster(k, dim3((unsigned)(a.rows * a.split)), dim3(kThreads), a.split, kSmem, s, a);
}

}  // namespace csa2
