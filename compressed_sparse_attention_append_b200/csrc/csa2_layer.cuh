// csa2_layer.cuh -- arguments of the kernels behind include/csa2_layer.h.
#pragma once

#include "../../include/csa2_layer.h"
#include "csa2_internal.cuh"

namespace csa2 {

// ---- rope.cu ---------------------------------------------------------------------------------------
struct RotateArgs {
    csa2_heads q, k;         // k.heads == 0: none
    const int64_t* pos;      // [tokens] (NULL: no rotation)
    const double* inv_freq;  // [rot / 2]
    int64_t tokens;
    int heads;               // q.heads + k.heads
    int d, rot, offset, layout, transposed;
    float mscale, eps, inv_d;
    int in_place;            // out is x and there is no norm: only the rotated channels are touched
    int lanes, rounds;       // lanes per row; rows in turn per group of lanes, over those in flight
    float inv_heads, inv_half;  // 1 / heads, 2 / rot
};
cudaError_t launch_rotate(const RotateArgs& a, int dtype, bool norm, cudaStream_t s);

// ---- paged.cu --------------------------------------------------------------------------------------
struct AppendRow {           // one of the three rows of a token
    const uint16_t* x;       // NULL: not appended
    int64_t x_batch, x_token;
    const uint16_t* weight;
    const double* inv_freq;  // NULL: no rotation
    int rot, offset, layout;
    double mscale;
};
struct PagedAppendArgs {
    csa2_paged_cache c;
    PageMap pg;
    int batch, t;
    const int64_t* pos;
    const int32_t* len;
    const int64_t* rpos;
    double eps;
    AppendRow row[3];        // latent, indexer key, window
    int kinds, kind[3];      // those that are appended
    unsigned first[3];       // and the first block of each
    int warp_bytes;          // shared memory of a warp
    uint32_t* status;
};
cudaError_t launch_paged_append(PagedAppendArgs a, cudaStream_t s);

struct PagedGatherArgs {
    csa2_paged_cache c;
    PageMap pg;
    int64_t rows;            // batch * n
    int n;
    const int32_t* idx;
    uint16_t* latent;
    uint16_t* key;
    uint32_t* status;
};
cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t s);

// ---- fp8.cu ----------------------------------------------------------------------------------------
cudaError_t launch_fp8_rows(int64_t rows, int k, const uint16_t* x, int64_t x_stride, uint8_t* data, float* scale,
                            cudaStream_t s);
cudaError_t launch_fp8_weight(int64_t n, int k, const uint16_t* w, uint8_t* data, float* scale, cudaStream_t s);

struct Fp8GemmArgs {
    int64_t m, n;
    int k;
    const uint8_t* x;
    const float* xs;
    const uint8_t* w;
    const float* ws;
    void* out;
    int64_t out_stride;
    int out_f32;
    uint32_t* status;
};
cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t s);

}  // namespace csa2
