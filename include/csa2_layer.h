/*
 * csa2_layer.h -- the operators around the CSA2 core of csa2.h, in the same library (libcsa2): the
 * FP8 projections before and after the layer step, the norms and rotary positions between a
 * projection and the cache, and a paged form of the latent cache with the append, the selection and
 * the attention that read it.
 *
 * The tags [B], [C] and the conventions (device pointers, ownership, streams, errors, workspaces) are
 * those of csa2.h. Nothing here allocates, synchronises or keeps state between calls; every call can
 * be captured into a CUDA graph. A call runs on the device that is current when it is made.
 *
 * A layer of the pages' own shape, one decode step of `batch` sequences:
 *   csa2_fp8_quantize, csa2_fp8_gemm      hidden state -> queries, latent, indexer queries and key
 *   csa2_norm_rope                        queries and indexer queries
 *   csa2_paged_append                     latent, indexer key, window row: norm, rotation, codec, write
 *   csa2_paged_index_topk                 the selection
 *   csa2_paged_attend                     attention over selected entries and the window
 *   csa2_rope (transposed, 1 / mscale)    the output turned back (K = V carries the keys' rotation and scale)
 *   csa2_fp8_quantize, csa2_fp8_gemm      output projection
 */
#ifndef CSA2_LAYER_H
#define CSA2_LAYER_H

#include "csa2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the calls that take more than one. */
#define CSA2_BF16 0
#define CSA2_F32  1

/* Device status bit (csa2_get_device_status), next to those of csa2.h: a page of the table that an
 * entry falls in, or a window slot, is outside the cache; the entry is skipped. */
#define CSA2_DEV_BAD_PAGE 0x10

/* ---- rotary positions ------------------------------------------------------------------------ */

/* Which channels of a rotated range of `rot` channels form pair j (0 <= j < rot / 2). */
#define CSA2_ROPE_HALF        0 /* j and j + rot / 2  */
#define CSA2_ROPE_INTERLEAVED 1 /* 2 j and 2 j + 1    */

/*
 * A rotation: pair j of the channels offset .. offset + rot - 1 of a head turns by the angle
 * t = position * inv_freq[j],
 *     (a, b) -> mscale * (a cos t - b sin t, b cos t + a sin t);
 * the other channels stay as they are. With `transposed` the sine changes its sign: with the same
 * mscale that is the transposed matrix, the gradient; with 1 / mscale it is the inverse, which undoes
 * the rotation. Angles are reduced in 64 bits with their rounding errors carried along, so they hold to
 * 64-bit accuracy at any position below 2^31.
 */
typedef struct {
    const double* inv_freq; /* device [rot / 2]: radians per position, 8-byte aligned */
    int rot;                /* rotated channels: even, 0 .. d                          */
    int offset;             /* the first of them: 0 .. d - rot                         */
    int layout;             /* CSA2_ROPE_HALF or CSA2_ROPE_INTERLEAVED                 */
    int transposed;         /* 0 or 1                                                  */
    float mscale;           /* 0 gives 1                                               */
} csa2_rope_spec;

/* How the frequencies of a longer context follow from those of the original one. */
#define CSA2_ROPE_PLAIN  0 /* f_j = base^(-2 j / rot)                                                      */
#define CSA2_ROPE_LINEAR 1 /* f_j / factor                                                                 */
#define CSA2_ROPE_NTK    2 /* the base times factor^(rot / (rot - 2)): slow channels stretched by `factor` */
#define CSA2_ROPE_YARN   3 /* channels that turn more than beta_fast times in orig_ctx positions keep f_j,
                              those below beta_slow turns take f_j / factor, a ramp linear in the channel
                              between; *mscale = 0.1 ln(factor) + 1                                        */

/*
 * The frequencies of a rotation, on the host: inv_freq [rot / 2] and *mscale (1 but for
 * CSA2_ROPE_YARN). factor >= 1; orig_ctx, beta_fast and beta_slow are read for CSA2_ROPE_YARN alone
 * (beta_fast > beta_slow > 0). The published stretching rules, the YaRN ramp in the channel number
 * between the (rounded) channels of beta_fast and beta_slow.
 * Returns CSA2_ERR_INVALID_ARG for an odd or negative rot, base <= 1, factor < 1 or a bad kind.
 */
CSA2_API csa2_status csa2_rope_frequencies(int rot, double base, int kind, double factor, int64_t orig_ctx,
                                           double beta_fast, double beta_slow, double* inv_freq /* host */,
                                           float* mscale /* host */);

/*
 * The heads of `tokens` tokens: head h of token i is the d elements at x + i * x_token + h * x_head
 * (strides in elements, any value >= 0 for which the rows stay apart; out likewise). `out` may be `x`
 * itself with the same strides; any other overlap is not allowed. weight [d]: the norm's, of the same
 * element type (csa2_norm_rope; NULL there is a norm without weights).
 */
typedef struct {
    const void* x;
    void* out;
    int64_t x_token, x_head;
    int64_t out_token, out_head;
    const void* weight;
    int heads;
} csa2_heads;

/*
 * Rotary positions: out = R_pos(x), d channels a head (1 <= d <= 1024), dtype CSA2_BF16 or CSA2_F32.
 *   pos [tokens] int64; a token with a negative position is padding: its rows of `out` are not written
 * The arithmetic is fp32 with one rounding to bf16. Called with out == x it touches the rotated
 * channels alone. Rows that allow 16-byte accesses (pointers, strides, d, offset, and rot or rot / 2
 * with CSA2_ROPE_HALF) take them, others narrower ones.
 */
CSA2_API csa2_status csa2_rope(const csa2_rope_spec* rope, int dtype, int64_t tokens, int d, const int64_t* pos,
                               const csa2_heads* h, void* stream);

/*
 * Norm of each head and its rotation in one pass, queries and keys in one launch:
 *   out = R_pos(x * w / sqrt(mean(x^2) + eps))   for the heads of q and of k (k may be NULL)
 * rope may be NULL (the norm alone; pos may then be NULL too). No rounding between norm and rotation;
 * the sum of squares is fp32 (rows beyond about 1e19 overflow it); otherwise as csa2_rope. eps >= 0.
 */
CSA2_API csa2_status csa2_norm_rope(const csa2_rope_spec* rope, int dtype, int64_t tokens, int d, const int64_t* pos,
                                    float eps, const csa2_heads* q, const csa2_heads* k, void* stream);

/* ---- products in 8-bit floating point ---------------------------------------------------------- */

/*
 * Rows in E4M3 with one fp32 scale per 128 channels: x [rows][k] bf16, row r at x + r * x_stride
 * (elements) -> data [rows][k] E4M3 bytes, scale [ceil(k / 128)][rows] fp32 (channel block major, so
 * that the rows' scales of one block lie together):
 *   s = amax / 448 (fp32 quotient), code = E4M3_RNE_satfinite(x / s) (of the fp32 quotient); s == 0
 *   gives codes +0. A block with a NaN becomes NaN whole; one with infinities has scale infinity, NaN in their
 *   places and zeros in the others (its products are not finite).
 * k a positive multiple of 16, x_stride a multiple of 8, x and data 16-byte aligned.
 */
CSA2_API csa2_status csa2_fp8_quantize(int64_t rows, int k, const uint16_t* x, int64_t x_stride, uint8_t* data,
                                       float* scale, void* stream);

/*
 * Weights in E4M3 with one fp32 scale per 128 x 128 block: w [n][k] bf16 (dense) -> data [n][k],
 * scale [ceil(n / 128)][ceil(k / 128)] fp32, the rule of csa2_fp8_quantize over the block.
 */
CSA2_API csa2_status csa2_fp8_quantize_weight(int64_t n, int k, const uint16_t* w, uint8_t* data, float* scale,
                                              void* stream);

/*
 * out[i][j] = sum over blocks b of xs[b][i] ws[j / 128][b] * (sum of x[i][c] w[j][c] over the 128
 * channels c of block b), x and w as the two calls above write them:
 *   x [m][k], xs [ceil(k / 128)][m]; w [n][k], ws [ceil(n / 128)][ceil(k / 128)]
 *   out [m][n], row i at out + i * out_stride (elements), bf16 or fp32 by out_dtype
 * Tensor cores (E4M3 products are exact, a block's sum is kept in fp32), the blocks' sums scaled and
 * added in fp32, one rounding to bf16. The result of a row does not depend on timing.
 * The two scales of a block are multiplied with each other before they meet its sum: where xs * ws
 * leaves fp32's normal range (2^-126 .. 2^128; operands of extreme sizes on both sides), the block loses
 * bits, vanishes or is not finite even where its share of the result could be held.
 * k a positive multiple of 16, x and w 16-byte aligned, out aligned to its elements, out_stride >= n.
 * m and n any size >= 0, below 2^31. status: at least 256 bytes from csa2_workspace_init (its status
 * word receives CSA2_DEV_TIMEOUT if a tensor-core wait ran out), or NULL.
 */
CSA2_API csa2_status csa2_fp8_gemm(int64_t m, int64_t n, int k, const uint8_t* x, const float* xs, const uint8_t* w,
                                   const float* ws, int out_dtype, void* out, int64_t out_stride, void* status,
                                   size_t status_bytes, void* stream);

/* ---- the paged latent cache ---------------------------------------------------------------------- */

/*
 * The latent cache of csa2.h (csa2_latent_cache) in pages of `page` entries (a power of two, 8 ..
 * 65536): entry p of sequence b lies in slot p % page of page table[b * max_pages + p / page], and
 * row r = that page * page + slot has the codes and scales of csa2_latent_cache's position r:
 *   l_data + r*256, l_scale + r*32, k_data + r*64, k_scale + r*4
 * Window rows are a ring per window slot, as there: token p of sequence b at
 *   swa + (s*swa_cap + (p & (swa_cap-1)))*512 with s = swa_slot ? swa_slot[b] : b.
 * A table entry outside [0, n_pages) (-1, say) is a page that is not there. Pages may be shared by
 * sequences that only read them. n_pages * page <= 2^31 - 1, max_pages * page <= 2^30; planes 16-byte
 * aligned; planes that a call does not touch may be NULL.
 */
typedef struct {
    uint8_t* l_data;
    uint8_t* l_scale;
    uint8_t* k_data;
    uint8_t* k_scale;
    uint8_t* swa;
    const int32_t* table;    /* device [batch][max_pages] */
    const int32_t* swa_slot; /* device [batch] or NULL    */
    int64_t n_pages;
    int64_t max_pages;       /* table entries of a sequence */
    int64_t n_slots;         /* window rings (>= batch when swa_slot is NULL) */
    int64_t swa_cap;         /* ring slots, power of two */
    int page;
} csa2_paged_cache;

/* A row to append: x [batch][t][channels] bf16, token (b, i) at x + b * x_batch + i * x_token (strides
 * in elements, multiples of 8; x 16-byte aligned); weight [channels] bf16 (16-byte aligned) norms the
 * row on the way (NULL: no norm); rope rotates it (NULL: no rotation; transposed is not allowed). */
typedef struct {
    const uint16_t* x;
    int64_t x_batch, x_token;
    const uint16_t* weight;
    const csa2_rope_spec* rope;
} csa2_append_row;

/*
 * Append with norm and rotation on the way ([C] sec. XI: cached values are quantised after the
 * rotation): entries pos[b] .. pos[b] + len[b] - 1 of each sequence,
 *   latent (512 channels) -> E2M1 codes + E4M3 scale per 16, idx_k (128) -> MXFP4, swa (512) -> window
 *   row in E4M3; each may be NULL, and its plane is then not touched
 *   y = R(x * w / sqrt(mean(x^2) + eps)), then the codecs of csa2.h, with no rounding in between:
 *   every code and scale is the one that y in real arithmetic (to 64-bit accuracy) has
 *   pos [batch] int64; len [batch] int32 or NULL (= t): tokens behind len[b] are padding
 *   rpos [batch][t] int64 or NULL: the tokens' positions for the rotation (NULL: pos[b] + i)
 * A sequence whose entries leave [0, max_pages * page), or with len outside [0, t], sets
 * CSA2_DEV_BAD_POS and is skipped (window rows need pos >= 0 alone); a token whose page is not there
 * sets CSA2_DEV_BAD_PAGE and is skipped. ws: at least 256 bytes from csa2_workspace_init for these
 * bits, or NULL. Two tokens of a call that share a slot (sequences with a common page, say) leave its
 * contents undefined.
 */
CSA2_API csa2_status csa2_paged_append(const csa2_paged_cache* cache, int batch, int t, const int64_t* pos,
                                       const int32_t* len, const int64_t* rpos, float eps,
                                       const csa2_append_row* latent, const csa2_append_row* idx_k,
                                       const csa2_append_row* swa, void* ws, size_t ws_bytes, void* stream);

/*
 * Entries read back as values: idx [batch][n] int32 -> latent [batch][n][512] and key
 * [batch][n][128] bf16 (exact: every code times its scale is a bf16 value; either may be NULL, both
 * 16-byte aligned). An index -1 gives zeros; one outside [-1, max_pages * page) sets
 * CSA2_DEV_BAD_INDEX, one whose page is not there CSA2_DEV_BAD_PAGE, and gives zeros.
 */
CSA2_API csa2_status csa2_paged_gather(const csa2_paged_cache* cache, int batch, int n, const int32_t* idx,
                                       uint16_t* latent, uint16_t* key, void* ws, size_t ws_bytes, void* stream);

/*
 * csa2_latent_attend over the pages: the same arguments, outputs and precision; an entry whose page
 * is not there sets CSA2_DEV_BAD_PAGE and is skipped (as is a window whose ring is not there). k >= 0:
 * k == 0 attends to the window alone (idx may then be NULL).
 * A head with a logit that is not finite gives NaN in out and lse.
 */
CSA2_API csa2_status csa2_paged_attend(const csa2_paged_cache* cache, int batch, int tq, const int64_t* qpos,
                                       const uint16_t* q, const int32_t* idx, int k, const int64_t* swa_begin, int win,
                                       int ratio, float sm_scale, uint16_t* out, float* out_f32, float* lse, void* ws,
                                       size_t ws_bytes, void* stream);

/*
 * csa2_latent_index_topk over the pages: the same arguments, workspace (csa2_latent_index_workspace_size)
 * and selection. An entry whose page is not there sets CSA2_DEV_BAD_PAGE and ranks below every other.
 */
CSA2_API csa2_status csa2_paged_index_topk(const csa2_paged_cache* cache, int batch, int tq, const int64_t* qpos,
                                           const uint16_t* idx_q, int hi, int k, int ratio, int64_t max_ctx,
                                           uint32_t flags, int32_t* out_idx, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA2_LAYER_H */
