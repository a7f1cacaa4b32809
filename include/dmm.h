/*
 * dmm.h -- C ABI of libdmm, an fp8 a8w8 GEMM library for AMD Instinct MI355X
 * (gfx950).
 *
 * The user sequence follows mori PR 809 ("mori.ops.ag_gemm"), section Using
 * it: quantise the activations per token, preshuffle the fp8 weight once,
 * then call the GEMM with both operands and their scales; the result is a
 * contiguous bf16 [M, N] tensor.  The GEMM computes
 *
 *     C[m, n] = bf16( sum_k (A[m, k] * sa(m, k)) * (B[n, k] * sb(n, k)) )
 *
 * with fp32 accumulation, where A [M, K] and B [N, K] hold OCP FP8 E4M3 codes
 * and sa / sb depend on the scaling mode (ptpc, blockscale, mxfp8) named in
 * mori PR 785 ("fix(gemm-ar): drain the peeled tail's producers instead of
 * tightening the loop"), section Cost.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers owned by the caller.  The library
 *     allocates nothing and keeps no state beyond a per-device arch check.
 *   - Every call is asynchronous on `stream` (a hipStream_t passed as void*;
 *     NULL is the default stream).  Nothing synchronises the host.
 *   - Layouts are row-major and contiguous.  e4m3 codes are uint8_t (OCP
 *     FP8 E4M3, max 448, NaN = S.1111.111); bf16 values are uint16_t bit
 *     patterns; E8M0 scales are uint8_t (2^(b-127)).
 *   - Argument errors return DMM_EINVAL before any HIP call is made;
 *     dmm_last_error() then describes the first violated rule.  A device that
 *     is not gfx950 returns DMM_ENODEV.  A failed launch returns DMM_ELAUNCH.
 *   - Every pointer must be 16-byte aligned, and every operand (A, B, C,
 *     scales) must be smaller than 2^31 bytes: the kernels address operands
 *     through 32-bit buffer offsets.
 *   - Calls on one stream are ordered; calls on different streams that write
 *     the same buffer race, as with any kernel.
 */
#ifndef DMM_H
#define DMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DMM_OK = 0,
    DMM_EINVAL = 1,  /* an argument breaks a documented rule */
    DMM_ENODEV = 2,  /* the current device is not gfx950 */
    DMM_ELAUNCH = 3  /* the HIP runtime reported an error */
} dmm_status;

/* Name of a status code ("DMM_OK", ...). */
const char* dmm_status_str(int status);

/* Detail for the last non-OK return on the calling thread ("" if none). */
const char* dmm_last_error(void);

/* ---------------------------------------------------------------- quantise */

/* Per-row E4M3 quantisation (mori PR 809, Using it: quantize_per_token; the
 * workloads use scale = amax / 448).  For each row r of x [rows, cols] fp32:
 *   scale[r] = amax_r / 448 (IEEE fp32 division; 1.0 when the row is zero),
 *   q[r, c]  = E4M3(x[r, c] / scale[r]), round to nearest even, saturating
 *              to +-448.
 * Used per token for A and per output channel for B [N, K].
 * Rules: rows >= 1, cols >= 16, cols % 16 == 0.  q [rows, cols] u8, scale
 * [rows] fp32, both written. */
dmm_status quantize_per_token(const float* x, uint8_t* q, float* scale, int64_t rows, int64_t cols,
                              void* stream);

/* The same for bf16 activations: x [rows, cols] bf16 (uint16_t bit
 * patterns), each value widened exactly to fp32, then the rule above.
 * Same rules and outputs. */
dmm_status quantize_per_token_bf16(const uint16_t* x, uint8_t* q, float* scale, int64_t rows, int64_t cols,
                                   void* stream);

/* Blockscale A: one fp32 scale per row per 128-wide K block (mori PR 785,
 * Cost: blockscale; the A scale is K-block major, mori PR 809, Not done yet).
 *   scale[kb * m + r] = amax(x[r, 128kb .. 128kb+127]) / 448 (1.0 if zero),
 *   q[r, c] = E4M3(x[r, c] / scale[c/128 * m + r]).
 * Rules: m >= 1, k >= 128, k % 128 == 0. */
dmm_status quantize_blockscale_a(const float* x, uint8_t* q, float* scale, int64_t m, int64_t k, void* stream);

/* Blockscale B [n, k]: one fp32 scale per 128 x 128 block, stored
 * scale[nb * (k/128) + kb]; a partial last row block uses only the rows it
 * has.  Rules: n >= 16, n % 16 == 0, k >= 128, k % 128 == 0. */
dmm_status quantize_blockscale_b(const float* x, uint8_t* q, float* scale, int64_t n, int64_t k, void* stream);

/* mxfp8: one E8M0 scale per 32 consecutive K values of a row (mori PR 785,
 * Cost: mxfp8).  e = ceil(log2(amax / 448)) clamped to [-127, 127] (0 for a
 * zero group), stored scale[(c/32) * rows + r] = e + 127;
 * q[r, c] = E4M3(x[r, c] * 2^-e).  Used for both A [M, K] and B [N, K].
 * Rules: rows >= 1, k >= 128, k % 128 == 0. */
dmm_status quantize_mxfp8(const float* x, uint8_t* q, uint8_t* scale, int64_t rows, int64_t k, void* stream);

/* ------------------------------------------------------------- preshuffle */

/* Reorders B [n, k] E4M3 codes (one row per output channel) into the byte
 * order the GEMM's matrix-core operands use (aiter PR 6539 names the kernels
 * "bpreshuffle"; mori PR 809, Using it, calls preshuffle_b once per weight).
 * The layout is library-defined: b_shuf has the same size as b (n * k
 * bytes) and is only meant to be passed to the gemm_a8w8_* calls.  (For
 * reference: 2 KiB chunk (j, kt) at (j * k/128 + kt) * 2048 holds block j of
 * 16 fragment rows for K tile kt; byte 16 l + t of its half h is
 * B[src(j, l % 16)][128 kt + 64 h + 16 (l / 16) + t].  Blocks come in groups
 * of four, 64 output columns; in group G = j / 4 of p blocks, fragment row r
 * of block nb = j % 4 is B row 64 G + 32 (nb / 2) + 8 (r / 4) + 4 (nb % 2) +
 * r % 4, except that the last block of a group with an odd p keeps row
 * order, 64 G + 16 nb + r.)
 * b and b_shuf must not overlap.  Rules: n >= 16, n % 16 == 0, k >= 128,
 * k % 128 == 0. */
dmm_status preshuffle_b(const uint8_t* b, uint8_t* b_shuf, int64_t n, int64_t k, void* stream);

/* --------------------------------------------------------------- the GEMM */

/* Rules shared by the three fp8 GEMMs:
 *   m >= 1; n >= 16 and n % 16 == 0 (the last 256-column tile may be
 *   partial; mori PR 809, Using it); k >= 128 and k % 128 == 0 (k = 256
 *   runs the peeled tail only; mori PR 785, Why the existing A+B-1 did not
 *   fix it).  a [m, k] u8 codes; b_shuf from preshuffle_b; c [m, n] bf16 is
 *   fully overwritten and nothing outside it is written. */

/* ptpc: a_scale [m] fp32 per token, b_scale [n] fp32 per output channel.
 *   C[m, n] = bf16(a_scale[m] * b_scale[n] * sum_k A[m, k] B[n, k]). */
dmm_status gemm_a8w8_ptpc(const uint8_t* a, const uint8_t* b_shuf, const float* a_scale, const float* b_scale,
                          uint16_t* c, int64_t m, int64_t n, int64_t k, void* stream);

/* ptpc with an explicit output-tile shape, the same result as
 * gemm_a8w8_ptpc: tile 1 = 256 x 256 (four waves), 2 = 128 x 256 (eight
 * waves), 3 = 128 x 128 (four waves), 0 = the choice gemm_a8w8_ptpc makes:
 * the tile whose waves over the compute units cost least, a 128 x 256 tile
 * costing 0.625 and a 128 x 128 tile 0.34 of a wide tile's time (so the
 * smaller tiles win only where the wide grid would leave many compute units
 * idle).  The pages size the
 * tile to the problem in the same spirit (mori PR 785, Cost: the table's
 * shapes; aiter PR 6539, Motivation and its review thread: the tuned rows,
 * one kernel configuration per shape).  Other values of tile return
 * DMM_EINVAL. */
dmm_status gemm_a8w8_ptpc_tile(const uint8_t* a, const uint8_t* b_shuf, const float* a_scale,
                               const float* b_scale, uint16_t* c, int64_t m, int64_t n, int64_t k, int tile,
                               void* stream);

/* ptpc over a gathered A: the GEMM half of an all-gather + GEMM (mori PR
 * 809, How it works: the tile order and the wait), on one GPU.  A [m, k] and
 * a_scale [m] are m / src_rows source slabs of src_rows rows; slab `own` is
 * resident when the call starts, and every other slab arrives in nchunks
 * row bands of src_rows / nchunks rows: band s * nchunks + c (rows
 * s * src_rows + c * src_rows / nchunks ...) may be read once
 * flags[s * nchunks + c] has reached epoch, compared wrap-safe as
 * (int32_t)(flags[band] - epoch) >= 0, so a caller advances epoch per call
 * and never resets the flags.  Tiles of the own slab run first, never
 * waiting; then, for each chunk c, the sources own+1, own+2, ... (mod the
 * source count).  A workgroup polls a band's flag with system-scope loads
 * before any load of its rows and fences (acquire) after seeing it; flags
 * may live in device memory or in pinned host memory that a host thread
 * writes.  After spin_limit polls (each about 0.3 us) for one band the wait
 * gives up: *status (device int, zeroed by the caller) becomes the largest
 * 1 + band that timed out and the result is undefined; the kernel still
 * finishes.  The result is otherwise bitwise that of gemm_a8w8_ptpc.
 * Rules beyond gemm_a8w8_ptpc's: src_rows a positive multiple of
 * 256 * nchunks; m a multiple of src_rows; at most 64 bands; 0 <= own <
 * m / src_rows; spin_limit >= 0; flags and status non-null, 4-byte aligned. */
dmm_status gemm_a8w8_ptpc_gathered(const uint8_t* a, const uint8_t* b_shuf, const float* a_scale,
                                   const float* b_scale, uint16_t* c, int64_t m, int64_t n, int64_t k,
                                   const uint32_t* flags, int64_t src_rows, int nchunks, int own, uint32_t epoch,
                                   int64_t spin_limit, int* status, void* stream);

/* blockscale: a_scale [k/128][m] fp32 (1x128 blocks, K-block major),
 * b_scale [ceil(n/128)][k/128] fp32 (128x128 blocks).
 *   C[m, n] = bf16(sum_kb a_scale[kb][m] b_scale[n/128][kb] sum_{k in kb} A B). */
dmm_status gemm_a8w8_blockscale(const uint8_t* a, const uint8_t* b_shuf, const float* a_scale,
                                const float* b_scale, uint16_t* c, int64_t m, int64_t n, int64_t k,
                                void* stream);

/* blockscale with an explicit output-tile shape, the same result as
 * gemm_a8w8_blockscale: tile 1 = 128 x 256 (eight waves, two per SIMD),
 * 2 = 128 x 128 (four waves), 0 = the choice gemm_a8w8_blockscale makes
 * (128 x 128 when its waves over the compute units cost less than the
 * 128 x 256 tile's, by the rule gemm_a8w8_mxfp8_tile describes; the pages
 * tune one configuration per shape: aiter PR 6539, Motivation and the tuned
 * rows of its review thread).  Other values of tile return DMM_EINVAL. */
dmm_status gemm_a8w8_blockscale_tile(const uint8_t* a, const uint8_t* b_shuf, const float* a_scale,
                                     const float* b_scale, uint16_t* c, int64_t m, int64_t n, int64_t k, int tile,
                                     void* stream);

/* mxfp8: a_scale [k/32][m] and b_scale [k/32][n] E8M0 bytes, one per 32
 * consecutive K values.
 *   C[m, n] = bf16(sum_g 2^(a_scale[g][m]-127) 2^(b_scale[g][n]-127) sum_{k in g} A B).
 * Scale byte 255 (NaN) is outside the contract. */
dmm_status gemm_a8w8_mxfp8(const uint8_t* a, const uint8_t* b_shuf, const uint8_t* a_scale,
                           const uint8_t* b_scale, uint16_t* c, int64_t m, int64_t n, int64_t k, void* stream);

/* mxfp8 with an explicit output-tile shape, the same result as
 * gemm_a8w8_mxfp8: tile 1 = 256 x 256, 2 = 256 x 128 (four waves, each
 * owning all 256 rows and 32 columns: the A tile that goes through LDS is
 * twice the B tile -- the narrow mxfp8 shape whose A side outgrows its B
 * side, mori PR 785, review thread), 0 = the choice gemm_a8w8_mxfp8 makes (256 x 128 when its
 * waves over the compute units cost less than the 256 x 256 tile's, e.g.
 * when the wide grid leaves most CUs idle).  The same choice rule picks
 * between gemm_a8w8_ptpc's two tiles.  Other values of tile return
 * DMM_EINVAL. */
dmm_status gemm_a8w8_mxfp8_tile(const uint8_t* a, const uint8_t* b_shuf, const uint8_t* a_scale,
                                const uint8_t* b_scale, uint16_t* c, int64_t m, int64_t n, int64_t k, int tile,
                                void* stream);

/* bf16 GEMM with fp32 accumulation (DeepGEMM PR 453, "Fix SM120 BF16 GEMM
 * shared-memory reuse ordering", Reproduction and validation: [4096, 1024]
 * x [1024, 896]).  a [m, k] bf16, b [n, k] bf16 (the weight given one row
 * per output column), c [m, n] bf16 = bf16(sum_k a[m, k] b[n, k]).
 * Rules: m >= 1; n >= 16, n % 16 == 0; k >= 64, k % 64 == 0. */
dmm_status gemm_bf16(const uint16_t* a, const uint16_t* b, uint16_t* c, int64_t m, int64_t n, int64_t k,
                     void* stream);

/* gemm_bf16 with an explicit output-tile shape, the same result: tile 1 =
 * 128 x 128, 2 = 64 x 64, 0 = gemm_bf16's choice (64 x 64 when the problem
 * has at most one 128 x 128 tile per two compute units).  Other values
 * return DMM_EINVAL. */
dmm_status gemm_bf16_tile(const uint16_t* a, const uint16_t* b, uint16_t* c, int64_t m, int64_t n, int64_t k,
                          int tile, void* stream);

/* ------------------------------------------- around the dense products */

/* The operators below belong to a feed-forward sublayer around the products
 * above.  They follow the conventions of this file with two differences: a
 * batch may be empty (rows or m = 0: nothing is read, outputs that do not
 * depend on the batch's size are written as the empty sum, and pointers to
 * empty arrays may be NULL), and operands may exceed 2^31 bytes (one row of
 * a matrix may have at most 2^21 elements).  The _workspace queries make no HIP
 * call: a size depends on the arguments alone. */

enum { DMM_BF16 = 0, DMM_FP32 = 1 };
enum {
    DMM_ACT_SILU = 0, /* z / (1 + exp(-z)) */
    DMM_ACT_GELU = 1  /* 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
};

/* Layer norm over the rows of x [rows, cols]:
 *   y = (x - mu) r weight + bias,  mu = mean of the row,
 *   r = 1 / sqrt(mean((x - mu)^2) + eps),
 * with statistics in fp32.  x, weight, bias [cols] and y share one dtype
 * (DMM_BF16 or DMM_FP32).  bias may be NULL (no bias).  mean and rstd [rows]
 * fp32 receive mu and r for the backward pass; both may be NULL.
 * Rules: rows >= 0; cols a multiple of 8 from 8 to 16384; eps >= 0. */
dmm_status layer_norm(const void* x, const void* weight, const void* bias, void* y, float* mean, float* rstd,
                      int64_t rows, int64_t cols, float eps, int dtype, void* stream);

/* Bytes of workspace that layer_norm_backward needs (-1 if rows or cols
 * break its rules). */
int64_t layer_norm_backward_workspace(int64_t rows, int64_t cols);

/* Gradients of layer_norm from dy [rows, cols] and the forward pass's x,
 * mean and rstd.  With xh = (x - mean) rstd and g = dy weight:
 *   dx = rstd (g - mean_row(g) - xh mean_row(g xh)),
 *   dweight = sum over rows of dy xh,  dbias = sum over rows of dy.
 * dx, dweight [cols] and dbias [cols] have dy's dtype; dbias may be NULL.
 * The sums over rows are in fp32 and in a fixed order: the result does not
 * change from call to call.  workspace is overwritten.  Rules as layer_norm. */
dmm_status layer_norm_backward(const void* dy, const void* x, const void* weight, const float* mean, const float* rstd,
                               void* dx, void* dweight, void* dbias, void* workspace, int64_t workspace_bytes,
                               int64_t rows, int64_t cols, int dtype, void* stream);

/* The gated feed-forward block, bf16 with fp32 sums:
 *   g = x w_gate^T,  u = x w_up^T,  h = act(g) u,  y = h w_down^T,
 * x and y [m, d], w_gate and w_up [f, d], w_down [d, f].  Both projections,
 * the activation and the product are one kernel (few tokens over a long d: K
 * is shared out, and a second kernel joins the shares); g and u are kept in
 * fp32 up to h, which is rounded to bf16 once, as the operand of the second
 * product.  gate and up [m, f] receive g and u rounded to bf16 for the
 * backward pass; both may be NULL.  workspace: overwritten, at least
 * gated_ffn_workspace(m, d, f) bytes (-1 if the sizes break a rule).
 * Rules: m >= 0; d and f positive multiples of 8; act DMM_ACT_SILU or
 * DMM_ACT_GELU. */
int64_t gated_ffn_workspace(int64_t m, int64_t d, int64_t f);
dmm_status gated_ffn_bf16(const uint16_t* x, const uint16_t* w_gate, const uint16_t* w_up, const uint16_t* w_down,
                          uint16_t* gate, uint16_t* up, uint16_t* y, void* workspace, int64_t workspace_bytes,
                          int64_t m, int64_t d, int64_t f, int act, void* stream);

/* Gradients of gated_ffn_bf16 from dy [m, d] and the forward pass's x, gate
 * and up.  With dh = dy w_down (kept in fp32):
 *   dgate = dh up act'(gate),  dup = dh act(gate),  h = act(gate) up,
 *   dx = dgate w_gate + dup w_up,  dw_gate = dgate^T x,  dw_up = dup^T x,
 *   dw_down = dy^T h.
 * dgate, dup and h are rounded to bf16 once, as the operands of the products
 * that follow; dx [m, d] and the weights' gradients, shaped as the weights,
 * are the results (m = 0: the weights' gradients are zero).  Every sum has a
 * fixed order.  workspace: overwritten, at least
 * gated_ffn_backward_workspace(m, d, f) bytes.  Rules as gated_ffn_bf16. */
int64_t gated_ffn_backward_workspace(int64_t m, int64_t d, int64_t f);
dmm_status gated_ffn_backward_bf16(const uint16_t* dy, const uint16_t* x, const uint16_t* w_gate, const uint16_t* w_up,
                                   const uint16_t* w_down, const uint16_t* gate, const uint16_t* up, uint16_t* dx,
                                   uint16_t* dw_gate, uint16_t* dw_up, uint16_t* dw_down, void* workspace,
                                   int64_t workspace_bytes, int64_t m, int64_t d, int64_t f, int act, void* stream);

/* The first half of the block over fp8 operands with the scales of
 * gemm_a8w8_ptpc (one per token, one per output channel):
 *   g[m, f] = a_scale[m] gate_scale[f] sum_d A[m, d] Wg[f, d],  u likewise,
 *   h = bf16(act(g) u),
 * the sum times a_scale first, then times the channel's scale, as there.
 * a [m, d], w_gate and w_up [f, d] are E4M3 codes in row order, as
 * quantize_per_token writes them (not preshuffled).  h [m, f] is what
 * quantize_per_token_bf16 takes for the down projection.  workspace:
 * overwritten, at least gated_up_a8w8_ptpc_workspace(m, d, f) bytes (0 for
 * most sizes; NULL then).
 * Rules: m >= 0; d a positive multiple of 16, f of 8; act as above. */
int64_t gated_up_a8w8_ptpc_workspace(int64_t m, int64_t d, int64_t f);
dmm_status gated_up_a8w8_ptpc(const uint8_t* a, const uint8_t* w_gate, const uint8_t* w_up, const float* a_scale,
                              const float* gate_scale, const float* up_scale, uint16_t* h, void* workspace,
                              int64_t workspace_bytes, int64_t m, int64_t d, int64_t f, int act, void* stream);

/* Low-rank adapters of many requests at once, beside a shared projection:
 *   y[t] = x[t] w^T + scales[i] (x[t] lora_a[i]^T) lora_b[i]^T,
 *   i = adapter_ids[t],
 * x [m, k], w [n, k], y [m, n] bf16; lora_a [adapters, r, k] and lora_b
 * [adapters, n, r] bf16; adapter_ids [m] int32, one per token in any order
 * (a request's tokens repeat its id); scales [adapters] fp32.  An id outside
 * [0, adapters) names no adapter: that token gets the shared part alone.  An
 * adapter's values (infinities and NaN too) reach its own tokens only.  The
 * value scales[i] x[t] lora_a[i]^T stays in fp32 for up to 256 tokens and is
 * rounded to bf16 once beyond, as the operand of the second product; the two
 * parts are summed in fp32 and rounded once.  So a token's last bits may depend
 * on how many tokens the call has, not on their order or on each other.
 * workspace: overwritten, at least lora_gemm_workspace(m, n, k, r) bytes (-1
 * if the sizes break a rule).
 * Rules: m >= 0; n and k positive multiples of 8; r a multiple of 8 up to
 * 1024; adapters >= 0 (with 0, lora_a, lora_b and scales may be NULL);
 * adapter_ids 4-byte aligned, so that it may be part of a longer batch's. */
int64_t lora_gemm_workspace(int64_t m, int64_t n, int64_t k, int64_t r);
dmm_status lora_gemm_bf16(const uint16_t* x, const uint16_t* w, const uint16_t* lora_a, const uint16_t* lora_b,
                          const int* adapter_ids, const float* scales, uint16_t* y, void* workspace,
                          int64_t workspace_bytes, int64_t m, int64_t n, int64_t k, int64_t r, int64_t adapters,
                          void* stream);

/* The same beside a projection computed elsewhere (one of the fp8 GEMMs
 * above, say): y[t] = c[t] + scales[i] (x[t] lora_a[i]^T) lora_b[i]^T, c and
 * y [m, n] bf16.  y may be c.  workspace: at least lora_add_workspace bytes.
 * Rules as lora_gemm_bf16. */
int64_t lora_add_workspace(int64_t m, int64_t n, int64_t k, int64_t r);
dmm_status lora_add_bf16(const uint16_t* c, const uint16_t* x, const uint16_t* lora_a, const uint16_t* lora_b,
                         const int* adapter_ids, const float* scales, uint16_t* y, void* workspace,
                         int64_t workspace_bytes, int64_t m, int64_t n, int64_t k, int64_t r, int64_t adapters,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DMM_H */
