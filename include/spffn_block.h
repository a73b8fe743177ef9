/*
 * spffn_block.h — the dense half of a batched decode block on one NVIDIA B200
 * (sm_100a), around the activation-sparse FFN of spffn.h:
 *
 *   spffn_norm_quant   residual addition, RMS norm, 8-bit rows with a scale per token
 *   spffn_mm8_*        product of 8-bit integer rows and weights, scales per token and channel
 *   spffn_kv4_append   rotary positions on q and k, and k, v appended to a paged 4-bit cache
 *   spffn_kv4_attend   attention of each sequence's new tokens over that cache
 *
 * One block over T tokens of B sequences (x the 16-bit residual stream):
 *   norm_quant(x, y) -> mm8 (q/k/v) -> kv4_append -> kv4_attend -> quantize_rows -> mm8
 *   (output projection) -> norm_quant (residual) -> spffn_step (sparse FFN) -> norm_quant ...
 * spffn_step takes rows in the storage type: between norm_quant and it the caller multiplies q by scale
 * (this library has no kernel for that).
 *
 * Conventions are those of spffn.h: device pointers into caller-owned memory, the
 * library allocates nothing on the device, `stream` is a cudaStream_t as void*,
 * argument errors return before anything is enqueued, device-side problems are
 * latched in the context's workspace and reported by its _last_device_error.  A
 * context is bound to the device that was current when it was created (its calls, _last_device_error
 * among them, are refused where another one is current), is used by
 * one stream at a time, and two contexts (or two captured graphs) that share a
 * workspace must not run concurrently.  A call may be captured in a CUDA graph:
 * lengths, positions and page tables are read on the device at replay.
 * Row strides (ld...) are in elements, at least the row's width; rows themselves
 * are contiguous.  Pointers need their element's alignment only, unless stated;
 * 16-byte aligned pointers and row strides of whole 16-byte pieces take the wide path.
 * T = 0 (or B = 0) is a valid call that does nothing.
 */
#ifndef SPFFN_BLOCK_H
#define SPFFN_BLOCK_H

#include <stddef.h>
#include <stdint.h>
#include "spffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- RMS norm with the residual's addition and 8-bit rows ------------------------------
 * For each of T rows of width d (1 <= d <= 16384):
 *   u     = x + y                                  (fp32; y == NULL: u = x)
 *   x_out = round(u)                               (storage dtype; skipped where x_out == NULL)
 *   w     = u g,  a = max_c |w_c|                  (fp32; g == NULL: w = u)
 *   rs    = 1 / sqrt(mean_c u_c^2 + eps)           (fp32 sums)
 *   q     = rint(w (127 / a))                      (int8 in -127..127, ties to even)
 *   scale = a rs / 127                             (fp32)
 * so q scale is the normalised row u g rs in 8 bits; q does not depend on rs.  A row of
 * a < 2^-119 (127 / a would overflow) gives q = 0 and scale = 0.  A row that holds a NaN or
 * an infinity in u or in w (a gain that is not finite: every row), or whose sum of squares overflows
 * fp32, gives q = 0 and scale = NaN.
 * x [T][ldx] storage dtype; y [T][ldy] fp32 if y_f32 else storage dtype; g [d] storage
 * dtype; x_out [T][ldo] (may be x itself, or y where it has the same type and stride;
 * no other overlap); q [T][ldq]; scale [T]; eps > 0, finite. */
spffn_status spffn_norm_quant(int32_t T, int32_t d, int32_t dtype, const void* x, int64_t ldx, const void* y,
                              int64_t ldy, int32_t y_f32, const void* g, float eps, void* x_out, int64_t ldo,
                              int8_t* q, int64_t ldq, float* scale, void* stream);

/* The same rows without addition and norm (weights by channel, attention outputs by token):
 * a = max|x|, q = rint(x (127 / a)), scale = a / 127; 1 <= d <= 131072; x holds fp32 if
 * x_f32, else the storage dtype.  A row with a NaN or an infinity: q = 0, scale = NaN. */
spffn_status spffn_quantize_rows(int32_t T, int32_t d, int32_t dtype, const void* x, int64_t ldx, int32_t x_f32,
                                 int8_t* q, int64_t ldq, float* scale, void* stream);

/* ---- product of 8-bit integers, scales per token and channel ---------------------------
 *   y[t][n] = round( a_scale[t] w_scale[n] sum_k A[t][k] W[n][k] + bias[n] )
 * The sum is exact for any int8 values (a 32-bit integer, and 2^31 where all of K = 131072 are -128); scales and bias are
 * applied in fp32, one rounding to the storage dtype.
 *   K  inner width; K % 16 == 0, 16 <= K <= 131072
 *   N  channels; 1 <= N <= 262144;  max_tokens 1..1048576 (largest T of a call)
 *   dtype  type of y and bias;  flags 0 */
typedef struct {
    int32_t K, N, max_tokens, dtype;
    uint32_t flags;
} spffn_mm8_config;

/* W [N][K] int8, 16-byte aligned; w_scale [N] fp32; bias [N] storage dtype or NULL.
 * Borrowed until spffn_mm8_destroy. */
typedef struct {
    const int8_t* W;
    const float* w_scale;
    const void* bias;
} spffn_mm8_weights;

typedef struct spffn_mm8_ctx spffn_mm8_ctx;

size_t spffn_mm8_workspace_bytes(const spffn_mm8_config* cfg);
/* workspace: device, zero-filled before first use, 256-byte aligned, borrowed (int32 parts of tiles that
 * several SMs share, and their counts). */
spffn_status spffn_mm8_create(const spffn_mm8_config* cfg, const spffn_mm8_weights* w, void* workspace,
                              size_t workspace_bytes, spffn_mm8_ctx** out);
spffn_status spffn_mm8_destroy(spffn_mm8_ctx* ctx);
/* A [T][lda] int8, 16-byte aligned, lda % 16 == 0; a_scale [T]; y [T][ldy].  One kernel; calls of up
 * to 256 tokens read each weight once.  Every wait in it is bounded
 * (2 s); one that runs out latches SPFFN_ERR_TIMEOUT, and _last_device_error makes the context usable again. */
spffn_status spffn_mm8_forward(spffn_mm8_ctx* ctx, const int8_t* A, int64_t lda, const float* a_scale, int32_t T,
                               void* y, int64_t ldy, void* stream);
spffn_status spffn_mm8_last_device_error(spffn_mm8_ctx* ctx, uint32_t* code, void* stream);

/* ---- paged cache of keys and values in 4 bits -------------------------------------------
 * pool[page][kv head][block of 16 tokens][640 NG bytes], NG = dh / 32 groups of 32 dims.
 * A block holds, one after the other (byte offsets in units of NG):
 *   0    K codes  [token 16][c 4][g NG][byte i 4]        dims 32g+8c+2i (low 4 bits), +1 (high)
 *   256  V codes  [half 2][r 8][token 8][g NG][byte i 2] dims 32g+4r+2i (low 4 bits), +1 (high);
 *                                                         token 8 half + t
 *   512  K steps  [token 16][g NG] fp16,   544  K zeros  [token 16][g NG] fp16
 *   576  V steps  [half 2][c 4][g NG][j 2] fp16,  608  V zeros, the same; token 8 half + 2c + j
 * A cached value is code step + zero.  A group x of 32 dims (fp32) is held as
 *   zero = fp16(min x), step = fp16((max x - min x) (1/15), 1/15 in fp32), code = clamp(rint((x - zero) / step), 0, 15)
 * (code 0 where step = 0); zero and step are clamped to +-65504, and a group that holds a
 * NaN or an infinity gets step = NaN, which every row that attends to it shows.
 * The layout is the one the attention kernel's matrix instructions read without shuffles.
 *
 * config:
 *   pages      pages of the pool, 1 .. 2^24;   page_size tokens a page: 16, 32, 64, 128 or 256
 *   nh, kvh    query heads and key/value heads; nh % kvh == 0, nh / kvh <= 64, nh <= 1024
 *   dh         head width: 64, 128 or 256
 *   max_seqs   1..4096 sequences and max_tokens 1..65536 new tokens of a call, at most
 *   dtype      type of q, k, v, q_out and out
 *   rope_dim   dims of a head that are rotated (even, 0 <= rope_dim <= dh; the first ones)
 *   rope_interleaved  pairs (2i, 2i+1) instead of (i, i + rope_dim/2)
 *   rope_amplitude    factor on cosine and sine (1 unless the scaling asks for another) */
typedef struct {
    int32_t pages, page_size, nh, kvh, dh, max_seqs, max_tokens, dtype, rope_dim, rope_interleaved;
    uint32_t flags;
    double rope_amplitude;
} spffn_kv4_config;

typedef struct spffn_kv4_ctx spffn_kv4_ctx;

/* Radians per position of the rope_dim / 2 pairs (host array `out`), from base^(-2i/rope_dim):
 *   SPFFN_ROPE_PLAIN   as they are
 *   SPFFN_ROPE_LINEAR  divided by factor (positions interpolated)
 *   SPFFN_ROPE_NTK     base raised to base factor^(rope_dim / (rope_dim - 2))
 *   SPFFN_ROPE_PARTS   pairs that turn more than 32 times over original_len positions as they
 *                      are, fewer than once divided by factor, a linear ramp between
 *                      (Peng et al., "YaRN: Efficient Context Window Extension of Large
 *                      Language Models", 2023); *amplitude = 0.1 ln(factor) + 1
 * *amplitude (may be NULL) is 1 otherwise.  Pure host function. */
typedef enum { SPFFN_ROPE_PLAIN = 0, SPFFN_ROPE_LINEAR = 1, SPFFN_ROPE_NTK = 2, SPFFN_ROPE_PARTS = 3 } spffn_rope_scaling;
spffn_status spffn_rope_frequencies(int32_t rope_dim, double base, int32_t scaling, double factor, double original_len,
                                    double* out, double* amplitude);

size_t spffn_kv4_pool_bytes(const spffn_kv4_config* cfg);
size_t spffn_kv4_workspace_bytes(const spffn_kv4_config* cfg);
/* pool: device, >= spffn_kv4_pool_bytes, 256-byte aligned, borrowed; its contents are the
 * caller's (nothing is read from it but what the calls' lengths cover).  rope_freqs: device
 * double [rope_dim / 2], radians per position, borrowed; may be NULL where rope_dim == 0.
 * workspace: zero-filled before first use, 256-byte aligned, borrowed. */
spffn_status spffn_kv4_create(const spffn_kv4_config* cfg, void* pool, size_t pool_bytes, const double* rope_freqs,
                              void* workspace, size_t workspace_bytes, spffn_kv4_ctx** out);
spffn_status spffn_kv4_destroy(spffn_kv4_ctx* ctx);

/* The batch, the same for append and attend (device int32 arrays):
 *   q_start [B + 1]  sequence b's new tokens are rows q_start[b] .. q_start[b+1] - 1 of q, k, v;
 *                    NULL: one new token for each, row b
 *   lens [B]         tokens of sequence b, its new ones included; new token i of n stands at
 *                    position lens[b] - n + i
 *   table [B][ld_table]  the pages of sequence b in order; position p is token p % page_size of
 *                    page table[b][p / page_size]; `width` columns are valid; entries beyond a
 *                    sequence's pages are not read
 * Rows behind q_start[B] (a padded batch) are neither read nor written.  A sequence whose rows
 * do not lie in 0 <= q_start[b] <= q_start[b+1] <= T is skipped; one whose length is below its
 * new tokens or above width page_size (or 2^30) is not appended and attends to nothing (its rows of out
 * become 0, those of q_out stay); a page outside [0, pages) is not written, and its tokens are left out of the
 * attention.  Each of these latches SPFFN_ERR_DEVICE_CHECK.
 * Sequences may share pages that only attend reads; two rows of one append must not name the
 * same place.  A row belongs to one sequence: where starts that fall back let two claim it, that row's
 * results are either's or a mixture (nothing out of range is touched).
 *
 * append: q_out = rotated q (storage dtype, fp32 arithmetic; may be q itself with the same
 * stride; q and q_out may both be NULL); k rotated, then k and v quantised, written to the cache.
 * Angles are taken in fp64 from the position, so far positions keep their accuracy.
 * q [T][ldq], row t holds nh heads of dh; k, v likewise with kvh heads. */
spffn_status spffn_kv4_append(spffn_kv4_ctx* ctx, const void* q, int64_t ldq, const void* k, int64_t ldk,
                              const void* v, int64_t ldv, int32_t T, const int32_t* table, int64_t ld_table,
                              int32_t width, const int32_t* lens, const int32_t* q_start, int32_t B, void* q_out,
                              int64_t ldqo, void* stream);

/* attend: for each new token (position p of its sequence) and query head h, over the cached
 * keys and values of kv head h / (nh / kvh) at positions 0..p:
 *   out = sum_j softmax_j(scale q . K_j) V_j
 * Scores, maxima, sums and outputs are held in fp32.  To fp16 (2^-11) are rounded: q, scaled by a power of two a
 * row (a value below 2^-19 of its row's largest may lose bits); each probability times a V step, and for a
 * bf16 output the probability before that.  The output is rounded once.
 * q [T][ldq] as append left it in q_out, out [T][ldo] (not q).  A row with nothing to attend to gives 0; a row
 * whose q is not finite, or that sees a key that is not a number or a value that is not finite, gives NaN, and no
 * other row does.  Two kernels; the same inputs give the same bits. */
spffn_status spffn_kv4_attend(spffn_kv4_ctx* ctx, const void* q, int64_t ldq, int32_t T, const int32_t* table,
                              int64_t ld_table, int32_t width, const int32_t* lens, const int32_t* q_start, int32_t B,
                              float scale, void* out, int64_t ldo, void* stream);

/* The values of n pages (device int32 ids; an id outside [0, pages) leaves its part unwritten
 * and latches): K, V [n][page_size][kvh][dh] storage dtype, 16-byte aligned, rounded once.
 * Every token of a page is read, whether it was ever appended or not. */
spffn_status spffn_kv4_read(spffn_kv4_ctx* ctx, const int32_t* page_ids, int32_t n, void* K, void* V, void* stream);

spffn_status spffn_kv4_last_device_error(spffn_kv4_ctx* ctx, uint32_t* code, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPFFN_BLOCK_H */
