/*
 * nmattn.h -- C ABI of libnmspmv, second part: what a decode layer does between
 * its q+k+v and o projections (nm_spmv_multi and nm_spmv of nmspmv.h).
 *
 *   nm_qk_norm_rope   per-head norms of queries and keys, and the position
 *                     rotation, in one pass over the projections' outputs
 *   nm_kv_write       new keys and values into a paged cache, 16-bit or
 *                     quantised to 8 or 4 bits as they are written
 *   nm_kv_read        rows of that cache back as 16-bit values
 *   nm_attn_decode    single-token attention over that cache for a batch, a
 *                     prefix that the whole batch shares being read once
 *
 * ---- Conventions ------------------------------------------------------------
 * Those of nmspmv.h: device pointers, caller-owned buffers, NM_* status codes,
 * every check before any work is queued, calls only enqueue on `stream` (a
 * hipStream_t of the current device) and are thread-safe.  dtype is NM_FP16 or
 * NM_BF16: q, k, v, the weights and the outputs all use it.  No call allocates,
 * waits or copies to the host, so all of them can be captured into a graph.
 * Calls that may run at the same time must not write the same cache rows,
 * outputs or workspace.
 *
 * Strided rows: q, k and v are [rows][heads][D] with heads and columns
 * contiguous and a row stride in elements (heads * D or more, a multiple of 8),
 * so that they can lie inside a fused q+k+v buffer.  The stride of a single row
 * is not looked at.  Outputs are contiguous.
 */
#ifndef NMATTN_H
#define NMATTN_H

#include <stdint.h>

#include "nmspmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * nm_qk_norm_rope -- for every row t and every head of q and k:
 *   n_d = x_d * w_d / sqrt(mean over d of x_d^2 + eps)   (w = wq or wk; n = x if it is NULL)
 *   pair i < rot / 2 of columns (a, b):  y_a = n_a cos(t_i) - n_b sin(t_i),
 *                                        y_b = n_b cos(t_i) + n_a sin(t_i),
 *   t_i = positions[t] * inv_freq[i];  columns rot..D-1: y = n.
 *   interleaved 0: pair i is columns (i, i + rot / 2); 1: columns (2i, 2i + 1).
 *   q [T][Hq][D], k [T][Hk][D]  strided rows (see above), 16-byte aligned.
 *   wq, wk [D]                  16-byte aligned, or NULL (both or either).
 *   positions [T] int32, inv_freq [rot / 2] fp32 (may be NULL when rot is 0).
 *   q_out [T][Hq][D], k_out [T][Hk][D]  contiguous, 16-byte aligned.  q_out may
 *     be q itself and k_out k itself when their rows are contiguous; no other
 *     overlap of an output with an input or the other output.
 * D a multiple of 8 up to 512; rot a multiple of 16 up to D, or 0; T below 2^31,
 * Hq and Hk 0..65535 (0: that side is absent, its pointers are not looked at);
 * eps finite and >= 0.  Norms and rotations are formed in fp32 and rounded once,
 * to nearest even; the angle is formed and reduced in double precision, so far
 * positions keep their phase.
 */
int nm_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t T, int Hq, int Hk, int D,
                    int dtype, const void* wq, const void* wk, float eps, const int32_t* positions,
                    const float* inv_freq, int rot, int interleaved, void* q_out, void* k_out, void* stream);

/*
 * ---- The cache ----------------------------------------------------------------
 * n_pages pages of page_size tokens (16, 32, 64, 128 or 256), heads key heads,
 * D = 64, 128 or 256 columns.  A slot is page * page_size + place in the page.
 *   NM_KV_16   the 16-bit values themselves.
 *   NM_KV_MX8  8-bit codes (e4m3: sign, 4 exponent and 3 mantissa bits), one
 *              power-of-two scale 2^e per 32 consecutive columns of a token's head.
 *   NM_KV_MX4  4-bit codes (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and sign), scales
 *              as for MX8.
 * e is the least integer with max|x| <= M 2^e over the 32 columns, M = 448 (e4m3)
 * or 6 (e2m1), but at least -126 in a bfloat16 cache, -14 (MX8) or -22 (MX4) in an
 * fp16 one; a code is x / 2^e rounded to nearest, ties to the even code.  32
 * columns that hold a NaN or an infinity read back as NaN, all of them.
 *
 * k, v       nm_kv_bytes(...) bytes each, 16-byte aligned.
 * k_scale, v_scale   nm_kv_scale_bytes(...) bytes each, 16-byte aligned (NULL for
 *            NM_KV_16, which has none).
 * The order of the bytes inside is the library's: a page's head is cut into
 * tiles of 16 tokens, and a tile is stored in the order in which a wave's lanes
 * feed it to the matrix cores (keys by 8 columns of a token, values by tokens),
 * so that attention reads full cache lines straight into operand registers.
 */
typedef enum { NM_KV_16 = 0, NM_KV_MX8 = 1, NM_KV_MX4 = 2 } nm_kv_format;

typedef struct {
    void* k;
    void* v;
    uint8_t* k_scale;
    uint8_t* v_scale;
    int64_t n_pages;   /* 1 .. 2^31 - 1 */
    int page_size;     /* 16, 32, 64, 128 or 256 */
    int heads;         /* 1 .. 65535 */
    int D;             /* 64, 128 or 256 */
    int dtype;         /* NM_FP16 or NM_BF16 */
    int format;        /* nm_kv_format */
} nm_kv_cache;

/* Sizes of a cache's buffers in bytes (0 scale bytes for NM_KV_16); -1 for
 * sizes outside the ranges above or a cache of 2^46 bytes and more. */
int64_t nm_kv_bytes(int64_t n_pages, int page_size, int heads, int D, int format);
int64_t nm_kv_scale_bytes(int64_t n_pages, int page_size, int heads, int D, int format);

/*
 * nm_kv_write -- row t of k and v [T][heads][D] (strided rows, 16-byte aligned)
 * into slot slots[t] (int64, 8-byte aligned).  A slot outside the cache (a
 * negative one: a padding row) is skipped.  Each slot at most once a call: one
 * that is listed twice ends with some mixture of its rows.  All other slots
 * keep their contents.  T below 2^31, T * heads * D below 2^40 (nm_kv_read too).
 */
int nm_kv_write(const nm_kv_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T,
                const int64_t* slots, void* stream);

/*
 * nm_kv_read -- k and v [T][heads][D] (contiguous, 16-byte aligned) from slots
 * slots[t] (any order, repeats allowed); zeros for a slot outside the cache.
 * Quantised values are rounded to the cache's dtype, to nearest even,
 * saturating at its largest finite value.  (The least e of an fp16 cache costs
 * 2^-24 of a value at most.)
 */
int nm_kv_read(const nm_kv_cache* cache, const int64_t* slots, int64_t T, void* k, void* v, void* stream);

/*
 * nm_attn_decode -- one query token per sequence.  Sequence b sees the first
 * prefix_len tokens of the shared pages, then lens[b] tokens of its own:
 *   o[b][h] = sum_t softmax_t(scale * q[b][h] . k[t][h / (Hq / heads)]) v[t][...]
 *   q [B][Hq][D]       strided rows, 16-byte aligned; Hq a multiple of heads.
 *   prefix_pages       int32 [ceil(prefix_len / page_size)] page numbers, the
 *                      same for the whole batch (NULL when prefix_len is 0).
 *   page_table         int32 [B][table_stride]; row b lists b's own pages (at
 *                      least ceil(max_len / page_size) entries a row, of which
 *                      those behind lens[b] are not followed); NULL if max_len is 0.
 *   lens [B] int32     tokens of b behind the prefix, at most max_len (a larger
 *                      one counts as max_len).  Negative: b is a padding row;
 *                      its rows of o and lse are left as they are.
 *   max_len            the work is cut into ranges by it, since lens is on the
 *                      device: one far above the lengths leaves most of the GPU
 *                      without tokens.
 *   o [B][Hq][D]       contiguous, 16-byte aligned; a sequence without a token
 *                      to see gets zeros.
 *   lse [B][Hq]        fp32 (natural log of the softmax's sum; -inf without a
 *                      token), or NULL.
 *   workspace          nm_attn_workspace_bytes(...) bytes of device memory,
 *                      256-byte aligned, any contents; may be NULL when that is 0.
 *                      So many bytes also serve every call with the same Hq,
 *                      heads, D and format and no larger B, prefix_len and max_len.
 * Several query tokens of a sequence (a draft, a piece of a prompt) are a batch
 * row each, with the same pages and a length that ends at the token.
 * A page number outside the cache is not followed: its tokens count as absent.
 * Scores, softmax statistics and sums are fp32; the weights of the sum go into
 * the matrix cores as two operands of dtype each (2^-16 of a weight is lost in
 * bfloat16; in fp16 2^-22 of it, or 2^-32 of the row's largest one if that is
 * more), and o is rounded once to dtype.
 * Results do not depend on other calls and repeat bit for bit.
 * Infinities and NaN in a token that is seen have the effect that the formula
 * gives them (a score of -inf weighs nothing; a row with no other scores gets
 * zeros), and so have fp32 sums that overflow, in which a bfloat16 token's value
 * counts once at most; in a token that is not seen they have none.  (In a
 * quantised bfloat16 cache magnitudes of 2^127 and more count as infinities here.)
 * B and Hq 1..65535, B * Hq below 2^26, prefix_len and max_len 0..2^30, |scale| <= 1e30.  o, lse
 * and workspace must not overlap anything else.
 */
int64_t nm_attn_workspace_bytes(int64_t B, int Hq, int heads, int D, int format, int64_t prefix_len, int64_t max_len);
int nm_attn_decode(const void* q, int64_t q_stride, int64_t B, int Hq, const nm_kv_cache* cache,
                   const int32_t* prefix_pages, int64_t prefix_len, const int32_t* page_table, int64_t table_stride,
                   const int32_t* lens, int64_t max_len, float scale, void* o, float* lse, void* workspace,
                   int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NMATTN_H */
