/*
 * nmserve.h -- C ABI of libnmspmv, third part: what a server does around the
 * decode step of nmattn.h.
 *
 *   nm_kv_plan        page tables, slots, positions and row starts from the
 *                     sequences' lengths and requests, on the device
 *   nm_attn_prompt    causal attention over whole prompts (or pieces of them
 *                     behind earlier tokens), packed one after the other
 *   nm_attn_tree      attention of a tree of drafted tokens over the paged cache
 *
 * ---- Conventions ------------------------------------------------------------
 * Those of nmattn.h: device pointers, caller-owned buffers, NM_* status codes,
 * every check before any work is queued, calls only enqueue on `stream` and are
 * thread-safe; no call allocates, waits or copies to the host, so all of them can
 * be captured into a graph.  Strided rows are what they are there.
 */
#ifndef NMSERVE_H
#define NMSERVE_H

#include <stdint.h>

#include "nmattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ---- Pages ---------------------------------------------------------------------
 * The book of a cache's pages: which pages each sequence has, and which are free.
 *   table   int32 [B][width]  row b lists b's pages in order (nm_attn_decode's
 *           page_table with table_stride = width); entries behind a sequence's
 *           last page mean nothing and are left as they are.
 *   lens    int32 [B]  tokens held; negative: a padding row.
 *   free    int32 [n_pages]  a stack of free page numbers, n_free[0] of them, the
 *           top one last.  (n_free is taken for 0 .. n_pages where it is not.)
 *   scratch nm_kv_plan_scratch_bytes(B) bytes, any contents, used within a call.
 * B 1 .. 65535, width 1 .. 2^24, B * width below 2^31, n_pages 1 .. 2^31 - 1,
 * page_size as in a cache (16, 32, 64, 128 or 256).  Pointers 4-byte, scratch 8-byte aligned.
 */
typedef struct {
    int32_t* table;
    int32_t* lens;
    int32_t* free;
    int32_t* n_free;
    void* scratch;
    int64_t B;
    int64_t width;
    int64_t n_pages;
    int page_size;
} nm_kv_pages;

int64_t nm_kv_plan_scratch_bytes(int64_t B);

/*
 * nm_kv_plan -- one step of the book.  adds[b] (int32 [B]) is what sequence b asks
 * for: tokens to come (positive), tokens to drop from its end (negative; all it has
 * at most: a sequence that ends, drafts that are refused), or nothing.
 *   1. Dropped tokens' pages go back onto the stack: the first one (lowest b, then
 *      lowest place in b's row) comes to lie on top.
 *   2. Then each sequence in turn gets the tokens it asks for, its new pages taken
 *      off the top of the stack one by one.  A sequence whose row of the table is too
 *      short gets none.  The first one for which the pages or the `rows` rows do not
 *      suffice gets none, and no later one does: none is overtaken.
 *   3. lens is brought up to date.
 * Outputs:
 *   granted   int32 [B]  tokens that b got (positive) or lost (negative).
 *   starts    int32 [B + 1]  b's new tokens are rows starts[b] .. starts[b+1] - 1.
 *   slots     int64 [rows]  a row's slot (page * page_size + place), for nm_kv_write;
 *             -1 behind the last row, and where a page number is negative.
 *   positions int32 [rows]  a row's place in its sequence; 0 behind the last row.
 * New rows are packed: a sequence that gets nothing has none.  nm_attn_prompt takes them
 * as they lie; nm_attn_decode (N = 1) and nm_attn_tree take rows b N .. b N + N - 1 for
 * sequence b.  Where one may get nothing (a padding row, a row of the table that is too short,
 * no pages), a step of N tokens a sequence is laid out by b N: row b N + i has slot
 * slots[starts[b] + i], or -1 where granted[b] is not positive, and such a sequence goes into
 * attention with the length -1.  A row's place is its position in the text, but for the drafts
 * of a tree with branches: draft i's is lens[b] - N + its depth (a root's is 0).  Dropping takes the last tokens;
 * kept drafts behind refused ones are moved to their places first (nm_kv_read, nm_kv_write).
 * Dropping what was just granted leaves the stack and lens as they were.
 * Padding rows get and lose nothing.  rows 0 .. 2^31 - 1; lens plus adds must stay below
 * 2^31.  No output or part of the book may overlap anything else.  Calls on one book
 * must follow each other (they share its scratch, too).
 */
int nm_kv_plan(const nm_kv_pages* pages, const int32_t* adds, int64_t rows, int32_t* starts, int64_t* slots,
               int32_t* positions, int32_t* granted, void* stream);

/*
 * nm_attn_prompt -- B sequences, packed: the queries of b are rows starts[b] ..
 * starts[b+1] - 1 of q, its keys and values rows k_starts[b] .. k_starts[b+1] - 1 of
 * k and v.  A sequence's last query stands at its last key: of nq queries and nk
 * keys, query i sees keys j <= i + nk - nq,
 *   o[i][h] = sum_j softmax_j(scale * q[i][h] . k[j][h / (Hq / heads)]) v[j][...]
 *   q [T][Hq][D], k, v [Tk][heads][D]  strided rows, 16-byte aligned; Hq a multiple
 *     of heads, D 64, 128 or 256.  More keys than queries: a piece of a prompt
 *     behind nk - nq earlier tokens (nm_kv_read gives their rows).
 *   starts, k_starts   int32 [B + 1], not decreasing, 0 .. T and 0 .. Tk (bounds
 *     outside count as the nearest of these, a sequence that ends before it starts
 *     as empty; starts that decrease say nothing about which rows of o are written,
 *     but no others than o's and lse's are).  k_starts NULL: starts, and Tk is T.
 *   o [T][Hq][D]       contiguous, 16-byte aligned; a query that sees no key gets
 *     zeros.  Rows that no sequence has are left as they are.
 *   lse [T][Hq]        fp32 (natural log of the softmax's sum; -inf where no key is
 *     seen), or NULL.
 *   workspace          nm_attn_prompt_call_bytes(...) bytes of device memory,
 *     256-byte aligned, any contents; may be NULL when that is 0.  So many serve
 *     calls of exactly these sizes; nm_attn_prompt_workspace_bytes(...) bytes serve
 *     every call with the same Hq, heads and D and no larger T, Tk and B.
 * Few rows behind many keys are cut into ranges of keys by the average Tk / B, since lengths
 * are on the device: one long sequence among many short ones is not cut, and is faster in
 * a call of its own (a query on 16384 keys beside 31 on 16: 278 us, alone 28).
 * Scores, softmax statistics and sums are fp32.  The weights of the sum are rounded
 * to dtype, and so the sum that they are divided by adds the rounded ones (nm_attn_decode and
 * nm_attn_tree keep more of them: a token's results as a prompt and as a decode step differ by that).
 * Infinities and NaN in a key or value that a query does not see do not reach it; in
 * one that it sees they have the effect that the formula gives them (a score of -inf weighs
 * nothing; a query with no other scores gets zeros), and so have fp32 sums that overflow.
 * Results do not depend on other calls and repeat bit for bit.
 * B 0 .. 65535, Hq and heads 1 .. 65535, B * heads below 2^30, T * Hq / heads and Tk
 * below 2^31 - 2^16, T * Hq * D and Tk * heads * D below 2^40, row strides up to 2^28
 * elements, |scale| <= 1e30.  o, lse and workspace must not overlap anything else.
 */
int64_t nm_attn_prompt_workspace_bytes(int64_t T, int64_t Tk, int64_t B, int Hq, int heads, int D);
int64_t nm_attn_prompt_call_bytes(int64_t T, int64_t Tk, int64_t B, int Hq, int heads, int D);
int nm_attn_prompt(const void* q, int64_t q_stride, int64_t T, const void* k, int64_t k_stride, const void* v,
                   int64_t v_stride, int64_t Tk, const int32_t* starts, const int32_t* k_starts, int64_t B, int Hq,
                   int heads, int D, int dtype, float scale, void* o, float* lse, void* workspace,
                   int64_t workspace_bytes, void* stream);

/*
 * nm_attn_tree -- N drafted tokens a sequence, arranged as a tree, over the cache.
 * Sequence b holds lens[b] tokens in its pages, the last N of which are the drafts.
 * Draft i sees every token before the drafts, and draft j where bit j of
 * visible[b][i] is set (itself and the drafts that lead to it, in a tree):
 *   o[b][i][h] = sum_t softmax_t(scale * q[b][i][h] . k[t][h / (Hq / heads)]) v[t][...]
 *   q [B * N][Hq][D]   strided rows, 16-byte aligned; Hq a multiple of heads.  Sequence b's
 *     drafts are rows b N .. b N + N - 1, whatever nm_kv_plan granted to those before it.
 *   visible [B][N]     64-bit masks, 8-byte aligned; bits N and above are not looked at.
 *   page_table, table_stride, lens, max_len, lse: as for nm_attn_decode (lens counts
 *     the drafts; a length above max_len counts as max_len; one below N lacks the first
 *     drafts; negative: a padding row, whose rows of o and lse stay).
 *   workspace: as for nm_attn_prompt, nm_attn_tree_call_bytes(...) for calls of exactly
 *     these sizes, nm_attn_tree_workspace_bytes(...) for those of no larger B and max_len.
 *     (max_len also decides the form of the work: 16 sequences of 24 drafts and up to 512 tokens,
 *     MX8, take 16 us with the longest length, 33 with four times that or more.)
 *   o [B][N][Hq][D], lse [B][N][Hq]; zeros and -inf for a draft that sees no token.
 * Types, rounding, absent pages, infinities and NaN: as for nm_attn_decode; what one
 * draft does not see does not reach it.
 * B and Hq 1..65535, N 1..64, B * N * Hq below 2^26, max_len 0..2^30, |scale| <= 1e30.
 */
int64_t nm_attn_tree_workspace_bytes(int64_t B, int N, int Hq, int heads, int D, int format, int64_t max_len);
int64_t nm_attn_tree_call_bytes(int64_t B, int N, int Hq, int heads, int D, int format, int64_t max_len);
int nm_attn_tree(const void* q, int64_t q_stride, int64_t B, int N, int Hq, const nm_kv_cache* cache,
                 const uint64_t* visible, const int32_t* page_table, int64_t table_stride, const int32_t* lens,
                 int64_t max_len, float scale, void* o, float* lse, void* workspace, int64_t workspace_bytes,
                 void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NMSERVE_H */
