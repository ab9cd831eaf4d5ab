// nmserve_api.cpp -- the C entry points of include/nmserve.h: argument checks,
// then the kernel side (nm_serve.h).  Host-only C++, as nmapi.cpp is.
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "nm_attn_rules.h"
#include "nm_serve.h"
#include "nmserve.h"

using namespace nmh;

namespace {

constexpr int64_t kMaxElements = int64_t(1) << 40;
constexpr int64_t kMaxWidth = int64_t(1) << 24;

bool heads_ok(int Hq, int heads, int D)
{
    return Hq >= 1 && Hq <= 65535 && heads >= 1 && heads <= 65535 && Hq % heads == 0 && (D == 64 || D == 128 || D == 256);
}

bool prompt_shape_ok(int64_t T, int64_t Tk, int64_t B, int Hq, int heads, int D)
{
    return heads_ok(Hq, heads, D) && T >= 0 && T <= INT32_MAX && Tk >= 0 && Tk < nms::kPromptMaxRows && B >= 0 &&
           B <= 65535 && B * heads < nms::kPromptMaxHeads && T * (Hq / heads) < nms::kPromptMaxRows &&
           T * Hq * D < kMaxElements && Tk * heads * D < kMaxElements;
}

bool tree_shape_ok(int64_t B, int N, int Hq, int heads, int D, int format, int64_t max_len)
{
    return heads_ok(Hq, heads, D) && B >= 1 && B <= 65535 && N >= 1 && N <= 64 && B * N * Hq < nma::kMaxRows &&
           format >= NM_KV_16 && format <= NM_KV_MX4 && max_len >= 0 && max_len <= nma::kMaxTokens;
}

}  // namespace

extern "C" {

int64_t nm_kv_plan_scratch_bytes(int64_t B) { return B >= 1 && B <= 65535 ? nms::plan_scratch(B) : -1; }

int nm_kv_plan(const nm_kv_pages* pages, const int32_t* adds, int64_t rows, int32_t* starts, int64_t* slots,
               int32_t* positions, int32_t* granted, void* stream)
{
    if (!pages)
        return NM_ERR_INVALID_ARG;
    const nm_kv_pages& p = *pages;
    if (p.B < 1 || p.B > 65535 || p.width < 1 || p.width > kMaxWidth || p.B * p.width > INT32_MAX || p.n_pages < 1 ||
        p.n_pages > INT32_MAX || p.page_size < 16 || p.page_size > 256 || (p.page_size & (p.page_size - 1)) != 0 ||
        rows < 0 || rows > INT32_MAX)
        return NM_ERR_BAD_SHAPE;
    const size_t B = (size_t)p.B, n = (size_t)rows;
    const Buf outs[9] = {{p.table, B * (size_t)p.width * 4}, {p.lens, B * 4}, {p.free, (size_t)p.n_pages * 4},
                         {p.n_free, 4}, {p.scratch, (size_t)nms::plan_scratch(p.B)}, {starts, (B + 1) * 4},
                         {slots, n * 8}, {positions, n * 4}, {granted, B * 4}};
    const Buf in = {adds, B * 4};
    if (!ptr_ok(p.table, outs[0].n, 4) || !ptr_ok(p.lens, outs[1].n, 4) || !ptr_ok(p.free, outs[2].n, 4) ||
        !ptr_ok(p.n_free, 4, 4) || !ptr_ok(p.scratch, outs[4].n, 8) || !ptr_ok(starts, outs[5].n, 4) ||
        !ptr_ok(slots, outs[6].n, 8) || !ptr_ok(positions, outs[7].n, 4) || !ptr_ok(granted, outs[8].n, 4) ||
        !ptr_ok(adds, in.n, 4))
        return NM_ERR_INVALID_ARG;
    if (!disjoint(outs, 9, &in, 1))
        return NM_ERR_INVALID_ARG;
    return nmk::kv_plan(p, adds, rows, starts, slots, positions, granted, stream);
}

int64_t nm_attn_prompt_workspace_bytes(int64_t T, int64_t Tk, int64_t B, int Hq, int heads, int D)
{
    return prompt_shape_ok(T, Tk, B, Hq, heads, D) ? nms::prompt_workspace_bound(T, Tk, B, Hq, heads, D) : -1;
}

int64_t nm_attn_prompt_call_bytes(int64_t T, int64_t Tk, int64_t B, int Hq, int heads, int D)
{
    return prompt_shape_ok(T, Tk, B, Hq, heads, D)
               ? nms::prompt_workspace(nms::prompt_plan(T, Tk, B, Hq, heads, D), heads, D)
               : -1;
}

int nm_attn_prompt(const void* q, int64_t q_stride, int64_t T, const void* k, int64_t k_stride, const void* v,
                   int64_t v_stride, int64_t Tk, const int32_t* starts, const int32_t* k_starts, int64_t B, int Hq,
                   int heads, int D, int dtype, float scale, void* o, float* lse, void* workspace,
                   int64_t workspace_bytes, void* stream)
{
    if (check_dtype(dtype) != NM_OK)
        return NM_ERR_UNSUPPORTED;
    if (!prompt_shape_ok(T, Tk, B, Hq, heads, D) || (!k_starts && Tk != T))
        return NM_ERR_BAD_SHAPE;
    const int64_t qw = (int64_t)Hq * D, kw = (int64_t)heads * D;
    if (!stride_ok(T, q_stride, qw, nms::kPromptMaxStride) || !stride_ok(Tk, k_stride, kw, nms::kPromptMaxStride) ||
        !stride_ok(Tk, v_stride, kw, nms::kPromptMaxStride) || !(std::fabs(scale) <= 1e30f))
        return NM_ERR_BAD_SHAPE;
    const nms::PromptPlan plan = nms::prompt_plan(T, Tk, B, Hq, heads, D);
    const int64_t need = nms::prompt_workspace(plan, heads, D);
    const size_t sb = B > 0 ? (size_t)(B + 1) * 4 : 0;
    const Buf ins[5] = {{q, rows_bytes(T, q_stride, qw)}, {k, rows_bytes(Tk, k_stride, kw)},
                        {v, rows_bytes(Tk, v_stride, kw)}, {starts, sb}, {k_starts, k_starts ? sb : 0}};
    const Buf outs[3] = {{o, (size_t)T * (size_t)qw * 2}, {lse, lse ? (size_t)T * (size_t)Hq * 4 : 0},
                         {workspace, workspace && workspace_bytes > 0 ? (size_t)workspace_bytes : 0}};
    if (!ptr_ok(q, ins[0].n, 16) || !ptr_ok(k, ins[1].n, 16) || !ptr_ok(v, ins[2].n, 16) || !ptr_ok(starts, sb, 4) ||
        !aligned(k_starts, 4) || !ptr_ok(o, outs[0].n, 16) || !aligned(lse, 4) || workspace_bytes < 0 ||
        (need > 0 && (!workspace || workspace_bytes < need)) || !aligned(workspace, 256))
        return NM_ERR_INVALID_ARG;
    if (!disjoint(outs, 3, ins, 5))
        return NM_ERR_INVALID_ARG;
    if (T == 0 || B == 0)
        return NM_OK;
    return nmk::attn_prompt(plan, q, q_stride, T, k, k_stride, v, v_stride, Tk, starts, k_starts ? k_starts : starts, B,
                            Hq, heads, D, dtype, scale, o, lse, workspace, stream);
}

int64_t nm_attn_tree_workspace_bytes(int64_t B, int N, int Hq, int heads, int D, int format, int64_t max_len)
{
    return tree_shape_ok(B, N, Hq, heads, D, format, max_len)
               ? nms::tree_workspace_bound(B, N, Hq, heads, D, max_len)
               : -1;
}

int64_t nm_attn_tree_call_bytes(int64_t B, int N, int Hq, int heads, int D, int format, int64_t max_len)
{
    return tree_shape_ok(B, N, Hq, heads, D, format, max_len)
               ? nms::tree_workspace(nms::tree_plan(B, N, Hq, heads, D, format, max_len), D)
               : -1;
}

int nm_attn_tree(const void* q, int64_t q_stride, int64_t B, int N, int Hq, const nm_kv_cache* cache,
                 const uint64_t* visible, const int32_t* page_table, int64_t table_stride, const int32_t* lens,
                 int64_t max_len, float scale, void* o, float* lse, void* workspace, int64_t workspace_bytes,
                 void* stream)
{
    int st = check_cache(cache);
    if (st != NM_OK)
        return st;
    const int64_t width = (int64_t)Hq * cache->D;
    if (!tree_shape_ok(B, N, Hq, cache->heads, cache->D, cache->format, max_len) || !stride_ok(B * N, q_stride, width) ||
        !(std::fabs(scale) <= 1e30f))
        return NM_ERR_BAD_SHAPE;
    const nms::TreePlan plan = nms::tree_plan(B, N, Hq, cache->heads, cache->D, cache->format, max_len);
    const int64_t need = nms::tree_workspace(plan, cache->D), pages = nma::ceil_div(max_len, cache->page_size);
    if (max_len > 0 && B > 1 && (table_stride < pages || table_stride > kMaxStride))
        return NM_ERR_BAD_SHAPE;
    const size_t rows = (size_t)(B * N);
    const size_t tb = max_len > 0 ? ((size_t)(B - 1) * (size_t)(B > 1 ? table_stride : 0) + (size_t)pages) * 4 : 0;
    Buf ins[8];
    cache_bufs(*cache, ins);
    ins[4] = {q, rows_bytes(B * N, q_stride, width)};
    ins[5] = {visible, rows * 8};
    ins[6] = {page_table, tb};
    ins[7] = {lens, (size_t)B * 4};
    const Buf outs[3] = {{o, rows * (size_t)width * 2}, {lse, lse ? rows * (size_t)Hq * 4 : 0},
                         {workspace, workspace && workspace_bytes > 0 ? (size_t)workspace_bytes : 0}};
    if (!ptr_ok(q, ins[4].n, 16) || !ptr_ok(visible, ins[5].n, 8) || !ptr_ok(page_table, tb, 4) ||
        !ptr_ok(lens, ins[7].n, 4) || !ptr_ok(o, outs[0].n, 16) || !aligned(lse, 4) || workspace_bytes < 0 ||
        (need > 0 && (!workspace || workspace_bytes < need)) || !aligned(workspace, 256))
        return NM_ERR_INVALID_ARG;
    if (!disjoint(outs, 3, ins, 8))
        return NM_ERR_INVALID_ARG;
    return nmk::attn_tree(plan, q, q_stride, B, N, Hq, *cache, visible, page_table, table_stride, lens, max_len, scale, o,
                          lse, workspace, stream);
}

}  // extern "C"
