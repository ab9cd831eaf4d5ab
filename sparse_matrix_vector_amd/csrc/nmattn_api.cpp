// nmattn_api.cpp -- the C entry points of include/nmattn.h: argument checks,
// then the kernel side (nm_attn.h).  Host-only C++, as nmapi.cpp is.
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "nm_attn.h"
#include "nm_rules.h"
#include "nmattn.h"

using namespace nmh;

namespace {

constexpr int64_t kMaxCacheBytes = int64_t(1) << 46;
constexpr int64_t kMaxStride = int64_t(1) << 30;    // elements; keeps every byte count below 2^63

struct Buf {
    const void* p;
    size_t n;
};

// No output shares a byte with an input or with another output.
bool disjoint(const Buf* outs, int n_outs, const Buf* ins, int n_ins)
{
    for (int i = 0; i < n_outs; ++i) {
        for (int j = 0; j < n_ins; ++j)
            if (overlaps(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
                return false;
        for (int j = i + 1; j < n_outs; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return false;
    }
    return true;
}

bool stride_ok(int64_t rows, int64_t stride, int64_t width)
{
    return rows <= 1 || (stride >= width && stride % 8 == 0 && stride <= kMaxStride);
}

// Bytes from the first to the last element of strided rows.
size_t rows_bytes(int64_t rows, int64_t stride, int64_t width)
{
    return rows == 0 || width == 0 ? 0 : ((size_t)(rows - 1) * (size_t)(rows > 1 ? stride : 0) + (size_t)width) * 2;
}

int check_cache(const nm_kv_cache* c)
{
    if (!c)
        return NM_ERR_INVALID_ARG;
    if (check_dtype(c->dtype) != NM_OK || c->format < NM_KV_16 || c->format > NM_KV_MX4)
        return NM_ERR_UNSUPPORTED;
    const int64_t bytes = nm_kv_bytes(c->n_pages, c->page_size, c->heads, c->D, c->format);
    if (bytes < 0)
        return NM_ERR_BAD_SHAPE;
    const int64_t sb = nm_kv_scale_bytes(c->n_pages, c->page_size, c->heads, c->D, c->format);
    if (!ptr_ok(c->k, (size_t)bytes, 16) || !ptr_ok(c->v, (size_t)bytes, 16) || !ptr_ok(c->k_scale, (size_t)sb, 16) ||
        !ptr_ok(c->v_scale, (size_t)sb, 16))
        return NM_ERR_INVALID_ARG;
    return NM_OK;
}

void cache_bufs(const nm_kv_cache& c, Buf* out)
{
    const size_t b = (size_t)nm_kv_bytes(c.n_pages, c.page_size, c.heads, c.D, c.format);
    const size_t s = (size_t)nm_kv_scale_bytes(c.n_pages, c.page_size, c.heads, c.D, c.format);
    out[0] = {c.k, b};
    out[1] = {c.v, b};
    out[2] = {c.k_scale, s};
    out[3] = {c.v_scale, s};
}

bool attn_shape_ok(int64_t B, int Hq, int heads, int D, int format, int64_t prefix_len, int64_t max_len)
{
    return B >= 1 && B <= 65535 && Hq >= 1 && Hq <= 65535 && heads >= 1 && heads <= 65535 && Hq % heads == 0 &&
           B * Hq < nma::kMaxRows && (D == 64 || D == 128 || D == 256) && format >= NM_KV_16 && format <= NM_KV_MX4 &&
           prefix_len >= 0 && prefix_len <= nma::kMaxTokens && max_len >= 0 && max_len <= nma::kMaxTokens;
}

}  // namespace

extern "C" {

int nm_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t T, int Hq, int Hk, int D,
                    int dtype, const void* wq, const void* wk, float eps, const int32_t* positions,
                    const float* inv_freq, int rot, int interleaved, void* q_out, void* k_out, void* stream)
{
    if (check_dtype(dtype) != NM_OK)
        return NM_ERR_UNSUPPORTED;
    if (T < 0 || T > INT32_MAX || Hq < 0 || Hq > 65535 || Hk < 0 || Hk > 65535 || D < 8 || D > 512 || D % 8 != 0 ||
        rot < 0 || rot > D || rot % 16 != 0 || !std::isfinite(eps) || eps < 0.0f)
        return NM_ERR_BAD_SHAPE;
    const int64_t qw = (int64_t)Hq * D, kw = (int64_t)Hk * D;
    if ((Hq > 0 && !stride_ok(T, q_stride, qw)) || (Hk > 0 && !stride_ok(T, k_stride, kw)))
        return NM_ERR_BAD_SHAPE;
    const size_t qb = rows_bytes(T, q_stride, qw), kb = rows_bytes(T, k_stride, kw);
    const size_t qo = (size_t)T * (size_t)qw * 2, ko = (size_t)T * (size_t)kw * 2;
    const size_t wb = (size_t)D * 2;
    const bool any = T > 0 && Hq + Hk > 0;
    const size_t pb = any && rot > 0 ? (size_t)T * 4 : 0, fb = any ? (size_t)(rot / 2) * 4 : 0;
    if (!ptr_ok(q, qb, 16) || !ptr_ok(k, kb, 16) || !ptr_ok(q_out, qo, 16) || !ptr_ok(k_out, ko, 16) ||
        !ptr_ok(positions, pb, 4) || !ptr_ok(inv_freq, fb, 4) || !aligned(wq, 16) || !aligned(wk, 16))
        return NM_ERR_INVALID_ARG;
    if (!any)
        return NM_OK;
    // In place: the very same rows, contiguous.
    const bool q_inplace = q_out == q && (T <= 1 || q_stride == qw), k_inplace = k_out == k && (T <= 1 || k_stride == kw);
    const Buf bq = {q, qb}, bk = {k, kb}, oq = {q_out, qo}, ok = {k_out, ko};
    const Buf rest[4] = {{wq, wb}, {wk, wb}, {positions, pb}, {inv_freq, fb}};
    const Buf outs[2] = {oq, ok};
    if (!disjoint(outs, 2, rest, 4) || (!q_inplace && overlaps(oq.p, oq.n, bq.p, bq.n)) ||
        (!k_inplace && overlaps(ok.p, ok.n, bk.p, bk.n)) || overlaps(oq.p, oq.n, bk.p, bk.n) ||
        overlaps(ok.p, ok.n, bq.p, bq.n))
        return NM_ERR_INVALID_ARG;
    return nmk::qk_norm_rope(q, q_stride, k, k_stride, T, Hq, Hk, D, dtype, wq, wk, eps, positions, inv_freq, rot,
                             interleaved, q_out, k_out, stream);
}

int64_t nm_kv_bytes(int64_t n_pages, int page_size, int heads, int D, int format)
{
    if (n_pages < 1 || n_pages > INT32_MAX || heads < 1 || heads > 65535 || page_size < 16 || page_size > 256 ||
        (page_size & (page_size - 1)) != 0 || (D != 64 && D != 128 && D != 256) || format < NM_KV_16 ||
        format > NM_KV_MX4)
        return -1;
    const int64_t page = (int64_t)heads * (page_size / nma::kTile) * nma::tile_bytes(D, nma::format_bits(format));
    return n_pages >= kMaxCacheBytes / page ? -1 : n_pages * page;
}

int64_t nm_kv_scale_bytes(int64_t n_pages, int page_size, int heads, int D, int format)
{
    if (nm_kv_bytes(n_pages, page_size, heads, D, format) < 0)
        return -1;
    return format == NM_KV_16 ? 0 : n_pages * heads * (page_size / nma::kTile) * nma::scale_tile_bytes(D);
}

int nm_kv_write(const nm_kv_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T,
                const int64_t* slots, void* stream)
{
    int st = check_cache(cache);
    if (st != NM_OK)
        return st;
    const int64_t width = (int64_t)cache->heads * cache->D;
    if (T < 0 || T > INT32_MAX || !stride_ok(T, k_stride, width) || !stride_ok(T, v_stride, width))
        return NM_ERR_BAD_SHAPE;
    const Buf ins[3] = {{k, rows_bytes(T, k_stride, width)}, {v, rows_bytes(T, v_stride, width)}, {slots, (size_t)T * 8}};
    if (!ptr_ok(k, ins[0].n, 16) || !ptr_ok(v, ins[1].n, 16) || !ptr_ok(slots, ins[2].n, 8))
        return NM_ERR_INVALID_ARG;
    Buf outs[4];
    cache_bufs(*cache, outs);
    if (!disjoint(outs, 4, ins, 3))
        return NM_ERR_INVALID_ARG;
    if (T == 0)
        return NM_OK;
    return nmk::kv_write(*cache, k, k_stride, v, v_stride, T, slots, stream);
}

int nm_kv_read(const nm_kv_cache* cache, const int64_t* slots, int64_t T, void* k, void* v, void* stream)
{
    int st = check_cache(cache);
    if (st != NM_OK)
        return st;
    if (T < 0 || T > INT32_MAX)
        return NM_ERR_BAD_SHAPE;
    const size_t n = (size_t)T * (size_t)cache->heads * (size_t)cache->D * 2;
    if (!ptr_ok(k, n, 16) || !ptr_ok(v, n, 16) || !ptr_ok(slots, (size_t)T * 8, 8))
        return NM_ERR_INVALID_ARG;
    Buf ins[5];
    cache_bufs(*cache, ins);
    ins[4] = {slots, (size_t)T * 8};
    const Buf outs[2] = {{k, n}, {v, n}};
    if (!disjoint(outs, 2, ins, 5))
        return NM_ERR_INVALID_ARG;
    if (T == 0)
        return NM_OK;
    return nmk::kv_read(*cache, slots, T, k, v, stream);
}

int64_t nm_attn_workspace_bytes(int64_t B, int Hq, int heads, int D, int format, int64_t prefix_len, int64_t max_len)
{
    return attn_shape_ok(B, Hq, heads, D, format, prefix_len, max_len)
               ? nma::attn_workspace_bound(B, Hq, heads, D, format, prefix_len, max_len)
               : -1;
}

int nm_attn_decode(const void* q, int64_t q_stride, int64_t B, int Hq, const nm_kv_cache* cache,
                   const int32_t* prefix_pages, int64_t prefix_len, const int32_t* page_table, int64_t table_stride,
                   const int32_t* lens, int64_t max_len, float scale, void* o, float* lse, void* workspace,
                   int64_t workspace_bytes, void* stream)
{
    int st = check_cache(cache);
    if (st != NM_OK)
        return st;
    const int64_t width = (int64_t)Hq * cache->D;
    if (!attn_shape_ok(B, Hq, cache->heads, cache->D, cache->format, prefix_len, max_len) || !stride_ok(B, q_stride, width) ||
        !(std::fabs(scale) <= 1e30f))
        return NM_ERR_BAD_SHAPE;
    const nma::AttnPlan plan = nma::attn_plan(B, Hq, cache->heads, cache->D, cache->format, prefix_len, max_len);
    const int64_t need = nma::attn_workspace(plan, cache->D);
    const int64_t own_pages = nma::ceil_div(max_len, cache->page_size);
    if (max_len > 0 && B > 1 && (table_stride < own_pages || table_stride > kMaxStride))
        return NM_ERR_BAD_SHAPE;
    const size_t tb = max_len > 0 ? ((size_t)(B - 1) * (size_t)(B > 1 ? table_stride : 0) + (size_t)own_pages) * 4 : 0;
    const size_t pb = (size_t)nma::ceil_div(prefix_len, cache->page_size) * 4;
    Buf ins[8];
    cache_bufs(*cache, ins);
    ins[4] = {q, rows_bytes(B, q_stride, width)};
    ins[5] = {prefix_pages, pb};
    ins[6] = {page_table, tb};
    ins[7] = {lens, (size_t)B * 4};
    const Buf outs[3] = {{o, (size_t)B * (size_t)width * 2}, {lse, lse ? (size_t)B * (size_t)Hq * 4 : 0},
                         {workspace, workspace && workspace_bytes > 0 ? (size_t)workspace_bytes : 0}};
    if (!ptr_ok(q, ins[4].n, 16) || !ptr_ok(prefix_pages, pb, 4) || !ptr_ok(page_table, tb, 4) ||
        !ptr_ok(lens, ins[7].n, 4) || !ptr_ok(o, outs[0].n, 16) || !ptr_ok(lse, outs[1].n, 4) ||
        workspace_bytes < 0 || (need > 0 && (!workspace || workspace_bytes < need)) || !aligned(workspace, 256))
        return NM_ERR_INVALID_ARG;
    if (!disjoint(outs, 3, ins, 8))
        return NM_ERR_INVALID_ARG;
    return nmk::attn_decode(plan, q, q_stride, B, Hq, *cache, prefix_pages, prefix_len, page_table, table_stride, lens,
                            max_len, scale, o, lse, workspace, stream);
}

}  // extern "C"
