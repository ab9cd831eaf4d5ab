// nm_attn_rules.h -- argument rules that the entry points of include/nmattn.h and
// include/nmserve.h share: strided rows, buffers that must lie apart, caches.
// Host-only C++, as nm_rules.h is.
#ifndef NM_ATTN_RULES_H
#define NM_ATTN_RULES_H

#include "nm_attn.h"
#include "nm_rules.h"

namespace nmh {

constexpr int64_t kMaxCacheBytes = int64_t(1) << 46;
constexpr int64_t kMaxStride = int64_t(1) << 30;    // elements; keeps every byte count below 2^63

struct Buf {
    const void* p;
    size_t n;
};

// No output shares a byte with an input or with another output.
inline bool disjoint(const Buf* outs, int n_outs, const Buf* ins, int n_ins)
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

inline bool stride_ok(int64_t rows, int64_t stride, int64_t width, int64_t most = kMaxStride)
{
    return rows <= 1 || (stride >= width && stride % 8 == 0 && stride <= most);
}

// Bytes from the first to the last element of strided rows.
inline size_t rows_bytes(int64_t rows, int64_t stride, int64_t width)
{
    return rows == 0 || width == 0 ? 0 : ((size_t)(rows - 1) * (size_t)(rows > 1 ? stride : 0) + (size_t)width) * 2;
}

inline int check_cache(const nm_kv_cache* c)
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

inline void cache_bufs(const nm_kv_cache& c, Buf* out)
{
    const size_t b = (size_t)nm_kv_bytes(c.n_pages, c.page_size, c.heads, c.D, c.format);
    const size_t s = (size_t)nm_kv_scale_bytes(c.n_pages, c.page_size, c.heads, c.D, c.format);
    out[0] = {c.k, b};
    out[1] = {c.v, b};
    out[2] = {c.k_scale, s};
    out[3] = {c.v_scale, s};
}

}  // namespace nmh

#endif  // NM_ATTN_RULES_H
