// nmtree.hip -- nm_attn_tree: attention of drafted tokens over the paged cache.
//
// A sequence's rows are its drafts' query heads of one key head, N G of them, and a
// unit takes 16 to 256 of them over a range of its tokens, so that the cache is read
// once for all drafts (once for every 256 rows), as a shared prefix is in
// nm_attn_decode; the units are the same (nm_attn_units.h): up to 32 rows a wave
// reads the cache itself and the block's waves take tiles in turn, beyond that 4 or 8
// waves of 32 rows share it through LDS.  Only tiles with drafts among their tokens
// look at the masks.
//   Up to some 64 rows the cache's bytes bound it, then the matrix cores and the vector
// work beside them.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "nm_attn_units.h"
#include "nm_serve.h"

namespace {

using namespace nmu;

// Units = (range, row group, sequence, key head).
template <int DT, int BITS, int D, int MT, int W>
__global__ __launch_bounds__((W ? W : nma::kWaves) * 64, 2) void tree_kernel(const AttnArgs A, int blocks, int direct)
{
    constexpr int NW = W ? W : nma::kWaves;
    constexpr int kLds = W ? staged_bytes<BITS, D, W ? W : 4>() : join_bytes(D, MT, NW);
    __shared__ __align__(16) uint8_t lds[kLds];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int block = (int)flat_block();
    if (block >= blocks)
        return;
    const unsigned unit = block;
    const int h = unit % A.heads, b = unit / A.heads % A.B;
    const int group = unit / A.heads / A.B % A.own_groups, split = unit / A.heads / A.B / A.own_groups;
    const int start = split * A.own_chunk;
    const int32_t* pages = A.page_table + (int64_t)b * A.table_stride;
    const int len = __builtin_amdgcn_readfirstlane(min(A.lens[b], A.max_len));
    if (len < 0 || (start >= len && !direct))       // combine looks at the ranges that hold tokens only
        return;
    const int end = min(start + A.own_chunk, len);
    const int64_t part_row = ((int64_t)split * A.B + b) * A.Hq + (int64_t)h * A.G;
    if constexpr (W > 0) {
        attend_staged<Drafts, DT, BITS, D, MT, W>(A, pages, h, b, group, A.G, start, end, direct != 0, part_row, lds);
    } else {
        const int at = start / nma::kTile + 2 * wave, row0 = group * 16 * MT;
        Seen<Drafts, MT> seen;
        seen.load(A, b, len, row0, A.G, threadIdx.x % 16);
        attend<Drafts, DT, BITS, D, MT, NW>(A, pages, h, b, row0, A.G, start, end, A.max_len,
                                            page_of(A, pages, at, A.max_len), page_of(A, pages, at + 1, A.max_len),
                                            direct != 0, part_row, seen, reinterpret_cast<float*>(lds));
    }
}

template <int DT, int D, int NW>
__global__ __launch_bounds__(NW * 64) void tree_join_kernel(const AttnArgs A)
{
    combine<Drafts, DT, D, NW>(A);
}

template <int DT, int BITS, int D, int MT, int W>
void launch_units(const AttnArgs& A, int64_t blocks, bool direct, hipStream_t s)
{
    hipLaunchKernelGGL((tree_kernel<DT, BITS, D, MT, W>), flat_grid(blocks), dim3((W ? W : nma::kWaves) * 64), 0, s, A,
                       (int)blocks, direct ? 1 : 0);
}

template <int DT, int BITS, int D>
int launch(const nms::TreePlan& P, const AttnArgs& A, hipStream_t s)
{
    const int64_t blocks = P.splits * P.groups * A.B * (int64_t)A.heads;
    const int64_t join = nma::ceil_div((int64_t)A.B * A.G, 16) * A.heads * (D / 16);
    if (blocks > INT32_MAX || join > INT32_MAX)
        return NM_ERR_BAD_SHAPE;
    (void)hipGetLastError();
    constexpr int kMt = D == 256 ? 1 : 2;
    if (P.waves == 0 && P.mt == 1)
        launch_units<DT, BITS, D, 1, 0>(A, blocks, P.direct, s);
    else if (P.waves == 8)
        launch_units<DT, BITS, D, kMt, 8>(A, blocks, P.direct, s);
    else if constexpr (D != 256) {
        if (P.waves == 4)
            launch_units<DT, BITS, D, 2, 4>(A, blocks, P.direct, s);
        else
            launch_units<DT, BITS, D, 2, 0>(A, blocks, P.direct, s);
    }
    if (!P.direct) {
        // Few tiles of rows have many parts each: more waves share them then.
        if (join < 2 * nma::kCus && P.splits > 16)
            hipLaunchKernelGGL((tree_join_kernel<DT, D, 16>), flat_grid(join), dim3(1024), 0, s, A);
        else
            hipLaunchKernelGGL((tree_join_kernel<DT, D, 4>), flat_grid(join), dim3(256), 0, s, A);
    }
    return hipGetLastError() == hipSuccess ? NM_OK : NM_ERR_HIP;
}

template <int DT, int BITS>
int launch_width(const nms::TreePlan& P, const AttnArgs& A, int D, hipStream_t s)
{
    switch (D) {
    case 64: return launch<DT, BITS, 64>(P, A, s);
    case 128: return launch<DT, BITS, 128>(P, A, s);
    default: return launch<DT, BITS, 256>(P, A, s);
    }
}

template <int DT>
int launch_format(const nms::TreePlan& P, const AttnArgs& A, int format, int D, hipStream_t s)
{
    switch (format) {
    case NM_KV_16: return launch_width<DT, 16>(P, A, D, s);
    case NM_KV_MX8: return launch_width<DT, 8>(P, A, D, s);
    default: return launch_width<DT, 4>(P, A, D, s);
    }
}

}  // namespace

int nmk::attn_tree(const nms::TreePlan& plan, const void* q, int64_t q_stride, int64_t B, int N, int Hq,
                   const nm_kv_cache& cache, const uint64_t* visible, const int32_t* page_table, int64_t table_stride,
                   const int32_t* lens, int64_t max_len, float scale, void* o, float* lse, void* workspace, void* stream)
{
    AttnArgs A = {};
    A.q = static_cast<const uint16_t*>(q);
    A.k = static_cast<const uint8_t*>(cache.k);
    A.v = static_cast<const uint8_t*>(cache.v);
    A.k_scale = cache.k_scale;
    A.v_scale = cache.v_scale;
    A.page_table = page_table;
    A.lens = lens;
    A.o = static_cast<uint16_t*>(o);
    A.lse = lse;
    A.part_o = static_cast<float*>(workspace);
    A.part_ml = reinterpret_cast<f32x2*>(A.part_o + plan.parts * cache.D);
    A.q_stride = B * N > 1 ? q_stride : 0;
    A.table_stride = B > 1 && max_len > 0 ? table_stride : 0;
    A.n_pages = (int)cache.n_pages;
    A.B = (int)B;
    A.Hq = N * Hq;
    A.heads = cache.heads;
    A.G = (int)plan.rows;
    A.page_shift = __builtin_ctz((unsigned)cache.page_size);
    A.max_len = (int)max_len;
    A.prefix_rows = (int)(B * plan.rows);
    A.own_groups = (int)plan.groups;
    A.own_splits = (int)plan.splits;
    A.own_chunk = (int)plan.chunk;
    // Codes of an fp16 cache become halves of their values (nm_attn.h: scale bytes).
    A.o_scale = cache.format != NM_KV_16 && cache.dtype == NM_FP16 ? 2.0f : 1.0f;
    A.scale = scale == 0.0f ? 1.0f : fabsf(scale) * kLog2e * A.o_scale;
    A.q_and = scale == 0.0f ? 0u : 0xFFFFFFFFu;
    A.q_xor = scale < 0.0f ? 0x80008000u : 0u;
    A.visible = visible;
    A.drafts = N;
    A.heads_g = Hq / cache.heads;
    A.heads_q = Hq;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return cache.dtype == NM_FP16 ? launch_format<NM_FP16>(plan, A, cache.format, cache.D, s)
                                  : launch_format<NM_BF16>(plan, A, cache.format, cache.D, s);
}
