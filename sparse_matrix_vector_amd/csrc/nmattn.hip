// nmattn.hip -- nm_attn_decode: single-token attention over the paged cache.
//
// For the rows (query heads) q of a unit and its tokens t, with scores
// s_t = scale * q . k_t, one pass keeps a reference m near the running maximum, the
// sum l = sum exp(s_t - m) and the vector o = sum exp(s_t - m) v_t, multiplying l and
// o by exp(m_old - m_new) where m is raised (Weights); units of one row are joined by
// the same rule (combine_kernel).
//
// Everything runs on the matrix cores with the cache as the left operand, 16
// tokens or 16 columns by 16 rows (v_mfma_f32_16x16x32):
//   scores  S^T[token][row]  = sum over columns of K[token][d] q[row][d]
//   output  O^T[d][row]     += sum over tokens of V[token][d] p[row][token]
// In both a lane's column is its row of q (lane % 16), so the softmax statistics
// and the rescaling of o are per lane.  The score tile's layout (lane quarter kg,
// register r: token 4 kg + r) is the second product's right operand as it
// stands when a step takes two 16-token tiles: its k index (kg, i) is token
// 4 kg + i of the first tile for i < 4, of the second for i >= 4.  The values are
// stored in that order, the keys in the order of the first product's left
// operand (nm_attn.h), so nothing passes through LDS and a wave's loads are
// contiguous pieces of 512 or 1024 bytes.
//
// Own tokens are bound by HBM: 32 sequences of 4096 tokens, 8 key heads of 128
// columns, MX8, take 45.5 us, 6.1 TB/s; with few or very different sequences the
// start of the blocks and the joining of ranges show (16 of 0 .. 8192: 29 + 4 us, 5.1
// TB/s; one of 131071, MX4: 27 + 4, 5.2).  A shared prefix of many rows is bound by the
// matrix cores and the vector instructions beside them (attend_staged), one of few rows
// by HBM.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "nm_attn_units.h"

namespace {

using namespace nmu;

int hip_status(hipError_t e) { return e == hipSuccess ? NM_OK : NM_ERR_HIP; }

// One launch for all units: the first prefix_blocks blocks take prefix units, staged
// with W waves or (W = 0) like own tokens, the others own-token units = (range, row
// group, sequence, key head).  Two waves a SIMD: with more than 256 registers to
// spend the compiler keeps sums in accumulation registers and moves them to and fro, a
// thousand moves beside 64 products (tests/test_attn_registers.py holds the build to none).
// That costs time only: in such a build, too, what reaches each key and value operand of a
// product is its own loads, conversions and masks and nothing else, by the assembly of all
// these kernels.
template <int DT, int BITS, int D, int MT, int W>
__global__ __launch_bounds__((W ? W : nma::kWaves) * 64, 2) void units_kernel(const AttnArgs A, int prefix_blocks, int blocks, int direct)
{
    constexpr int NW = W ? W : nma::kWaves;
    constexpr int kJoin = join_bytes(D, W ? 1 : MT, NW), kLds = W && staged_bytes<BITS, D, W ? W : 4>() > kJoin
                                                                    ? staged_bytes<BITS, D, W ? W : 4>() : kJoin;
    __shared__ __align__(16) uint8_t lds[kLds];
    float* const join = reinterpret_cast<float*>(lds);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int block = (int)flat_block();
    if (block >= blocks)
        return;
    if (block < prefix_blocks) {
        const int unit = block;
        if constexpr (W > 0) {
            attend_staged<DT, BITS, D, MT, W>(A, unit, lds);
        } else {
            const int h = unit % A.heads, split = unit / A.heads % A.prefix_splits, group = unit / A.heads / A.prefix_splits;
            const int start = split * A.prefix_chunk, end = min(start + A.prefix_chunk, A.prefix_len);
            const int at = start / nma::kTile + 2 * wave;
            attend<OneToken, DT, BITS, D, MT, NW>(A, A.prefix_pages, h, 0, group * 16 * MT, A.prefix_rows, start, end,
                                                  end, page_of(A, A.prefix_pages, at, end),
                                                  page_of(A, A.prefix_pages, at + 1, end), false,
                                                  ((int64_t)split * A.heads + h) * A.prefix_rows, {}, join);
        }
        return;
    }
    const unsigned unit = block - prefix_blocks;
    const int h = unit % A.heads, b = unit / A.heads % A.B;
    const int group = unit / A.heads / A.B % A.own_groups, split = unit / A.heads / A.B / A.own_groups;
    const int start = split * A.own_chunk, at = start / nma::kTile + 2 * wave;
    // The length and the first page numbers come together: the table's entries behind
    // the length may be read, they are only not followed.
    const int32_t* pages = A.page_table + (int64_t)b * A.table_stride;
    const int held = A.lens[b], page0 = page_of(A, pages, at, A.max_len), page1 = page_of(A, pages, at + 1, A.max_len);
    asm volatile("" ::"s"(held), "s"(page0), "s"(page1));
    const int len = min(held, A.max_len);
    if (len < 0 || (start >= len && !direct))   // combine looks at the ranges that hold tokens only
        return;
    attend<OneToken, DT, BITS, D, 1, NW>(A, pages, h, b, group * 16, A.G, start, min(start + A.own_chunk, len),
                                         A.max_len, page0, page1, direct != 0,
                                         A.own_base + ((int64_t)split * A.B + b) * A.Hq + (int64_t)h * A.G, {}, join);
}

template <int DT, int D, int NW>
__global__ __launch_bounds__(NW * 64) void combine_kernel(const AttnArgs A)
{
    combine<OneToken, DT, D, NW>(A);
}

template <int DT, int BITS, int D, int MT, int W>
void launch_units(const AttnArgs& A, int64_t prefix_blocks, int64_t blocks, bool direct, hipStream_t s)
{
    hipLaunchKernelGGL((units_kernel<DT, BITS, D, MT, W>), flat_grid(blocks), dim3((W ? W : nma::kWaves) * 64), 0, s, A,
                       (int)prefix_blocks, (int)blocks, direct ? 1 : 0);
}

template <int DT, int BITS, int D>
int launch(const nma::AttnPlan& P, const AttnArgs& A, hipStream_t s)
{
    (void)hipGetLastError();
    const int64_t prefix_blocks = P.prefix_groups * P.prefix_splits * A.heads;
    const int64_t all = prefix_blocks + (P.direct ? 1 : P.own_splits) * P.own_groups * A.B * (int64_t)A.heads;
    if (all > INT32_MAX)
        return NM_ERR_BAD_SHAPE;
    constexpr int kMt = D == 256 ? 1 : 2;           // of the larger prefix units (attn_plan)
    if (prefix_blocks == 0 || (P.waves == 0 && P.mt == 1))
        launch_units<DT, BITS, D, 1, 0>(A, prefix_blocks, all, P.direct, s);
    else if (P.waves == 8)
        launch_units<DT, BITS, D, kMt, 8>(A, prefix_blocks, all, false, s);
    else if constexpr (D != 256) {
        if (P.waves == 4)
            launch_units<DT, BITS, D, 2, 4>(A, prefix_blocks, all, false, s);
        else
            launch_units<DT, BITS, D, 2, 0>(A, prefix_blocks, all, false, s);
    }
    if (!P.direct) {
        const int64_t blocks = nma::ceil_div(P.prefix_rows, 16) * A.heads * (D / 16);
        if (blocks > INT32_MAX)
            return NM_ERR_BAD_SHAPE;
        // Few tiles of rows have many parts each: more waves share them then.
        if (blocks < 2 * nma::kCus && P.prefix_splits + P.own_splits > 16)
            hipLaunchKernelGGL((combine_kernel<DT, D, 16>), flat_grid(blocks), dim3(1024), 0, s, A);
        else
            hipLaunchKernelGGL((combine_kernel<DT, D, 4>), flat_grid(blocks), dim3(256), 0, s, A);
    }
    return hip_status(hipGetLastError());
}

template <int DT, int BITS>
int launch_width(const nma::AttnPlan& P, const AttnArgs& A, int D, hipStream_t s)
{
    switch (D) {
    case 64: return launch<DT, BITS, 64>(P, A, s);
    case 128: return launch<DT, BITS, 128>(P, A, s);
    default: return launch<DT, BITS, 256>(P, A, s);
    }
}

template <int DT>
int launch_format(const nma::AttnPlan& P, const AttnArgs& A, int format, int D, hipStream_t s)
{
    switch (format) {
    case NM_KV_16: return launch_width<DT, 16>(P, A, D, s);
    case NM_KV_MX8: return launch_width<DT, 8>(P, A, D, s);
    default: return launch_width<DT, 4>(P, A, D, s);
    }
}

}  // namespace

int nmk::attn_decode(const nma::AttnPlan& plan, const void* q, int64_t q_stride, int64_t B, int Hq,
                     const nm_kv_cache& cache, const int32_t* prefix_pages, int64_t prefix_len,
                     const int32_t* page_table, int64_t table_stride, const int32_t* lens, int64_t max_len, float scale,
                     void* o, float* lse, void* workspace, void* stream)
{
    AttnArgs A = {};
    A.q = static_cast<const uint16_t*>(q);
    A.k = static_cast<const uint8_t*>(cache.k);
    A.v = static_cast<const uint8_t*>(cache.v);
    A.k_scale = cache.k_scale;
    A.v_scale = cache.v_scale;
    A.prefix_pages = prefix_pages;
    A.page_table = page_table;
    A.lens = lens;
    A.o = static_cast<uint16_t*>(o);
    A.lse = lse;
    A.part_o = static_cast<float*>(workspace);
    A.part_ml = reinterpret_cast<f32x2*>(A.part_o + (plan.prefix_parts + plan.own_parts) * cache.D);
    A.q_stride = B > 1 ? q_stride : 0;
    A.table_stride = B > 1 && max_len > 0 ? table_stride : 0;
    A.n_pages = (int)cache.n_pages;
    A.own_base = plan.prefix_parts;
    A.B = (int)B;
    A.Hq = Hq;
    A.heads = cache.heads;
    A.G = plan.G;
    A.page_shift = __builtin_ctz((unsigned)cache.page_size);
    A.prefix_len = (int)prefix_len;
    A.max_len = (int)max_len;
    A.prefix_rows = (int)plan.prefix_rows;
    A.prefix_groups = (int)plan.prefix_groups;
    A.prefix_splits = (int)plan.prefix_splits;
    A.prefix_chunk = (int)plan.prefix_chunk;
    A.own_groups = (int)plan.own_groups;
    A.own_splits = (int)plan.own_splits;
    A.own_chunk = (int)plan.own_chunk;
    // Codes of an fp16 cache become halves of their values (nm_attn.h: scale bytes).
    A.o_scale = cache.format != NM_KV_16 && cache.dtype == NM_FP16 ? 2.0f : 1.0f;
    A.scale = scale == 0.0f ? 1.0f : fabsf(scale) * kLog2e * A.o_scale;
    A.q_and = scale == 0.0f ? 0u : 0xFFFFFFFFu;
    A.q_xor = scale < 0.0f ? 0x80008000u : 0u;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return cache.dtype == NM_FP16 ? launch_format<NM_FP16>(plan, A, cache.format, cache.D, s)
                                  : launch_format<NM_BF16>(plan, A, cache.format, cache.D, s);
}
