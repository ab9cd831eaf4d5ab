// nmtree.hip -- nm_attn_tree: attention of drafted tokens over the paged cache.
//
// A sequence's rows are its drafts' query heads of one key head, N G of them, and a
// unit takes up to 128 of them over a range of its tokens, so that the cache comes from
// memory once for all drafts.  Two forms:
//   up to 32 rows of up to 128 columns: as in nm_attn_decode (nm_attn_units.h), each wave
//     reads the cache itself, straight into operands, and takes pairs of tiles in turn;
//   else (shared_kernel) a block of four waves shares it through LDS, each wave 32 rows:
//     four tiles at a time are loaded by the block, turned into operands once and written
//     to one of two buffers, the next four being on their way meanwhile.  One wave's 32
//     rows are the columns of 32 x 32 products (32 keys, or 32 columns of v, by 32 rows);
//     with 64 rows or fewer two waves share a row group and take the tile pairs in turn.
// Only pairs of tiles with drafts, or with fewer tokens than they could hold, look at the
// masks.  Units of one row are joined by a second launch.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nm_attn_units.h"
#include "nm_serve.h"

namespace {

using namespace nmu;

// Units = (range, row group, sequence, key head).
template <int DT, int BITS, int D, int MT>
__global__ __launch_bounds__(nma::kWaves * 64, 2) void tree_kernel(const AttnArgs A, int blocks, int direct)
{
    constexpr int NW = nma::kWaves;
    __shared__ __align__(16) float join[join_bytes(D, MT, NW) / 4];
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
    if (len < 0 || (start >= len && !direct))       // the join looks at the ranges that hold tokens only
        return;
    const int at = start / nma::kTile + 2 * wave, row0 = group * 16 * MT;
    Seen<Drafts, MT> seen;
    seen.load(A, b, len, row0, A.G, threadIdx.x % 16);
    attend<Drafts, DT, BITS, D, MT, NW>(A, pages, h, b, row0, A.G, start, min(start + A.own_chunk, len), A.max_len,
                                        page_of(A, pages, at, A.max_len), page_of(A, pages, at + 1, A.max_len),
                                        direct != 0, ((int64_t)split * A.B + b) * A.Hq + (int64_t)h * A.G, seen, join);
}

// ---- units that share the cache through LDS --------------------------------------

typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;

// Partial results of a row group, in the workspace: lane (g, m) holds of row m the columns
// c = 8 a + 4 g + i of each of the D / 16 in a group (value operands lie that way, see below).
// They are kept in pieces of four, [4 a + i][quarter of the group][g][row of the tile's nr]
// 16 bytes, so that a wave's store (and the load that joins them) is one contiguous piece.
__device__ __forceinline__ int64_t piece_at(int piece, int g, int nr, int m)
{
    return ((int64_t)(piece * 2 + g) * nr + m) * 4;
}

template <int DT, int BITS, int D>
__global__ __launch_bounds__(nms::kTreeWaves * 64, D == 256 ? 1 : 2) void shared_kernel(const AttnArgs A, int units,
                                                                                       int groups_w, int direct)
{
    constexpr int NW = nms::kTreeWaves;
    using S = Stage<DT, BITS, D, NW>;
    using C = typename S::C;
    constexpr int NT = S::kTiles, kPer = D / 16, kSteps = D / 16, kCols = D / 32;
    constexpr float kBelow = Weights<DT, 1, 2>::kBelow, kRoom = Weights<DT, 1, 2>::kRoom;
    static_assert(NT == NW, "a wave loads a tile");
    __shared__ __align__(1024) uint8_t lds[2 * S::kBytes];
    __shared__ int count[2][NT];
    const int lane = threadIdx.x % 64, m = lane % 32, g = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    // Row groups of one range lie on one XCD (blocks go round the eight), one after the other.
    const unsigned block = flat_block(), turn = block / 8;
    const unsigned unit = turn / A.own_groups * 8 + block % 8;
    if (unit >= (unsigned)units)
        return;
    const int group = turn % A.own_groups;
    const int h = unit % A.heads, b = unit / A.heads % A.B, split = unit / A.heads / A.B;
    const int start = split * A.own_chunk;
    const int32_t* pages = A.page_table + (int64_t)b * A.table_stride;
    const int len = __builtin_amdgcn_readfirstlane(min(A.lens[b], A.max_len));
    if (len < 0 || (start >= len && !direct))       // the join looks at the ranges that hold tokens only
        return;
    const int end = min(start + A.own_chunk, len), R = A.G;

    // groups_w row groups in the block's waves; with one or two, two waves have the same rows and a
    // pair of tiles of every four each (share), of one, two waves only load.
    const int share = wave / groups_w, shares = groups_w == 4 ? 1 : 2;
    const int row0 = (group * groups_w + wave % groups_w) * 32;
    const bool busy = row0 < R && share < shares;
    const int r = min(row0 + m, R - 1);

    u32x4 q[kSteps];
    {
        const uint16_t* row = A.q + Drafts::q_at(A, h, b, r, D);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            q[s] = (*reinterpret_cast<const u32x4*>(row + C::column(s / 2, s % 2 * 2 + g)) & A.q_and) ^ A.q_xor;
    }
    const int first_draft = len - A.drafts;
    const uint64_t bits = A.visible[(int64_t)b * A.drafts + r / A.heads_g];

    f32x16 acc[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[c][i] = 0.0f;
    float mx = NM_NEG_INF, sum = 0.0f;

    // A pair's score rows: row 16 x + 8 y + 4 z + c is token 8 x + 4 z + c of its tile y, so that the
    // lane's scores 8 x .. 8 x + 7 are tokens 4 (2 x + g) .. + 3 of both tiles: the k indices of the
    // value operands as they are staged.  Keys of odd tiles are staged 8 lanes along (banks).
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int tile = m / 8 % 2, token = m / 16 * 8 + m % 8;
    const uint32_t k_at = base + tile * S::kTileBytes + g * 256 + (token ^ 8 * tile) * 16;
    const uint32_t v_at = base + NT * S::kTileBytes + m / 16 * 1024 + g * 256 + m % 16 * 16;

    // Scores of pair `pair` of the buffer at `buf`, weights from them, and the weighted values.
    const auto attend_pair = [&](uint32_t buf, int pair, auto masked, const int (&n)[2], int first) {
        f32x16 s;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
            s = mfma32<DT>(*(lds_u32x4*)(uintptr_t)(k_at + buf + pair * 2 * S::kTileBytes + c * 512), q[c], s);
        const auto sees4 = [&](int x, int y) {          // whether the row sees its tokens of scores 8 x + 4 y ..
            const int in = 8 * x + 4 * g;
            const int t = first + y * nma::kTile + in, draft = t - first_draft, before = min(max(-draft, 0), 4);
            const uint32_t held = (1u << min(max(n[y] - in, 0), 4)) - 1u;
            return ((uint32_t)((bits >> (max(draft, 0) & 63)) << before) | ((1u << before) - 1u)) & held;
        };
        if constexpr (masked()) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[i] = sees4(i / 8, i / 4 % 2) >> i % 4 & 1 ? s[i] : NM_NEG_INF;
        }
        float top = NM_NEG_INF;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            top = fmaxf(top, s[i]);
        top *= A.scale;
        if (__any(top > mx + kRoom)) {
            top = halves_max(top);
            top = top > mx + kRoom ? top - kBelow : mx;
            const float f = mx == top ? 1.0f : __builtin_amdgcn_exp2f(mx - top);
            sum *= f;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                acc[c] *= f;
            mx = top;
        }
        const float ref = mx == NM_NEG_INF ? 0.0f : mx;
        // A weight is the sum of two operands, its rounding and the rest (nm_attn_units.h, Weights).
        u32x4 p[2], rest[2];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], A.scale, -ref));
            const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i + 1], A.scale, -ref));
            sum += w0 + w1;
            const uint32_t w = pack2<DT>(w0, w1);
            p[i / 8][i % 8 / 2] = w;
            rest[i / 8][i % 8 / 2] = left_out<DT>(w, w0, w1);
        }
        const auto value = [&](int x, int c) {
            return *(lds_u32x4*)(uintptr_t)(v_at + buf + (pair * kPer + 2 * c) * 1024 + x * 512);
        };
        if constexpr (masked()) {
            // 0 * NaN must not reach a row that does not see the token: value operands with
            // infinities or NaN are taken token by token, rows that do not see it keep their sums.
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const u32x4 v = value(x, c);
                    float odd = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        odd = dot2<DT>(v[i], 0u, odd);
                    if (!__any(odd != 0.0f)) {
                        acc[c] = mfma32<DT>(v, rest[x], mfma32<DT>(v, p[x], acc[c]));
                        continue;
                    }
#pragma unroll 1
                    for (int k = 0; k < 16; ++k) {                  // k index (k / 8, k % 8)
                        const uint32_t keep = k / 8 == g ? (k % 2 ? 0xFFFF0000u : 0xFFFFu) : 0u;
                        u32x4 one;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            one[i] = i == k % 8 / 2 ? v[i] & keep : 0u;
                        const int y = k / 4 % 2, in = 8 * x + 4 * (k / 8) + k % 4;
                        const int t = first + y * nma::kTile + in, draft = t - first_draft;
                        const bool sees = (draft < 0) | (int)((bits >> (max(draft, 0) & 63)) & 1);
                        const f32x16 with = mfma32<DT>(one, rest[x], mfma32<DT>(one, p[x], acc[c]));
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[c][i] = sees ? with[i] : acc[c][i];
                    }
                }
        } else {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const u32x4 v = value(x, c);
                    acc[c] = mfma32<DT>(v, rest[x], mfma32<DT>(v, p[x], acc[c]));
                }
        }
    };

    S stage;
    int at = start / nma::kTile + wave;
    const int steps = (end - start + nma::kStaged - 1) / nma::kStaged;
    stage.load(A, tile_ref(A, page_of(A, pages, at, end), at, end, h), 0, lane);
    int page = page_of(A, pages, at + NT, end);
    const auto put = [&](int which) {
        stage.put(lds + which * S::kBytes, wave, 0, lane, true);
        if (lane == 0)
            count[which][wave] = stage.n;
    };
    // The four tiles after those of step i begin their way.
    const auto fetch = [&](int i) {
        if (i + 1 >= steps)
            return;
        at += NT;
        stage.load(A, tile_ref(A, page, at, end, h), 0, lane);
        page = page_of(A, pages, at + NT, end);
    };
    const auto arrived = [&](int i) {
        if (i + 1 < steps)
            put((i + 1) & 1);                       // that buffer's readers passed the barrier before this step
        __syncthreads();
    };
    const auto counted = [&](int i, int pair, int (&n)[2]) {
        n[0] = __builtin_amdgcn_readfirstlane(count[i & 1][2 * pair]);
        n[1] = __builtin_amdgcn_readfirstlane(count[i & 1][2 * pair + 1]);
    };
    const int pair0 = share, pairs = NT / 2 / shares;
    put(0);
    __syncthreads();
    for (int i = 0; i < steps;) {
        // whole pairs, then, where there are others, with their masks
        for (; i < steps; ++i) {
            int n[NT / 2][2];
            bool whole = start + (i + 1) * nma::kStaged <= first_draft;
#pragma unroll
            for (int pair = 0; pair < NT / 2; ++pair) {
                counted(i, pair, n[pair]);
                whole = whole && n[pair][0] == nma::kTile && n[pair][1] == nma::kTile;
            }
            if (!whole)
                break;
            fetch(i);
            if (busy) {
                const uint32_t buf = (i & 1) * S::kBytes;
                attend_pair(buf, pair0, std::false_type(), n[0], 0);
                if (pairs == 2)
                    attend_pair(buf, 1, std::false_type(), n[0], 0);
            }
            arrived(i);
        }
        if (i < steps) {
            fetch(i);
            if (busy)
#pragma unroll 1
                for (int pair = pair0; pair < pair0 + pairs; ++pair) {
                    int n[2];
                    counted(i, pair, n);
                    attend_pair((i & 1) * S::kBytes, pair, std::true_type(), n,
                                start + i * nma::kStaged + pair * 2 * nma::kTile);
                }
            arrived(i);
            ++i;
        }
    }
    sum = halves_sum(sum);

    // Two waves of the same rows are joined through LDS, lane to lane.
    if (shares == 2) {
        float* const box = reinterpret_cast<float*>(lds) + wave % groups_w * (16 * kCols + 2) * 64 + lane;
        if (share == 1) {
            box[16 * kCols * 64] = mx;
            box[(16 * kCols + 1) * 64] = sum;
#pragma unroll
            for (int i = 0; i < 16 * kCols; ++i)
                box[i * 64] = acc[i / 16][i % 16];
        }
        __syncthreads();
        if (share == 0) {
            const float om = box[16 * kCols * 64], os = box[(16 * kCols + 1) * 64];
            const float top = fmaxf(mx, om), ref = top == NM_NEG_INF ? 0.0f : top;
            const float f0 = __builtin_amdgcn_exp2f(mx - ref), f1 = __builtin_amdgcn_exp2f(om - ref);
            sum = sum * f0 + os * f1;
            mx = top;
#pragma unroll
            for (int i = 0; i < 16 * kCols; ++i)
                acc[i / 16][i % 16] = acc[i / 16][i % 16] * f0 + box[i * 64] * f1;
        }
    }
    if (share != 0 || row0 + m >= R)
        return;
    // Value operand rows 16 z + c of tile `t` of columns are column 2 t + z of group c (of D / 16 columns):
    // the lane holds column j of group 8 a + 4 g + i in acc[j / 2][8 (j % 2) + 4 a + i].
    if (direct) {
        const float f = sum > 0.0f || sum != sum ? A.o_scale / sum : 0.0f;
        const int64_t row = Drafts::out_row(A, h, b, r);
        uint16_t* o = A.o + row * D + 4 * g * kPer;
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int j = 0; j < kPer; j += 4) {
                const int i = e / 4 * 4 + e % 4;
                *reinterpret_cast<u32x2*>(o + (e / 4 * 8 + e % 4) * kPer + j) =
                    u32x2{pack2<DT>(acc[j / 2][i] * f, acc[j / 2][i + 8] * f),
                          pack2<DT>(acc[j / 2 + 1][i] * f, acc[j / 2 + 1][i + 8] * f)};
            }
        if (A.lse && g == 0)
            A.lse[row] = (mx + __builtin_amdgcn_logf(sum)) * kLn2;
        return;
    }
    const int64_t part = ((int64_t)split * A.B + b) * A.Hq + (int64_t)h * R + row0;
    const int nr = min(32, R - row0);
    float* o = A.part_o + part * D;
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int j = 0; j < kPer; j += 4)
            *reinterpret_cast<f32x4*>(o + piece_at(e * (kPer / 4) + j / 4, g, nr, m)) =
                f32x4{acc[j / 2][e], acc[j / 2][e + 8], acc[j / 2 + 1][e], acc[j / 2 + 1][e + 8]};
    if (g == 0)
        A.part_ml[part + m] = f32x2{mx, sum};
}

// Joins the ranges of 32 rows of one sequence and key head: a block takes one piece of them, a
// lane (g, m) row m as in the partial results.  NW waves share the ranges, each keeps a reference
// and sums of its own, and they meet in LDS.
template <int DT, int D, int NW>
__global__ __launch_bounds__(NW * 64) void shared_join_kernel(const AttnArgs A, int blocks)
{
    constexpr int kBatch = 4, kPer = D / 16, kPieces = D / 8;
    __shared__ float tops[NW][64], sums[NW][64];
    __shared__ f32x4 box[NW][64];
    const int lane = threadIdx.x % 64, m = lane % 32, g = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const unsigned block = flat_block();
    if (block >= (unsigned)blocks)
        return;
    const int R = A.G, tiles = (R + 31) / 32;
    const int piece = block % kPieces, tile = block / kPieces % tiles;
    const int h = block / kPieces / tiles % A.heads, b = block / kPieces / tiles / A.heads;
    const int len = __builtin_amdgcn_readfirstlane(min(A.lens[b], A.max_len));
    if (len < 0)
        return;
    const int parts = (len + A.own_chunk - 1) / A.own_chunk, row0 = tile * 32, nr = min(32, R - row0);
    const int row = min(m, nr - 1);
    const int64_t first = (int64_t)b * A.Hq + (int64_t)h * R + row0, step = (int64_t)A.B * A.Hq;
    float mx = NM_NEG_INF, sum = 0.0f;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = wave; i < parts; i += kBatch * NW) {
        f32x2 x[kBatch];
        f32x4 o[kBatch];
        float top = mx;
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            const int at = i + c * NW;
            x[c] = f32x2{NM_NEG_INF, 0.0f};
            o[c] = acc * 0.0f;
            if (at < parts) {
                const int64_t part = first + at * step;
                x[c] = A.part_ml[part + row];
                o[c] = *reinterpret_cast<const f32x4*>(A.part_o + part * D + piece_at(piece, g, nr, row));
            }
            top = fmaxf(top, x[c].x);
        }
        const float ref = top == NM_NEG_INF ? 0.0f : top, f = __builtin_amdgcn_exp2f(mx - ref);
        mx = top;
        sum *= f;
        acc *= f;
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
            if (i + c * NW < parts) {
                const float w = __builtin_amdgcn_exp2f(x[c].x - ref);
                sum += x[c].y * w;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[e] += o[c][e] * w;
            }
    }
    tops[wave][lane] = mx;
    sums[wave][lane] = sum;
    box[wave][lane] = acc;
    __syncthreads();
    if (wave > 0 || m >= nr)
        return;
#pragma unroll
    for (int w = 1; w < NW; ++w)
        mx = fmaxf(mx, tops[w][lane]);
    const float ref = mx == NM_NEG_INF ? 0.0f : mx;
    sum = 0.0f;
    acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float f = __builtin_amdgcn_exp2f(tops[w][lane] - ref);
        sum += sums[w][lane] * f;
        acc += box[w][lane] * f;
    }
    acc *= sum > 0.0f || sum != sum ? A.o_scale / sum : 0.0f;
    const int64_t out = Drafts::out_row(A, h, b, row0 + m);
    const int e = piece / (kPer / 4), column = (e / 4 * 8 + 4 * g + e % 4) * kPer + piece % (kPer / 4) * 4;
    *reinterpret_cast<u32x2*>(A.o + out * D + column) = u32x2{pack2<DT>(acc[0], acc[1]), pack2<DT>(acc[2], acc[3])};
    if (A.lse && g == 0 && piece == 0)
        A.lse[out] = (mx + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <int DT, int D, int NW>
__global__ __launch_bounds__(NW * 64) void tree_join_kernel(const AttnArgs A)
{
    combine<Drafts, DT, D, NW>(A);
}

template <int DT, int BITS, int D>
int launch(const nms::TreePlan& P, const AttnArgs& A, hipStream_t s)
{
    const int64_t units = P.splits * A.B * (int64_t)A.heads;
    const int64_t blocks = P.shared ? nma::ceil_div(units, 8) * 8 * P.groups : units * P.groups;
    const int64_t join = P.shared ? (int64_t)A.B * A.heads * nma::ceil_div(A.G, 32) * (D / 8)
                                  : nma::ceil_div((int64_t)A.B * A.G, 16) * A.heads * (D / 16);
    if (blocks > INT32_MAX || join > INT32_MAX)
        return NM_ERR_BAD_SHAPE;
    const int direct = P.direct ? 1 : 0;
    constexpr int kThreads = nms::kTreeWaves * 64;
    (void)hipGetLastError();
    if (P.shared) {
        hipLaunchKernelGGL((shared_kernel<DT, BITS, D>), flat_grid(blocks), dim3(kThreads), 0, s, A, (int)units, P.waves,
                           direct);
        if (!direct)
            hipLaunchKernelGGL((shared_join_kernel<DT, D, 4>), flat_grid(join), dim3(256), 0, s, A, (int)join);
        return hipGetLastError() == hipSuccess ? NM_OK : NM_ERR_HIP;
    }
    if constexpr (D != 256) {
        if (P.mt == 1)
            hipLaunchKernelGGL((tree_kernel<DT, BITS, D, 1>), flat_grid(blocks), dim3(kThreads), 0, s, A, (int)blocks, direct);
        else
            hipLaunchKernelGGL((tree_kernel<DT, BITS, D, 2>), flat_grid(blocks), dim3(kThreads), 0, s, A, (int)blocks, direct);
        // Few tiles of rows have many parts each: more waves share them then.
        if (!direct && join < 2 * nma::kCus && P.splits > 16)
            hipLaunchKernelGGL((tree_join_kernel<DT, D, 16>), flat_grid(join), dim3(1024), 0, s, A);
        else if (!direct)
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
