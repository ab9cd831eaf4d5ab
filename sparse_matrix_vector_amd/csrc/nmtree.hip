// nmtree.hip -- nm_attn_tree: attention of drafted tokens over the paged cache.
//
// A sequence's rows are its drafts' query heads of one key head, N G of them, and a
// unit takes up to 128 of them over a range of its tokens, so that the cache comes from
// memory once for all drafts.  Two forms:
//   up to 32 rows of up to 128 columns, or more where there is little work (tree_shared in
//     nm_serve.h): as in nm_attn_decode (nm_attn_units.h), each wave reads the cache itself,
//     straight into operands, and takes pairs of tiles in turn;
//   else (shared_kernel) a block of four waves shares it through LDS, each wave 32 rows:
//     four tiles at a time are loaded by the block, turned into operands once and written
//     to one of two buffers, the next four being on their way meanwhile.  One wave's 32
//     rows are the columns of 32 x 32 products (32 keys, or 32 columns of v, by 32 rows).
//     A pair of tiles is worked on in three rounds, as in nmprompt.hip: its scores beside
//     the weights of the pair before, its sums beside the scores of the next.  With 64 rows
//     or fewer two waves share a row group and take a pair of every four tiles each.
// Many rows are bound by the products (one sequence of 131071 tokens, 64 drafts of 64 heads on 8
// of 128 columns, MX4: 404 us, 680 TFLOP/s of the formula, half as much again with the weights'
// second operand), few by the cache's way through LDS and the barriers (32 sequences of 12 drafts, 40
// heads, up to 2048 tokens, 16-bit: 40.6 us, 3.6 TB/s; 16 of 24, 32 heads, up to 8192, MX8: 100).
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

// One wave's tile on its way to LDS.  16-bit rows go there directly (global_load_lds, 1 KB an
// instruction), as they lie in the cache; codes through registers, as operands.  In LDS:
//   keys    [tile][column piece of 8, token] 16 bytes; the tokens m of odd tiles are stored at m ^ 8 (banks)
//   values  16-bit: [tile][column j of a group][quarter][group] 8 bytes (four tokens);
//           codes: [pair][column j][quarter][group] 16 bytes (four tokens of each tile)
template <int DT, int BITS, int D>
struct Way {
    using S = Stage<DT, BITS, D, nms::kTreeWaves>;
    static constexpr bool kCodes = BITS != 16;
    static constexpr int kBytes = nms::kTreeWaves * S::kTileBytes;        // keys, or values, of four tiles
    S stage;

    static __device__ __forceinline__ void direct(uint32_t lds, const uint8_t* tile, int lane, int turned)
    {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(
                             __builtin_amdgcn_readfirstlane(lds + i * 1024)),
                         "v"((lane ^ turned) * 16), "s"(tile + i * 1024)
                         : "memory");
    }
    __device__ __forceinline__ void load_k(const AttnArgs& A, const TileRef& t, uint32_t lds, int wave, int lane)
    {
        if constexpr (kCodes)
            stage.load_k(A, t, 0, lane);
        else
            direct(lds + wave * S::kTileBytes, A.k + t.tile * nma::tile_bytes(D, BITS), lane, wave % 2 * 8);
    }
    __device__ __forceinline__ void load_v(const AttnArgs& A, const TileRef& t, uint32_t lds, int wave, int lane)
    {
        if constexpr (kCodes)
            stage.load_v(A, t, 0, lane);
        else
            direct(lds + wave * S::kTileBytes, A.v + t.tile * nma::tile_bytes(D, BITS), lane, 0);
    }
    __device__ __forceinline__ void put_k(uint8_t* buf, int wave, int lane) const { stage.put_k(buf, wave, 0, lane, true); }
    __device__ __forceinline__ void put_v(uint8_t* buf, int wave, int lane) const { stage.put_v(buf, wave, 0, lane); }
};

template <int DT, int BITS, int D, int SHARES>
__global__ __launch_bounds__(nms::kTreeWaves * 64, D == 256 ? 1 : 2) void shared_kernel(const AttnArgs A, int units,
                                                                                       int groups_w, int direct)
{
    constexpr int NW = nms::kTreeWaves;
    using W = Way<DT, BITS, D>;
    using C = Cache<DT, BITS, D>;
    constexpr int kTileBytes = W::S::kTileBytes, kBytes = W::kBytes;
    constexpr int NT = NW, kPer = D / 16, kSteps = D / 16, kCols = D / 32, kQuarter = kSteps / 4;
    constexpr float kBelow = Weights<DT, 1, 2>::kBelow, kRoom = Weights<DT, 1, 2>::kRoom;
    static_assert(W::S::kTiles == NT, "a wave loads a tile");
    __shared__ __align__(1024) uint8_t lds[4 * kBytes];         // two buffers of keys, two of values
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
    const int end = min(start + A.own_chunk, len), R = A.G, first_draft = len - A.drafts;

    // groups_w row groups in the block's waves; with one or two, two waves have the same rows and a
    // pair of tiles of every four each (share), of one, two waves only load.
    const int share = SHARES == 2 ? wave / groups_w : 0;
    const int row0 = (group * groups_w + wave % groups_w) * 32;
    const bool busy = row0 < R && share < SHARES;
    const int r = min(row0 + m, R - 1);

    // Four tiles (a stage) by their pages: which are there, and where the wave's own is.
    struct Pages {
        int page[NT];
    };
    const int tile0 = start / nma::kTile;
    const auto pages_of = [&](int stage) {
        Pages x;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            x.page[j] = page_of(A, pages, tile0 + stage * NT + j, end);
        return x;
    };
    const auto tokens = [&](const Pages& x, int stage, int j) {         // that count in tile j
        const bool inside = (unsigned)x.page[j] < (unsigned)A.n_pages;
        return inside ? min(max(end - (tile0 + stage * NT + j) * nma::kTile, 0), nma::kTile) : 0;
    };
    const auto own_tile = [&](const Pages& x, int stage) {
        const int page = wave == 0 ? x.page[0] : wave == 1 ? x.page[1] : wave == 2 ? x.page[2] : x.page[3];
        return tile_ref(A, page, tile0 + stage * NT + wave, end, h);
    };
    const auto is_whole = [&](const Pages& x, int stage) {
        bool whole = start + (stage + 1) * nma::kStaged <= min(end, first_draft);
#pragma unroll
        for (int j = 0; j < NT; ++j)
            whole = whole && (unsigned)x.page[j] < (unsigned)A.n_pages;
        return whole;
    };

    const uint32_t k_buf = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds, v_buf = k_buf + 2 * kBytes;
    W way;
    const int steps = (end - start + nma::kStaged - 1) / nma::kStaged;      // stages
    // of stages t .. t + 3 in round t (begin)
    Pages x2 = pages_of(0), x3 = pages_of(1), x0 = x2, x1 = x2;
    way.load_k(A, own_tile(x2, 0), k_buf, wave, lane);

    u32x4 q[kSteps];
    {
        const uint16_t* row = A.q + Drafts::q_at(A, h, b, r, D);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            q[s] = (*reinterpret_cast<const u32x4*>(row + C::column(s / 2, s % 2 * 2 + g)) & A.q_and) ^ A.q_xor;
    }
    const uint64_t bits = A.visible[(int64_t)b * A.drafts + r / A.heads_g];

    f32x16 acc[kCols], s, w;                                    // s: scores of the coming pair, w: weights of the one before
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        s[i] = w[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
            acc[c][i] = 0.0f;
    }
    float mx = NM_NEG_INF, sum = 0.0f;

    // A pair's score rows: row 16 x + 8 y + 4 z + c is token 8 x + 4 z + c of its tile y, so that the
    // lane's scores 8 x .. 8 x + 7 are tokens 4 (2 x + g) .. + 3 of both tiles: the k indices of the
    // value operands as they are staged.  Value operand rows 16 z + i of tile c of columns are column
    // 2 c + z of group i (of D / 16 columns).  Keys of stage t + 1, values of stage t:
    const int tile = m / 8 % 2, token = m / 16 * 8 + m % 8;
    uint32_t k_at = k_buf + tile * kTileBytes + g * 256 + (token ^ 8 * tile) * 16;
    uint32_t v_at = v_buf + kBytes + (BITS == 16 ? m / 16 * 512 + g * 128 + m % 16 * 8
                                                 : m / 16 * 1024 + g * 256 + m % 16 * 16);
    const auto key = [&](int c, int part) {
        return *(lds_u32x4*)(uintptr_t)(k_at + part * 2 * kTileBytes + c * 512);
    };
    const auto value = [&](int x, int c, int part) {
        if constexpr (BITS == 16) {
            typedef __attribute__((address_space(3))) const u32x2 lds_u32x2;
            const uint32_t at = v_at + part * 2 * kTileBytes + c * 1024 + x * 256;
            const u32x2 lo = *(lds_u32x2*)(uintptr_t)at, hi = *(lds_u32x2*)(uintptr_t)(at + kTileBytes);
            return u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
            return *(lds_u32x4*)(uintptr_t)(v_at + (part * kPer + 2 * c) * 1024 + x * 512);
        }
    };
    // Room for the scores s: raises the reference of rows that need it.
    const auto make_room = [&]() {
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
            w *= f;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                acc[c] *= f;
            mx = top;
        }
    };
    // s = weights of its scores i .. i + n - 1, added to the sum
    const auto weigh = [&](int i, int n) {
        const float ref = mx == NM_NEG_INF ? 0.0f : mx;
#pragma unroll
        for (int j = i; j < i + n; ++j) {
            s[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], A.scale, -ref));
            sum += s[j];
        }
    };
    // Weights 8 x .. 8 x + 7 as operands: each is the sum of two, its rounding and the rest
    // (nm_attn_units.h, Weights).
    const auto pack = [&](const f32x16& w, int x, u32x4& p, u32x4& rest) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[i] = pack2<DT>(w[8 * x + 2 * i], w[8 * x + 2 * i + 1]);
            rest[i] = left_out<DT>(p[i], w[8 * x + 2 * i], w[8 * x + 2 * i + 1]);
        }
    };
    // Whole tiles, a pair of every stage for each of two waves: the next pair's scores beside this one's weights.
    const auto hot_share = [&]() {
        u32x4 ka[2][kQuarter], va[2][kCols], p[2], rest[2];
#pragma unroll
        for (int c = 0; c < kQuarter; ++c)
            ka[0][c] = key(c, share);
        make_room();
        f32x16 next;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            next[i] = 0.0f;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x < 3)
#pragma unroll
                for (int c = 0; c < kQuarter; ++c)
                    ka[(x + 1) % 2][c] = key((x + 1) * kQuarter + c, share);
            if (x == 1)
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    va[0][c] = value(0, c, share);
            weigh(4 * x, 4);
#pragma unroll
            for (int c = 0; c < kQuarter; ++c)
                next = mfma32<DT>(ka[x % 2][c], q[x * kQuarter + c], next);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c)
            va[1][c] = value(1, c, share);
        pack(s, 0, p[0], rest[0]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                acc[c] = mfma32<DT>(va[x][c], p[x], acc[c]);
            if (x == 0)
                pack(s, 1, p[1], rest[1]);
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                acc[c] = mfma32<DT>(va[x][c], rest[x], acc[c]);
        }
        s = next;
    };
    // Whole tiles, all pairs: scores of the next (keys of stage t + 1), weights, sums of the one before
    // (values of stage t), all independent of each other.
    const auto hot = [&](auto part_) {
        constexpr int part = part_();
        u32x4 ka[2][kQuarter], va[2][kQuarter], p[2], rest[2];
        const auto read = [&](int x) {
#pragma unroll
            for (int c = 0; c < kQuarter; ++c) {
                const int at = x * kQuarter + c;
                ka[x % 2][c] = key(at, part);
                va[x % 2][c] = value(at / kCols, at % kCols, part);
            }
        };
        read(0);
        make_room();
        pack(w, 0, p[0], rest[0]);
        f32x16 next;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            next[i] = 0.0f;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x < 3)
                read(x + 1);
            if (x == 1)
                pack(w, 1, p[1], rest[1]);
#pragma unroll
            for (int c = 0; c < kQuarter; ++c) {
                const int at = x * kQuarter + c;
                next = mfma32<DT>(ka[x % 2][c], q[at], next);
                acc[at % kCols] = mfma32<DT>(va[x % 2][c], p[at / kCols], acc[at % kCols]);
            }
            weigh(4 * x, 4);
#pragma unroll
            for (int c = 0; c < kQuarter; ++c) {
                const int at = x * kQuarter + c;
                acc[at % kCols] = mfma32<DT>(va[x % 2][c], rest[at / kCols], acc[at % kCols]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        w = s;
        s = next;
    };

    // Whether the row sees its tokens of scores 8 x + 4 y .. + 3 of a pair: bits 0 .. 3.
    const auto sees4 = [&](int x, int y, int n, int first) {
        const int in = 8 * x + 4 * g;
        const int draft = first + y * nma::kTile + in - first_draft, before = min(max(-draft, 0), 4);
        const uint32_t held = (1u << min(max(n - in, 0), 4)) - 1u;
        return ((uint32_t)((bits >> (max(draft, 0) & 63)) << before) | ((1u << before) - 1u)) & held;
    };
    const auto mask = [&](int n0, int n1, int first) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[i] = sees4(i / 8, i / 4 % 2, i / 4 % 2 ? n1 : n0, first) >> i % 4 & 1 ? s[i] : NM_NEG_INF;
    };
    // The values of a pair, of whose tiles n[.] tokens count, times the weights x.
    const auto add = [&](const f32x16& weights, int part, int n0, int n1, int first) {
        u32x4 p[2], rest[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            pack(weights, x, p[x], rest[x]);
        // 0 * NaN must not reach a row that does not see the token: value operands with
        // infinities or NaN are taken token by token, rows that do not see it keep their sums.
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const u32x4 v = value(x, c, part);
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
                    const int draft = first + y * nma::kTile + in - first_draft;
                    const bool sees = ((draft < 0) | (int)((bits >> (max(draft, 0) & 63)) & 1)) & (in < (y ? n1 : n0));
                    const f32x16 with = mfma32<DT>(one, rest[x], mfma32<DT>(one, p[x], acc[c]));
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[c][i] = sees ? with[i] : acc[c][i];
                }
            }
    };
    const auto scores = [&](int part) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
            s = mfma32<DT>(key(c, part), q[c], s);
    };
    // The same rounds with all conditions and masks.  (Arrays that are indexed as they run would go to LDS here, and
    // finding their place there takes a read of the launch's packet from host memory, some 10 us a block.)
    const auto cold_share = [&](int t) {
        if (t >= 0) {
            const int n0 = share ? tokens(x0, t, 2) : tokens(x0, t, 0), n1 = share ? tokens(x0, t, 3) : tokens(x0, t, 1);
            const int first = start + t * nma::kStaged + share * 2 * nma::kTile;
            mask(n0, n1, first);
            make_room();
            weigh(0, 16);
            add(s, share, n0, n1, first);
        }
        if (t + 1 < steps)
            scores(share);
    };
    const auto cold = [&](int t, int part) {
        // pair 2 t + 1 + part: of stage t, or (part 1) of stage t + 1
        const int stage = t + part, side = 1 - part;
        if (stage >= 0 && stage < steps) {
            const int n0 = part == 0 ? tokens(x0, t, 2) : tokens(x1, t + 1, 0);
            const int n1 = part == 0 ? tokens(x0, t, 3) : tokens(x1, t + 1, 1);
            mask(n0, n1, start + stage * nma::kStaged + side * 2 * nma::kTile);
            make_room();
        }
        if (t >= 0) {
            const int n0 = part == 0 ? tokens(x0, t, 0) : tokens(x0, t, 2), n1 = part == 0 ? tokens(x0, t, 1) : tokens(x0, t, 3);
            add(w, part, n0, n1, start + t * nma::kStaged + part * 2 * nma::kTile);
        }
        if (stage >= 0 && stage < steps) {
            weigh(0, 16);
            w = s;
        }
        if (t + 1 < steps)
            scores(part);
    };

    // Round t: keys of stage t + 1 and values of stage t lie in LDS, keys of t + 2 and values of t + 1 begin their
    // way.  (Codes without conditions: behind the last stage they are page 0's, which nobody looks at.  With
    // branches between the products and the loop's end the compiler keeps the sums twice and spills.  Codes
    // loaded a whole round ahead, at the end of the one before or through LDS, take as long: 102 to 105 us for 100.)
    const auto begin = [&](int t) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        x0 = x1;
        x1 = x2;
        x2 = x3;
        x3 = pages_of(t + 3);
        if (W::kCodes || t + 2 < steps)
            way.load_k(A, own_tile(x2, t + 2), k_buf + (t & 1) * kBytes, wave, lane);
        if (W::kCodes || t + 1 < steps)
            way.load_v(A, own_tile(x1, t + 1), v_buf + (~t & 1) * kBytes, wave, lane);
    };
    const auto finish = [&](int t) {
        if constexpr (W::kCodes) {
            way.put_k(lds + (t & 1) * kBytes, wave, lane);
            way.put_v(lds + (2 + (~t & 1)) * kBytes, wave, lane);
        }
        k_at ^= kBytes;
        v_at ^= kBytes;
    };
    if constexpr (W::kCodes)
        way.put_k(lds, wave, lane);
    if (!busy)                                      // a wave without rows only loads
        for (int t = -1; t < steps; ++t) {
            begin(t);
            finish(t);
        }
    for (int t = busy ? -1 : steps; t < steps;) {
        begin(t);
        if constexpr (SHARES == 2) {
            cold_share(t);
        } else {
#pragma unroll 1
            for (int part = 0; part < 2; ++part)
                cold(t, part);
        }
        finish(t);
        ++t;
        if constexpr (SHARES == 2) {
            for (; t + 1 < steps && is_whole(x1, t); ++t) {
                begin(t);
                hot_share();
                finish(t);
            }
        } else {
            for (; t + 1 < steps && is_whole(x1, t) && is_whole(x2, t + 1); ++t) {
                begin(t);
                hot(std::integral_constant<int, 0>());
                hot(std::integral_constant<int, 1>());
                finish(t);
            }
        }
    }
    sum = halves_sum(sum);

    // Two waves of the same rows are joined through LDS, lane to lane.
    if constexpr (SHARES == 2) {
        __syncthreads();                            // the last readers of what lay there
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
    // The lane holds column j of group 8 a + 4 g + i in acc[j / 2][8 (j % 2) + 4 a + i].
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

// Joins the ranges of 32 rows of one sequence and key head: NW waves take one piece of them, a
// lane (g, m) row m as in the partial results.  They share the ranges, each keeps a reference and
// sums of its own, and they meet in LDS.
template <int DT, int D, int NW>
__global__ __launch_bounds__(256) void shared_join_kernel(const AttnArgs A, int units)
{
    constexpr int kBatch = 4, kPer = D / 16, kPieces = D / 8;
    __shared__ float tops[4][64], sums[4][64];
    __shared__ f32x4 box[4][64];
    const int lane = threadIdx.x % 64, m = lane % 32, g = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), w0 = wave % NW;
    const unsigned unit = flat_block() * (4 / NW) + wave / NW;
    if (unit >= (unsigned)units)
        return;
    const int R = A.G, tiles = (R + 31) / 32;
    const int piece = unit % kPieces, tile = unit / kPieces % tiles;
    const int h = unit / kPieces / tiles % A.heads, b = unit / kPieces / tiles / A.heads;
    const int len = __builtin_amdgcn_readfirstlane(min(A.lens[b], A.max_len));
    if (len < 0)
        return;
    const int parts = (len + A.own_chunk - 1) / A.own_chunk, row0 = tile * 32, nr = min(32, R - row0);
    const int row = min(m, nr - 1);
    const int64_t first = (int64_t)b * A.Hq + (int64_t)h * R + row0, step = (int64_t)A.B * A.Hq;
    float mx = NM_NEG_INF, sum = 0.0f;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = w0; i < parts; i += kBatch * NW) {
        f32x2 x[kBatch];
        f32x4 o[kBatch];
        float top = mx;
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            const int64_t part = first + min(i + c * NW, parts - 1) * step;     // (others are not added)
            x[c] = A.part_ml[part + row];
            o[c] = *reinterpret_cast<const f32x4*>(A.part_o + part * D + piece_at(piece, g, nr, row));
        }
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
            top = i + c * NW < parts ? fmaxf(top, x[c].x) : top;
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
    if constexpr (NW > 1) {
        tops[wave][lane] = mx;
        sums[wave][lane] = sum;
        box[wave][lane] = acc;
        __syncthreads();
        if (w0 > 0)
            return;
#pragma unroll
        for (int w = 1; w < NW; ++w)
            mx = fmaxf(mx, tops[wave + w][lane]);
        const float ref = mx == NM_NEG_INF ? 0.0f : mx;
        sum = 0.0f;
        acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = __builtin_amdgcn_exp2f(tops[wave + w][lane] - ref);
            sum += sums[wave + w][lane] * f;
            acc += box[wave + w][lane] * f;
        }
    }
    if (m >= nr)
        return;
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
    const int direct = P.direct ? 1 : 0;
    constexpr int kThreads = nms::kTreeWaves * 64;
    (void)hipGetLastError();
    if (P.shared) {
        if (P.waves == 4)
            hipLaunchKernelGGL((shared_kernel<DT, BITS, D, 1>), flat_grid(blocks), dim3(kThreads), 0, s, A, (int)units, 4,
                               direct);
        else
            hipLaunchKernelGGL((shared_kernel<DT, BITS, D, 2>), flat_grid(blocks), dim3(kThreads), 0, s, A, (int)units,
                               P.waves, direct);
        // One wave joins up to 8 ranges, four share more.
        if (!direct && P.splits <= 8)
            hipLaunchKernelGGL((shared_join_kernel<DT, D, 1>), flat_grid(nma::ceil_div(join, 4)), dim3(256), 0, s, A,
                               (int)join);
        else if (!direct)
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
