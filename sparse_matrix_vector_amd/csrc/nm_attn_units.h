// nm_attn_units.h -- device code of attention over the paged cache, shared by
// nmattn.hip (one query token a sequence) and nmtree.hip (a tree of drafted
// tokens): a block's work on one unit, and the joining of units.  What a unit
// computes and how it is laid out stands at the head of nmattn.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nm_attn.h"
#include "nm_device.h"

namespace nmu {

using namespace nmd;


constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
#define NM_NEG_INF (-__builtin_inff())

struct AttnArgs {
    const uint16_t* q;
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* k_scale;
    const uint8_t* v_scale;
    const int32_t* prefix_pages;
    const int32_t* page_table;
    const int32_t* lens;
    uint16_t* o;
    float* lse;
    float* part_o;              // [rows][D] partial sums: prefix rows first, own rows behind them
    f32x2* part_ml;             // [rows] (maximum, sum)
    int64_t q_stride, table_stride, own_base;            // own_base: first partial row of the own-token units
    int n_pages, B, Hq, heads, G, page_shift;
    int prefix_len, max_len;
    int prefix_rows, prefix_groups, prefix_splits, prefix_chunk;
    int own_groups, own_splits, own_chunk;
    // Scores are kept in base 2: q . k times `scale` = |scale| log2(e) > 0, the sign
    // (and a scale of zero) being put into q, which is exact.
    float scale;
    uint32_t q_and, q_xor;
    float o_scale;              // 2 where the operands are half the cached values, else 1
    // Trees only, where a sequence's rows are draft * heads_g + head (G, Hq and B * G rows count them all):
    const uint64_t* visible;    // [B][drafts]
    int drafts, heads_g, heads_q;
};

// What a sequence's rows are: query heads of one token (r is head h G + r of row b0), also
// of a whole batch (r is head h G + r % G of row b0 + r / G), or of its drafts.
struct OneToken {
    static constexpr bool kTree = false;
    static __device__ __forceinline__ int64_t q_at(const AttnArgs& A, int h, int b0, int r, int D)
    {
        return (int64_t)(b0 + r / A.G) * A.q_stride + (int64_t)(h * A.G + r % A.G) * D;
    }
    static __device__ __forceinline__ int64_t out_row(const AttnArgs& A, int h, int b, int r)
    {
        return (int64_t)b * A.Hq + (int64_t)h * A.G + r;
    }
};

struct Drafts {
    static constexpr bool kTree = true;
    static __device__ __forceinline__ int64_t q_at(const AttnArgs& A, int h, int b, int r, int D)
    {
        return ((int64_t)b * A.drafts + r / A.heads_g) * A.q_stride + (int64_t)(h * A.heads_g + r % A.heads_g) * D;
    }
    static __device__ __forceinline__ int64_t out_row(const AttnArgs& A, int h, int b, int r)
    {
        return ((int64_t)b * A.drafts + r / A.heads_g) * A.heads_q + h * A.heads_g + r % A.heads_g;
    }
};

// Which of the tokens that count each of a lane's MT rows sees: all of them, or, in a
// tree, those before the drafts (token `first_draft` on) and the drafts of its mask.
template <class P, int MT>
struct Seen {
};

template <int MT>
struct Seen<Drafts, MT> {
    int first_draft;
    uint64_t bits[MT];

    __device__ __forceinline__ void load(const AttnArgs& A, int b, int len, int row0, int R, int m)
    {
        first_draft = len - A.drafts;
#pragma unroll
        for (int g = 0; g < MT; ++g)
            bits[g] = A.visible[(int64_t)b * A.drafts + min(row0 + 16 * g + m, R - 1) / A.heads_g];
    }
    // Bits 0 .. 3: whether row g sees tokens t .. t + 3.  Plain arithmetic: where conditions with
    // || chose the scores to mask, the compiler (of ROCm 7.2) lost one of them in units of two row tiles.
    __device__ __forceinline__ uint32_t four(int g, int t) const
    {
        const int draft = t - first_draft, before = min(max(-draft, 0), 4);
        return (uint32_t)((bits[g] >> (max(draft, 0) & 63)) << before) | ((1u << before) - 1u);
    }
};

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (DT == NM_FP16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

// Maximum / sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48 (one row's quarters).
__device__ __forceinline__ float quarters_max(float v)
{
    u32x2 p = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(f32_bits(v), f32_bits(v), false, false));
    v = fmaxf(bits_f32(p.x), bits_f32(p.y));
    p = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(f32_bits(v), f32_bits(v), false, false));
    return fmaxf(bits_f32(p.x), bits_f32(p.y));
}

__device__ __forceinline__ float quarters_sum(float v)
{
    u32x2 p = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(f32_bits(v), f32_bits(v), false, false));
    v = bits_f32(p.x) + bits_f32(p.y);
    p = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(f32_bits(v), f32_bits(v), false, false));
    return bits_f32(p.x) + bits_f32(p.y);
}

// Two neighbouring codes of a word times a power of two, as two 16-bit floats.
template <int DT, bool HIGH>
__device__ __forceinline__ uint32_t from_fp8(uint32_t w, float f)
{
    if constexpr (DT == NM_FP16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, f, HIGH));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, f, HIGH));
}

template <int DT, int BYTE>
__device__ __forceinline__ uint32_t from_fp4(uint32_t w, float f)
{
    if constexpr (DT == NM_FP16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, BYTE));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, BYTE));
}

// One lane's part of a 16-token tile of keys or values as loaded, and how it
// becomes operands of the cache's dtype.  BITS 16: as it is.  Codes: converted with
// the scale applied, which is exact (nm_attn.h: scale bytes).
template <int DT, int BITS, int D>
struct Cache {
    static constexpr int kCb = nma::k_chunk_bytes(D, BITS);
    static constexpr int kVb = nma::v_chunk_bytes(D, BITS);
    static constexpr int kWords = nma::lane_bytes(D, BITS) / 4;
    static constexpr int kE = kCb * 8 / BITS;          // elements of a chunk
    static constexpr int kBlocks = D / nma::kBlock;    // scales of a token
    static constexpr int kPer = D / 16;                // value columns of a lane

    struct Raw {
        uint32_t w[kWords];
    };

    template <int CB>
    static __device__ __forceinline__ void load(Raw& raw, const uint8_t* tile, int lane)
    {
        typedef uint32_t chunk __attribute__((ext_vector_type(CB / 4)));
#pragma unroll
        for (int c = 0; c < kWords * 4 / CB; ++c) {
            const chunk x = __builtin_nontemporal_load(reinterpret_cast<const chunk*>(tile + c * 64 * CB + lane * CB));
#pragma unroll
            for (int i = 0; i < CB / 4; ++i)
                raw.w[CB / 4 * c + i] = x[i];
        }
    }

    // The scale bytes of the lane's token (keys; kBlocks bytes, up to two words).
    struct KScale {
        uint32_t w[kBlocks > 4 ? 2 : 1];
    };
    static __device__ __forceinline__ void load_k_scale(KScale& s, const uint8_t* tile, int m)
    {
        if constexpr (BITS != 16) {
            if constexpr (kBlocks == 2)
                s.w[0] = *reinterpret_cast<const uint16_t*>(tile + m * 2);
            else if constexpr (kBlocks == 4)
                s.w[0] = *reinterpret_cast<const uint32_t*>(tile + m * 4);
            else {
                const u32x2 x = *reinterpret_cast<const u32x2*>(tile + m * 8);
                s.w[0] = x.x;
                s.w[1] = x.y;
            }
        }
    }

    // The scale bytes of the lane's four tokens in its column group's block (values).
    static __device__ __forceinline__ void load_v_scale(uint32_t& s, const uint8_t* tile, int m, int kg)
    {
        if constexpr (BITS != 16)
            s = *reinterpret_cast<const uint32_t*>(tile + nma::v_scale_offset(4 * kg, m * kPer / nma::kBlock));
    }

    // Key operand of k-step s: columns column(s, kg) .. + 7 of the lane's token.
    static __device__ __forceinline__ int column(int s, int kg) { return s * 8 / kE * 4 * kE + kg * kE + s * 8 % kE; }

    static __device__ __forceinline__ u32x4 k_operand(const Raw& raw, const KScale& sc, int s, int kg)
    {
        if constexpr (BITS == 16) {
            return u32x4{raw.w[4 * s], raw.w[4 * s + 1], raw.w[4 * s + 2], raw.w[4 * s + 3]};
        } else {
            return k_codes(raw.w + s * BITS / 4, sc, s, kg);
        }
    }

    // The same from k-step s's codes (BITS bytes).
    static __device__ __forceinline__ u32x4 k_codes(const uint32_t* w, const KScale& sc, int s, int kg)
    {
        u32x4 out = {0u, 0u, 0u, 0u};
        if constexpr (BITS != 16) {
            // the block of columns c 4E + kg E + ..: the first part is known here, the second by kg
            const int block = s * 8 / kE * (4 * kE / nma::kBlock) + kg * kE / nma::kBlock;
            const uint32_t word = kBlocks > 4 && block >= 4 ? sc.w[kBlocks > 4 ? 1 : 0] : sc.w[0];
            const float f = scale_value((word >> (8 * (block % 4))) & 255u);
            if constexpr (BITS == 8)
                out = u32x4{from_fp8<DT, false>(w[0], f), from_fp8<DT, true>(w[0], f), from_fp8<DT, false>(w[1], f),
                            from_fp8<DT, true>(w[1], f)};
            else
                out = u32x4{from_fp4<DT, 0>(w[0], f), from_fp4<DT, 1>(w[0], f), from_fp4<DT, 2>(w[0], f),
                            from_fp4<DT, 3>(w[0], f)};
        }
        return out;
    }

    // Value operands: out[2 j], out[2 j + 1] = column j of the lane's group, its
    // four tokens.
    static __device__ __forceinline__ void v_operands(uint32_t (&out)[2 * kPer], const Raw& raw, uint32_t sc)
    {
        if constexpr (BITS == 16) {
#pragma unroll
            for (int i = 0; i < 2 * kPer; ++i)
                out[i] = raw.w[i];
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t half[kPer];
                v_codes(half, raw.w + i * kPer * BITS / 16, sc >> (16 * i));
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    out[2 * j + i] = half[j];
            }
        }
    }

    // out[j] = column j of the lane's group, tokens (2 i, 2 i + 1), from the pair's
    // codes (kPer BITS / 4 bytes) and scale bytes (the low two of sc).
    static __device__ __forceinline__ void v_codes(uint32_t (&out)[kPer], const uint32_t* w, uint32_t sc)
    {
        uint32_t pair[2][kPer / 2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float f = scale_value((sc >> (8 * r)) & 255u);
#pragma unroll
            for (int p = 0; p < kPer / 2; ++p) {
                const int at = (r * kPer + 2 * p) * BITS / 8;
                const uint32_t x = w[at / 4];
                if constexpr (BITS == 8)
                    pair[r][p] = at % 4 ? from_fp8<DT, true>(x, f) : from_fp8<DT, false>(x, f);
                else
                    pair[r][p] = at % 4 == 0   ? from_fp4<DT, 0>(x, f)
                                 : at % 4 == 1 ? from_fp4<DT, 1>(x, f)
                                 : at % 4 == 2 ? from_fp4<DT, 2>(x, f)
                                               : from_fp4<DT, 3>(x, f);
            }
        }
        // (column 2p, column 2p + 1) by token -> (token 2i, token 2i + 1) by column
#pragma unroll
        for (int p = 0; p < kPer / 2; ++p) {
            out[2 * p] = __builtin_amdgcn_perm(pair[1][p], pair[0][p], 0x05040100u);
            out[2 * p + 1] = __builtin_amdgcn_perm(pair[1][p], pair[0][p], 0x07060302u);
        }
    }
};

// Everything one wave needs of a step's tile: where it lies and how many of its
// 16 tokens count (a prefix of them).
struct TileRef {
    int64_t tile;
    int n;
    int first;          // its first token
};

// Page number of tile `a` (16-token index within its sequence or prefix, the same
// for the whole wave) of a list that holds `limit` tokens: a scalar load, which
// takes no part in the counts of vector loads outstanding.
__device__ __forceinline__ int page_of(const AttnArgs& A, const int32_t* pages, int a, int limit)
{
    typedef __attribute__((address_space(4))) const int32_t constant_i32;
    return a * nma::kTile < limit ? ((constant_i32*)pages)[a >> (A.page_shift - 4)] : -1;
}

// That tile of key head h, where tokens from `end` on do not count.  A page number
// outside the cache is not followed: its tokens are absent.
__device__ __forceinline__ TileRef tile_ref(const AttnArgs& A, int page, int a, int end, int h)
{
    const bool inside = (unsigned)page < (unsigned)A.n_pages;
    TileRef t;
    t.n = inside ? min(max(end - a * nma::kTile, 0), nma::kTile) : 0;
    t.n = __builtin_amdgcn_readfirstlane(t.n);
    t.first = a * nma::kTile;
    page = __builtin_amdgcn_readfirstlane(inside ? page : 0);
    const int per = 1 << (A.page_shift - 4);
    t.tile = ((int64_t)page * A.heads + h) * per + (a & (per - 1));
    return t;
}

// The lane's row of each of MT row tiles, as right operands of the score product.
template <class P, int DT, int BITS, int D, int MT>
struct Rows {
    static constexpr int kSteps = D / 32;                            // k-steps of the score product
    u32x4 op[MT][kSteps];

    __device__ __forceinline__ void load(const AttnArgs& A, int h, int b0, int row0, int R, int m, int kg)
    {
#pragma unroll
        for (int g = 0; g < MT; ++g) {
            const int r = row0 + 16 * g + m;
            const uint16_t* row = A.q + P::q_at(A, h, b0, r, D);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                op[g][s] = u32x4{0u, 0u, 0u, 0u};
                if (r < R)
                    op[g][s] =
                        (*reinterpret_cast<const u32x4*>(row + Cache<DT, BITS, D>::column(s, kg)) & A.q_and) ^ A.q_xor;
            }
        }
    }
};

// Scores of tokens that do not count: n[u] of tile u's 16 do.
template <int MT, int NT>
__device__ __forceinline__ void mask_scores(f32x4 (&sc)[MT][NT], const int (&n)[NT], int kg)
{
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (4 * kg + r >= n[u])
#pragma unroll
                for (int g = 0; g < MT; ++g)
                    sc[g][u][r] = NM_NEG_INF;               // whatever lies there, NaN included
}

// The same for tiles with drafts among their tokens: first[u] is tile u's first one.
template <int MT, int NT>
__device__ __forceinline__ void mask_scores(f32x4 (&sc)[MT][NT], const int (&n)[NT], const int (&first)[NT],
                                            const Seen<Drafts, MT>& seen, int kg)
{
#pragma unroll
    for (int u = 0; u < NT; ++u) {
        const uint32_t held = (1u << min(max(n[u] - 4 * kg, 0), 4)) - 1u;
#pragma unroll
        for (int g = 0; g < MT; ++g) {
            const uint32_t sees = seen.four(g, first[u] + 4 * kg) & held;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                sc[g][u][r] = sees >> r & 1 ? sc[g][u][r] : NM_NEG_INF;
        }
    }
}

// acc[g] += v w[.][g] for one column's operand v of a pair of tiles (first tokens `first`) of
// which some rows do not see all.  If it holds infinities or NaN, token by token, each row
// keeping its sums where it does not see the token: 0 * NaN must not reach them.
template <int DT, int MT>
__device__ __forceinline__ void add_seen(f32x4 (&acc)[MT], u32x4 v, const u32x4 (&w)[2][MT], const int (&first)[2],
                                         const Seen<Drafts, MT>& seen, int kg)
{
    float odd = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        odd = dot2<DT>(v[i], 0u, odd);
    if (!__any(odd != 0.0f)) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int g = 0; g < MT; ++g)
                acc[g] = mfma<DT>(v, w[p][g], acc[g]);
        return;
    }
#pragma unroll 1
    for (int x = 0; x < 2 * nma::kTile; ++x) {
        const int in = x % nma::kTile, word = x / nma::kTile * 2 + in % 4 / 2;
        const uint32_t keep = in / 4 == kg ? (in % 2 ? 0xFFFF0000u : 0xFFFFu) : 0u;
        const int t = (x < nma::kTile ? first[0] : first[1]) + in;
        u32x4 one;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            one[i] = i == word ? v[i] & keep : 0u;
#pragma unroll
        for (int g = 0; g < MT; ++g) {
            const bool sees = seen.four(g, t) & 1;
            const f32x4 with = mfma<DT>(one, w[1][g], mfma<DT>(one, w[0][g], acc[g]));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[g][i] = sees ? with[i] : acc[g][i];
        }
    }
}

// What a dword of two 16-bit floats, `whole`, leaves out of the fp32 a and b that were
// rounded to it, as another such dword.  The differences are exact, each one dot product
// of two 16-bit floats with (-1, 0) or (0, -1).  These come from scalar registers: of
// bfloat16 constants the compiler makes the first the instruction's inline -1.0, which
// the hardware takes for (0, -1).
template <int DT>
__device__ __forceinline__ uint32_t left_out(uint32_t whole, float a, float b)
{
    constexpr uint32_t kMinusOne = DT == NM_FP16 ? 0xBC00u : 0xBF80u;
    uint32_t low = kMinusOne, high = kMinusOne << 16;
    asm("" : "+s"(low), "+s"(high));
    return pack2<DT>(dot2<DT>(whole, low, a), dot2<DT>(whole, high, b));
}

// The softmax weights of a step of NT tiles, in place of its scores; updates the rows'
// references (mx), sums and, where a reference grows, what has been added up so far.
template <int DT, int MT, int NT>
struct Weights {
    // Weights are relative to a row's reference `mx` (base 2), which need not be its maximum.
    // It is raised where a score passes it by more than kRoom, and is then put kBelow under
    // that score, so that the largest weight lies between 2^kBelow and 2^kRoom.
    //   It may lag, so that in long ranges the sums are hardly ever multiplied: 32 sequences
    // of 64 heads behind 32768 tokens, 16-bit: 67.5 us with the maximum itself, 63.7 with
    // it up to 2^8 behind; MX8 and 4096 own tokens 82.6 / 78.6 (both with a weight's first
    // operand alone).
    //   In fp16 it stays below: the operands' range then ends at 2^-32 of the largest weight,
    // not at 2^-25, where the tokens behind a first one that takes most of the weight would
    // be lost; 2^15 is the last power of two that fits (65504).  bfloat16 has fp32's range,
    // and values near its end: the reference stays above, and no value is added more than
    // once.
    static constexpr float kBelow = DT == NM_FP16 ? 7.0f : -8.0f;
    static constexpr float kRoom = DT == NM_FP16 ? 15.0f : 0.0f;

    f32x4 p[MT][NT];

    template <int PER>
    __device__ __forceinline__ void find(float (&mx)[MT], float (&sum)[MT], f32x4 (&acc)[MT][PER], float scale)
    {
#pragma unroll
        for (int g = 0; g < MT; ++g) {
            float top = NM_NEG_INF;
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    top = fmaxf(top, p[g][u][r]);
            top = quarters_max(top) * scale;
            if (__any(top > mx[g] + kRoom)) {
                top = fmaxf(mx[g], top - kBelow);
                const float f = mx[g] == top ? 1.0f : __builtin_amdgcn_exp2f(mx[g] - top);
                sum[g] *= f;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    acc[g][j] *= f;
                mx[g] = top;
            }
            const float base = mx[g] == NM_NEG_INF ? 0.0f : mx[g];
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    p[g][u][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[g][u][r], scale, -base));
                    sum[g] += p[g][u][r];
                }
        }
    }

    // Right operands of the second product for tiles 2 t, 2 t + 1: a weight is the sum of
    // two 16-bit floats, its own rounding (whole) and what that leaves out (rest).  That
    // keeps it to 2^-16 of itself in bfloat16 and 2^-22 in fp16; one alone would leave
    // 2^-8 and 2^-11, as much as o's own rounding.  Own tokens, bound by HBM, hardly
    // notice the second product (32 sequences of 4096, us with one / two: 16-bit 83.7 / 83.7,
    // MX8 45.6 / 45.4, MX4 34.3 / 37.2); staged prefix units, bound by the matrix cores,
    // do (32 sequences of 64 heads behind 32768 tokens 64.5 / 75.7, of 32 heads behind 8192
    // 23.4 / 25.0).
    __device__ __forceinline__ void whole(u32x4 (&out)[MT], int t) const
    {
#pragma unroll
        for (int g = 0; g < MT; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                out[g][i] = pack2<DT>(p[g][2 * t + i / 2][i % 2 * 2], p[g][2 * t + i / 2][i % 2 * 2 + 1]);
    }

    __device__ __forceinline__ void rest(u32x4 (&out)[MT], const u32x4 (&w)[MT], int t) const
    {
#pragma unroll
        for (int g = 0; g < MT; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                out[g][i] = left_out<DT>(w[g][i], p[g][2 * t + i / 2][i % 2 * 2], p[g][2 * t + i / 2][i % 2 * 2 + 1]);
    }
};

// Partial results of a row tile, in the workspace: the lane (kg, m) holds columns
// kg D/4 + r D/16 + j of row m in acc[j][r]; they are kept as
//   [r D/64 + j / 4][kg][row of the tile's nr] 16 bytes,
// so that a wave's store (and the load that joins them) is one contiguous piece.
__device__ __forceinline__ int64_t part_at(int chunk, int kg, int nr, int m)
{
    return ((int64_t)(chunk * 4 + kg) * nr + m) * 4;
}

template <int D>
__device__ __forceinline__ void store_part(const AttnArgs& A, int64_t row0, int nr, int m, int kg,
                                           const f32x4 (&acc)[D / 16], float mx, float sum)
{
    constexpr int kPer = D / 16;
    float* o = A.part_o + row0 * D;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < kPer; j += 4)
            *reinterpret_cast<f32x4*>(o + part_at(c * (kPer / 4) + j / 4, kg, nr, m)) =
                f32x4{acc[j][c], acc[j + 1][c], acc[j + 2][c], acc[j + 3][c]};
    if (kg == 0)
        A.part_ml[row0 + m] = f32x2{mx, sum};
}

// A row's outputs, from the lanes that hold its columns kg D/4 + r D/16 + j in acc[j][r].
template <class P, int DT, int D>
__device__ __forceinline__ void store_out(const AttnArgs& A, int h, int b, int r, int kg, const f32x4 (&acc)[D / 16],
                                          float mx, float sum)
{
    constexpr int kPer = D / 16;
    const float f = sum > 0.0f || sum != sum ? A.o_scale / sum : 0.0f;
    const int64_t row = P::out_row(A, h, b, r);
    uint16_t* o = A.o + row * D + kg * (D / 4);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < kPer; j += 4)
            *reinterpret_cast<u32x2*>(o + c * kPer + j) = u32x2{pack2<DT>(acc[j][c] * f, acc[j + 1][c] * f),
                                                                pack2<DT>(acc[j + 2][c] * f, acc[j + 3][c] * f)};
    if (A.lse && kg == 0)
        A.lse[row] = (mx + __builtin_amdgcn_logf(sum)) * kLn2;
}

// One unit: 16 MT rows from row0 of the R rows of key head h, tokens
// [start, end) of a page list that holds `limit` tokens.  Page numbers are loaded
// a step before the tiles they lead to; the wave's first two are page0 and page1.
template <class P, int DT, int BITS, int D, int MT, int NW>
__device__ __forceinline__ void attend(const AttnArgs& A, const int32_t* pages, int h, int b0, int row0, int R,
                                       int start, int end, int limit, int page0, int page1, bool direct,
                                       int64_t part_row, const Seen<P, MT>& seen, float* lds)
{
    using C = Cache<DT, BITS, D>;
    constexpr int kSteps = D / 32;                                   // k-steps of the score product
    constexpr int kPer = D / 16;
    const int lane = threadIdx.x % 64, m = lane % 16, kg = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    int at = start / nma::kTile + 2 * wave;             // the wave's next pair of tiles
    int page[2] = {page0, page1};
    Rows<P, DT, BITS, D, MT> rows;
    rows.load(A, h, b0, row0, R, m, kg);

    f32x4 acc[MT][kPer];
    float mx[MT], sum[MT];
#pragma unroll
    for (int g = 0; g < MT; ++g) {
        mx[g] = NM_NEG_INF;
        sum[g] = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            acc[g][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    typename C::Raw kr[2], vr[2];
    typename C::KScale ks[2];
    uint32_t vs[2] = {0u, 0u};
    TileRef cur[2], next[2];
    const auto load_k = [&](const TileRef(&t)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            C::template load<C::kCb>(kr[u], A.k + t[u].tile * nma::tile_bytes(D, BITS), lane);
            if constexpr (BITS != 16)
                C::load_k_scale(ks[u], A.k_scale + t[u].tile * nma::scale_tile_bytes(D), m);
        }
    };
    const auto load_v = [&](const TileRef(&t)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            C::template load<C::kVb>(vr[u], A.v + t[u].tile * nma::tile_bytes(D, BITS), lane);
            if constexpr (BITS != 16)
                C::load_v_scale(vs[u], A.v_scale + t[u].tile * nma::scale_tile_bytes(D), m, kg);
        }
    };

    const int last = (end + nma::kTile - 1) / nma::kTile;
    const auto fetch = [&]() {                          // the pages of pair `at`
        page[0] = page_of(A, pages, at, limit);
        page[1] = page_of(A, pages, at + 1, limit);
    };
    const auto refer = [&](TileRef(&t)[2]) {            // its tiles
        t[0] = tile_ref(A, page[0], at, end, h);
        t[1] = tile_ref(A, page[1], at + 1, end, h);
        at += 2 * NW;
    };
    // One step; with `more`, the loads of the wave's next one start as soon as the
    // registers they fill are free.  In a tree the caller says whether it is `masked`.
    const auto step = [&](auto more, auto masked) {
        if constexpr (more()) {
            refer(next);
            fetch();
        }
        // scores
        Weights<DT, MT, 2> w;
        auto& sc = w.p;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int g = 0; g < MT; ++g)
                sc[g][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const u32x4 a = C::k_operand(kr[u], ks[u], s, kg);
#pragma unroll
                for (int g = 0; g < MT; ++g) {
                    sc[g][u] = mfma<DT>(a, rows.op[g][s], sc[g][u]);
                }
            }
        }
        if constexpr (more())
            load_k(next);
        const int n[2] = {cur[0].n, cur[1].n}, first[2] = {cur[0].first, cur[1].first};
        const bool whole = P::kTree ? !masked() : n[0] == nma::kTile && n[1] == nma::kTile;
        if constexpr (P::kTree) {
            if constexpr (masked())
                mask_scores(sc, n, first, seen, kg);
        } else if (!whole) {
            mask_scores(sc, n, kg);
        }
        w.find(mx, sum, acc, A.scale);
        u32x4 wo[2][MT];
        w.whole(wo[0], 0);
        w.rest(wo[1], wo[0], 0);
        // values
        uint32_t vo[2][2 * kPer];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            C::v_operands(vo[u], vr[u], vs[u]);
        if (!whole) {
            // a token that does not count may hold anything: 0 * NaN must not reach o
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int left = cur[u].n - 4 * kg;
                const uint32_t keep[2] = {left >= 2 ? 0xFFFFFFFFu : left == 1 ? 0xFFFFu : 0u,
                                          left >= 4 ? 0xFFFFFFFFu : left == 3 ? 0xFFFFu : 0u};
#pragma unroll
                for (int i = 0; i < 2 * kPer; ++i)
                    vo[u][i] &= keep[i % 2];
            }
        }
        const auto products = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const u32x4 a = {vo[0][2 * j], vo[0][2 * j + 1], vo[1][2 * j], vo[1][2 * j + 1]};
#pragma unroll
                    for (int g = 0; g < MT; ++g)
                        acc[g][j] = mfma<DT>(a, wo[i][g], acc[g][j]);
                }
        };
        if constexpr (P::kTree) {
            if constexpr (masked()) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const u32x4 a = {vo[0][2 * j], vo[0][2 * j + 1], vo[1][2 * j], vo[1][2 * j + 1]};
                    f32x4 column[MT];
#pragma unroll
                    for (int g = 0; g < MT; ++g)
                        column[g] = acc[g][j];
                    add_seen<DT, MT>(column, a, wo, first, seen, kg);
#pragma unroll
                    for (int g = 0; g < MT; ++g)
                        acc[g][j] = column[g];
                }
            } else {
                products();
            }
        } else {
            products();
        }
        if constexpr (more()) {
            load_v(next);
            cur[0] = next[0];
            cur[1] = next[1];
        }
    };
    if (at < last) {
        refer(cur);
        load_k(cur);
        __builtin_amdgcn_sched_barrier(0);              // keys first: they are waited for first
        load_v(cur);
        fetch();
        if constexpr (P::kTree) {
            // drafts, and what else is not whole, lie behind the whole tiles
            const auto whole = [&]() {
                return cur[0].n == nma::kTile && cur[1].n == nma::kTile && cur[1].first + nma::kTile <= seen.first_draft;
            };
            while (at < last && whole())
                step(std::true_type(), std::false_type());
            while (at < last)
                step(std::true_type(), std::true_type());
            step(std::false_type(), std::true_type());
        } else {
            while (at < last)
                step(std::true_type(), std::false_type());
            step(std::false_type(), std::false_type());
        }
    }
#pragma unroll
    for (int g = 0; g < MT; ++g)
        sum[g] = quarters_sum(sum[g]);

    // The block's waves are joined two by two through LDS, lane to lane.
    constexpr int kRegs = MT * (4 * kPer + 2);
#pragma unroll
    for (int half = NW / 2; half >= 1; half /= 2) {
        float* box = lds + (wave % half) * kRegs * 64 + lane;
        if (half < NW / 2)
            __syncthreads();                            // the boxes' last readers are done
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int g = 0; g < MT; ++g) {
                box[(g * (4 * kPer + 2) + 4 * kPer) * 64] = mx[g];
                box[(g * (4 * kPer + 2) + 4 * kPer + 1) * 64] = sum[g];
#pragma unroll
                for (int i = 0; i < 4 * kPer; ++i)
                    box[(g * (4 * kPer + 2) + i) * 64] = acc[g][i / 4][i % 4];
            }
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int g = 0; g < MT; ++g) {
                const float om = box[(g * (4 * kPer + 2) + 4 * kPer) * 64];
                const float os = box[(g * (4 * kPer + 2) + 4 * kPer + 1) * 64];
                const float top = fmaxf(mx[g], om), base = top == NM_NEG_INF ? 0.0f : top;
                const float f0 = __builtin_amdgcn_exp2f(mx[g] - base), f1 = __builtin_amdgcn_exp2f(om - base);
                sum[g] = sum[g] * f0 + os * f1;
                mx[g] = top;
#pragma unroll
                for (int i = 0; i < 4 * kPer; ++i)
                    acc[g][i / 4][i % 4] = acc[g][i / 4][i % 4] * f0 + box[(g * (4 * kPer + 2) + i) * 64] * f1;
            }
        }
    }
    if (wave != 0)
        return;
#pragma unroll
    for (int g = 0; g < MT; ++g) {
        const int r = row0 + 16 * g + m;
        if (r >= R)
            continue;
        if (direct) {
            store_out<P, DT, D>(A, h, b0, r, kg, acc[g], mx[g], sum[g]);
        } else {
            store_part<D>(A, part_row + row0 + 16 * g, min(16, R - row0 - 16 * g), m, kg, acc[g], mx[g], sum[g]);
        }
    }
}

constexpr int join_bytes(int D, int mt, int waves) { return waves / 2 * mt * (D / 4 + 2) * 64 * 4; }

// ---- staged prefix units -----------------------------------------------------
//
// W waves with 16 MT rows each share every tile of the range: four tiles at a
// time are loaded by the block (each wave a half or a whole of one tile's keys and
// values), turned into operands once, and written to LDS in operand order, in two
// buffers; the next four are on their way while the current ones are multiplied.
//   keys    [tile][k-step][lane] 16 bytes
//   values  [tile pair][column j][lane] 16 bytes, 8 of each tile
template <int DT, int BITS, int D, int W>
struct Stage {
    using C = Cache<DT, BITS, D>;
    static constexpr int kTiles = nma::kStaged / nma::kTile;
    static constexpr int kShare = W / kTiles;                // waves that load one tile
    static constexpr int kSteps = D / 32, kPer = D / 16;
    static constexpr int kTileBytes = 32 * D;                // a tile's keys (or values) as operands
    static constexpr int kBytes = 2 * kTiles * kTileBytes;   // a buffer: all keys, then all values
    static constexpr int kMine = kSteps / kShare;            // k-steps of keys (and equal parts of values) a wave loads
    static_assert(kShare == 1 || kShare == 2, "a tile is loaded by one or two waves");

    // Raw loads of one wave.  16-bit: whole 1 KB pieces of the tile.  Codes: keys by
    // k-step (BITS bytes a lane), values by pairs of tokens.
    static constexpr int kVPairs = 2 / kShare;               // token pairs (of a lane's two) a wave loads
    static constexpr int kVBytes = kPer * BITS / 4;          // a lane's bytes of one pair
    static constexpr int kVLoad = kVBytes < C::kCb ? kVBytes : C::kCb;
    uint32_t k[BITS == 16 ? 4 * kMine : kMine * BITS / 4];
    uint32_t v[BITS == 16 ? 4 * kMine : kVPairs * kVBytes / 4];
    typename C::KScale ks;
    uint32_t vs;
    int n;

    template <int BYTES>
    static __device__ __forceinline__ void get(uint32_t* dst, const uint8_t* src)
    {
        typedef uint32_t piece __attribute__((ext_vector_type(BYTES / 4)));
        if constexpr (BYTES == 4) {
            dst[0] = *reinterpret_cast<const uint32_t*>(src);
        } else {
            const piece x = *reinterpret_cast<const piece*>(src);
#pragma unroll
            for (int i = 0; i < BYTES / 4; ++i)
                dst[i] = x[i];
        }
    }

    // Codes: keys and values by themselves.
    __device__ __forceinline__ void load_k(const AttnArgs& A, const TileRef& t, int part, int lane)
    {
        const uint8_t* kt = A.k + t.tile * nma::tile_bytes(D, BITS);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int at = (part * kMine + i) * BITS;
            get<BITS>(k + i * BITS / 4, kt + at / C::kCb * 64 * C::kCb + lane * C::kCb + at % C::kCb);
        }
        C::load_k_scale(ks, A.k_scale + t.tile * nma::scale_tile_bytes(D), lane % 16);
    }

    __device__ __forceinline__ void load_v(const AttnArgs& A, const TileRef& t, int part, int lane)
    {
        const uint8_t* vt = A.v + t.tile * nma::tile_bytes(D, BITS);
        n = t.n;
#pragma unroll
        for (int i = 0; i < kVPairs * kVBytes; i += kVLoad) {
            const int at = part * kVPairs * kVBytes + i;
            get<kVLoad>(v + i / 4, vt + at / C::kVb * 64 * C::kVb + lane * C::kVb + at % C::kVb);
        }
        C::load_v_scale(vs, A.v_scale + t.tile * nma::scale_tile_bytes(D), lane % 16, lane / 16);
    }

    // Both.  16-bit pieces of keys and values go in turn, to LDS too: all keys and then all values is slower
    // (64 heads of 32 sequences behind 32741 tokens and up to 1024 own, us in turn / apart: 72.8 / 74.4).
    __device__ __forceinline__ void load(const AttnArgs& A, const TileRef& t, int part, int lane)
    {
        if constexpr (BITS == 16) {
            const uint8_t* kt = A.k + t.tile * nma::tile_bytes(D, BITS);
            const uint8_t* vt = A.v + t.tile * nma::tile_bytes(D, BITS);
            n = t.n;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                get<16>(k + 4 * i, kt + (part * kMine + i) * 1024 + lane * 16);
                get<16>(v + 4 * i, vt + (part * kMine + i) * 1024 + lane * 16);
            }
        } else {
            load_k(A, t, part, lane);
            load_v(A, t, part, lane);
        }
    }

    // Operands of the codes that were loaded into the tile's place among keys, or values, of which those of
    // tokens that do not count become zeros (0 * NaN must not reach o).  With `turned`, the keys'
    // lanes of an odd tile change places (m with m ^ 8).  (The operand functions take a lane's whole
    // part; what this wave did not load is not used.)
    __device__ __forceinline__ void put_k(uint8_t* keys, int tile, int part, int lane, bool turned = false) const
    {
        uint8_t* kd = keys + tile * kTileBytes;
        const int to = lane ^ (turned ? tile % 2 * 8 : 0);
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            *reinterpret_cast<u32x4*>(kd + (part * kMine + i) * 1024 + to * 16) =
                C::k_codes(k + i * BITS / 4, ks, part * kMine + i, lane / 16);
    }

    __device__ __forceinline__ void put_v(uint8_t* values, int tile, int part, int lane) const
    {
        uint8_t* vd = values + tile / 2 * 2 * kTileBytes + tile % 2 * 8;
        const int left = n - 4 * (lane / 16);
        if constexpr (kVPairs == 2) {
            uint32_t lo[kPer], hi[kPer];
            C::v_codes(lo, v, vs);
            C::v_codes(hi, v + kVBytes / 4, vs >> 16);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                *reinterpret_cast<u32x2*>(vd + j * 1024 + lane * 16) =
                    u32x2{lo[j] & keep(left, 0), hi[j] & keep(left, 1)};
        } else {
            uint32_t out[kPer];
            C::v_codes(out, v, vs >> (16 * part));
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                *reinterpret_cast<uint32_t*>(vd + j * 1024 + lane * 16 + part * 4) = out[j] & keep(left, part);
        }
    }

    // Both, into a buffer of all keys, then all values.
    __device__ __forceinline__ void put(uint8_t* buf, int tile, int part, int lane) const
    {
        if constexpr (BITS == 16) {
            uint8_t* kd = buf + tile * kTileBytes;
            uint8_t* vd = buf + (kTiles + tile / 2 * 2) * kTileBytes + tile % 2 * 8;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                *reinterpret_cast<u32x4*>(kd + (part * kMine + i) * 1024 + lane * 16) =
                    u32x4{k[4 * i], k[4 * i + 1], k[4 * i + 2], k[4 * i + 3]};
                u32x4 x = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
                if (n < nma::kTile) {
                    // 16 bytes here are two lanes' halves of one column: quarter (lane % 32) / 8
                    const int left = n - 4 * (lane % 32 / 8);
                    x &= u32x4{keep(left, 0), keep(left, 1), keep(left, 0), keep(left, 1)};
                }
                uint8_t* to = vd + ((part * kMine + i) * 128 + lane * 2) * 16;
                *reinterpret_cast<u32x2*>(to) = u32x2{x.x, x.y};
                *reinterpret_cast<u32x2*>(to + 16) = u32x2{x.z, x.w};
            }
        } else {
            put_k(buf, tile, part, lane);
            put_v(buf + kTiles * kTileBytes, tile, part, lane);
        }
    }

    // Mask of the token pair (2 i, 2 i + 1) of a quarter of which `left` tokens count.
    static __device__ __forceinline__ uint32_t keep(int left, int i)
    {
        return left >= 2 * i + 2 ? 0xFFFFFFFFu : left == 2 * i + 1 ? 0xFFFFu : 0u;
    }
};

// Row group `group` of a page list's R rows, tokens [start, end); lds: two buffers and two counts of
// each tile's tokens (staged_bytes).
//   256 rows, 131072 tokens, 16-bit: 207 us at 2.1 GHz, 660 TFLOP/s of the formula.  A wave
// and step has 96 products (a third of them for the weights' second operands) and 234
// vector instructions, 32 of them exponentials; at 16, 4 and 16 cycles these are 1536 and
// 1320 of the 3380 cycles that it takes.  So the matrix cores are busy 45% of the time: the
// two waves of a SIMD leave each barrier together, and one's products hide little of the
// other's vector work.  On zeros, where the card's power does not count, 198 us for 222.
template <int BITS, int D, int W>
constexpr int staged_bytes()
{
    return 2 * Stage<NM_FP16, BITS, D, W>::kBytes + 2 * Stage<NM_FP16, BITS, D, W>::kTiles * 4;
}

template <int DT, int BITS, int D, int MT, int W>
__device__ __forceinline__ void attend_staged(const AttnArgs& A, int unit, uint8_t* lds)
{
    using S = Stage<DT, BITS, D, W>;
    constexpr int NT = S::kTiles, kSteps = S::kSteps, kPer = S::kPer;
    constexpr int kGroup = 4;                                // value operands read at a time
    int(*const count)[NT] = reinterpret_cast<int(*)[NT]>(lds + 2 * S::kBytes);
    const int lane = threadIdx.x % 64, m = lane % 16, kg = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int h = unit % A.heads, split = unit / A.heads % A.prefix_splits;
    const int row0 = (unit / A.heads / A.prefix_splits * W + wave) * 16 * MT;
    const int start = split * A.prefix_chunk, end = min(start + A.prefix_chunk, A.prefix_len);
    const int mine = wave % NT, part = wave / NT;            // the tile of each step that this wave loads
    const bool busy = row0 < A.prefix_rows;

    Rows<OneToken, DT, BITS, D, MT> rows;
    rows.load(A, h, 0, row0, A.prefix_rows, m, kg);
    f32x4 acc[MT][kPer];
    float mx[MT], sum[MT];
#pragma unroll
    for (int g = 0; g < MT; ++g) {
        mx[g] = NM_NEG_INF;
        sum[g] = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            acc[g][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    S stage;
    int at = start / nma::kTile + mine;
    const int steps = (end - start + nma::kStaged - 1) / nma::kStaged;
    const auto put = [&](int which) {
        stage.put(lds + which * S::kBytes, mine, part, lane);
        if (part == 0 && lane == 0)
            count[which][mine] = stage.n;
    };
    stage.load(A, tile_ref(A, page_of(A, A.prefix_pages, at, end), at, end, h), part, lane);
    int page = page_of(A, A.prefix_pages, at + NT, end);
    put(0);
    __syncthreads();
    for (int i = 0; i < steps; ++i) {
        const bool more = i + 1 < steps;
        if (more) {
            at += NT;
            stage.load(A, tile_ref(A, page, at, end, h), part, lane);
            page = page_of(A, A.prefix_pages, at + NT, end);
        }
        if (busy) {
            const uint8_t* kb = lds + (i & 1) * S::kBytes;
            const uint8_t* vb = kb + NT * S::kTileBytes;
            // Operands are read from LDS one tile (keys) or one group of columns (values)
            // ahead of the products that use them; the barriers keep the compiler from
            // moving the reads down to their uses.
            u32x4 ka[2][kSteps], va[2][kGroup];
            const auto read_k = [&](int u) {
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    ka[u % 2][s] = *reinterpret_cast<const u32x4*>(kb + u * S::kTileBytes + s * 1024 + lane * 16);
            };
            const auto read_v = [&](int x) {
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    va[x % 2][j] = *reinterpret_cast<const u32x4*>(vb + (x * kGroup + j) * 1024 + lane * 16);
            };
            Weights<DT, MT, NT> w;
            auto& sc = w.p;
            read_k(0);
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                if (u + 1 < NT)
                    read_k(u + 1);
                else
                    read_v(0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int g = 0; g < MT; ++g)
                    sc[g][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int g = 0; g < MT; ++g) {
                        sc[g][u] = mfma<DT>(ka[u % 2][s], rows.op[g][s], sc[g][u]);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
            int n[NT];
            bool whole = true;
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                n[u] = __builtin_amdgcn_readfirstlane(count[i & 1][u]);
                whole = whole && n[u] == nma::kTile;
            }
            if (!whole)
                mask_scores(sc, n, kg);
            w.find(mx, sum, acc, A.scale);
            constexpr int kGroups = NT / 2 * kPer / kGroup;
            u32x4 wo[2][MT];
#pragma unroll
            for (int x = 0; x < kGroups; ++x) {
                const bool first = x * kGroup % kPer == 0;
                const int t = x * kGroup / kPer;
                if (x + 1 < kGroups)
                    read_v(x + 1);
                if (first)
                    w.whole(wo[0], t);
                __builtin_amdgcn_sched_barrier(0);
                if (first)              // beside the first products
                    w.rest(wo[1], wo[0], t);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < kGroup; ++c)
#pragma unroll
                        for (int g = 0; g < MT; ++g) {
                            const int j = (x * kGroup + c) % kPer;
                            acc[g][j] = mfma<DT>(va[x % 2][c], wo[i][g], acc[g][j]);
                        }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (more)
            put((i + 1) & 1);           // that buffer's readers passed the barrier before this step
        __syncthreads();
    }
#pragma unroll
    for (int g = 0; g < MT; ++g) {
        const int r = row0 + 16 * g;
        const float total = quarters_sum(sum[g]);
        if (r + m < A.prefix_rows)
            store_part<D>(A, ((int64_t)split * A.heads + h) * A.prefix_rows + r, min(16, A.prefix_rows - r), m, kg,
                          acc[g], mx[g], total);
    }
}

// Joins the partial results: a block takes one chunk of a tile of 16 rows (r = b G
// + g) of one key head, a lane (kg, m) row m as in the partial results.  NW waves
// share the parts, each keeps a reference and sums of its own as the units do, and
// they meet in LDS.  A wave loads four parts at a time, with the next four on their
// way, and the first four before the sequence's length is known (units and join of 32
// sequences of 32 heads behind 8192 tokens, when this was measured: 28.4 us with the
// maxima looked at first, 27.1 this way; one sequence of 131071, MX4: 32.0 / 31.5).
template <class P, int DT, int D, int NW>
__device__ __forceinline__ void combine(const AttnArgs& A)
{
    constexpr int kBatch = 4;
    __shared__ float tops[NW][64], sums[NW][64];
    __shared__ f32x4 box[NW][64];
    const int lane = threadIdx.x % 64, m = lane % 16, kg = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int tiles = (A.prefix_rows + 15) / 16;
    const uint32_t block = flat_block();
    const int h = block % A.heads, tile = block / A.heads % tiles, chunk = block / A.heads / tiles;
    if (chunk >= D / 16)
        return;
    const int r = tile * 16 + m, rr = min(r, A.prefix_rows - 1), b = rr / A.G, g = rr % A.G;
    const int held = A.lens[b], np = A.prefix_splits;
    // Part i of the lane's row: first row of its tile, rows of the tile, row in it.
    const int p_rows = min(16, A.prefix_rows - tile * 16), o_rows = min(16, A.G - g / 16 * 16);
    const int64_t p0 = (int64_t)h * A.prefix_rows + tile * 16, p_step = (int64_t)A.heads * A.prefix_rows;
    const int64_t o_step = (int64_t)A.B * A.Hq;
    const int64_t o0 = A.own_base + (int64_t)b * A.Hq + (int64_t)h * A.G + g / 16 * 16 - np * o_step;
    f32x2 x[kBatch], next_x[kBatch];                    // (reference, sum)
    f32x4 o[kBatch], next_o[kBatch];
    // Parts i, i + NW, .. of those below `parts` (others are read from the first one and not added).
    const auto load = [&](int i, int parts) {
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            const int at = i + c * NW < parts ? i + c * NW : 0;
            const int in = (at < np ? rr : g) % 16;
            const int64_t row0 = at < np ? p0 + at * p_step : o0 + at * o_step;
            next_x[c] = A.part_ml[row0 + in];
            next_o[c] = *reinterpret_cast<const f32x4*>(A.part_o + row0 * D +
                                                        part_at(chunk, kg, at < np ? p_rows : o_rows, in));
        }
    };
    load(wave, np + A.own_splits);
    const int len = min(held, A.max_len);
    const int mine = np + (max(len, 0) + A.own_chunk - 1) / A.own_chunk;
    int total = mine;                                   // of the tile's longest row
#pragma unroll
    for (int i = 1; i < 64; i *= 2)
        total = max(total, __shfl_xor(total, i));
    total = __builtin_amdgcn_readfirstlane(total);

    float mx = NM_NEG_INF, sum = 0.0f;
    f32x4 acc = {};
    for (int i = wave; i < total; i += kBatch * NW) {
        float top = mx;
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            x[c] = next_x[c];
            o[c] = next_o[c];
            if (i + c * NW < mine)
                top = fmaxf(top, x[c].x);
        }
        if (i + kBatch * NW < total)
            load(i + kBatch * NW, mine);
        const float base = top == NM_NEG_INF ? 0.0f : top, f = __builtin_amdgcn_exp2f(mx - base);
        mx = top;
        sum *= f;
        acc *= f;
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            const bool live = i + c * NW < mine;        // a part that no block wrote may hold anything
            const float w = __builtin_amdgcn_exp2f(x[c].x - base);
            sum += live ? x[c].y * w : 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[e] += live ? o[c][e] * w : 0.0f;
        }
    }
    tops[wave][lane] = mx;
    sums[wave][lane] = sum;
    box[wave][lane] = acc;
    __syncthreads();
    if (wave > 0 || r >= A.prefix_rows || len < 0)      // a padding row stays as it was
        return;
#pragma unroll
    for (int w = 1; w < NW; ++w)
        mx = fmaxf(mx, tops[w][lane]);
    const float base = mx == NM_NEG_INF ? 0.0f : mx;
    sum = 0.0f;
    acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float f = __builtin_amdgcn_exp2f(tops[w][lane] - base);
        sum += sums[w][lane] * f;
        acc += box[w][lane] * f;
    }
    acc *= sum > 0.0f || sum != sum ? A.o_scale / sum : 0.0f;
    const int64_t row = P::out_row(A, h, b, g);
    *reinterpret_cast<u32x2*>(A.o + row * D + kg * (D / 4) + chunk * 4) =
        u32x2{pack2<DT>(acc[0], acc[1]), pack2<DT>(acc[2], acc[3])};
    if (A.lse && kg == 0 && chunk == 0)
        A.lse[row] = (mx + __builtin_amdgcn_logf(sum)) * kLn2;
}

}  // namespace nmu
