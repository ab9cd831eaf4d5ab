// nm_attn.h -- shared by the entry points of include/nmattn.h and their
// kernels: the cache's byte layout, the launch plan of nm_attn_decode, and the
// kernel-side declarations.  Host-only C++ (no HIP types): the checks and the
// plan also build with a plain compiler under sanitizers; the constexpr layout
// functions are used by the device code too.

#ifndef NM_ATTN_H
#define NM_ATTN_H

#include <cstdint>

#include "nmattn.h"

namespace nma {

// ---- cache layout -----------------------------------------------------------
//
// [page][head][page_size / 16] tiles of 16 tokens x D columns.  A tile is cut
// into `chunks` of 64 x cb bytes, cb (16, or 8 in the smallest case) bytes for
// each lane of a wave, in lane order: lane = quarter * 16 + m.  A load of one
// chunk by a wave is one contiguous read of full cache lines, and what it
// brings is that lane's part of a matrix-core operand:
//   keys    m = token, a lane's e = 8 cb / bits elements are consecutive columns,
//           chunk c, quarter q: columns c * 4e + q * e ..
//   values  m = column group (D / 16 columns), quarter q: tokens 4q .. 4q + 3;
//           16-bit: a chunk is a column's four tokens (half an operand as it is);
//           codes: a token's D / 16 columns side by side (one scale serves them).
constexpr int kTile = 16;

constexpr int format_bits(int format) { return format == NM_KV_16 ? 16 : format == NM_KV_MX8 ? 8 : 4; }
constexpr int tile_bytes(int D, int bits) { return kTile * D * bits / 8; }
constexpr int lane_bytes(int D, int bits) { return tile_bytes(D, bits) / 64; }              // 8 .. 128
constexpr int k_chunk_bytes(int D, int bits) { return lane_bytes(D, bits) < 16 ? lane_bytes(D, bits) : 16; }
constexpr int v_chunk_bytes(int D, int bits) { return bits == 16 ? 8 : k_chunk_bytes(D, bits); }

// Byte of a tile at which key element (token, d) lies; d a multiple of 8 (8
// columns always lie side by side, bits * 8 / 8 bytes).
constexpr int k_offset(int D, int bits, int token, int d)
{
    const int cb = k_chunk_bytes(D, bits), e = cb * 8 / bits;
    return d / (4 * e) * (64 * cb) + (d / e % 4 * 16 + token) * cb + d % e * bits / 8;
}

// Byte of a tile at which value element (token, d) lies (4-bit: d even, two
// columns a byte, the lower one in the low nibble).
constexpr int v_offset(int D, int bits, int token, int d)
{
    const int cb = v_chunk_bytes(D, bits), per = D / 16, j = d % per, r = token % 4;
    const int at = (bits == 16 ? j * 4 + r : r * per + j) * bits / 8;
    return at / cb * (64 * cb) + (token / 4 * 16 + d / per) * cb + at % cb;
}

// Scale bytes: one per 32 columns of a token's head; D / 2 per tile.  Keys:
// [token][block] (a lane reads its token's), values: [block][token] (a lane
// reads its four tokens' of one block).
constexpr int kBlock = 32;
constexpr int scale_tile_bytes(int D) { return kTile * D / kBlock; }
constexpr int k_scale_offset(int D, int token, int block) { return token * (D / kBlock) + block; }
constexpr int v_scale_offset(int token, int block) { return block * kTile + token; }

// A scale byte b stands for codes times 2^(b - bias).  Attention turns codes into
// operands of the cache's dtype times 2^(b - 127), and that has to be exact.  It is
// in bfloat16, whose range is fp32's; fp16 ends at 65504, below the 65536 to which a
// large value may be rounded, and at multiples of 2^-24.  So an fp16 cache's operands
// are half its values (bias 126, made good in the scores' scale and in the output),
// and its e stays where the smallest codes, 2^-9 (e4m3) and 2^-1 (e2m1), do not fall
// below 2^-23: values are off by 2^-24 at most for that, one step of fp16's own least
// numbers.  255 marks a block that held a NaN or an infinity.
constexpr int scale_bias(int dtype) { return dtype == NM_FP16 ? 126 : 127; }
constexpr int least_exponent(int dtype, int bits) { return dtype == NM_BF16 ? -126 : bits == 8 ? -14 : -22; }

// ---- the plan of nm_attn_decode ----------------------------------------------
//
// Work is cut into units of (row group, key head, range of tokens), one block
// each.  Own-token units: one sequence's query heads of one key head, 16 rows;
// the block's kWaves waves take pairs of tiles of the range in turn and add their
// results up in LDS.  Prefix units: rows are the whole batch's query heads of one
// key head.  Up to 32 rows they are worked like own-token units (16 mt rows);
// beyond, a block of `waves` waves holds 16 mt rows in each wave, and all its
// waves read the range's tiles from LDS, staged once for the block.
// Ranges of one row are added up by a second launch (combine), through fp32
// partial results in the workspace; with a single range per row there is none
// and no workspace.
constexpr int kWaves = 4;
constexpr int kStep = 2 * kTile;            // tokens a wave takes at a time
constexpr int kStaged = 4 * kTile;          // tokens staged at a time
constexpr int kCus = 256;
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxRows = int64_t(1) << 26;      // B * Hq

struct AttnPlan {
    int G;                                        // query heads per key head
    int mt;                                       // row tiles of a prefix unit's wave
    int waves;                                    // of a staged prefix unit; 0: worked like own tokens
    int64_t prefix_rows;                          // B * G
    int64_t prefix_groups, prefix_splits, prefix_chunk;
    int64_t own_groups, own_splits, own_chunk;
    bool direct;                                  // no combine: units write o
    int64_t prefix_parts, own_parts;              // partial rows of each kind
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Cuts `tokens` into ranges of whole steps for every wave, so that `units` row
// groups make about `blocks` blocks, and into ranges of at most `longest` where
// that takes no more than 64 (a batch of very different lengths would otherwise
// wait for its longest sequence's block).
constexpr int64_t kMaxRanges = 64, kMaxBlocks = int64_t(1) << 24;

inline void cut(int64_t tokens, int64_t units, int64_t blocks, int64_t longest, int64_t* splits, int64_t* chunk)
{
    const int64_t grain = kWaves * kStep;
    if (tokens == 0) {
        *splits = 0;
        *chunk = grain;
        return;
    }
    int64_t want = blocks > units ? ceil_div(blocks, units) : 1;
    int64_t even = ceil_div(tokens, longest);
    if (even > kMaxRanges)
        even = kMaxRanges;
    if (even > kMaxBlocks / units)
        even = kMaxBlocks / units;
    if (want < even)
        want = even;
    if (want > ceil_div(tokens, grain))
        want = ceil_div(tokens, grain);
    *chunk = ceil_div(ceil_div(tokens, want), grain) * grain;
    *splits = ceil_div(tokens, *chunk);
}

inline AttnPlan attn_plan(int64_t B, int Hq, int heads, int D, int format, int64_t prefix_len, int64_t max_len)
{
    AttnPlan p;
    p.G = Hq / heads;
    p.prefix_rows = B * p.G;
    p.mt = p.prefix_rows <= 16 || D == 256 ? 1 : 2;
    p.waves = p.prefix_rows <= 16 * p.mt ? 0 : p.prefix_rows <= 64 * p.mt && D != 256 ? 4 : 8;
    p.prefix_groups = ceil_div(p.prefix_rows, 16 * p.mt * (p.waves ? p.waves : 1));
    p.own_groups = ceil_div(p.G, 16);
    // Prefix units of eight waves have a CU to themselves, and the matrix cores limit
    // them; own-token units are limited by HBM.  So they share the GPU side by side,
    // the prefix taking as many CUs as its share of the work: a token of a key head
    // counts 52 in a staged block and 22 in an own-token block (16-bit; by its bytes), of
    // which two thirds, since the batch is rarely full to max_len.  (52 was a staged block's
    // time before weights had a second operand; 65, its time since, gives the prefix more
    // CUs and is slower, 52 / 65: 32741 + up to 1024 below 73.8 / 78.6, MX8, 32768 + up to
    // 4096 85.1 / 95.3, 16384 + up to 1024 48.2 / 53.1, but 8192 + up to 2048 39.6 / 35.9.)
    // 32 sequences of 64 heads on 8 of 128 columns, us for 256 / 192 / 160 prefix blocks:
    // 16-bit, 32741 tokens + up to 1024 82.7 / 75.2 / 82.3, 8192 + up to 1024 49.4 / 45.3 /
    // 39.6; MX8, 32768 + up to 4096 100.4 / 99.0 / 85.3; 32768 alone 68.7 / 74.6 / 81.8.
    // Short own tokens have an eighth of the CUs left to them all the same, or they would
    // wait for the prefix (16-bit, 16 own tokens, 256 / 224 blocks: 4096 + 29.7 / 24.7,
    // 8192 + 35.0 / 31.7, 32768 + 67.5 / 69.6).
    const double staged = 52.0 * (double)(prefix_len * heads * p.prefix_groups);
    const double own = 22.0 * 2 / 3 * format_bits(format) / 16 * (double)(B * heads * p.own_groups) * (double)max_len;
    int64_t cus = kCus;
    if (max_len > 0) {
        cus = (int64_t)(kCus * (staged / (staged + own)));
        if (cus > kCus * 7 / 8)
            cus = kCus * 7 / 8;
    }
    // Smaller prefix units: one block a CU, since every further range of a row costs its
    // partial sums' way to memory and back; but two where ranges are long all the same,
    // a block alone does not keep its CU busy (staged by four waves, or 4-bit) and few
    // own tokens want the room.  us with one / two, 8 key heads of 128 columns (other widths
    // and head counts go by the same rule, unmeasured): 64 rows, MX8, 8192 tokens 18.9 /
    // 20.4, 16384 27.2 / 26.2, 32768 42.6 / 36.0; 128 rows, 16-bit, 8192 22.3 / 27.9, 32768
    // 49.4 / 46.8, 65536 82.6 / 71.1; 32 rows, MX8, 32768 21.9 / 24.3; 16 rows, MX4, 8192
    // 11.0 / 11.7, 32768 17.4 / 15.8, MX8, 131072 50.2 / 51.6.  With up to 2048 own tokens:
    // 64 rows, MX8, 32768 44.4 / 42.0, 65536 77.5 / 62.2; 128 rows, MX8, 32768 48.5 / 50.9,
    // 65536 81.6 / 76.3; 16 rows, MX4, 32768 17.8 / 16.8.
    const int64_t prefix_units = heads * p.prefix_groups, longish = format == NM_KV_16 ? 1024 : 512;
    const bool two = (p.waves == 4 || format == NM_KV_MX4) && prefix_len * prefix_units >= longish * 2 * kCus &&
                     max_len * 32 <= prefix_len;
    cut(prefix_len, prefix_units, p.waves == 8 ? cus : two ? 2 * kCus : kCus, kMaxTokens, &p.prefix_splits,
        &p.prefix_chunk);
    // Own tokens (us; 8 key heads, MX8, x blocks for each CU): 32 sequences of up to
    // 1024 tokens, one unit per CU: 1 block 12.3, 2 blocks 14.2, 3 blocks 14.8; 16 of up
    // to 8192: 38.3 / 34.2 / 35.8; 8 of up to 32768: 69.8 / 58.1 / 61.8.  Longest range
    // for 32 sequences of up to 16384: 2048 tokens 95.7, 4096 97.2, 8192 110.3; of
    // 4096 each: 49.8 / 45.7 / 45.7.
    const int64_t units = B * heads * p.own_groups;
    cut(max_len, units, units >= kCus ? kCus : 2 * kCus, 4096, &p.own_splits, &p.own_chunk);
    // Up to 512 tokens a single range without a second launch is no slower than several
    // (one sequence, 16-bit: 200 tokens 5.4 / 7.4 us, 400 6.5 / 7.6, 800 8.5 / 7.9).
    if (prefix_len == 0 && max_len > 0 && max_len <= 512) {
        p.own_splits = 1;
        p.own_chunk = 512;
    }
    p.direct = p.prefix_splits == 0 && p.own_splits <= 1;
    p.prefix_parts = p.direct ? 0 : p.prefix_splits * heads * p.prefix_rows;
    p.own_parts = p.direct ? 0 : p.own_splits * B * Hq;
    return p;
}

// Workspace: every partial row's D sums, then every row's (maximum, sum).
inline int64_t attn_workspace(const AttnPlan& p, int D) { return (p.prefix_parts + p.own_parts) * (D + 2) * 4; }

// A workspace that serves every call of no larger B, prefix_len and max_len.  A plan's own
// is no such thing: a longer max_len leaves the prefix fewer CUs, and ranges are rounded up
// to whole steps, so that one sequence of 32 heads on 8 takes 1 064 960 bytes at 8192 tokens
// and 549 120 at 8193.  From the rules of attn_plan and cut:
//   own tokens, u = units of a sequence: a sequence has at most ceil(max_len / 128) ranges,
//   and B sequences together ceil(512 / (B u)) B <= 512 / u + B while B u < 256, or B times
//   the ranges of at most 4096 tokens (64; kMaxBlocks units in all);
//   prefix: at most ceil(prefix_len / 128) ranges of heads * B G rows, and `blocks` blocks of
//   at most 16 mt waves rows, beside one more range of every row for rounding up.
inline int64_t attn_workspace_bound(int64_t B, int Hq, int heads, int D, int format, int64_t prefix_len, int64_t max_len)
{
    if (prefix_len == 0 && max_len <= 512)
        return 0;
    const auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
    const auto most = [](int64_t a, int64_t b) { return a > b ? a : b; };
    const int64_t grain = kWaves * kStep, G = Hq / heads, rows = B * G, u = heads * ceil_div(G, 16);
    const int64_t even = most(1, least(kMaxRanges, ceil_div(max_len, 4096)));
    int64_t own = least(B * even, most(B, kMaxBlocks / u));
    if (u < kCus)
        own = most(own, 2 * kCus / u + least(B, (kCus - 1) / u));
    own = least(own, B * ceil_div(max_len, grain)) * Hq;
    const int64_t narrow = D == 256 ? 16 : 32;          // rows of a prefix unit's wave
    int64_t prefix = (format == NM_KV_MX4 ? 2 * kCus : kCus) * least(rows, narrow);
    if (rows > narrow && D != 256)
        prefix = most(prefix, 2 * kCus * least(rows, 4 * narrow));
    if (rows > narrow)
        prefix = most(prefix, kCus * least(rows, 8 * narrow));
    prefix = least(prefix + rows * heads, rows * heads * ceil_div(prefix_len, grain));
    return (prefix + own) * (D + 2) * 4;
}

}  // namespace nma

namespace nmk {

// The kernel side of the calls of the same names, on checked arguments with
// work to do (rows > 0).
int qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t T, int Hq, int Hk, int D,
                 int dtype, const void* wq, const void* wk, float eps, const int32_t* positions,
                 const float* inv_freq, int rot, int interleaved, void* q_out, void* k_out, void* stream);
int kv_write(const nm_kv_cache& cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T,
             const int64_t* slots, void* stream);
int kv_read(const nm_kv_cache& cache, const int64_t* slots, int64_t T, void* k, void* v, void* stream);
int attn_decode(const nma::AttnPlan& plan, const void* q, int64_t q_stride, int64_t B, int Hq,
                const nm_kv_cache& cache, const int32_t* prefix_pages, int64_t prefix_len, const int32_t* page_table,
                int64_t table_stride, const int32_t* lens, int64_t max_len, float scale, void* o, float* lse,
                void* workspace, void* stream);

}  // namespace nmk

#endif  // NM_ATTN_H
