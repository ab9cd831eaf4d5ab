// nm_serve.h -- shared by the entry points of include/nmserve.h and their
// kernels: launch plans and the kernel-side declarations.  Host-only C++ (no HIP
// types), so that the checks and plans also build with a plain compiler.
#ifndef NM_SERVE_H
#define NM_SERVE_H

#include <cstdint>

#include "nm_attn.h"
#include "nmserve.h"

namespace nms {

using nma::ceil_div;

// ---- nm_kv_plan -----------------------------------------------------------------
constexpr int kPlanThreads = 1024;              // of the deciding block
constexpr int64_t kPlanRows = 8192;             // most rows that it deals with itself

constexpr int64_t plan_scratch(int64_t B) { return (B + 2) / 2 * 8; }       // B + 1 int32, in whole 8 bytes

// ---- nm_attn_prompt -----------------------------------------------------------
//
// Work is cut into tiles of kPromptRows rows, a row being one query head of one query of
// a sequence and key head (row r: query r / G, head r % G).  Lengths are on the
// device, so the grid has room for every way of cutting T queries into B sequences:
// sequence b's tiles are numbers from starts[b] G / kPromptRows + b on (rounded down), which
// leaves each at least as many as it needs.
constexpr int kPromptWave = 32;                 // rows of a wave
// Waves of a block: two blocks of four share a CU and do not wait for each other.  One of
// eight stages keys and values once for twice the rows, but its waves go in step and its
// tiles are coarser (us with four / eight: 16 prompts of up to 1024 tokens 106 / 116, one of
// 2048 61 / 69, one of 8192 on 64 heads 1165 / 1120; before the products were made to overlap).
constexpr int kPromptWaves = 4;
constexpr int kPromptRows = kPromptWave * kPromptWaves;
constexpr int64_t kPromptMaxStride = int64_t(1) << 28;
constexpr int64_t kPromptMaxRows = (int64_t(1) << 31) - (int64_t(1) << 16);     // T * G, and Tk
constexpr int64_t kPromptMaxHeads = int64_t(1) << 30;                           // B * heads

struct PromptPlan {
    int G;
    int64_t tiles;                              // per key head, most that may be needed
    int64_t splits;                             // ranges of each tile's keys, joined by a second launch
};

// Few rows behind many keys leave most of the GPU idle: their keys are cut into ranges (each
// tile's own into equal ones, on the device).  A tile of 64 keys takes a lone block about 1 us,
// the second launch about 6, and partial results go through memory at about 4.5 TB/s both ways
// together (16 queries behind 16384 tokens, 32 heads on 8 of 128 columns: 283 us in one range,
// 27.5 in 32).  On the host only the average of the keys is known, so that one long sequence among
// many short ones is not cut (32 sequences of a query, one of 16384 keys and 31 of 16: 278 us, 28
// for the long one alone; one of 131072 among 64: 2270 and 126).
constexpr int64_t kPromptKeys = 64;             // of a tile of keys
constexpr int64_t kPromptRanges = 64, kPromptBlocks = 512;

inline PromptPlan prompt_plan(int64_t T, int64_t Tk, int64_t B, int Hq, int heads, int D)
{
    PromptPlan p;
    p.G = Hq / heads;
    p.tiles = T * p.G / kPromptRows + B;
    p.splits = 1;
    const int64_t blocks = p.tiles * heads, keys = B > 0 ? Tk / B / kPromptKeys : 0;
    double best = (double)keys;
    for (int64_t s = 2; s <= kPromptRanges && s * blocks <= kPromptBlocks && 2 * s <= keys; s *= 2) {
        const double bytes = (double)(s * blocks * kPromptRows) * (D + 4) * 8;
        const double t = (double)keys / (double)s + 6.0 + bytes / 4.5e6;
        if (t < best) {
            best = t;
            p.splits = s;
        }
    }
    return p;
}

// Workspace: every partial row's (reference, sums), then its D sums.
inline int64_t prompt_workspace(const PromptPlan& p, int heads, int D)
{
    return p.splits > 1 ? p.splits * p.tiles * heads * kPromptRows * (D + 4) * 4 : 0;
}

// For every call of no larger T, Tk and B: ranges there are only while all blocks are no more
// than kPromptBlocks and a sequence has 4 tiles of keys.
inline int64_t prompt_workspace_bound(int64_t T, int64_t Tk, int64_t B, int Hq, int heads, int D)
{
    const int64_t blocks = (T * (Hq / heads) / kPromptRows + B) * heads;
    if (Tk < 4 * kPromptKeys || B == 0)
        return 0;
    return (blocks * kPromptRanges < kPromptBlocks ? blocks * kPromptRanges : kPromptBlocks) * kPromptRows * (D + 4) * 4;
}

// ---- nm_attn_tree ----------------------------------------------------------------
//
// Units of (rows of a sequence and key head, range of its tokens), one block each, in two
// forms (nmtree.hip).
constexpr int kTreeWaves = 4;
// Tokens of a range at most.  Shorter ones would share out sequences of different lengths better, but each costs
// a block's start and a partial result (us with 1024 / 2048 / 4096, 32 heads on 8 of 128 columns: 16 sequences of 24
// drafts and up to 8192 tokens, MX8 104.5 / 103.5 / 102.7, all of 8192 122.5 / 116.1 / 114.0; 8 of 8 drafts, up to 32768,
// MX4 81.4 / 71.6 / 67.2; 4 of 64 drafts, 16384 tokens, 16-bit 138.5 / 123.6 / 124.0; 64 heads, 64 drafts behind 131071,
// MX4 427 / 427 / 408; slower only where there are many: 48 of 24 drafts, up to 8192, 16-bit 239.8 / 239.1 / 259.0).
constexpr int64_t kTreeRange = 4096;

// Blocks that fill the GPU: two a CU, but one where a block of the shared form takes a CU's registers and
// LDS (256 columns), and one where the plain form has enough units without ranges to give each CU one.
inline int64_t tree_blocks(bool shared, int D, int64_t units)
{
    return shared && D == 256 ? nma::kCus : shared || units < nma::kCus ? 2 * nma::kCus : nma::kCus;
}

struct TreePlan {
    int64_t rows;                               // of a sequence and key head: N * G
    bool shared;                                // the form that shares the cache through LDS
    int mt;                                     // else: 16 mt rows
    int waves;                                  // shared: row groups of 32 in a block (1, 2 or 4)
    int64_t groups, splits, chunk;              // units of the rows, ranges of the tokens
    bool direct;                                // one range: units write o
    int64_t parts;                              // partial rows
};

// Row groups of 32 in a block of the shared form: with two (four waves, two on the same rows) blocks that
// hold four would leave half their waves without rows (64 rows, 8 sequences of 4096 tokens, us with two / four:
// 16-bit 34.5 / 38.2, MX8 31.5 / 39.9).
inline int tree_waves(int64_t rows) { return rows <= 32 ? 1 : rows <= 64 ? 2 : 4; }

// Whether the cache is shared through LDS.  The plain form reads it once for every 32 rows, and
// converts it as often, but has no barriers and a block has less before and behind its loop.  It is taken for
// 32 rows and for little work in all (us plain / shared; 128 columns, 8 key heads: 32 rows, 8 sequences of 4096
// tokens, 16-bit 30.3 / 31.3, MX8 21.8 / 27.7; MX8, 128 rows, 16 of 1024 23.0 / 36.3, 8 of 4096 41.7 / 47.6, 48 of
// 4096 265 / 197; 72 rows, 4 of 4096 26.8 / 31.3, 8 of 4096 44.5 / 41.6; 64 rows, 8 of 4096 29.9 / 31.5, 8 of
// 8192 45.0 / 44.3; 16-bit, 64 rows, 1 of 16384 24.2 / 26.3, 8 of 4096 39.0 / 34.5, 72 rows, 4 of 4096 32.4 / 30.7).
inline bool tree_shared(int64_t rows, int64_t tokens, int D, int format)
{
    return D == 256 || (rows > 32 && rows * tokens > (format == NM_KV_16 ? int64_t(1) << 23 : int64_t(1) << 24));
}

inline TreePlan tree_plan(int64_t B, int N, int Hq, int heads, int D, int format, int64_t max_len)
{
    TreePlan p;
    p.rows = (int64_t)N * (Hq / heads);
    p.shared = tree_shared(p.rows, B * heads * max_len, D, format);
    p.mt = p.rows <= 16 ? 1 : 2;
    p.waves = tree_waves(p.rows);
    p.groups = ceil_div(p.rows, p.shared ? 32 * p.waves : 16 * p.mt);
    const int64_t units = B * heads * p.groups;
    // Few tokens are one range: a second launch costs more than it spreads (8 key heads of 128
    // columns, 16-bit, us in one range / ranges of 128: one sequence of 32 rows, 256 tokens 8.5 / 10.4,
    // 512 10.3 / 10.5, 1024 14.0 / 10.6; shared, four of 128 rows, 256 tokens 17.0 / 18.6, 512 22.9 / 21.2).
    const int64_t blocks = max_len <= (p.shared ? 256 : 512) ? 1 : tree_blocks(p.shared, D, units);
    nma::cut(max_len, units, blocks, kTreeRange, &p.splits, &p.chunk);
    p.direct = p.splits <= 1;
    if (p.direct)
        p.splits = 1;
    p.parts = p.direct ? 0 : p.splits * B * N * Hq;
    return p;
}

inline int64_t tree_workspace(const TreePlan& p, int D) { return p.parts * (D + 2) * 4; }

// A workspace that serves every call of no larger B and max_len (and the same N).  Up to 256
// tokens no plan has ranges.  Else a sequence has at most ceil(max_len / 128) of them, and
// all sequences together at most 512 / u + B while they have fewer than 512 units (u of a
// sequence); with more units a sequence has one range, and so no partial results, unless
// tokens pass kTreeRange: then B times the ranges of so many (nma::cut).  The plain form has
// no fewer units than the shared.
inline int64_t tree_workspace_bound(int64_t B, int N, int Hq, int heads, int D, int64_t max_len)
{
    const auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
    const auto most = [](int64_t a, int64_t b) { return a > b ? a : b; };
    const int64_t grain = nma::kWaves * nma::kStep, rows = (int64_t)N * (Hq / heads);
    const int64_t u = heads * ceil_div(rows, 32 * tree_waves(rows));
    if (max_len <= 256)
        return 0;
    const int64_t even = least(nma::kMaxRanges, ceil_div(max_len, kTreeRange));
    int64_t ranges = even > 1 ? least(B * even, nma::kMaxBlocks / u) : 0;
    if (u < 2 * nma::kCus)
        ranges = most(ranges, 2 * nma::kCus / u + least(B, (2 * nma::kCus - 1) / u));
    ranges = least(ranges, B * ceil_div(max_len, grain));
    return ranges * N * Hq * (D + 2) * 4;
}

}  // namespace nms

namespace nmk {

// The kernel side of the calls of the same names, on checked arguments with
// work to do.
int kv_plan(const nm_kv_pages& pages, const int32_t* adds, int64_t rows, int32_t* starts, int64_t* slots,
            int32_t* positions, int32_t* granted, void* stream);

int attn_prompt(const nms::PromptPlan& plan, const void* q, int64_t q_stride, int64_t T, const void* k, int64_t k_stride,
                const void* v, int64_t v_stride, int64_t Tk, const int32_t* starts, const int32_t* k_starts, int64_t B,
                int Hq, int heads, int D, int dtype, float scale, void* o, float* lse, void* workspace, void* stream);
int attn_tree(const nms::TreePlan& plan, const void* q, int64_t q_stride, int64_t B, int N, int Hq,
              const nm_kv_cache& cache, const uint64_t* visible, const int32_t* page_table, int64_t table_stride,
              const int32_t* lens, int64_t max_len, float scale, void* o, float* lse, void* workspace, void* stream);

}  // namespace nmk

#endif  // NM_SERVE_H
