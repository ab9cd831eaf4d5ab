// serve_checks.cpp -- host code behind include/nmserve.h under sanitizers: the
// launch plans (ranges cover every token once, grids fit, what the *_bytes calls
// give holds every smaller call's partial rows), and the entry points' checks on
// random calls, linked with a stand-in for the kernel side that checks what
// nm_serve.h promises it.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "nm_serve.h"

namespace {

long g_launches[3] = {0, 0, 0};

void promise(bool ok, const char* what)
{
    if (!ok) {
        std::fprintf(stderr, "broken: %s\n", what);
        std::abort();
    }
}

bool al(const void* p, uintptr_t a) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0; }

using Wide = unsigned __int128;

struct Buf {
    const void* p;
    Wide n;
};

bool apart(Buf a, Buf b)
{
    if (!a.n || !b.n || !a.p || !b.p)
        return true;
    const Wide a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 + a.n <= b0 || b0 + b.n <= a0;
}

Wide strided(int64_t rows, int64_t stride, int64_t width)
{
    return rows <= 0 ? 0 : (Wide)((rows - 1) * (__int128)(rows > 1 ? stride : 0) + width) * 2;
}

void all_apart(const std::vector<Buf>& outs, const std::vector<Buf>& ins)
{
    for (size_t i = 0; i < outs.size(); ++i) {
        for (const Buf& b : ins)
            promise(apart(outs[i], b), "an output overlaps an input");
        for (size_t j = i + 1; j < outs.size(); ++j)
            promise(apart(outs[i], outs[j]), "two outputs overlap");
    }
}

bool power(int64_t x) { return x == 16 || x == 32 || x == 64 || x == 128 || x == 256; }

}  // namespace

namespace nmk {

int kv_plan(const nm_kv_pages& p, const int32_t* adds, int64_t rows, int32_t* starts, int64_t* slots, int32_t* positions,
            int32_t* granted, void*)
{
    promise(p.B >= 1 && p.B <= 65535 && p.width >= 1 && p.width <= (1 << 24) && p.B * p.width <= INT32_MAX, "book");
    promise(p.n_pages >= 1 && p.n_pages <= INT32_MAX && power(p.page_size) && rows >= 0 && rows <= INT32_MAX, "book sizes");
    promise(al(p.table, 4) && al(p.lens, 4) && al(p.free, 4) && al(p.n_free, 4) && al(p.scratch, 8) && al(adds, 4) &&
            al(starts, 4) && al(granted, 4), "book pointers");
    promise(rows == 0 || (al(slots, 8) && al(positions, 4)), "rows");
    promise(nm_kv_plan_scratch_bytes(p.B) >= (p.B + 1) * 4, "scratch");
    all_apart({{p.table, (Wide)(p.B * p.width) * 4}, {p.lens, (Wide)p.B * 4}, {p.free, (Wide)p.n_pages * 4}, {p.n_free, 4},
               {p.scratch, (Wide)nm_kv_plan_scratch_bytes(p.B)}, {starts, (Wide)(p.B + 1) * 4}, {slots, (Wide)rows * 8},
               {positions, (Wide)rows * 4}, {granted, (Wide)p.B * 4}}, {{adds, (Wide)p.B * 4}});
    ++g_launches[0];
    return NM_ERR_HIP;
}

int attn_prompt(const nms::PromptPlan& plan, const void* q, int64_t qs, int64_t T, const void* k, int64_t ks,
                const void* v, int64_t vs, int64_t Tk, const int32_t* starts, const int32_t* k_starts, int64_t B, int Hq,
                int heads, int D, int dtype, float scale, void* o, float* lse, void* ws, void*)
{
    const int64_t qw = (int64_t)Hq * D, kw = (int64_t)heads * D;
    promise(T >= 1 && B >= 1 && B <= 65535 && Tk >= 0 && heads >= 1 && Hq % heads == 0, "prompt shape");
    promise((D == 64 || D == 128 || D == 256) && (dtype == 0 || dtype == 1) && std::isfinite(scale), "prompt type");
    promise(T * plan.G < nms::kPromptMaxRows && Tk < nms::kPromptMaxRows, "rows and keys are counted in int32");
    promise(al(q, 16) && al(o, 16) && al(starts, 4) && al(k_starts, 4) && (!lse || al(lse, 4)), "prompt pointers");
    promise(Tk == 0 || (al(k, 16) && al(v, 16)), "keys");
    promise(T == 1 || (qs >= qw && qs % 8 == 0), "q stride");
    promise(Tk <= 1 || (ks >= kw && vs >= kw && ks % 8 == 0 && vs % 8 == 0 && std::max(ks, vs) * 2 * 7 <= UINT32_MAX), "k stride");
    const int64_t need = nms::prompt_workspace(plan, heads, D);
    promise(need == 0 || al(ws, 256), "prompt workspace");
    all_apart({{o, (Wide)T * qw * 2}, {lse, lse ? (Wide)T * Hq * 4 : 0}, {need ? ws : nullptr, (Wide)need}},
              {{q, strided(T, qs, qw)}, {k, strided(Tk, ks, kw)}, {v, strided(Tk, vs, kw)}, {starts, (Wide)(B + 1) * 4},
               {k_starts, (Wide)(B + 1) * 4}});
    ++g_launches[1];
    return NM_ERR_HIP;
}

int attn_tree(const nms::TreePlan& plan, const void* q, int64_t qs, int64_t B, int N, int Hq, const nm_kv_cache& c,
              const uint64_t* visible, const int32_t* table, int64_t ts, const int32_t* lens, int64_t ml, float scale,
              void* o, float* lse, void* ws, void*)
{
    const int64_t w = (int64_t)Hq * c.D, pages = (ml + c.page_size - 1) / c.page_size;
    promise(B >= 1 && B <= 65535 && N >= 1 && N <= 64 && c.heads >= 1 && Hq % c.heads == 0 && power(c.page_size), "tree shape");
    promise(ml >= 0 && ml <= (1 << 30) && std::isfinite(scale) && (c.D == 64 || c.D == 128 || c.D == 256), "tree type");
    promise(al(q, 16) && al(o, 16) && al(lens, 4) && al(visible, 8) && (!lse || al(lse, 4)), "tree pointers");
    promise(B * N == 1 || (qs >= w && qs % 8 == 0), "tree stride");
    promise(ml == 0 || (al(table, 4) && (B == 1 || ts >= pages)), "table");
    const int64_t need = nms::tree_workspace(plan, c.D);
    promise(need == 0 || al(ws, 256), "tree workspace");
    const Wide elems = (Wide)c.n_pages * c.page_size * c.heads * c.D;
    const Wide bytes = c.format == 0 ? elems * 2 : c.format == 1 ? elems : elems / 2, sb = c.format ? elems / 32 : 0;
    all_apart({{o, (Wide)(B * N) * w * 2}, {lse, lse ? (Wide)(B * N) * Hq * 4 : 0}, {need ? ws : nullptr, (Wide)need}},
              {{c.k, bytes}, {c.v, bytes}, {c.k_scale, sb}, {c.v_scale, sb}, {q, strided(B * N, qs, w)},
               {visible, (Wide)(B * N) * 8}, {lens, (Wide)B * 4},
               {table, ml ? (Wide)((B - 1) * (__int128)(B > 1 ? ts : 0) + pages) * 4 : 0}});
    ++g_launches[2];
    return NM_ERR_HIP;
}

// The calls of nmattn.h, which nothing here makes.
int qk_norm_rope(const void*, int64_t, const void*, int64_t, int64_t, int, int, int, int, const void*, const void*, float,
                 const int32_t*, const float*, int, int, void*, void*, void*) { std::abort(); }
int kv_write(const nm_kv_cache&, const void*, int64_t, const void*, int64_t, int64_t, const int64_t*, void*) { std::abort(); }
int kv_read(const nm_kv_cache&, const int64_t*, int64_t, void*, void*, void*) { std::abort(); }
int attn_decode(const nma::AttnPlan&, const void*, int64_t, int64_t, int, const nm_kv_cache&, const int32_t*, int64_t,
                const int32_t*, int64_t, const int32_t*, int64_t, float, void*, float*, void*, void*) { std::abort(); }

}  // namespace nmk

namespace {

std::mt19937_64 rng(17);
int64_t pick(std::initializer_list<int64_t> v) { return *(v.begin() + rng() % v.size()); }

// least .. top, spread over its logarithm, with the edges of the plans' rules among them.
int64_t size(int64_t least, int64_t top)
{
    static const int64_t edges[] = {0, 1, 2, 31, 32, 33, 64, 127, 128, 129, 255, 256, 257, 512, 513, 4096, 4097, 8192, 8193};
    const int64_t v = rng() % 3 == 0 ? edges[rng() % 19]
                                     : (int64_t)std::exp2(std::log2((double)std::max<int64_t>(top, 1)) * (double)(rng() % 100001) / 1e5);
    return std::min(std::max(v, least), top);
}

long prompts(long n)
{
    long checked = 0, ranges = 0;
    for (long i = 0; i < n; ++i) {
        const int heads = (int)size(1, i % 8 ? 64 : 65535), G = (int)size(1, i % 8 ? 64 : 65535 / heads), D = 64 << rng() % 3;
        const int64_t Hq = (int64_t)heads * G;
        const int64_t T = size(1, std::min((nms::kPromptMaxRows - 1) / G, ((int64_t(1) << 40) - 1) / (Hq * D)));
        const int64_t Tk = size(0, std::min(nms::kPromptMaxRows - 1, ((int64_t(1) << 40) - 1) / ((int64_t)heads * D)));
        const int64_t B = size(1, std::min<int64_t>(65535, (nms::kPromptMaxHeads - 1) / heads));
        const int64_t bound = nm_attn_prompt_workspace_bytes(T, Tk, B, (int)Hq, heads, D);
        promise(bound >= 0 && bound < (int64_t(1) << 40), "a size for every shape in the limits");
        for (int j = 0; j < 8; ++j) {
            const int64_t t = j & 1 ? size(1, T) : T, tk = j & 2 ? size(0, Tk) : Tk, b = j & 4 ? size(1, B) : B;
            const nms::PromptPlan p = nms::prompt_plan(t, tk, b, (int)Hq, heads, D);
            promise(p.splits >= 1 && p.splits <= nms::kPromptRanges, "prompt ranges");
            promise(p.splits == 1 || p.tiles * heads * p.splits <= nms::kPromptBlocks, "ranges of few rows only");
            promise(p.tiles * heads * p.splits <= INT32_MAX, "prompt grid");
            promise(p.tiles * nms::kPromptRows >= t * p.G, "tiles for every row");
            promise(nms::prompt_workspace(p, heads, D) <= bound, "prompt workspace of a smaller call");
            promise(nms::prompt_workspace_bound(t, tk, b, (int)Hq, heads, D) <= bound, "prompt sizes grow");
            ranges += p.splits > 1;
            ++checked;
        }
        // Any way of cutting T queries into B sequences: the tiles of each lie behind those of the one before.
        if (B <= 64) {
            std::vector<int64_t> at(B + 1, T);
            for (int64_t b = 0; b < B; ++b)
                at[b] = (int64_t)(rng() % (uint64_t)(T + 1));
            std::sort(at.begin(), at.end());
            at[0] = std::min<int64_t>(at[0], 7);
            const int64_t tiles = nms::prompt_plan(T, Tk, B, (int)Hq, heads, D).tiles;
            for (int64_t b = 0; b < B; ++b) {
                const int64_t first = at[b] * G / nms::kPromptRows + b, rows = (at[b + 1] - at[b]) * G;
                const int64_t next = b + 1 < B ? at[b + 1] * G / nms::kPromptRows + b + 1 : tiles;
                promise(first + (rows + nms::kPromptRows - 1) / nms::kPromptRows <= next, "room for a sequence's tiles");
            }
        }
    }
    promise(ranges > n / 100, "ranges are among the plans");
    return checked;
}

long trees(long n)
{
    long checked = 0, joined = 0;
    for (long i = 0; i < n; ++i) {
        const int heads = (int)size(1, i % 8 ? 64 : 65535), G = (int)size(1, i % 8 ? 64 : 65535 / heads), D = 64 << rng() % 3;
        const int64_t Hq = (int64_t)heads * G, most = nma::kMaxRows - 1;
        const int N = (int)size(1, std::min<int64_t>(64, most / Hq));
        const int64_t B = size(1, std::min<int64_t>(65535, most / (N * Hq)));
        const int64_t ml = size(0, nma::kMaxTokens);
        const int64_t bound = nm_attn_tree_workspace_bytes(B, N, (int)Hq, heads, D, (int)(i % 3), ml);
        promise(bound >= 0 && bound < (int64_t(1) << 46), "a size for every tree in the limits");
        for (int j = 0; j < 4; ++j) {
            const int64_t b = j & 1 ? size(1, B) : B, m = j & 2 ? size(0, ml) : ml;
            const nms::TreePlan p = nms::tree_plan(b, N, (int)Hq, heads, D, (int)(i % 3), m);
            promise(p.chunk > 0 && p.chunk % nma::kStep == 0 && p.splits * p.chunk >= m && (p.splits - 1) * p.chunk <= m,
                    "tree ranges");
            promise(p.splits * p.chunk <= int64_t(1) << 31, "tokens are counted in int32");
            promise(p.shared || p.mt * 16 * p.groups >= p.rows, "rows of the plain form");
            promise(!p.shared || p.waves * 32 * p.groups >= p.rows, "rows of the shared form");
            promise(p.direct ? p.splits == 1 && p.parts == 0 : p.parts == p.splits * b * N * Hq, "partial rows");
            promise(nma::ceil_div(p.splits * b * heads, 8) * 8 * p.groups <= INT32_MAX, "tree grid");
            promise(nma::ceil_div(b * p.rows, 16) * heads * (D / 16) <= INT32_MAX &&
                    b * heads * nma::ceil_div(p.rows, 32) * (D / 8) <= INT32_MAX, "tree join grids");
            promise(nms::tree_workspace(p, D) <= bound, "tree workspace of a smaller call");
            promise(nms::tree_workspace_bound(b, N, (int)Hq, heads, D, m) <= bound, "tree sizes grow");
            joined += !p.direct;
            ++checked;
        }
    }
    promise(joined > n / 100, "joined plans are among them");
    return checked;
}

void fuzz(long calls)
{
    char* const base = reinterpret_cast<char*>(uintptr_t(1) << 40);
    const auto ptr = [&]() -> char* {
        if (rng() % 80 == 0)
            return nullptr;
        return base + (rng() % 64) * (1 << 20) + (rng() % 10 ? 0 : pick({256, 16, 8, 4, 2, 1}));
    };
    const auto i32 = [&]() { return reinterpret_cast<int32_t*>(ptr()); };
    long ok = 0;
    for (long i = 0; i < calls; ++i) {
        const int64_t s1 = pick({64, 128, 256, 512, 12, 0, -8, INT64_MAX, int64_t(1) << 28, (int64_t(1) << 28) + 8});
        const int64_t s2 = pick({64, 128, 256, 1024, int64_t(1) << 28});
        const int64_t room = pick({0, 100, 4096, 1 << 20, -5, INT64_MAX >> 20});
        const float scale = rng() % 20 ? 0.5f : INFINITY;
        int st = 0;
        switch (rng() % 3) {
        case 0: {
            const nm_kv_pages p = {i32(), i32(), i32(), i32(), ptr(), pick({1, 2, 3, 64, 1000, 65535, 0, -1, 65536}),
                                   pick({1, 2, 9, 1 << 15, 1 << 24, 0, -1, INT64_MAX}), pick({1, 5, 1 << 12, INT32_MAX, 0, int64_t(1) << 31}),
                                   (int)pick({16, 32, 256, 64, 0, 24, 512, -16})};
            st = nm_kv_plan(rng() % 50 ? &p : nullptr, i32(), pick({0, 1, 7, 4096, INT32_MAX, -1, int64_t(1) << 31}), i32(),
                            reinterpret_cast<int64_t*>(ptr()), i32(), i32(), nullptr);
            break;
        }
        case 1: {
            const int64_t T = pick({0, 1, 2, 3, 5, 500, -1, INT32_MAX, int64_t(1) << 31, INT64_MIN, INT64_MAX});
            st = nm_attn_prompt(ptr(), s1, T, ptr(), s2, ptr(), pick({64, 128, 512, 1024}),
                                rng() % 2 ? T : pick({0, 1, 9, 2000, 5000, INT32_MAX, -1, INT64_MAX}), i32(), rng() % 2 ? i32() : nullptr,
                                pick({0, 1, 1, 2, 3, 65535, 65536, -1}), (int)pick({1, 2, 4, 3, 0, -2, 65535}), (int)pick({1, 1, 2, 0, -1, 65535}),
                                (int)pick({64, 64, 128, 256, 96, 0}), (int)pick({0, 1, 0, 1, 2}), scale, ptr(),
                                rng() % 2 ? reinterpret_cast<float*>(ptr()) : nullptr, ptr(), room, nullptr);
            break;
        }
        default: {
            nm_kv_cache c;
            c.k = ptr();
            c.v = ptr();
            c.k_scale = reinterpret_cast<uint8_t*>(ptr());
            c.v_scale = reinterpret_cast<uint8_t*>(ptr());
            c.n_pages = pick({1, 2, 2, 3, 5, 0, INT32_MAX, int64_t(1) << 40});
            c.page_size = (int)pick({16, 16, 32, 64, 256, 15, 0});
            c.heads = (int)pick({1, 1, 2, 2, 0, 65535, -1});
            c.D = (int)pick({64, 64, 128, 256, 96});
            c.dtype = (int)pick({0, 1, 0, 1, 2});
            c.format = (int)pick({0, 1, 2, 2, 3, -1});
            st = nm_attn_tree(ptr(), s1, pick({1, 1, 2, 3, 0, 65535, 65536, -1}), (int)pick({1, 4, 8, 64, 0, 65, -1}),
                              (int)pick({1, 2, 4, 3, 0, -2, 65535}), rng() % 50 ? &c : nullptr, reinterpret_cast<uint64_t*>(ptr()),
                              i32(), pick({0, 1, 4, 100, -1, INT64_MAX}), i32(), pick({0, 1, 33, 500, 5000, -1, INT64_MAX}), scale,
                              ptr(), rng() % 2 ? reinterpret_cast<float*>(ptr()) : nullptr, ptr(), room, nullptr);
        }
        }
        promise(st >= NM_OK && st <= NM_ERR_HIP, "status");
        ok += st == NM_OK;
    }
    std::printf("calls %ld, empty %ld, launches %ld %ld %ld\n", calls, ok, g_launches[0], g_launches[1], g_launches[2]);
    promise(g_launches[0] > 0 && g_launches[1] > 0 && g_launches[2] > 0 && ok > 0, "the random calls reach the kernels");
}

}  // namespace

int main(int argc, char** argv)
{
    const long n = argc > 1 ? std::atol(argv[1]) : 200000;
    std::printf("prompt plans checked %ld\n", prompts(n));
    std::printf("tree plans checked %ld\n", trees(n));
    fuzz(10 * n);
    return 0;
}
