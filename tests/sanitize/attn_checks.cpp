// attn_checks.cpp -- host code behind include/nmattn.h under sanitizers: the
// cache's byte layout (every element has bytes of its own, inside its tile),
// the launch plans of nm_attn_decode (ranges cover every token once, partial
// rows fit the workspace, grids fit), and the entry points' checks on random
// calls, linked with a stand-in for the kernel side that checks what nm_attn.h
// promises it.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "nm_attn.h"

namespace {

long g_launches = 0;

void promise(bool ok, const char* what)
{
    if (!ok) {
        std::fprintf(stderr, "broken: %s\n", what);
        std::abort();
    }
}

bool al(const void* p, uintptr_t a) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Buf {
    const void* p;
    unsigned __int128 n;
};

bool apart(Buf a, Buf b)
{
    if (!a.n || !b.n || !a.p || !b.p)
        return true;
    const unsigned __int128 a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 + a.n <= b0 || b0 + b.n <= a0;
}

unsigned __int128 strided(int64_t rows, int64_t stride, int64_t width)
{
    return rows <= 0 ? 0 : (unsigned __int128)((rows - 1) * (__int128)(rows > 1 ? stride : 0) + width) * 2;
}

std::vector<Buf> cache_ok(const nm_kv_cache& c)
{
    promise(c.page_size == 16 || c.page_size == 32 || c.page_size == 64 || c.page_size == 128 || c.page_size == 256, "page");
    promise(c.D == 64 || c.D == 128 || c.D == 256, "D");
    promise(c.n_pages >= 1 && c.n_pages <= INT32_MAX && c.heads >= 1 && c.heads <= 65535, "cache size");
    promise(c.dtype == 0 || c.dtype == 1, "dtype");
    promise(c.format >= 0 && c.format <= 2, "format");
    const unsigned __int128 elems = (unsigned __int128)c.n_pages * c.page_size * c.heads * c.D;
    const unsigned __int128 bytes = c.format == 0 ? elems * 2 : c.format == 1 ? elems : elems / 2;
    promise(bytes < ((unsigned __int128)1 << 46), "bytes");
    promise(al(c.k, 16) && al(c.v, 16), "cache pointers");
    if (c.format)
        promise(al(c.k_scale, 16) && al(c.v_scale, 16), "scale pointers");
    const unsigned __int128 sb = c.format ? elems / 32 : 0;
    return {{c.k, bytes}, {c.v, bytes}, {c.k_scale, sb}, {c.v_scale, sb}};
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

}  // namespace

namespace nmk {

int qk_norm_rope(const void* q, int64_t qs, const void* k, int64_t ks, int64_t T, int Hq, int Hk, int D, int dtype,
                 const void* wq, const void* wk, float eps, const int32_t* pos, const float* f, int rot, int, void* qo,
                 void* ko, void*)
{
    promise(T > 0 && T <= INT32_MAX && Hq >= 0 && Hk >= 0 && Hq + Hk > 0 && D >= 8 && D <= 512 && D % 8 == 0, "qk shape");
    promise(dtype == 0 || dtype == 1, "qk dtype");
    promise(rot >= 0 && rot <= D && rot % 16 == 0 && eps >= 0 && std::isfinite(eps), "qk rot, eps");
    const int64_t qw = (int64_t)Hq * D, kw = (int64_t)Hk * D;
    promise((!Hq || (al(q, 16) && al(qo, 16))) && (!Hk || (al(k, 16) && al(ko, 16))), "qk rows");
    promise(T == 1 || ((!Hq || (qs >= qw && qs % 8 == 0)) && (!Hk || (ks >= kw && ks % 8 == 0))), "qk strides");
    promise(rot == 0 || (al(pos, 4) && al(f, 4)), "positions");
    const Buf bq = {q, Hq ? strided(T, qs, qw) : 0}, bk = {k, Hk ? strided(T, ks, kw) : 0};
    const Buf oq = {qo, (unsigned __int128)T * qw * 2}, ok = {ko, (unsigned __int128)T * kw * 2};
    all_apart({oq, ok}, {{wq, (unsigned __int128)D * 2}, {wk, (unsigned __int128)D * 2},
                         {pos, rot ? (unsigned __int128)T * 4 : 0}, {f, (unsigned __int128)rot * 2}});
    promise((qo == q && (T == 1 || qs == qw)) || apart(oq, bq), "q_out on q");
    promise((ko == k && (T == 1 || ks == kw)) || apart(ok, bk), "k_out on k");
    promise(apart(oq, bk) && apart(ok, bq), "crossed outputs");
    ++g_launches;
    return NM_ERR_HIP;
}

int kv_write(const nm_kv_cache& c, const void* k, int64_t ks, const void* v, int64_t vs, int64_t T, const int64_t* slots,
             void*)
{
    const std::vector<Buf> outs = cache_ok(c);
    const int64_t w = (int64_t)c.heads * c.D;
    promise(T > 0 && T <= INT32_MAX && al(k, 16) && al(v, 16) && al(slots, 8), "write arguments");
    promise(T == 1 || (ks >= w && vs >= w && ks % 8 == 0 && vs % 8 == 0), "write strides");
    all_apart(outs, {{k, strided(T, ks, w)}, {v, strided(T, vs, w)}, {slots, (unsigned __int128)T * 8}});
    ++g_launches;
    return NM_ERR_HIP;
}

int kv_read(const nm_kv_cache& c, const int64_t* slots, int64_t T, void* k, void* v, void*)
{
    std::vector<Buf> ins = cache_ok(c);
    ins.push_back({slots, (unsigned __int128)T * 8});
    const unsigned __int128 n = (unsigned __int128)T * c.heads * c.D * 2;
    promise(T > 0 && T <= INT32_MAX && al(k, 16) && al(v, 16) && al(slots, 8), "read arguments");
    all_apart({{k, n}, {v, n}}, ins);
    ++g_launches;
    return NM_ERR_HIP;
}

int attn_decode(const nma::AttnPlan& p, const void* q, int64_t qs, int64_t B, int Hq, const nm_kv_cache& c,
                const int32_t* pp, int64_t P, const int32_t* table, int64_t ts, const int32_t* lens, int64_t ml,
                float scale, void* o, float* lse, void* ws, void*)
{
    std::vector<Buf> ins = cache_ok(c);
    promise(B >= 1 && B <= 65535 && Hq >= 1 && Hq % c.heads == 0, "attention shape");
    promise(P >= 0 && ml >= 0 && P <= (1 << 30) && ml <= (1 << 30) && std::isfinite(scale), "lengths");
    const int64_t w = (int64_t)Hq * c.D, pages = (ml + c.page_size - 1) / c.page_size;
    promise(al(q, 16) && al(o, 16) && al(lens, 4) && (!lse || al(lse, 4)), "attention pointers");
    promise(B == 1 || (qs >= w && qs % 8 == 0 && (ml == 0 || ts >= pages)), "attention strides");
    promise((P == 0 || al(pp, 4)) && (ml == 0 || al(table, 4)), "tables");
    const int64_t need = nma::attn_workspace(p, c.D);
    promise(need == 0 || (ws && reinterpret_cast<uintptr_t>(ws) % 256 == 0), "workspace");
    ins.push_back({q, strided(B, qs, w)});
    ins.push_back({pp, (unsigned __int128)((P + c.page_size - 1) / c.page_size) * 4});
    ins.push_back({table, ml ? (unsigned __int128)((B - 1) * (__int128)(B > 1 ? ts : 0) + pages) * 4 : 0});
    ins.push_back({lens, (unsigned __int128)B * 4});
    all_apart({{o, (unsigned __int128)B * w * 2}, {lse, lse ? (unsigned __int128)B * Hq * 4 : 0},
               {ws, (unsigned __int128)need}}, ins);
    ++g_launches;
    return NM_ERR_HIP;
}

}  // namespace nmk

namespace {

std::mt19937_64 rng(7);
int64_t pick(std::initializer_list<int64_t> v) { return *(v.begin() + rng() % v.size()); }

void layout()
{
    for (int bits : {16, 8, 4})
        for (int D : {64, 128, 256}) {
            const int nibbles = nma::tile_bytes(D, bits) * 2, per = bits / 4;
            std::vector<int> seen(nibbles, 0);
            for (int side = 0; side < 2; ++side) {
                std::fill(seen.begin(), seen.end(), 0);
                for (int t = 0; t < 16; ++t)
                    for (int d = 0; d < D; ++d) {
                        // keys are addressed by groups of eight columns, 4-bit values by pairs
                        const int step = side == 0 ? 8 : bits == 4 ? 2 : 1, d0 = d / step * step;
                        const int byte = side == 0 ? nma::k_offset(D, bits, t, d0) : nma::v_offset(D, bits, t, d0);
                        const int nib = byte * 2 + (d - d0) * per;
                        for (int i = 0; i < per; ++i) {
                            promise(nib + i >= 0 && nib + i < nibbles, "element outside its tile");
                            ++seen[nib + i];
                        }
                    }
                for (int n : seen)
                    promise(n == 1, "elements share bytes, or bytes are unused");
            }
            std::vector<int> scales(nma::scale_tile_bytes(D), 0), vscales(nma::scale_tile_bytes(D), 0);
            for (int t = 0; t < 16; ++t)
                for (int b = 0; b < D / 32; ++b) {
                    ++scales.at(nma::k_scale_offset(D, t, b));
                    ++vscales.at(nma::v_scale_offset(t, b));
                }
            for (size_t i = 0; i < scales.size(); ++i)
                promise(scales[i] == 1 && vscales[i] == 1, "scales share bytes");
        }
}

long plans()
{
    long n = 0;
    for (int64_t B : {1, 2, 7, 16, 33, 48, 500, 65535})
        for (int heads : {1, 2, 8, 16, 200})
            for (int G : {1, 3, 8, 16, 17, 64})
                for (int D : {64, 128, 256})
                    for (int64_t P : {int64_t(0), int64_t(1), int64_t(127), int64_t(129), int64_t(5000), int64_t(131071), int64_t(1) << 30})
                        for (int64_t ml : {int64_t(0), int64_t(1), int64_t(128), int64_t(777), int64_t(131072), int64_t(1) << 30}) {
                            const int64_t Hq = (int64_t)heads * G;
                            if (Hq > 65535 || B * Hq >= nma::kMaxRows)
                                continue;
                            const nma::AttnPlan p = nma::attn_plan(B, (int)Hq, heads, D, (int)(n % 3), P, ml);
                            const auto covers = [](int64_t splits, int64_t chunk, int64_t tokens) {
                                return chunk > 0 && chunk % nma::kStep == 0 && splits * chunk >= tokens &&
                                       (splits == 0 || (splits - 1) * chunk < tokens) && splits * chunk <= (int64_t(1) << 31);
                            };
                            promise(covers(p.prefix_splits, p.prefix_chunk, P), "prefix ranges");
                            promise(covers(p.own_splits, p.own_chunk, ml), "own ranges");
                            promise(p.prefix_groups * 16 * p.mt * (p.waves ? p.waves : 1) >= B * G && p.own_groups * 16 >= G, "row groups");
                            promise(p.direct == (P == 0 && p.own_splits <= 1), "direct");
                            if (!p.direct) {
                                promise(p.prefix_parts == p.prefix_splits * B * Hq, "prefix partial rows");
                                promise(p.own_parts == p.own_splits * B * Hq, "own partial rows");
                            }
                            promise(nma::attn_workspace(p, D) >= 0 && nma::attn_workspace(p, D) < (int64_t(1) << 46), "workspace size");
                            promise(p.prefix_groups * p.prefix_splits * heads <= INT32_MAX, "prefix grid");
                            promise(p.own_splits * p.own_groups * B * heads <= INT32_MAX, "own grid");
                            ++n;
                        }
    return n;
}

void fuzz(long calls)
{
    char* const base = reinterpret_cast<char*>(uintptr_t(1) << 40);
    const auto ptr = [&]() -> char* {
        if (rng() % 12 == 0)
            return nullptr;
        return base + (rng() % 40) * 4096 + pick({0, 0, 0, 0, 256, 16, 8, 4, 2, 1});
    };
    long ok = 0;
    for (long i = 0; i < calls; ++i) {
        nm_kv_cache c;
        c.k = ptr();
        c.v = ptr();
        c.k_scale = reinterpret_cast<uint8_t*>(ptr());
        c.v_scale = reinterpret_cast<uint8_t*>(ptr());
        c.n_pages = pick({1, 2, 2, 3, 0, -1, INT32_MAX, int64_t(1) << 40});
        c.page_size = (int)pick({16, 16, 16, 32, 64, 256, 15, 0, 512, -16});
        c.heads = (int)pick({1, 1, 2, 2, 0, 65535, 65536, -1});
        c.D = (int)pick({64, 64, 128, 256, 96, 0, -64});
        c.dtype = (int)pick({0, 1, 1, 2});
        c.format = (int)pick({0, 1, 2, 2, 3, -1});
        const int64_t T = pick({0, 1, 2, 3, 5, -1, INT32_MAX, int64_t(1) << 31, INT64_MIN, INT64_MAX});
        const int64_t s1 = pick({64, 128, 256, 512, 12, 0, -8, INT64_MAX, int64_t(1) << 30}), s2 = pick({64, 128, 256, 1024});
        int st = 0;
        switch (rng() % 4) {
        case 0:
            st = nm_kv_write(rng() % 50 ? &c : nullptr, ptr(), s1, ptr(), s2, T, reinterpret_cast<int64_t*>(ptr()), nullptr);
            break;
        case 1:
            st = nm_kv_read(rng() % 50 ? &c : nullptr, reinterpret_cast<int64_t*>(ptr()), T, ptr(), ptr(), nullptr);
            break;
        case 2: {
            char* q = ptr();
            char* k = ptr();
            st = nm_qk_norm_rope(q, s1, k, s2, T, (int)pick({0, 1, 2, 4, -1, 65535, 70000}), (int)pick({0, 1, 2, -1}),
                                 (int)pick({8, 64, 128, 512, 0, 12, 1024}), (int)pick({0, 1, 2}), ptr(), ptr(),
                                 (float)pick({0, 1, -1}), reinterpret_cast<int32_t*>(ptr()), reinterpret_cast<float*>(ptr()),
                                 (int)pick({0, 16, 64, 128, 8, -16}), (int)pick({0, 1}), rng() % 3 ? ptr() : q,
                                 rng() % 3 ? ptr() : k, nullptr);
            break;
        }
        default:
            st = nm_attn_decode(ptr(), s1, pick({1, 1, 2, 3, 0, 65536, -1}), (int)pick({1, 2, 4, 3, 0, -2, 65535}),
                                rng() % 50 ? &c : nullptr, reinterpret_cast<int32_t*>(ptr()),
                                pick({0, 0, 1, 40, 5000, -1, int64_t(1) << 31}), reinterpret_cast<int32_t*>(ptr()),
                                pick({0, 1, 4, 100, -1, INT64_MAX}), reinterpret_cast<int32_t*>(ptr()),
                                pick({0, 1, 33, 500, -1, INT64_MAX}), rng() % 20 ? 0.5f : INFINITY, ptr(),
                                reinterpret_cast<float*>(ptr()), ptr(), pick({0, 100, 4096, 1 << 20, -5, INT64_MAX >> 20}),
                                nullptr);
        }
        promise(st >= NM_OK && st <= NM_ERR_HIP, "status");
        ok += st == NM_OK;
    }
    std::printf("calls %ld, empty %ld, launches %ld\n", calls, ok, g_launches);
    promise(g_launches > 0 && ok > 0, "the random calls reach the kernels");
}

}  // namespace

int main(int argc, char** argv)
{
    layout();
    std::printf("plans checked %ld\n", plans());
    fuzz(argc > 1 ? std::atol(argv[1]) : 100000);
    return 0;
}
