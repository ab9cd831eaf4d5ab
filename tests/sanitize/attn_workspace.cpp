// attn_workspace.cpp -- nm_attn_workspace_bytes against the plans of nm_attn_decode: what it
// gives for a shape holds the partial rows of that shape and of every smaller one.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "nm_attn.h"

namespace {

std::mt19937_64 rng(11);

// 0 .. top, spread over its logarithm, with the edges of the plan's rules among them.
int64_t size(int64_t least, int64_t top)
{
    static const int64_t edges[] = {0, 1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 512, 513, 4096, 4097, 8192, 8193};
    const int64_t v = rng() % 3 == 0 ? edges[rng() % 18]
                                     : (int64_t)std::exp2(std::log2((double)top) * (double)(rng() % 100001) / 100000.0);
    return std::min(std::max(v, least), top);
}

}  // namespace

int main(int argc, char** argv)
{
    const long calls = argc > 1 ? std::atol(argv[1]) : 1000000;
    long shapes = 0;
    double over = 0.0;
    for (long i = 0; i < calls; ++i) {
        const int heads = (int)size(1, i % 10 ? 32 : 2000), G = (int)size(1, i % 10 ? 80 : 2000);
        const int D = 64 << rng() % 3, format = (int)(rng() % 3);
        const int64_t Hq = (int64_t)heads * G;
        if (Hq > 65535)
            continue;
        const int64_t rows = nma::kMaxRows - 1, top_b = std::min<int64_t>(65535, rows / Hq);
        const int64_t B = size(1, i % 4 ? std::min<int64_t>(top_b, 600) : top_b);
        const int64_t P = rng() % 2 ? size(0, nma::kMaxTokens) : rng() % 2 * size(0, 40000);
        const int64_t ml = rng() % 2 ? size(0, nma::kMaxTokens) : rng() % 4 ? size(0, 40000) : 0;
        const int64_t bound = nma::attn_workspace_bound(B, (int)Hq, heads, D, format, P, ml);
        for (int j = 0; j < 8; ++j) {
            const int64_t b = j & 1 ? size(1, B) : B, p = P && j & 2 ? size(0, P) : P, m = ml && j & 4 ? size(0, ml) : ml;
            const int64_t need = nma::attn_workspace(nma::attn_plan(b, (int)Hq, heads, D, format, p, m), D);
            const int64_t less = nma::attn_workspace_bound(b, (int)Hq, heads, D, format, p, m);
            if (need > bound || less > bound || bound < 0 || bound >= int64_t(1) << 46) {
                std::fprintf(stderr, "heads %d G %d D %d format %d: (%ld, %ld, %ld) has %ld bytes, (%ld, %ld, %ld) needs %ld\n",
                             heads, G, D, format, (long)B, (long)P, (long)ml, (long)bound, (long)b, (long)p, (long)m,
                             (long)std::max(need, less));
                return 1;
            }
            if (j == 0 && need > 0)
                over = std::max(over, (double)bound / (double)need);
        }
        ++shapes;
    }
    std::printf("shapes checked %ld, at most %.1f times a plan's own\n", shapes, over);
    return 0;
}
