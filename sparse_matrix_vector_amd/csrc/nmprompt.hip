// nmprompt.hip -- nm_attn_prompt: causal attention over packed prompts.
//
// A block holds 4 x 32 rows (query heads of one key head, nm_serve.h) and walks
// over the keys that its last row sees, 64 at a time.  Each wave keeps its 32 rows
// as matrix operands and, in one pass over the keys, a reference m near the running
// maximum of their scores, the sum l of the weights exp(s - m) and the vector
// o = sum exp(s - m) v; where a score passes the reference by too much, l and o are
// multiplied by exp(m_old - m_new).
//
// Both products run on the matrix cores with the rows of q as columns
// (v_mfma_f32_32x32x16: 32 keys or 32 columns of v by 32 rows):
//   scores  S^T[key][row]  = sum over columns of K[key][d] q[row][d]
//   output  O^T[d][row]   += sum over keys of V[key][d] p[row][key]
// A lane's column is its row of q (lane % 32) in both, so the softmax is per lane (and
// its other half, lane ^ 32).  The score tile's registers (half g, register i: key
// 8 (i / 4) + 4 g + i % 4) are the second product's right operand as they stand, when
// its k index (g, j) means key 4 g + j for j < 4 and 8 + 4 g + j - 4 for j >= 4; the
// values are read from LDS in that order by transposing reads.
//
// A weight enters the second product as one 16-bit operand, where the paged cache's attention has
// two (the rounding and the rest, nm_attn_units.h).  A prompt's products are what bounds it, and
// the second operand would make them half as many again; one loses half a step of each weight, in
// the order of what rounding the output does (root mean square error against 64 bits on the
// measured prompts: 1.08 to 1.29 times that of 32-bit arithmetic rounded once at the end).  So
// that the weights still add up to one, the sum they are divided by adds the rounded ones; lse
// adds them as they were.
//
// Keys and values go from memory to LDS directly (global_load_lds, 1 KB a wave and
// instruction), one tile ahead.  Rows lie in LDS as in memory but for an exclusive
// or of their 16-byte pieces' numbers with the row's, which keeps the banks apart:
// keys by row % 16 (reads of 16 rows' same piece), values by 2 (row % 8) (transposing
// reads of 4 rows' same 32 bytes).
//
// The work on a step of 32 keys is spread over three: its scores are formed during the
// step before, its weights (32 exponentials a pair of rows) beside other steps' products,
// its sums during the step after, so that a wave always has products that wait for
// nothing (one prompt of 8192 tokens, 64 heads on 8 of 128 columns: 1165 us with the three
// in a row, 1050 this way, 1047 TFLOP/s of the formula).

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nm_device.h"
#include "nm_serve.h"

namespace {

using namespace nmd;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
#define NM_NEG_INF (-__builtin_inff())

constexpr int kKeys = 64;                   // keys of a tile
constexpr int kPart = 32;                   // keys of a step

struct PromptArgs {
    const uint16_t* q;
    const uint8_t* k;
    const uint8_t* v;
    const int32_t* starts;
    const int32_t* k_starts;
    uint16_t* o;
    float* lse;
    int64_t q_stride;                       // elements
    int64_t k_stride, v_stride;             // bytes
    int T, Tk, B, Hq, heads, G;
    int tiles;                              // per key head
    int splits;                             // ranges of a tile's keys, one block each
    f32x4* part_o;                          // partial results (more than one range)
    f32x4* part_ml;
    // Scores are kept in base 2: q . k times `scale` = |scale| log2(e) > 0, the sign
    // (and a scale of zero) being put into q, which is exact.
    float scale;
    uint32_t q_and, q_xor;
};

// 1 KB from memory to LDS: the 16 bytes at lane i's address (base + offset) go to
// lds + 16 i.  The compiler does not know that LDS is written nor that a load is in
// flight: whoever reads waits (arrive) first.  (m0 is reserved: the compiler keeps nothing
// in it from one statement to the next.)
__device__ __forceinline__ void to_lds(uint32_t lds, const uint8_t* base, uint32_t offset)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base)
                 : "memory");
}

__device__ __forceinline__ void to_lds(uint32_t lds, const uint8_t* address)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(address) : "memory");
}

// All of this wave's loads into LDS are there, then all waves'; and all waves are
// past their reads from before.
__device__ __forceinline__ void arrive()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The sequence that tile `tile` belongs to: the last one whose first tile is not
// behind it.  A wave looks at 64 sequences at a time.
__device__ __forceinline__ int bound(int x, int most) { return min(max(x, 0), most); }

__device__ __forceinline__ int64_t first_tile(const PromptArgs& A, int b, int rows)
{
    return (int64_t)bound(A.starts[b], A.T) * A.G / rows + b;
}

__device__ __forceinline__ int find_sequence(const PromptArgs& A, int tile, int rows, int lane)
{
    int lo = 0, n = A.B;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int at = lane * step;
        const bool before = at < n && first_tile(A, lo + at, rows) <= tile;
        const int count = __popcll(__ballot(before));
        const int skip = max(count - 1, 0) * step;
        lo += skip;
        n = min(step, n - skip);
    }
    return lo;
}

// A tile's rows (keys or values) in LDS, and their way there.
template <int D, int NW>
struct Tile {
    static constexpr int kRow = 2 * D;                          // bytes of a row
    static constexpr int kBytes = kKeys * kRow;
    static constexpr int kRows = 1024 / kRow;                   // rows of a load
    static constexpr int kLanes = kRow / 16;                    // lanes of a row
    static constexpr int kLoads = kKeys / kRows / NW;           // of a wave
    static constexpr int kKinds = 16 / (kRows * NW) > 1 ? 16 / (kRows * NW) : 1;    // loads whose pieces lie differently
    static_assert(kLoads >= 1 && kKeys % (kRows * NW) == 0, "every wave loads as much");

    // The exclusive or of a piece's number in row `row`.
    static __device__ __forceinline__ int k_swap(int row) { return D == 64 ? row / 2 % 8 : row % 16; }
    static __device__ __forceinline__ int v_swap(int row) { return D == 64 ? 2 * (row % 4) : 2 * (row % 8); }

    const uint8_t* rows;        // the sequence's first row of this head
    int64_t stride;             // bytes
    uint32_t offset[kKinds];    // of the lane's 16 bytes from a load's first row
    int kind[kKinds];           // its piece

    template <bool KEYS>
    __device__ __forceinline__ void start(const uint8_t* first, int64_t stride_, int wave, int lane)
    {
        rows = first;
        stride = stride_;
#pragma unroll
        for (int x = 0; x < kKinds; ++x) {
            const int row = (wave + NW * x) * kRows + lane / kLanes;
            kind[x] = (lane % kLanes ^ (KEYS ? k_swap(row) : v_swap(row))) * 16;
            offset[x] = (uint32_t)(lane / kLanes) * (uint32_t)stride + kind[x];
        }
    }

    // Tile `tile` of a sequence of `n` rows; rows behind its last one are copies of that.
    __device__ __forceinline__ void load(uint32_t lds, int tile, int n, int wave, int lane) const
    {
        const int row0 = tile * kKeys;
        if (row0 + kKeys <= n) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int at = (wave + NW * j) * kRows;
                to_lds(lds + at * kRow, rows + (row0 + at) * stride, offset[j % kKinds]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int at = (wave + NW * j) * kRows;
                to_lds(lds + at * kRow, rows + min(row0 + at + lane / kLanes, n - 1) * stride + kind[j % kKinds]);
            }
        }
    }
};

template <int DT, int D, bool LSE>
__global__ __launch_bounds__(nms::kPromptWaves * 64, D == 256 ? 1 : 2) void prompt_kernel(const PromptArgs A, int blocks)
{
    constexpr int NW = nms::kPromptWaves;
    using L = Tile<D, NW>;
    constexpr int kSteps = D / 16;                              // k-steps of the score product
    constexpr int kCols = D / 32;                               // tiles of columns of the output
    constexpr int kQuarter = kSteps / 4;                        // products of each sort in a quarter of a step
    constexpr int kRows = NW * nms::kPromptWave;
    constexpr float kBelow = DT == NM_FP16 ? 7.0f : -8.0f, kRoom = DT == NM_FP16 ? 15.0f : 0.0f;
    constexpr uint32_t kOnes = DT == NM_FP16 ? 0x3C003C00u : 0x3F803F80u;
    __shared__ __align__(1024) uint8_t lds[4 * L::kBytes];      // two buffers of keys, two of values
    const int lane = threadIdx.x % 64, m = lane % 32, g = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int block = (int)flat_block();
    if (block >= blocks)
        return;
    // Key heads side by side, so that blocks of one share an XCD's cache where there are
    // eight; long tiles (the last ones of a sequence) first.
    const int h = block % A.heads, split = block / A.heads % A.splits;
    const int tile = A.tiles - 1 - block / A.heads / A.splits;
    const int b = find_sequence(A, tile, kRows, lane);
    const int q0 = bound(A.starts[b], A.T), nq = bound(A.starts[b + 1], A.T) - q0;
    const int k0 = bound(A.k_starts[b], A.Tk);
    const int all_keys = max(bound(A.k_starts[b + 1], A.Tk) - k0, 0);
    const int64_t r0 = ((int64_t)tile - first_tile(A, b, kRows)) * kRows;        // the block's first row
    if (nq <= 0 || r0 < 0 || r0 >= (int64_t)nq * A.G)           // (below 0: starts that decrease)
        return;
    const int R = nq * A.G, row0 = (int)r0 + wave * nms::kPromptWave;
    // The block's range: tiles of keys from `first` on, and keys counted from there.
    const int last_key = ((int)min(r0 + kRows, (int64_t)R) - 1) / A.G + all_keys - nq;
    const int all_tiles = max(last_key + kKeys, 0) / kKeys, per = (all_tiles + A.splits - 1) / A.splits;
    const int first = __builtin_amdgcn_readfirstlane(min(split * per, all_tiles));
    const int tiles = __builtin_amdgcn_readfirstlane(min(per, all_tiles - first));
    const int key0 = first * kKeys, nk = __builtin_amdgcn_readfirstlane(all_keys - key0);
    const int r = min(row0 + m, R - 1), query = r / A.G, head = h * A.G + r % A.G;
    const int limit = query + nk - nq;                                           // the last key the lane's row sees
    // Of the wave's steps of 32 keys the first n_whole are seen by all its rows, those from n_steps on by none.
    const int all = min(row0, R - 1) / A.G + nk - nq + 1, some = min(row0 + 31, R - 1) / A.G + nk - nq + 1;
    const int n_whole = __builtin_amdgcn_readfirstlane(max(all, 0) / kPart);
    const int n_steps = __builtin_amdgcn_readfirstlane(
        row0 < R ? min((max(some, 0) + kPart - 1) / kPart, tiles * (kKeys / kPart)) : 0);

    L keys, values;
    keys.template start<true>(A.k + ((int64_t)k0 + key0) * A.k_stride + (int64_t)h * 2 * D, A.k_stride, wave, lane);
    values.template start<false>(A.v + ((int64_t)k0 + key0) * A.v_stride + (int64_t)h * 2 * D, A.v_stride, wave, lane);
    const uint32_t k_buf = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const uint32_t v_buf = k_buf + 2 * L::kBytes;
    if (tiles > 0)
        keys.load(k_buf, 0, nk, wave, lane);

    u32x4 q[kSteps];
    {
        const uint16_t* row = A.q + (q0 + query) * A.q_stride + (int64_t)head * D + 8 * g;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            q[s] = (*reinterpret_cast<const u32x4*>(row + 16 * s) & A.q_and) ^ A.q_xor;
    }
    f32x16 acc[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[c][i] = 0.0f;
    float mx = NM_NEG_INF, sum = 0.0f, plain_sum = 0.0f;
    f32x16 s = acc[0];                                      // scores of the coming step
    f32x16 w = acc[0];                                      // weights of the step before

    // Where the lane's operands lie: keys of the buffer of tile t + 1, values of that of tile t.
    uint32_t k_at[kSteps], v_at[kCols];
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
        k_at[c] = k_buf + m * L::kRow + ((2 * c ^ g ^ L::k_swap(m)) << 4);
    const int vr = 4 * g + lane % 16 / 4;
#pragma unroll
    for (int c = 0; c < kCols; ++c)
        v_at[c] = v_buf + L::kBytes + vr * L::kRow + lane % 2 * 8 +
                  ((4 * c ^ (lane / 16 % 2 * 2 + lane % 4 / 2) ^ L::v_swap(vr)) << 4);
    const auto read_k = [&](int c, int part) {
        return *(lds_u32x4*)(uintptr_t)(k_at[c] + part * kPart * L::kRow);
    };
    const auto read_v = [&](int x, int c, int part) {
        const uint32_t at = v_at[c] + (part * kPart + 16 * x) * L::kRow;
        const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)at));
        const u32x2 hi = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(at + 8 * L::kRow)));
        return u32x4{lo.x, lo.y, hi.x, hi.y};
    };
    // The tile's loads, and the buffers' change of roles.
    const auto begin = [&](int t) {
        arrive();
        if (t + 2 < tiles)
            keys.load(k_buf + (t & 1) * L::kBytes, t + 2, nk, wave, lane);
        if (t + 1 < tiles)
            values.load(v_buf + (~t & 1) * L::kBytes, t + 1, nk, wave, lane);
    };
    const auto turn = [&]() {
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
            k_at[c] ^= L::kBytes;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
            v_at[c] ^= L::kBytes;
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
            plain_sum *= f;
            w *= f;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                acc[c] *= f;
            mx = top;
        }
    };
    // Two weights as operands, added to the sum.
    const auto pack = [&](int i) {
        const uint32_t x = pack2<DT>(w[i], w[i + 1]);
        sum = dot2<DT>(x, kOnes, sum);
        if constexpr (LSE)
            plain_sum += w[i] + w[i + 1];
        return x;
    };

    const auto hot = [&](auto part_) {
        constexpr int part = part_();
        make_room();
        const float ref = mx == NM_NEG_INF ? 0.0f : mx;
        f32x16 next;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            next[i] = 0.0f;
        // Operands are read one quarter ahead of the products that use them.
        u32x4 ka[2][kQuarter], va[2][kQuarter], p[2];
        const auto read = [&](int x) {
#pragma unroll
            for (int c = 0; c < kQuarter; ++c) {
                const int at = x * kQuarter + c;
                ka[x % 2][c] = read_k(at, part);
                va[x % 2][c] = read_v(at / kCols, at % kCols, part);
            }
        };
        read(0);
#pragma unroll
        for (int i = 0; i < 16; i += 2)
            p[i / 8][i % 8 / 2] = pack(i);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x < 3)
                read(x + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < kQuarter; ++c) {
                const int at = x * kQuarter + c;
                next = mfma32<DT>(ka[x % 2][c], q[at], next);
                acc[at % kCols] = mfma32<DT>(va[x % 2][c], p[at / kCols], acc[at % kCols]);
            }
#pragma unroll
            for (int i = 4 * x; i < 4 * x + 4; ++i)
                w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], A.scale, -ref));
            __builtin_amdgcn_sched_barrier(0);
        }
        s = next;
    };

    // Step u with all its conditions.
    const auto cold = [&](int u, int part) {
        if (u >= 0 && u < n_steps) {
            if (u >= n_whole)
#pragma unroll
                for (int i = 0; i < 16; ++i)                     // whatever lies there, NaN included
                    s[i] = u * kPart + 8 * (i / 4) + 4 * g + i % 4 > limit ? NM_NEG_INF : s[i];
            make_room();
        }
        if (u >= 1 && u <= n_steps) {
            u32x4 p0, p1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p0[i] = pack(2 * i);
                p1[i] = pack(8 + 2 * i);
            }
            float odd = 0.0f;
            if (u > n_whole)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        const u32x4 a = read_v(x, c, part);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            odd = dot2<DT>(a[i], 0u, odd);
                    }
            if (__any(odd != 0.0f)) {
                // 0 * NaN must not reach a row that does not see the value: steps with infinities
                // or NaN among the values take them key by key, and rows that do not see the key
                // keep their sums.
#pragma unroll
                for (int c = 0; c < kCols; ++c)
#pragma unroll 1
                    for (int key = 0; key < kPart; ++key) {
                        const int in = key % 16, word = (in % 4 + in / 8 * 4) / 2;
                        const uint32_t keep = in / 4 % 2 == g ? (key % 2 ? 0xFFFF0000u : 0xFFFFu) : 0u;
                        const bool sees = (u - 1) * kPart + key <= limit;
                        u32x4 a = read_v(key / 16, c, part), p;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            a[i] &= i == word ? keep : 0u;
                            p[i] = key < 16 ? p0[i] : p1[i];
                        }
                        const f32x16 with = mfma32<DT>(a, p, acc[c]);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[c][i] = sees ? with[i] : acc[c][i];
                    }
            } else {
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    acc[c] = mfma32<DT>(read_v(1, c, part), p1, mfma32<DT>(read_v(0, c, part), p0, acc[c]));
            }
        }
        if (u >= 0 && u < n_steps) {
            const float ref = mx == NM_NEG_INF ? 0.0f : mx;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], A.scale, -ref));
        }
        if (u + 1 < n_steps) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[i] = 0.0f;
#pragma unroll
            for (int c = 0; c < kSteps; ++c)
                s = mfma32<DT>(read_k(c, part), q[c], s);
        }
    };

    for (int t = -1; t < tiles;) {
        begin(t);
#pragma unroll 1
        for (int part = 0; part < 2; ++part)
            cold(2 * t + 1 + part, part);
        turn();
        for (++t; 2 * t + 2 < n_whole && 2 * t + 3 < n_steps; ++t) {
            begin(t);
            hot(std::integral_constant<int, 0>());
            hot(std::integral_constant<int, 1>());
            turn();
        }
    }
    sum = halves_sum(sum);
    if constexpr (LSE)
        plain_sum = halves_sum(plain_sum);
    if (row0 + m >= R)
        return;
    // The lane holds columns 32 c + 8 (i / 4) + 4 g + i % 4 of its row in acc[c][i].
    if (A.splits > 1) {
        // Partial results lie as the lanes hold them: [range][tile][key head][wave][four columns][lane] 16 bytes.
        const int64_t part = (((int64_t)split * A.tiles + tile) * A.heads + h) * NW + wave;
        f32x4* o = A.part_o + part * (kCols * 4) * 64 + lane;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[(c * 4 + i) * 64] = f32x4{acc[c][4 * i], acc[c][4 * i + 1], acc[c][4 * i + 2], acc[c][4 * i + 3]};
        if (g == 0)
            A.part_ml[part * 32 + m] = f32x4{mx, sum, plain_sum, 0.0f};
        return;
    }
    const float f = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    const int64_t row = (int64_t)(q0 + query) * A.Hq + head;
    uint16_t* o = A.o + row * D + 4 * g;
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<u32x2*>(o + 32 * c + 2 * i) =
                u32x2{pack2<DT>(acc[c][i] * f, acc[c][i + 1] * f), pack2<DT>(acc[c][i + 2] * f, acc[c][i + 3] * f)};
    if constexpr (LSE)
        if (g == 0)
            A.lse[row] = (mx + __builtin_amdgcn_logf(plain_sum)) * kLn2;
}

// Joins the ranges of a tile: a block takes four columns (piece) of every lane, a wave the rows
// that a wave of the tile's blocks had.
template <int DT, int D, bool LSE>
__global__ __launch_bounds__(nms::kPromptWaves * 64) void prompt_join_kernel(const PromptArgs A, int blocks)
{
    constexpr int NW = nms::kPromptWaves, kPieces = D / 8, kRows = NW * nms::kPromptWave, kBatch = 4;
    const int lane = threadIdx.x % 64, m = lane % 32, g = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int block = (int)flat_block();
    if (block >= blocks)
        return;
    const int piece = block % kPieces, h = block / kPieces % A.heads, tile = block / kPieces / A.heads;
    const int b = find_sequence(A, tile, kRows, lane);
    const int q0 = bound(A.starts[b], A.T), nq = bound(A.starts[b + 1], A.T) - q0;
    const int64_t r0 = ((int64_t)tile - first_tile(A, b, kRows)) * kRows, r = r0 + wave * nms::kPromptWave + m;
    if (nq <= 0 || r0 < 0 || r >= (int64_t)nq * A.G)
        return;
    const int64_t part0 = ((int64_t)tile * A.heads + h) * NW + wave, step = (int64_t)A.tiles * A.heads * NW;
    float mx = NM_NEG_INF, sum = 0.0f, plain_sum = 0.0f;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < A.splits; i += kBatch) {
        f32x4 x[kBatch], o[kBatch];
        float top = mx;
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            const int64_t part = part0 + min(i + c, A.splits - 1) * step;           // (others are not added)
            x[c] = A.part_ml[part * 32 + m];
            o[c] = A.part_o[(part * kPieces + piece) * 64 + lane];
        }
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
            top = i + c < A.splits ? fmaxf(top, x[c].x) : top;
        const float ref = top == NM_NEG_INF ? 0.0f : top, f = __builtin_amdgcn_exp2f(mx - ref);
        mx = top;
        sum *= f;
        plain_sum *= f;
        acc *= f;
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
            if (i + c < A.splits) {
                const float w = __builtin_amdgcn_exp2f(x[c].x - ref);
                sum += x[c].y * w;
                plain_sum += x[c].z * w;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[e] += o[c][e] * w;
            }
    }
    acc *= sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    const int64_t row = (q0 + r / A.G) * A.Hq + h * A.G + r % A.G;
    *reinterpret_cast<u32x2*>(A.o + row * D + piece / 4 * 32 + piece % 4 * 8 + 4 * g) =
        u32x2{pack2<DT>(acc[0], acc[1]), pack2<DT>(acc[2], acc[3])};
    if constexpr (LSE)
        if (g == 0 && piece == 0)
            A.lse[row] = (mx + __builtin_amdgcn_logf(plain_sum)) * kLn2;
}

template <int DT, int D>
int launch(const nms::PromptPlan& P, const PromptArgs& A, hipStream_t s)
{
    const int64_t blocks = P.tiles * P.splits * A.heads, join = P.tiles * A.heads * (D / 8);
    constexpr int kThreads = nms::kPromptWaves * 64;
    const auto run = [&](auto kernel, int64_t n) {
        hipLaunchKernelGGL(kernel, flat_grid(n), dim3(kThreads), 0, s, A, (int)n);
    };
    (void)hipGetLastError();
    if (A.lse)
        run(prompt_kernel<DT, D, true>, blocks);
    else
        run(prompt_kernel<DT, D, false>, blocks);
    if (P.splits > 1 && A.lse)
        run(prompt_join_kernel<DT, D, true>, join);
    else if (P.splits > 1)
        run(prompt_join_kernel<DT, D, false>, join);
    return hipGetLastError() == hipSuccess ? NM_OK : NM_ERR_HIP;
}

template <int DT>
int launch_width(const nms::PromptPlan& P, const PromptArgs& A, int D, hipStream_t s)
{
    switch (D) {
    case 64: return launch<DT, 64>(P, A, s);
    case 128: return launch<DT, 128>(P, A, s);
    default: return launch<DT, 256>(P, A, s);
    }
}

}  // namespace

int nmk::attn_prompt(const nms::PromptPlan& plan, const void* q, int64_t q_stride, int64_t T, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, int64_t Tk, const int32_t* starts,
                     const int32_t* k_starts, int64_t B, int Hq, int heads, int D, int dtype, float scale, void* o,
                     float* lse, void* workspace, void* stream)
{
    PromptArgs A;
    A.q = static_cast<const uint16_t*>(q);
    A.k = static_cast<const uint8_t*>(k);
    A.v = static_cast<const uint8_t*>(v);
    A.starts = starts;
    A.k_starts = k_starts;
    A.o = static_cast<uint16_t*>(o);
    A.lse = lse;
    A.q_stride = T > 1 ? q_stride : 0;
    A.k_stride = Tk > 1 ? k_stride * 2 : 0;
    A.v_stride = Tk > 1 ? v_stride * 2 : 0;
    A.T = (int)T;
    A.Tk = (int)Tk;
    A.B = (int)B;
    A.Hq = Hq;
    A.heads = heads;
    A.G = plan.G;
    A.tiles = (int)plan.tiles;
    A.splits = (int)plan.splits;
    A.part_ml = static_cast<f32x4*>(workspace);
    A.part_o = A.part_ml + plan.splits * plan.tiles * heads * nms::kPromptRows;
    A.scale = scale == 0.0f ? 1.0f : fabsf(scale) * kLog2e;
    A.q_and = scale == 0.0f ? 0u : 0xFFFFFFFFu;
    A.q_xor = scale < 0.0f ? 0x80008000u : 0u;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == NM_FP16 ? launch_width<NM_FP16>(plan, A, D, s) : launch_width<NM_BF16>(plan, A, D, s);
}
