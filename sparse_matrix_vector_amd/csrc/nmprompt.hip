// nmprompt.hip -- nm_attn_prompt: causal attention over packed prompts.
//
// A block holds NW x 32 rows (query heads of one key head, nm_serve.h) and walks
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
// Keys and values go from memory to LDS directly (global_load_lds, 1 KB a wave and
// instruction), one tile ahead.  Rows lie in LDS as in memory but for an exclusive
// or of their 16-byte pieces' numbers with the row's, which keeps the banks apart:
// keys by row % 16 (reads of 16 rows' same piece), values by 2 (row % 8) (transposing
// reads of 4 rows' same 32 bytes).

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "nm_device.h"
#include "nm_serve.h"

namespace {

using namespace nmd;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
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
    // Scores are kept in base 2: q . k times `scale` = |scale| log2(e) > 0, the sign
    // (and a scale of zero) being put into q, which is exact.
    float scale;
    uint32_t q_and, q_xor;
};

template <int DT>
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (DT == NM_FP16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
}

// sum + a.x + a.y of the two 16-bit floats (times b's).
template <int DT>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float sum)
{
    if constexpr (DT == NM_FP16)
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), sum, false);
    else
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), sum, false);
}

// Maximum / sum of a lane and lane ^ 32 (a row's two halves).
__device__ __forceinline__ float halves_max(float v)
{
    const u32x2 p = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(f32_bits(v), f32_bits(v), false, false));
    return fmaxf(bits_f32(p.x), bits_f32(p.y));
}

__device__ __forceinline__ float halves_sum(float v)
{
    const u32x2 p = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(f32_bits(v), f32_bits(v), false, false));
    return bits_f32(p.x) + bits_f32(p.y);
}

// 1 KB from memory to LDS: the 16 bytes at lane i's address go to lds + 16 i.  The
// compiler does not know that LDS is written nor that a load is in flight: whoever
// reads waits (arrive) first.  (m0 is reserved: the compiler keeps nothing in it from
// one statement to the next.)
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

// The keys and values of one tile in LDS, and their way there.
template <int D, int NW>
struct Tile {
    static constexpr int kRow = 2 * D;                          // bytes of a row
    static constexpr int kBytes = kKeys * kRow;                 // of the keys, and of the values
    static constexpr int kRows = 1024 / kRow;                   // rows of a load
    static constexpr int kLanes = kRow / 16;                    // lanes of a row
    static constexpr int kLoads = kKeys / kRows / NW;           // of a wave, keys and values each
    static_assert(kLoads >= 1 && kKeys % (kRows * NW) == 0, "every wave loads as much");

    // The exclusive or of a piece's number in row `row`.
    static __device__ __forceinline__ int k_swap(int row) { return D == 64 ? row / 2 % 8 : row % 16; }
    static __device__ __forceinline__ int v_swap(int row) { return D == 64 ? 2 * (row % 4) : 2 * (row % 8); }

    // Rows key0 .. of a sequence that ends at key `end`: rows from there on are copies of its last one.
    static __device__ __forceinline__ void load(uint32_t lds, const uint8_t* k, int64_t k_stride, const uint8_t* v,
                                                int64_t v_stride, int key0, int end, int wave, int lane)
    {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int row0 = (wave + NW * j) * kRows, row = row0 + lane / kLanes;
            const int key = min(key0 + row, end - 1);
            const int kc = lane % kLanes ^ k_swap(row), vc = lane % kLanes ^ v_swap(row);
            to_lds(lds + row0 * kRow, k + key * k_stride + kc * 16);
            to_lds(lds + kBytes + row0 * kRow, v + key * v_stride + vc * 16);
        }
    }
};

template <int DT, int D, int NW, bool LSE>
__global__ __launch_bounds__(NW * 64, NW == 8 ? 2 : 1) void prompt_kernel(const PromptArgs A, int blocks)
{
    using L = Tile<D, NW>;
    constexpr int kSteps = D / 16;                              // k-steps of the score product
    constexpr int kCols = D / 32;                               // tiles of columns of the output
    constexpr int kRows = NW * nms::kPromptWave;
    constexpr float kBelow = DT == NM_FP16 ? 7.0f : -8.0f, kRoom = DT == NM_FP16 ? 15.0f : 0.0f;
    __shared__ __align__(1024) uint8_t lds[4 * L::kBytes];
    const int lane = threadIdx.x % 64, m = lane % 32, g = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int block = (int)flat_block();
    if (block >= blocks)
        return;
    // Key heads side by side, so that blocks of one share an XCD's cache where there are
    // eight; long tiles (the last ones of a sequence) first.
    const int h = block % A.heads, tile = A.tiles - 1 - block / A.heads;
    const int b = find_sequence(A, tile, kRows, lane);
    const int q0 = bound(A.starts[b], A.T), nq = bound(A.starts[b + 1], A.T) - q0;
    const int k0 = bound(A.k_starts[b], A.Tk), nk = max(bound(A.k_starts[b + 1], A.Tk) - k0, 0);
    const int64_t r0 = ((int64_t)tile - first_tile(A, b, kRows)) * kRows;        // the block's first row
    if (nq <= 0 || r0 >= (int64_t)nq * A.G)
        return;
    const int R = nq * A.G, row0 = (int)r0 + wave * nms::kPromptWave;
    const int r = min(row0 + m, R - 1), query = r / A.G, head = h * A.G + r % A.G;
    const int limit = query + nk - nq;                                           // the last key the lane's row sees
    // Keys below `all` are seen by every row of the wave, from `some` on by none.
    const int all = __builtin_amdgcn_readfirstlane(min(row0, R - 1) / A.G + nk - nq + 1);
    const int some = __builtin_amdgcn_readfirstlane(row0 < R ? min(row0 + 31, R - 1) / A.G + nk - nq + 1 : 0);
    const int end = __builtin_amdgcn_readfirstlane(((int)min(r0 + kRows, (int64_t)R) - 1) / A.G + nk - nq + 1);

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

    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const uint8_t* kp = A.k + k0 * A.k_stride + (int64_t)h * 2 * D;
    const uint8_t* vp = A.v + k0 * A.v_stride + (int64_t)h * 2 * D;
    const int tiles = (end + kKeys - 1) / kKeys;
    if (tiles > 0)
        L::load(base, kp, A.k_stride, vp, A.v_stride, 0, nk, wave, lane);
    // Where the lane's operands lie in a tile.
    const uint32_t k_at = m * L::kRow, k_piece = g ^ L::k_swap(m);
    const int vr = 4 * g + lane % 16 / 4;
    const uint32_t v_at = vr * L::kRow + lane % 2 * 8;
    const uint32_t v_piece = (lane / 16 % 2 * 2 + lane % 4 / 2) ^ L::v_swap(vr);

    for (int t = 0; t < tiles; ++t) {
        arrive();
        if (t + 1 < tiles)
            L::load(base + ((t + 1) & 1) * 2 * L::kBytes, kp, A.k_stride, vp, A.v_stride, (t + 1) * kKeys, nk, wave, lane);
        const uint32_t kb = base + (t & 1) * 2 * L::kBytes, vb = kb + L::kBytes;
#pragma unroll
        for (int part = 0; part < kKeys / kPart; ++part) {
            const int key0 = t * kKeys + part * kPart;
            if (key0 >= some)
                break;
            const bool whole = key0 + kPart <= all;
            f32x16 s;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[i] = 0.0f;
#pragma unroll
            for (int c = 0; c < kSteps; ++c) {
                const u32x4 a = *(lds_u32x4*)(uintptr_t)(kb + part * kPart * L::kRow + k_at + ((2 * c ^ k_piece) << 4));
                s = mfma<DT>(a, q[c], s);
            }
            if (!whole)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key0 + 8 * (i / 4) + 4 * g + i % 4 > limit)
                        s[i] = NM_NEG_INF;                       // whatever lies there, NaN included
            float top = NM_NEG_INF;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                top = fmaxf(top, s[i]);
            top *= A.scale;
            if (__any(top > mx + kRoom)) {
                // rows that need no more room stay as they are, whatever stands beside them
                top = halves_max(top);
                top = top > mx + kRoom ? top - kBelow : mx;
                const float f = mx == top ? 1.0f : __builtin_amdgcn_exp2f(mx - top);
                sum *= f;
                plain_sum *= f;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    acc[c] *= f;
                mx = top;
            }
            const float ref = mx == NM_NEG_INF ? 0.0f : mx;
            u32x4 p[2];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], A.scale, -ref));
                const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i + 1], A.scale, -ref));
                const uint32_t w = pack2<DT>(w0, w1);
                if constexpr (LSE)
                    plain_sum += w0 + w1;
                p[i / 8][i % 8 / 2] = w;
                sum = dot2<DT>(w, DT == NM_FP16 ? 0x3C003C00u : 0x3F803F80u, sum);
            }
            u32x4 va[2][kCols];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const uint32_t at = vb + (part * kPart + 16 * x) * L::kRow + v_at + ((4 * c ^ v_piece) << 4);
                    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)at));
                    const u32x2 hi = __builtin_bit_cast(
                        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(at + 8 * L::kRow)));
                    va[x][c] = u32x4{lo.x, lo.y, hi.x, hi.y};
                }
            if (!whole) {
                // 0 * NaN must not reach a row that does not see the value.  Steps with
                // infinities or NaN among the values take them key by key and keep the sums of
                // the rows that do not see the key.
                float odd = 0.0f;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            odd = dot2<DT>(va[x][c][i], 0u, odd);
                if (__any(odd != 0.0f)) {
#pragma unroll 1
                    for (int key = 0; key < kPart; ++key) {
                        const int in = key % 16, word = (in % 4 + in / 8 * 4) / 2;
                        const uint32_t keep = in / 4 % 2 == g ? (key % 2 ? 0xFFFF0000u : 0xFFFFu) : 0u;
                        u32x4 mask;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mask[i] = i == word ? keep : 0u;
                        const u32x4 w = key < 16 ? p[0] : p[1];
#pragma unroll
                        for (int c = 0; c < kCols; ++c) {
                            const u32x4 a = (key < 16 ? va[0][c] : va[1][c]) & mask;
                            const f32x16 with = mfma<DT>(a, w, acc[c]);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                acc[c][i] = key0 + key <= limit ? with[i] : acc[c][i];
                        }
                    }
                    continue;
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    acc[c] = mfma<DT>(va[x][c], p[x], acc[c]);
        }
    }
    sum = halves_sum(sum);
    if constexpr (LSE)
        plain_sum = halves_sum(plain_sum);
    if (row0 + m >= R)
        return;
    // The lane holds columns 32 c + 8 (i / 4) + 4 g + i % 4 of its row in acc[c][i].
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

template <int DT, int D, int NW>
int launch(const nms::PromptPlan& P, const PromptArgs& A, hipStream_t s)
{
    const int64_t blocks = P.tiles * A.heads;
    if (blocks > INT32_MAX)
        return NM_ERR_BAD_SHAPE;
    (void)hipGetLastError();
    if (A.lse)
        hipLaunchKernelGGL((prompt_kernel<DT, D, NW, true>), flat_grid(blocks), dim3(NW * 64), 0, s, A, (int)blocks);
    else
        hipLaunchKernelGGL((prompt_kernel<DT, D, NW, false>), flat_grid(blocks), dim3(NW * 64), 0, s, A, (int)blocks);
    return hipGetLastError() == hipSuccess ? NM_OK : NM_ERR_HIP;
}

template <int DT>
int launch_width(const nms::PromptPlan& P, const PromptArgs& A, int D, hipStream_t s)
{
    switch (D) {
    case 64: return launch<DT, 64, 8>(P, A, s);
    case 128: return launch<DT, 128, 8>(P, A, s);
    default: return launch<DT, 256, 4>(P, A, s);
    }
}

}  // namespace

int nmk::attn_prompt(const nms::PromptPlan& plan, const void* q, int64_t q_stride, int64_t T, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, int64_t Tk, const int32_t* starts,
                     const int32_t* k_starts, int64_t B, int Hq, int heads, int D, int dtype, float scale, void* o,
                     float* lse, void*, void* stream)
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
    A.scale = scale == 0.0f ? 1.0f : fabsf(scale) * kLog2e;
    A.q_and = scale == 0.0f ? 0u : 0xFFFFFFFFu;
    A.q_xor = scale < 0.0f ? 0x80008000u : 0u;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == NM_FP16 ? launch_width<NM_FP16>(plan, A, D, s) : launch_width<NM_BF16>(plan, A, D, s);
}
