// nmcache.hip -- the row-wise kernels of include/nmattn.h: per-head norm with
// the position rotation, and the paged cache's write and read.
//
// All three move each byte once and compute little on it; what bounds them is
// HBM for long prompts and the launch for decode steps (about 3 us).  A thread
// holds eight consecutive columns (one 16-byte load), so a head is D / 8
// neighbouring lanes and its reductions are lane exchanges within a wave.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "nm_attn.h"
#include "nm_device.h"

namespace {

using namespace nmd;

int hip_status(hipError_t e) { return e == hipSuccess ? NM_OK : NM_ERR_HIP; }

// ---- per-head norm and rotation ----------------------------------------------

constexpr int kQkThreads = 256;

struct QkArgs {
    const uint16_t* x[2];       // q, k
    uint16_t* y[2];
    const uint16_t* w[2];       // norm weights or NULL
    int64_t stride[2];          // of x, elements
    int heads[2];
    int64_t T;
    int D, rot, blocks_per_row;
    float eps;
    const int32_t* positions;
    const float* inv_freq;
};

// LPH lanes (a power of two, at least D / 8) hold one head; a block takes one
// row's heads hb, hb + blocks_per_row, ... in groups of 256 / LPH.  The row's
// sines and cosines are computed once per block and kept in LDS; a thread's next
// load is always in flight (16384 rows of 64 + 8 heads, 604 MB: 172 us with each
// load waited for at once, 125 with the next one started first, 115 to 121 with the
// rows non-temporal as well; a non-temporal copy of as many bytes takes 100).
//   y = n cos -+ n' sin  with n' the pair's other column: the same thread's for
// neighbouring pairs, the one rot / 16 lanes away for pairs (i, i + rot / 2).
template <int DT, int LPH, bool INTERLEAVED, bool ONCE>
__global__ __launch_bounds__(kQkThreads) void qk_kernel(const QkArgs A)
{
    __shared__ float cs[2][256];
    const uint32_t block = flat_block();
    const int64_t t = block / A.blocks_per_row;
    const int part = block % A.blocks_per_row;
    if (t >= A.T)
        return;
    const int half = A.rot / 2;
    constexpr int kPerPass = kQkThreads / LPH;
    const int lane = threadIdx.x % LPH, d0 = lane * 8;
    const bool live = d0 < A.D;
    const int total = A.heads[0] + A.heads[1], stride = A.blocks_per_row * kPerPass;
    const auto load = [&](int hh) {
        u32x4 raw = {0u, 0u, 0u, 0u};
        if (live && hh < total) {
            const int side = hh >= A.heads[0], h = side ? hh - A.heads[0] : hh;
            const u32x4* at = reinterpret_cast<const u32x4*>(A.x[side] + t * A.stride[side] + (int64_t)h * A.D + d0);
            raw = ONCE ? __builtin_nontemporal_load(at) : *at;
        }
        return raw;
    };
    int hh = part * kPerPass + threadIdx.x / LPH;
    u32x4 next = load(hh);          // in flight while the sines are computed
    if ((int)threadIdx.x < half) {
        // Turns in double: a position's product with its frequency keeps its phase
        // (fp32 would lose it from some thousand positions on).
        const double turns = (double)A.positions[t] * (double)A.inv_freq[threadIdx.x] * 0.15915494309189533577;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[0][threadIdx.x] = c;
        cs[1][threadIdx.x] = s;
    }
    __syncthreads();
    for (; hh < total; hh += stride) {      // whole groups of LPH lanes leave together
        const u32x4 raw = next;
        next = load(hh + stride);
        const int side = hh >= A.heads[0];
        const int h = side ? hh - A.heads[0] : hh;
        float n[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 p = unpack2<DT>(raw[i]);
            n[2 * i] = p.x;
            n[2 * i + 1] = p.y;
        }
        if (A.w[side]) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss += n[i] * n[i];
#pragma unroll
            for (int m = 1; m < LPH; m *= 2)
                ss += __shfl_xor(ss, m, LPH);
            const float r = 1.0f / sqrtf(ss / (float)A.D + A.eps);
            if (live) {
                const u32x4 raw = *reinterpret_cast<const u32x4*>(A.w[side] + d0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x2 p = unpack2<DT>(raw[i]);
                    n[2 * i] *= r * p.x;
                    n[2 * i + 1] *= r * p.y;
                }
            }
        }
        float y[8];
        const bool turned = d0 < A.rot;         // all eight columns or none: rot is a multiple of 16
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = turned ? d0 / 2 + i : 0;
                const float c = cs[0][p], s = cs[1][p];
                y[2 * i] = n[2 * i] * c - n[2 * i + 1] * s;
                y[2 * i + 1] = n[2 * i + 1] * c + n[2 * i] * s;
            }
        } else {
            const int away = A.rot / 16;
            const bool low = d0 < half;
            const int from = low ? lane + away : turned ? lane - away : lane;
            const int p = low ? d0 : turned ? d0 - half : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float other = __shfl(n[i], from, LPH);
                const float c = cs[0][p + i], s = cs[1][p + i];
                y[i] = low ? n[i] * c - other * s : n[i] * c + other * s;
            }
        }
        if (!turned)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = n[i];
        if (live) {
            u32x4 out;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                out[i] = pack2<DT>(y[2 * i], y[2 * i + 1]);
            u32x4* at = reinterpret_cast<u32x4*>(A.y[side] + (t * A.heads[side] + h) * A.D + d0);
            if constexpr (ONCE)
                __builtin_nontemporal_store(out, at);
            else
                *at = out;
        }
    }
}

template <int DT, int LPH, bool ONCE>
int launch_qk(const QkArgs& A, bool interleaved, int64_t blocks, hipStream_t s)
{
    (void)hipGetLastError();
    if (interleaved)
        hipLaunchKernelGGL((qk_kernel<DT, LPH, true, ONCE>), flat_grid(blocks), dim3(kQkThreads), 0, s, A);
    else
        hipLaunchKernelGGL((qk_kernel<DT, LPH, false, ONCE>), flat_grid(blocks), dim3(kQkThreads), 0, s, A);
    return hip_status(hipGetLastError());
}

template <int DT, int LPH>
int launch_qk(const QkArgs& A, bool interleaved, bool once, int64_t blocks, hipStream_t s)
{
    return once ? launch_qk<DT, LPH, true>(A, interleaved, blocks, s) : launch_qk<DT, LPH, false>(A, interleaved, blocks, s);
}

template <int DT>
int launch_qk_dt(QkArgs A, bool interleaved, int64_t T, hipStream_t s)
{
    int lph = 4;
    while (lph * 8 < A.D)
        lph *= 2;
    const int passes = (A.heads[0] + A.heads[1] + kQkThreads / lph - 1) / (kQkThreads / lph);
    // One block per pass of a row while the rows are few (every head's loads in
    // flight at once), one block for the whole row when rows fill the GPU.
    A.blocks_per_row = T >= 2 * nma::kCus ? 1 : passes;
    // Non-temporal from 64 MB of rows on (64 + 8 heads, us without / with: 16384 rows 125.1
    // / 120.3, with the cache write behind it 143.5 / 137.8; 4096 36.6 / 34.3; 1237 13.5 /
    // 13.9, 17.3 / 18.0).
    const bool once = T * (A.heads[0] + A.heads[1]) * A.D * 2 >= int64_t(64) << 20;
    const int64_t row_limit = INT32_MAX / A.blocks_per_row;
    if (T > row_limit)
        return NM_ERR_BAD_SHAPE;
    const int64_t blocks = T * A.blocks_per_row;
    switch (lph) {
    case 4: return launch_qk<DT, 4>(A, interleaved, once, blocks, s);
    case 8: return launch_qk<DT, 8>(A, interleaved, once, blocks, s);
    case 16: return launch_qk<DT, 16>(A, interleaved, once, blocks, s);
    case 32: return launch_qk<DT, 32>(A, interleaved, once, blocks, s);
    default: return launch_qk<DT, 64>(A, interleaved, once, blocks, s);
    }
}

// ---- the cache -----------------------------------------------------------------

constexpr int kCacheThreads = 256;

struct CacheArgs {
    uint8_t* codes[2];          // k, v
    uint8_t* scales[2];
    const int64_t* slots;
    int64_t n_slots, T;
    int page_shift, heads;
};

// Where slot's (head) tile of 16 tokens starts, in tiles, and the token in it.
__device__ __forceinline__ int64_t tile_of(const CacheArgs& A, int64_t slot, int h, int& token)
{
    const int64_t page = slot >> A.page_shift;
    const int place = (int)(slot & ((1 << A.page_shift) - 1));
    token = place % nma::kTile;
    return (page * A.heads + h) * ((1 << A.page_shift) / nma::kTile) + place / nma::kTile;
}

// Scale byte of the 32 columns whose largest magnitude is `top`: the least e with
// top <= M 2^e, M = 1.75 * 2^8 or 1.5 * 2^2, so top's own exponent minus 8 (2), and one
// more if its fraction is above M's.
template <int DT, int BITS>
__device__ __forceinline__ int scale_byte(float top)
{
    const uint32_t b = f32_bits(top);
    const int e = (int)(b >> 23) - 127 - (BITS == 8 ? 8 : 2) +
                  ((b & 0x7FFFFFu) > (BITS == 8 ? 0x600000u : 0x400000u) ? 1 : 0);
    return max(e, nma::least_exponent(DT, BITS)) + nma::scale_bias(DT);
}

// The cache kernels' work: a wave takes kRows rows by kCols columns, a lane eight
// columns of one row, of k and of v.  The four neighbouring lanes that share a
// scale find it by two exchanges.  Eight rows by 64 columns: a row's piece is one
// cache line on the rows' side, and on the cache's side eight tokens of a tile
// make up whole lines.  32768 rows of 8 x 128 in MX8, write / read of 65536 back:
// 4 rows x 128 columns 51 / 85 us, 8 x 64 48 / 81, 16 x 32 51 / 94 (a thread a
// unit with 64-bit divisions, before: 63 / 128; all by one unit a wave).
// The rows are touched once, so they are loaded and stored non-temporally and the caches
// are left to the codes' pieces (us; written rows just produced / long ago, 32768 rows,
// 16-bit: 52.0 / 69.5 without, 52.0 / 58.4 with; MX8 41.7 / 56.1, 38.6 / 44.2; MX4 31.3 /
// 49.6, 32.4 / 39.5; 4096 rows, MX8: 10.2 / 13.2, 11.0 / 7.6; 65536 rows read back, MX8 77 ->
// 62, MX4 68 -> 51, 16-bit 105).
// With all of it, write / read back in a kernel trace: MX8 39 / 61 to 72, MX4 38 / 50 (a
// non-temporal copy of as many bytes: 34 / 67, 28 / 56).
constexpr int kRows = 8, kCols = 64;

// Units of a wave that reads codes back: two, eight rows apart, their loads in flight
// together (as above, MX8 81.8 -> 74.7 us, MX4 86.5 -> 71.3; four 76.0 / 73.6).  Not for
// 16-bit values (2474 rows 6.2 -> 6.7), and not for writes (32768 rows, MX8 47.9 -> 50.2).
constexpr int read_units(int bits) { return bits == 16 ? 1 : 2; }

struct Lane {
    int64_t t;          // row
    int col;            // column of the row (heads D of them); h and d0 from it
    bool live;
};

template <int UNITS>
__device__ __forceinline__ Lane lane_of(int64_t T, int width)
{
    const uint32_t lane = threadIdx.x % 64, per = (uint32_t)(width + kCols - 1) / kCols;
    const uint32_t item = flat_block() * (kCacheThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t group = item / per;          // uniform; cache_grid keeps items in 31 bits
    Lane l;
    l.t = (int64_t)group * (kRows * UNITS) + lane / (kCols / 8);
    l.col = (int)(item - group * per) * kCols + (int)(lane % (kCols / 8)) * 8;
    l.live = l.t < T && l.col < width;
    return l;
}

// Eight columns d0 .. d0 + 7 of a token into its tile.
template <int DT, int BITS, int D>
__device__ __forceinline__ void write_unit(const CacheArgs& A, int side, int64_t tile, int token, int d0, u32x4 raw)
{
    uint8_t* dst = A.codes[side] + tile * nma::tile_bytes(D, BITS);
    if constexpr (BITS == 16) {
        if (side == 0) {
            *reinterpret_cast<u32x4*>(dst + nma::k_offset(D, BITS, token, d0)) = raw;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint16_t*>(dst + nma::v_offset(D, BITS, token, d0 + j)) =
                    (uint16_t)(raw[j / 2] >> (16 * (j % 2)));
        }
    } else {
        float x[8], top = 0.0f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 p = unpack2<DT>(raw[j]);
            x[2 * j] = p.x;
            x[2 * j + 1] = p.y;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bad |= (f32_bits(x[j]) & 0x7F800000u) == 0x7F800000u;
            top = fmaxf(top, fabsf(x[j]));
        }
        if (bad)
            top = bits_f32(0x7F800000u);
        top = fmaxf(top, __shfl_xor(top, 1));
        top = fmaxf(top, __shfl_xor(top, 2));
        bad = f32_bits(top) == 0x7F800000u;
        const int byte = bad ? 255 : scale_byte<DT, BITS>(top);
        // x 2^-e is exact (a code's subnormals lie far above fp32's), so one rounding
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = bad ? 0.0f : ldexpf(x[j], nma::scale_bias(DT) - byte);
        if constexpr (BITS == 8) {
            u32x2 c = {0u, 0u};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                c[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * j], x[4 * j + 1], (int)c[j], false);
                c[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * j + 2], x[4 * j + 3], (int)c[j], true);
            }
            if (side == 0 || D >= 128) {
                const int at = side ? nma::v_offset(D, BITS, token, d0) : nma::k_offset(D, BITS, token, d0);
                *reinterpret_cast<u32x2*>(dst + at) = c;
            } else {
                *reinterpret_cast<uint32_t*>(dst + nma::v_offset(D, BITS, token, d0)) = c[0];
                *reinterpret_cast<uint32_t*>(dst + nma::v_offset(D, BITS, token, d0 + 4)) = c[1];
            }
        } else {
            uint32_t c = 0u;
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], 1.0f, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], 1.0f, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], 1.0f, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], 1.0f, 3);
            if (side == 0 || D >= 128) {
                const int at = side ? nma::v_offset(D, BITS, token, d0) : nma::k_offset(D, BITS, token, d0);
                *reinterpret_cast<uint32_t*>(dst + at) = c;
            } else {
                *reinterpret_cast<uint16_t*>(dst + nma::v_offset(D, BITS, token, d0)) = (uint16_t)c;
                *reinterpret_cast<uint16_t*>(dst + nma::v_offset(D, BITS, token, d0 + 4)) = (uint16_t)(c >> 16);
            }
        }
        if (d0 % nma::kBlock == 0) {
            const int at = side ? nma::v_scale_offset(token, d0 / nma::kBlock) : nma::k_scale_offset(D, token, d0 / nma::kBlock);
            A.scales[side][tile * nma::scale_tile_bytes(D) + at] = (uint8_t)byte;
        }
    }
}

template <int DT, int BITS, int D>
__global__ __launch_bounds__(kCacheThreads) void kv_write_kernel(const CacheArgs A, const uint16_t* __restrict__ k,
                                                                 const uint16_t* __restrict__ v, int64_t k_stride,
                                                                 int64_t v_stride)
{
    const Lane l = lane_of<1>(A.T, A.heads * D);
    if (!l.live)                    // rows and blocks of 32 columns leave whole, and with them the lanes of a scale
        return;
    const u32x4 kr = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(k + l.t * k_stride + l.col));
    const u32x4 vr = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(v + l.t * v_stride + l.col));
    const int64_t slot = A.slots[l.t];
    if (slot < 0 || slot >= A.n_slots)
        return;
    int token;
    const int64_t tile = tile_of(A, slot, l.col / D, token);
    write_unit<DT, BITS, D>(A, 0, tile, token, l.col % D, kr);
    write_unit<DT, BITS, D>(A, 1, tile, token, l.col % D, vr);
}

// Largest finite value of a 16-bit type, as fp32.
template <int DT>
__device__ __forceinline__ float finite_max()
{
    return DT == NM_FP16 ? 65504.0f : bits_f32(0x7F7F0000u);
}

template <int DT>
__device__ __forceinline__ float saturate(float v)
{
    const float m = finite_max<DT>();
    return v > m ? m : v < -m ? -m : v;         // a NaN stays one
}

// Eight columns of a token out of its tile.
template <int DT, int BITS, int D>
__device__ __forceinline__ u32x4 read_unit(const CacheArgs& A, int side, int64_t tile, int token, int d0)
{
    u32x4 out = {0u, 0u, 0u, 0u};
    const uint8_t* src = A.codes[side] + tile * nma::tile_bytes(D, BITS);
    if constexpr (BITS == 16) {
        if (side == 0) {
            out = *reinterpret_cast<const u32x4*>(src + nma::k_offset(D, BITS, token, d0));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                out[j / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(src + nma::v_offset(D, BITS, token, d0 + j))
                              << (16 * (j % 2));
        }
    } else {
        const int at = side ? nma::v_scale_offset(token, d0 / nma::kBlock) : nma::k_scale_offset(D, token, d0 / nma::kBlock);
        const uint32_t byte = A.scales[side][tile * nma::scale_tile_bytes(D) + at];
        float x[8];
        const int p0 = side ? nma::v_offset(D, BITS, token, d0) : nma::k_offset(D, BITS, token, d0);
        const int p1 = side ? nma::v_offset(D, BITS, token, d0 + 4) : p0 + 4 * BITS / 8;
        // the eight columns lie side by side but for values of D = 64 (four and four)
        const bool whole = side == 0 || D >= 128;
        if constexpr (BITS == 8) {
            u32x2 c;
            if (whole)
                c = *reinterpret_cast<const u32x2*>(src + p0);
            else
                c = u32x2{*reinterpret_cast<const uint32_t*>(src + p0), *reinterpret_cast<const uint32_t*>(src + p1)};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], false);
                const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], true);
                x[4 * j] = lo.x, x[4 * j + 1] = lo.y, x[4 * j + 2] = hi.x, x[4 * j + 3] = hi.y;
            }
        } else {
            const uint32_t c = whole ? *reinterpret_cast<const uint32_t*>(src + p0)
                                     : (uint32_t)*reinterpret_cast<const uint16_t*>(src + p0) |
                                           (uint32_t)*reinterpret_cast<const uint16_t*>(src + p1) << 16;
            const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0),
                                __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1),
                                __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2),
                                __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3)};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[2 * j] = p[j].x, x[2 * j + 1] = p[j].y;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = byte == 255u ? scale_value(byte) : saturate<DT>(ldexpf(x[j], (int)byte - nma::scale_bias(DT)));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            out[j] = pack2<DT>(x[2 * j], x[2 * j + 1]);
    }
    return out;
}

template <int DT, int BITS, int D>
__global__ __launch_bounds__(kCacheThreads) void kv_read_kernel(const CacheArgs A, uint16_t* __restrict__ k,
                                                                uint16_t* __restrict__ v)
{
    constexpr int UNITS = read_units(BITS);
    const Lane l = lane_of<UNITS>(A.T, A.heads * D);
    if (!l.live)
        return;
    int64_t slot[UNITS];
    u32x4 kr[UNITS], vr[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
        slot[u] = l.t + u * kRows < A.T ? A.slots[l.t + u * kRows] : -1;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        kr[u] = vr[u] = u32x4{0u, 0u, 0u, 0u};
        if (slot[u] >= 0 && slot[u] < A.n_slots) {
            int token;
            const int64_t tile = tile_of(A, slot[u], l.col / D, token);
            kr[u] = read_unit<DT, BITS, D>(A, 0, tile, token, l.col % D);
            vr[u] = read_unit<DT, BITS, D>(A, 1, tile, token, l.col % D);
        }
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        if (l.t + u * kRows >= A.T)
            break;
        const int64_t at = (l.t + u * kRows) * A.heads * D + l.col;
        __builtin_nontemporal_store(kr[u], reinterpret_cast<u32x4*>(k + at));
        __builtin_nontemporal_store(vr[u], reinterpret_cast<u32x4*>(v + at));
    }
}

CacheArgs cache_args(const nm_kv_cache& c, const int64_t* slots, int64_t T)
{
    CacheArgs A;
    A.codes[0] = static_cast<uint8_t*>(c.k);
    A.codes[1] = static_cast<uint8_t*>(c.v);
    A.scales[0] = c.k_scale;
    A.scales[1] = c.v_scale;
    A.slots = slots;
    A.n_slots = c.n_pages * c.page_size;
    A.T = T;
    A.page_shift = __builtin_ctz((unsigned)c.page_size);
    A.heads = c.heads;
    return A;
}

// Calls fn.template operator()<DT, BITS, D>() for a cache's type, format and width.
template <typename Fn>
int by_cache(const nm_kv_cache& c, Fn fn)
{
    auto by_width = [&](auto dt, auto bits) {
        switch (c.D) {
        case 64: return fn(dt, bits, std::integral_constant<int, 64>());
        case 128: return fn(dt, bits, std::integral_constant<int, 128>());
        default: return fn(dt, bits, std::integral_constant<int, 256>());
        }
    };
    auto by_bits = [&](auto dt) {
        switch (nma::format_bits(c.format)) {
        case 16: return by_width(dt, std::integral_constant<int, 16>());
        case 8: return by_width(dt, std::integral_constant<int, 8>());
        default: return by_width(dt, std::integral_constant<int, 4>());
        }
    };
    return c.dtype == NM_FP16 ? by_bits(std::integral_constant<int, NM_FP16>())
                              : by_bits(std::integral_constant<int, NM_BF16>());
}

int cache_grid(const nm_kv_cache& c, int64_t T, int units, dim3* grid)
{
    const int64_t items = nma::ceil_div(T, kRows * units) * nma::ceil_div((int64_t)c.heads * c.D, kCols);
    if (items > INT32_MAX)
        return NM_ERR_BAD_SHAPE;
    *grid = flat_grid(nma::ceil_div(items, kCacheThreads / 64));
    return NM_OK;
}

}  // namespace

int nmk::qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t T, int Hq, int Hk,
                      int D, int dtype, const void* wq, const void* wk, float eps, const int32_t* positions,
                      const float* inv_freq, int rot, int interleaved, void* q_out, void* k_out, void* stream)
{
    QkArgs A;
    A.x[0] = static_cast<const uint16_t*>(q);
    A.x[1] = static_cast<const uint16_t*>(k);
    A.y[0] = static_cast<uint16_t*>(q_out);
    A.y[1] = static_cast<uint16_t*>(k_out);
    A.w[0] = static_cast<const uint16_t*>(wq);
    A.w[1] = static_cast<const uint16_t*>(wk);
    A.stride[0] = T > 1 ? q_stride : 0;
    A.stride[1] = T > 1 ? k_stride : 0;
    A.heads[0] = Hq;
    A.heads[1] = Hk;
    A.T = T;
    A.D = D;
    A.rot = rot;
    A.eps = eps;
    A.positions = positions;
    A.inv_freq = inv_freq;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == NM_FP16 ? launch_qk_dt<NM_FP16>(A, interleaved != 0, T, s)
                            : launch_qk_dt<NM_BF16>(A, interleaved != 0, T, s);
}

int nmk::kv_write(const nm_kv_cache& cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T,
                  const int64_t* slots, void* stream)
{
    dim3 grid;
    if (cache_grid(cache, T, 1, &grid) != NM_OK)
        return NM_ERR_BAD_SHAPE;
    const CacheArgs A = cache_args(cache, slots, T);
    return by_cache(cache, [&](auto dt, auto bits, auto d) {
        (void)hipGetLastError();
        hipLaunchKernelGGL((kv_write_kernel<dt(), bits(), d()>), grid, dim3(kCacheThreads), 0,
                           static_cast<hipStream_t>(stream), A, static_cast<const uint16_t*>(k),
                           static_cast<const uint16_t*>(v), T > 1 ? k_stride : 0, T > 1 ? v_stride : 0);
        return hip_status(hipGetLastError());
    });
}

int nmk::kv_read(const nm_kv_cache& cache, const int64_t* slots, int64_t T, void* k, void* v, void* stream)
{
    dim3 grid;
    if (cache_grid(cache, T, read_units(nma::format_bits(cache.format)), &grid) != NM_OK)
        return NM_ERR_BAD_SHAPE;
    const CacheArgs A = cache_args(cache, slots, T);
    return by_cache(cache, [&](auto dt, auto bits, auto d) {
        (void)hipGetLastError();
        hipLaunchKernelGGL((kv_read_kernel<dt(), bits(), d()>), grid, dim3(kCacheThreads), 0,
                           static_cast<hipStream_t>(stream), A, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
        return hip_status(hipGetLastError());
    });
}
