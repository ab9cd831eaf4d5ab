// nm_device.h -- device helpers shared by the kernels behind include/nmattn.h:
// 16-bit floats, quantised codes and their scales, lane exchanges.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "nmspmv.h"

namespace nmd {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float bits_f32(uint32_t b) { return __builtin_bit_cast(float, b); }
__device__ __forceinline__ uint32_t f32_bits(float v) { return __builtin_bit_cast(uint32_t, v); }

// The two 16-bit floats of a dword (low half first).
template <int DT>
__device__ __forceinline__ f32x2 unpack2(uint32_t w)
{
    if constexpr (DT == NM_FP16) {
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        return f32x2{(float)h.x, (float)h.y};
    } else {
        return f32x2{bits_f32(w << 16), bits_f32(w & 0xFFFF0000u)};
    }
}

// Two fp32 to a dword of 16-bit floats, to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (DT == NM_FP16)
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    else
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// 2^(byte - 127) for scale bytes 1 .. 254; NaN for 255 (a block that held a NaN
// or an infinity).
__device__ __forceinline__ float scale_value(uint32_t byte)
{
    return bits_f32(byte == 255u ? 0x7FC00000u : byte << 23);
}

// 32 x 32 += 32 x 16 times 16 x 32: lane l holds row (of a) or column (of b) l % 32 and eight
// k indices from 8 (l / 32) on; of c column l % 32 and rows 8 (i / 4) + 4 (l / 32) + i % 4.
template <int DT>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (DT == NM_FP16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
}

// sum + the products of two pairs of 16-bit floats.
template <int DT>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float sum)
{
    if constexpr (DT == NM_FP16)
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), sum, false);
    else
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), sum, false);
}

// Maximum / sum of a lane and lane ^ 32.
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

// A grid of `blocks` blocks.  A grid dimension holds less than 2^32 threads, so many
// blocks are laid out in rows of kGridRow; flat_block() is the block's number, which
// may be `blocks` or more in the last row.
constexpr int64_t kGridRow = int64_t(1) << 22;

inline dim3 flat_grid(int64_t blocks)
{
    return blocks <= kGridRow ? dim3((unsigned)blocks)
                              : dim3((unsigned)kGridRow, (unsigned)((blocks + kGridRow - 1) / kGridRow));
}

__device__ __forceinline__ uint32_t flat_block() { return blockIdx.y * gridDim.x + blockIdx.x; }

}  // namespace nmd
