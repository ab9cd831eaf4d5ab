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
