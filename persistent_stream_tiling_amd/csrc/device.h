// Device helpers of the kernels whose rows choose their matrix: vector types,
// raw buffer descriptors and the rounding stores of C.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gsk {
namespace dev {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kOutOfRange = 0x80000000u;  // a buffer offset that is never in range

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, 0x7fffffff,
                                             0x00020000);
}

// Reinterpretations are by value: a bit cast applied to one subscripted
// element of a vector lvalue has been lowered to a read of element 0.
__device__ __forceinline__ uint32_t bits_of(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ uint32_t f16_bits(float x)
{
    return __builtin_bit_cast(uint16_t, (_Float16)x);
}
__device__ __forceinline__ uint32_t bf16_bits(float x)
{
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// Four consecutive columns n .. n + 3 of a row of C, at byte offset `row_off`
// of the descriptor's base; ok: the row is inside C.  c_dtype: 0 fp32, 1 fp16,
// 2 bf16, rounded to nearest even from the fp32 sums.  vec (uniform): the four
// are all inside C or all outside.  Elements outside get an out-of-range
// offset, which drops the write.
__device__ __forceinline__ void store_four(const f32x4 &v, __amdgpu_buffer_rsrc_t c,
                                           uint32_t row_off, int n, int N, bool ok, bool vec,
                                           int c_dtype)
{
    if (c_dtype != 0) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = c_dtype == 1 ? f16_bits(v[e]) : bf16_bits(v[e]);
        const uint32_t off = row_off + (uint32_t)n * 2;
        if (vec) {
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)}, c,
                                                  (int)(ok && n < N ? off : kOutOfRange), 0, 0);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                __builtin_amdgcn_raw_buffer_store_b16(
                    (uint16_t)h[e], c, (int)(ok && n + e < N ? off + 2 * e : kOutOfRange), 0, 0);
        }
        return;
    }
    const uint32_t off = row_off + (uint32_t)n * 4;
    const u32x4 u = u32x4{bits_of(v[0]), bits_of(v[1]), bits_of(v[2]), bits_of(v[3])};
    if (vec) {
        __builtin_amdgcn_raw_buffer_store_b128(u, c, (int)(ok && n < N ? off : kOutOfRange), 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            __builtin_amdgcn_raw_buffer_store_b32(
                u[e], c, (int)(ok && n + e < N ? off + 4 * e : kOutOfRange), 0, 0);
    }
}

}  // namespace dev
}  // namespace gsk
