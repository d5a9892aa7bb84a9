// Device helpers of the kernels whose rows choose their matrix: vector types,
// raw buffer descriptors and the rounding stores of C.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gsk {
namespace dev {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

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

__device__ __forceinline__ f32x4 as_floats(u32x4 x) { return __builtin_bit_cast(f32x4, x); }

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

// One 32x32 accumulator block (rows brow .., columns col .. of C; rows_ok: how
// many rows from the descriptor's base exist).  Lane l holds row brow + l % 32
// at columns col + 8g + 4(l / 32) + e in register 4g + e.  For vector stores,
// quads 2j and 2j + 1 are exchanged first (v_permlane16_swap: lanes 16-31 and
// 48-63 of the one with lanes 0-15 and 32-47 of the other), so that each store
// covers 16 rows with 64 contiguous bytes (32 for 16-bit C) instead of 32 rows
// with 32.
__device__ __forceinline__ void store_block(const f32x16 &blk, __amdgpu_buffer_rsrc_t c,
                                            uint32_t row_bytes, int brow, int rows_ok, int col,
                                            int N, bool vec, int c_dtype)
{
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // (as in store_lines)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const f32x4 q0 = f32x4{blk[8 * j], blk[8 * j + 1], blk[8 * j + 2], blk[8 * j + 3]};
        const f32x4 q1 = f32x4{blk[8 * j + 4], blk[8 * j + 5], blk[8 * j + 6], blk[8 * j + 7]};
        if (vec) {
            f32x4 lo, hi;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const auto r =
                    __builtin_amdgcn_permlane16_swap(bits_of(q0[e]), bits_of(q1[e]), false, false);
                lo[e] = __builtin_bit_cast(float, (uint32_t)r[0]);
                hi[e] = __builtin_bit_cast(float, (uint32_t)r[1]);
            }
            const int row = brow + (lane & 15);
            const int n = col + 16 * j + 8 * ((lane >> 4) & 1) + 4 * (lane >> 5);
            store_four(lo, c, (uint32_t)row * row_bytes, n, N, row < rows_ok, true, c_dtype);
            store_four(hi, c, (uint32_t)(row + 16) * row_bytes, n, N, row + 16 < rows_ok, true,
                       c_dtype);
        } else {
            const int row = brow + (lane & 31), n = col + 16 * j + 4 * (lane >> 5);
            store_four(q0, c, (uint32_t)row * row_bytes, n, N, row < rows_ok, false, c_dtype);
            store_four(q1, c, (uint32_t)row * row_bytes, n + 8, N, row < rows_ok, false, c_dtype);
        }
    }
}

// A wave's 32 rows by 64 columns (two accumulator blocks side by side) to C, in
// whole 128-byte lines: the caches take a store line by line, and from the
// accumulators' order a store would touch 16 lines for 512 or 1024 bytes (a
// 256x256 bf16 tile took 9 us to store, all CUs at it).  So 32 rows of 128
// bytes (64 columns of 16 bits, or 32 of 32) pass through 4 KiB of LDS of the
// wave's own: 16-byte chunk c of row r sits at c ^ (r & 7), which keeps writes
// and reads free of bank conflicts, and each store covers 8 rows.  Where a
// chunk could straddle C's last column (`whole` false) blocks are stored as
// they lie.
__device__ __forceinline__ void store_lines(const f32x16 &left, const f32x16 &right, uint8_t *lds,
                                            __amdgpu_buffer_rsrc_t c, uint32_t row_bytes, int brow,
                                            int rows_ok, int col, int N, bool whole, bool vec,
                                            int c_dtype)
{
    if (!whole) {
        store_block(left, c, row_bytes, brow, rows_ok, col, N, vec, c_dtype);
        store_block(right, c, row_bytes, brow, rows_ok, col + 32, N, vec, c_dtype);
        return;
    }
    // (opaque, so that the addresses below are formed here: formed once, ahead of
    // a loop over tiles, they would occupy registers its products need)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int row = lane & 31, half = lane >> 5;
    const auto at = [](int r, int chunk) { return (uint32_t)(r * 128 + ((chunk ^ (r & 7)) << 4)); };
    // the rows' 128 bytes from column n on
    const auto send = [&](int n, int columns_per_chunk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 3), chunk = (lane & 7) ^ (r & 7);
            const u32x4 v = *(const u32x4 *)(lds + r * 128 + ((lane & 7) << 4));
            const int cn = n + chunk * columns_per_chunk;
            const uint32_t off = (uint32_t)(brow + r) * row_bytes + (uint32_t)cn * (16 / columns_per_chunk);
            __builtin_amdgcn_raw_buffer_store_b128(
                v, c, (int)(brow + r < rows_ok && cn < N ? off : kOutOfRange), 0, 0);
        }
    };
    if (c_dtype != 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x16 &b = j ? right : left;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    h[e] = c_dtype == 1 ? f16_bits(b[4 * g + e]) : bf16_bits(b[4 * g + e]);
                *(u32x2 *)(lds + at(row, 4 * j + g) + 8 * half) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
            }
        }
        send(col, 8);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x16 &b = j ? right : left;
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *(u32x4 *)(lds + at(row, 2 * g + half)) = u32x4{bits_of(b[4 * g]), bits_of(b[4 * g + 1]),
                                                              bits_of(b[4 * g + 2]), bits_of(b[4 * g + 3])};
            send(col + 32 * j, 4);
        }
    }
}

// ---- direct global -> LDS copies and the rings they fill

__device__ __forceinline__ void barrier_only()
{
    // no memory fence: the callers' s_waitcnt order what they need; the asm
    // keeps the compiler from moving LDS accesses across it
    asm volatile("s_barrier" ::: "memory");
}

// A compile-time index as an argument.
template <int V>
struct IC {
    static constexpr int value = V;
};

template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void wait_lds()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// A raw buffer descriptor (base, no stride, 2^31 - 1 bytes, untyped) as words.
__device__ __forceinline__ i32x4 rsrc_words(const void *base)
{
    const uint64_t b = (uint64_t)base;
    return i32x4{(int)(uint32_t)b, (int)((uint32_t)(b >> 32) & 0xffff), 0x7fffffff, 0x00020000};
}

// 16 bytes per lane from buffer offset voff (kOutOfRange: zeros) into LDS at
// lds_addr + 16 * lane (lds_addr wave-uniform).  Inline assembly, so that the
// compiler does not wait for every copy in flight before each transposing LDS
// read; the callers' s_waitcnt vmcnt() and barriers order the copies.
__device__ __forceinline__ void copy16(i32x4 rsrc, uint32_t voff, uint32_t lds_addr)
{
    asm volatile("s_mov_b32 m0, %0\n\t"
                 "s_nop 0\n\t"
                 "buffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(voff), "s"(rsrc)
                 : "m0");
}

#define GSK_LDS_PTR(T, p) ((__attribute__((address_space(3))) T *)(p))

__device__ __forceinline__ uint32_t lds_address(const uint8_t *p)
{
    return (uint32_t)(uintptr_t)GSK_LDS_PTR(const uint8_t, p);
}

// 16-byte chunk c of a 128-byte LDS row r sits at c ^ swz_row(r): eight rows
// read at one chunk index then touch all 32 bank pairs.
__device__ __forceinline__ uint32_t swz_row(int row) { return (uint32_t)(row ^ (row >> 3)) & 7; }

// Chunk c of k-row r of a slab stored k-row by k-row sits at c ^ swz_krow(r)
// ({0, 6, 10, 12} by r mod 4): the four k-rows that one half of a transposing
// read touches fall on distinct banks.
__device__ __forceinline__ uint32_t swz_krow(int krow) { return (0xCA60u >> ((krow & 3) * 4)) & 0xF; }

// acc += a . b^T for one 16-deep step of a 32x32 block, operands swapped so
// that the accumulator holds the transposed block (see store_block).
template <int DT>
__device__ __forceinline__ void mfma16(f32x16 &acc, const u32x4 &b, const u32x4 &a)
{
    if constexpr (DT == 1)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b),
                                                     __builtin_bit_cast(f16x8, a), acc, 0, 0, 0);
    else
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b),
                                                      __builtin_bit_cast(bf16x8, a), acc, 0, 0, 0);
}

}  // namespace dev
}  // namespace gsk
