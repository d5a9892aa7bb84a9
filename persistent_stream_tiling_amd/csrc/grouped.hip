// Products whose rows choose their matrix: C[r] = A[r] . B[group of r] for
// rows sorted by group, and the gradient of the matrices, C[g] = A_g^T . D_g.
// gfx950.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "device.h"
#include "errors.h"
#include "gemm_sk.h"
#include "grouped.h"

namespace gsk {

using namespace dev;

namespace {

// ---------------------------------------------------------------------------
// Exact-product kernel: operands are widened to fp32 in LDS and multiplied by
// the fp32 matrix instruction, 128x128 tiles, any sizes and alignments.
//
// An operand is a slab of 128 rows (m or n) by 16 k per iteration.  It lies in
// memory either with k contiguous (KC: 8 consecutive k per thread) or with
// m / n contiguous (8 consecutive m per thread), and in LDS always as
// [k][m], the order the 32x32x2 instruction reads (lane l: row l % 32, k = l /
// 32).  LDS rows are 160 floats apart: the two k rows that one read touches
// are then 32 banks apart.  Two LDS buffers; the next slab's loads are in
// flight while the current one is multiplied.
constexpr int kXTile = 128, kXDeep = 16, kXThreads = 256, kXPitch = 160;

template <typename T>
struct Packed8 {
    struct __attribute__((packed, aligned(sizeof(T)))) Words {
        uint32_t w[8 * sizeof(T) / 4];
    };
};

// Eight consecutive elements at p, of which the first n (0 .. 8) exist.
template <typename T>
__device__ __forceinline__ void load8(float (&x)[8], const T *p, int n)
{
    T t[8];
    if (n >= 8) {
        const auto w = *(const typename Packed8<T>::Words *)p;
        __builtin_memcpy(t, &w, sizeof(t));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            t[e] = e < n ? p[e] : (T)0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = (float)t[e];
}

// One thread's share of a slab: rows [0, rows) x k [0, k) exist at p.
template <typename T, bool KC>
__device__ __forceinline__ void load_slab(float (&x)[8], const T *p, int64_t ld, int rows, int k)
{
    const int tid = threadIdx.x;
    const int r = KC ? tid >> 1 : (tid & 15) * 8, kk = KC ? (tid & 1) * 8 : tid >> 4;
    const int n = KC ? (r < rows ? k - kk : 0) : (kk < k ? rows - r : 0);
    load8(x, KC ? p + r * ld + kk : p + kk * ld + r, n);
}

template <bool KC>
__device__ __forceinline__ void park_slab(float *lds, const float (&x)[8])
{
    const int tid = threadIdx.x;
    if constexpr (KC) {
        const int r = tid >> 1, kk = (tid & 1) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            lds[(kk + e) * kXPitch + r] = x[e];
    } else {
        float *p = lds + (tid >> 4) * kXPitch + (tid & 15) * 8;
        *(f32x4 *)p = f32x4{x[0], x[1], x[2], x[3]};
        *(f32x4 *)(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
    }
}

// acc (2 x 2 blocks of 32x32 per wave, 2 x 2 waves) = the tile's sums over k
// in [0, k).  The operands are swapped in the instruction, so lane l holds
// C[32*mt + l % 32][32*nt + 8*g + 4*(l / 32) + e] in register 4*g + e.
template <typename T, bool A_KC, bool B_KC>
__device__ __forceinline__ void exact_tile(f32x16 (&acc)[2][2], float *lds, const T *a, int64_t lda,
                                           int m, const T *b, int64_t ldb, int n, int k)
{
    constexpr int kSlab = kXDeep * kXPitch;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int half = lane >> 5, l32 = lane & 31;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const int64_t a_step = A_KC ? kXDeep : kXDeep * lda, b_step = B_KC ? kXDeep : kXDeep * ldb;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        acc[i >> 1][i & 1] = f32x16{};
    float xa[8], xb[8];
    if (k > 0) {
        load_slab<T, A_KC>(xa, a, lda, m, k);
        load_slab<T, B_KC>(xb, b, ldb, n, k);
    }
    for (int k0 = 0, buf = 0; k0 < k; k0 += kXDeep, buf ^= 1) {
        float *sa = lds + buf * 2 * kSlab, *sb = sa + kSlab;
        park_slab<A_KC>(sa, xa);
        park_slab<B_KC>(sb, xb);
        // one barrier per slab: a wave two slabs on would overwrite this
        // buffer, and to get there it has to pass the next barrier
        __syncthreads();
        if (k0 + kXDeep < k) {
            a += a_step;
            b += b_step;
            load_slab<T, A_KC>(xa, a, lda, m, k - k0 - kXDeep);
            load_slab<T, B_KC>(xb, b, ldb, n, k - k0 - kXDeep);
        }
#pragma unroll
        for (int kk = 0; kk < kXDeep; kk += 2) {
            const int row = (kk + half) * kXPitch + l32;
            float fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = sa[row + wm + 32 * i];
                fb[i] = sb[row + wn + 32 * i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i >> 1][i & 1] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[i & 1], fa[i >> 1],
                                                                          acc[i >> 1][i & 1], 0, 0, 0);
        }
    }
}

// Rows m0 .. and columns n0 .. of the tile to C, whose row m0 starts at c.
__device__ __forceinline__ void store_exact(const f32x16 (&acc)[2][2], uint8_t *c, int64_t ldc,
                                            int m, int n0, int N, int c_dtype, bool c_vec)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int half = lane >> 5, l32 = lane & 31;
    const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(c);
    const bool vec = c_vec || n0 + kXTile <= N;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
        const int row = (wave >> 1) * 64 + 32 * mt + l32;
        const uint32_t row_off = (uint32_t)(row * ldc * (c_dtype ? 2 : 4));
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                store_four(f32x4{acc[mt][nt][4 * g], acc[mt][nt][4 * g + 1], acc[mt][nt][4 * g + 2],
                                 acc[mt][nt][4 * g + 3]},
                           rsrc, row_off, n0 + (wave & 1) * 64 + 32 * nt + 8 * g + 4 * half, N,
                           row < m, vec, c_dtype);
    }
}

template <typename T, bool B_KC>
__global__ __launch_bounds__(kXThreads) void rows_exact_kernel(GroupedArgs a)
{
    __shared__ __attribute__((aligned(16))) float lds[4 * kXDeep * kXPitch];
    RowTile t;
    if (!find_row_tile<kXTile>(a, blockIdx.x, &t))
        return;
    const int n0 = t.tn * kXTile, m = t.m_end - t.m0 < kXTile ? t.m_end - t.m0 : kXTile;
    const T *A = (const T *)a.A + (int64_t)t.m0 * a.lda;
    // (the rows past the last group multiply nothing: depth 0)
    const T *B = (const T *)a.B + (t.g < a.groups ? t.g * a.b_stride : 0) +
                 (B_KC ? (int64_t)n0 * a.ldb : n0);
    f32x16 acc[2][2];
    exact_tile<T, true, B_KC>(acc, lds, A, a.lda, m, B, a.ldb, a.N - n0, t.g < a.groups ? a.K : 0);
    store_exact(acc, a.C + (int64_t)t.m0 * a.N * (a.c_dtype ? 2 : 4), a.N, m, n0, a.N, a.c_dtype,
                a.c_vec);
}

template <typename T>
__global__ __launch_bounds__(kXThreads) void wgrad_exact_kernel(GroupedArgs a)
{
    __shared__ __attribute__((aligned(16))) float lds[4 * kXDeep * kXPitch];
    const int64_t per = (int64_t)a.tiles_m * a.tiles_n;
    const int32_t g = (int32_t)(blockIdx.x / per);
    const int32_t in = (int32_t)(blockIdx.x - g * per);
    const int m0 = in / a.tiles_n * kXTile, n0 = in % a.tiles_n * kXTile;
    int32_t lo, hi;
    group_rows(a.offsets, g, a.groups, a.rows, &lo, &hi);
    f32x16 acc[2][2];
    exact_tile<T, false, false>(acc, lds, (const T *)a.A + (int64_t)lo * a.lda + m0, a.lda, a.M - m0,
                                (const T *)a.B + (int64_t)lo * a.ldb + n0, a.ldb, a.N - n0, hi - lo);
    store_exact(acc, a.C + ((int64_t)g * a.M + m0) * a.N * (a.c_dtype ? 2 : 4), a.N, a.M - m0, n0,
                a.N, a.c_dtype, a.c_vec);
}

int elem_bytes(int dtype)
{
    return dtype == GEMM_F32 ? 4 : (dtype == GEMM_F16 || dtype == GEMM_BF16 ? 2 : 0);
}

constexpr int kMaxGroups = 4096;

// Shared argument checks of both products; 0 or -1.
int check(const gemm_grouped *p)
{
    if (!p) {
        set_error("NULL problem");
        return -1;
    }
    if (p->op != GEMM_GROUPED_ROWS && p->op != GEMM_GROUPED_ROWS_BT && p->op != GEMM_GROUPED_WGRAD) {
        set_error("unknown grouped product %d", p->op);
        return -1;
    }
    if (!elem_bytes(p->dtype)) {
        set_error("grouped products take fp32, fp16 or bf16; got dtype %d", p->dtype);
        return -1;
    }
    if (p->flags & ~(uint32_t)GEMM_FLAG_C_INPUT_DTYPE) {
        set_error("grouped products take no flag but GEMM_FLAG_C_INPUT_DTYPE (flags 0x%x)", p->flags);
        return -1;
    }
    if (p->rows < 0 || p->K < 0 || p->N < 0 || p->groups < 1) {
        set_error("rows, K and N must not be negative and groups at least 1");
        return -1;
    }
    if (p->groups > kMaxGroups) {
        set_error("groups must be at most %d, got %d", kMaxGroups, p->groups);
        return -1;
    }
    // the kernels address inside a tile's rows and inside one k slab with
    // 32-bit byte offsets
    const int64_t widest = (int64_t)1 << 20;
    if (p->rows >= ((int64_t)1 << 31) - 1024 || p->K >= widest || p->N >= widest) {
        set_error("rows must stay below 2^31 - 1024, K and N below 2^20");
        return -1;
    }
    return 0;
}

}  // namespace
}  // namespace gsk

using namespace gsk;

extern "C" {

size_t gemm_grouped_workspace_size(const gemm_grouped *p)
{
    (void)p;
    return 0;
}

int gemm_grouped_run(const gemm_grouped *p, const int32_t *offsets, const void *A, const void *B,
                     void *C, void *workspace, void *stream)
{
    if (check(p))
        return -1;
    const bool wgrad = p->op == GEMM_GROUPED_WGRAD;
    const int64_t c_rows = wgrad ? p->groups * p->K : p->rows;
    if (c_rows == 0 || p->N == 0)
        return 0;
    const int c_dtype = (p->flags & GEMM_FLAG_C_INPUT_DTYPE) ? p->dtype : GEMM_F32;
    const int E = elem_bytes(p->dtype), CE = elem_bytes(c_dtype);
    const bool reads = p->rows > 0 && p->K > 0;
    if (!offsets || !C || (reads && (!A || !B))) {
        set_error("NULL argument");
        return -1;
    }
    if (((uintptr_t)offsets & 3) || ((uintptr_t)C & (CE - 1)) || ((uintptr_t)A & (E - 1)) ||
        ((uintptr_t)B & (E - 1))) {
        set_error("misaligned pointer");
        return -1;
    }
    (void)workspace;
    GroupedArgs a{};
    a.A = (const uint8_t *)A;
    a.B = (const uint8_t *)B;
    a.C = (uint8_t *)C;
    a.offsets = offsets;
    a.rows = (int32_t)p->rows;
    a.groups = p->groups;
    a.N = (int32_t)p->N;
    a.K = (int32_t)p->K;
    a.M = (int32_t)p->K;
    a.b_stride = p->K * p->N;
    a.lda = (int32_t)p->K;
    a.ldb = (int32_t)(p->op == GEMM_GROUPED_ROWS_BT ? p->K : p->N);
    a.c_dtype = c_dtype;
    a.c_vec = p->N % 4 == 0 && ((uintptr_t)C & (4 * CE - 1)) == 0;
    a.xcds = 8;
    a.tiles_n = (int32_t)((p->N + kXTile - 1) / kXTile);
    a.tiles_m = (int32_t)((p->K + kXTile - 1) / kXTile);
    int64_t tiles;
    if (wgrad) {
        tiles = (int64_t)p->groups * a.tiles_m * a.tiles_n;
    } else {
        // a group's rows, and those past the last group, end inside a tile
        const int64_t ends = p->groups + 1 < p->rows ? p->groups + 1 : p->rows;
        tiles = (p->rows / kXTile + ends) * a.tiles_n;
        tiles = (tiles + a.xcds - 1) / a.xcds * a.xcds;
    }
    if (tiles >= ((int64_t)1 << 32) / kXThreads) {
        set_error("too many tiles for one launch (%lld)", (long long)tiles);
        return -1;
    }
    const hipStream_t s = (hipStream_t)stream;
#define GSK_EXACT(T)                                                                             \
    do {                                                                                         \
        if (wgrad)                                                                               \
            hipLaunchKernelGGL((wgrad_exact_kernel<T>), dim3((unsigned)tiles), dim3(kXThreads),  \
                               0, s, a);                                                         \
        else if (p->op == GEMM_GROUPED_ROWS_BT)                                                  \
            hipLaunchKernelGGL((rows_exact_kernel<T, true>), dim3((unsigned)tiles),              \
                               dim3(kXThreads), 0, s, a);                                        \
        else                                                                                     \
            hipLaunchKernelGGL((rows_exact_kernel<T, false>), dim3((unsigned)tiles),             \
                               dim3(kXThreads), 0, s, a);                                        \
    } while (0)
    if (p->dtype == GEMM_F32)
        GSK_EXACT(float);
    else if (p->dtype == GEMM_F16)
        GSK_EXACT(_Float16);
    else
        GSK_EXACT(__bf16);
#undef GSK_EXACT
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        set_error("grouped product launch failed: %s", hipGetErrorString(e));
        return -3;
    }
    return 0;
}

}  // extern "C"
