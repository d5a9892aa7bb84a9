// Low-rank adapters of many requests beside a shared projection:
//   Y[t] = X[t] . W + s[a] (X[t] . A[a]^T) . B[a]^T,   a = ids[t],
// in two launches: the rows' projections to rank r, H[t] = s[a] X[t] . A[a]^T,
// then the shared product, whose tiles add H[t] . B[a]^T to their sums before
// they are stored.  gfx950.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "errors.h"
#include "gemm_sk.h"
#include "kernels.h"
#include "tiles.h"

namespace gsk {

using namespace dev;

namespace {

typedef float f32x2v __attribute__((ext_vector_type(2)));

struct AdapterArgs {
    const uint8_t *X;        // rows x ldx
    const uint8_t *W;        // K x ldw, or N x ldw (linear-layer weights)
    const uint8_t *x_plain;  // X as the caller's (rows x K): the rank projection's operand
    const uint8_t *A;        // adapters x rank x K
    const uint8_t *B;        // adapters x N x rank
    const int32_t *ids;
    const float *scales;     // or NULL: all 1
    uint8_t *C;
    float *H;                // slices x rows x rank_pad
    float *partials;         // parts x tiles x (32 MT x 128), when parts > 1
    int32_t *counters;       // parts of a tile done; zeroed by the first launch
    int32_t rows, N, K, rank, rank_pad, adapters;
    int32_t ldx, ldw;
    int32_t slices, slice_k; // of the rank projection's depth
    int32_t parts, part_k;   // of the shared product's depth
    int32_t terms;           // 16-bit terms that H is split into
    int32_t tiles_m, tiles_n;
    int32_t c_dtype, c_vec, xcds;
};

// The row's adapter, -1 for none.
__device__ __forceinline__ int adapter_of(const AdapterArgs &a, int row)
{
    const int id = row < a.rows ? a.ids[row] : -1;
    return id >= 0 && id < a.adapters ? id : -1;
}

template <int DT>
struct Elem;
template <>
struct Elem<0> {
    typedef float T;
};
template <>
struct Elem<1> {
    typedef _Float16 T;
};
template <>
struct Elem<2> {
    typedef __bf16 T;
};

template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Words16 {
    uint32_t w[4];
};

// 16 bytes of elements at p, of which the first n exist (rows need not be
// whole 16-byte words: unaligned access is enabled).
template <typename T>
__device__ __forceinline__ u32x4 load_some(const T *p, int n)
{
    constexpr int V = 16 / (int)sizeof(T);
    if (n >= V) {
        const Words16<T> w = *(const Words16<T> *)p;
        return u32x4{w.w[0], w.w[1], w.w[2], w.w[3]};
    }
    T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
        t[e] = e < n ? p[e] : (T)0.0f;
    u32x4 r;
    __builtin_memcpy(&r, t, 16);
    return r;
}

// ---------------------------------------------------------------------------
// H[t] = s[a] X[t] . A[a]^T, 16 rows and one slice of the depth per workgroup
// of eight waves.
//
// The waves share the adapters present among the 16 rows out between them, and
// where there are fewer than eight, the depth as well; a wave multiplies all 16
// rows by one adapter's A (16x16 matrix instruction: 16 ranks by 16 rows) and
// keeps the rows that chose it.  So a row's sums hold nothing of another
// adapter's values, and neither does a row without one.  Operands go straight
// from memory to registers, 16 bytes per lane and load: each is used once.
// Bound by the reads of X and of the A present; a decoding step (32 rows of K =
// 4096, each with its own adapter) spreads them over 2 x 16 workgroups by
// slices, whose sums the second launch adds in order.
constexpr int kShrinkRows = 16, kShrinkWaves = 8;

template <int DT, int RT>  // RT: 16-rank blocks
__global__ __launch_bounds__(64 * kShrinkWaves) void shrink_kernel(AdapterArgs a)
{
    using T = typename Elem<DT>::T;
    constexpr int V = 16 / (int)sizeof(T);  // elements per load; a step is 4 V deep
    constexpr int kPitch = RT * 16 + 4;
    __shared__ __attribute__((aligned(16))) float red[kShrinkWaves][kShrinkRows][kPitch];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const int row0 = (int)blockIdx.x * kShrinkRows;
    if (a.parts > 1)
        for (int i = (int)(blockIdx.y * gridDim.x + blockIdx.x) * 64 * kShrinkWaves +
                     (int)threadIdx.x;
             i < a.tiles_m * a.tiles_n; i += (int)(gridDim.x * gridDim.y) * 64 * kShrinkWaves)
            a.counters[i] = 0;

    const int id = adapter_of(a, row0 + r16);
    uint64_t left = __builtin_amdgcn_ballot_w64(id >= 0) & 0xffff;
    int n = 0;
    for (uint64_t m = left; m; ++n)
        m &= ~__builtin_amdgcn_ballot_w64(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(m)));
    if (n == 0)
        return;  // nobody reads these rows' H
    const int ways = n < kShrinkWaves ? kShrinkWaves / n : 1;  // of the depth, per adapter
    const int k_lo = (int)blockIdx.y * a.slice_k;
    const int k_hi = k_lo + a.slice_k < a.K ? k_lo + a.slice_k : a.K;
    const int way = wave / n;  // (n < 8: waves past n * ways idle)
    const int per = ((k_hi - k_lo + ways - 1) / ways + 4 * V - 1) / (4 * V) * (4 * V);
    const int k0 = k_lo + way * per;
    const int k1 = k0 + per < k_hi ? k0 + per : k_hi;

    const T *x = (const T *)a.x_plain + (int64_t)(row0 + r16) * a.K;
    const bool x_ok = row0 + r16 < a.rows;
    int nth = 0;
    for (uint64_t m = left; m; ++nth) {
        const int mine = __builtin_amdgcn_readlane(id, __builtin_ctzll(m));
        m &= ~__builtin_amdgcn_ballot_w64(id == mine);
        if (n < kShrinkWaves ? (way >= ways || wave - way * n != nth) : nth % kShrinkWaves != wave)
            continue;
        f32x4 acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
            acc[t] = f32x4{};
        const T *A = (const T *)a.A + (int64_t)mine * a.rank * a.K;
#pragma unroll 2
        for (int k = k0; k < k1; k += 4 * V) {
            const int kk = k + q * V;
            const u32x4 fx = load_some(x + kk, x_ok ? k1 - kk : 0);
            u32x4 fa[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int r = t * 16 + r16;
                fa[t] = load_some(A + (int64_t)r * a.K + kk, r < a.rank ? k1 - kk : 0);
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                if constexpr (DT == 1) {
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        __builtin_bit_cast(f16x8, fa[t]), __builtin_bit_cast(f16x8, fx), acc[t], 0, 0, 0);
                } else if constexpr (DT == 2) {
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, fa[t]), __builtin_bit_cast(bf16x8, fx), acc[t], 0, 0, 0);
                } else {
                    // element e of both operands: the same k meets the same k
                    const f32x4 af = __builtin_bit_cast(f32x4, fa[t]), xf = __builtin_bit_cast(f32x4, fx);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(af[e], xf[e], acc[t], 0, 0, 0);
                }
            }
        }
        // lane: row r16, ranks 16 t + 4 q .. + 3
        if (id == mine)
#pragma unroll
            for (int t = 0; t < RT; ++t)
                *(f32x4 *)&red[n < kShrinkWaves ? way : 0][r16][t * 16 + 4 * q] = acc[t];
    }
    __syncthreads();
    float *h = a.H + (int64_t)blockIdx.y * a.rows * a.rank_pad;
    for (int i = threadIdx.x; i < kShrinkRows * RT * 16; i += 64 * kShrinkWaves) {
        const int row = i / (RT * 16), r = i % (RT * 16);
        const int of = adapter_of(a, row0 + row);
        if (of < 0 || r >= a.rank_pad)
            continue;
        float sum = red[0][row][r];
        for (int w = 1; w < ways; ++w)
            sum += red[w][row][r];
        h[(int64_t)(row0 + row) * a.rank_pad + r] = sum * (a.scales ? a.scales[of] : 1.0f);
    }
}

// ---------------------------------------------------------------------------
// acc += H . B^T for the rows that have an adapter: row blocks of 32 from row0
// on, column blocks of 32 from col0 on.  Of the adapters met in a wave's rows,
// this call takes those numbered `part`, part + parts, ...
//
// Per adapter and 16 ranks, one matrix product of all the block's rows is
// formed in registers of its own, and the rows that chose the adapter add it
// to theirs: another adapter's infinities and NaN never reach them.  H is fp32
// and the instruction takes 16 bits, so H is scaled by a power of two per row
// (largest magnitude of the 16 near 2^10: inside fp16's range, the terms above
// its subnormals) and split into 16-bit terms, each the rounding of what the
// earlier ones leave: two for fp16 (22 bits) and for bf16 with bf16 results
// (16 bits, against the 8 of the result), three for bf16 with fp32 results (24).
// The fp32 kernel multiplies H as it is.
template <int DT, int MT, int NT>
__device__ __forceinline__ void add_adapters(f32x16 (&acc)[MT][NT], const AdapterArgs &a, int row0,
                                             int col0, int part, int parts)
{
    using T = typename Elem<DT>::T;
    constexpr int kTerms = DT == 2 ? 3 : 2;
    const int lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
    int id[MT];
    uint64_t any = 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        id[i] = adapter_of(a, row0 + 32 * i + l32);
        any |= __builtin_amdgcn_ballot_w64(id[i] >= 0);
    }
    if (!any)
        return;
    for (int r0 = 0; r0 < a.rank; r0 += 16) {
        // the lane's H values: row l32 of each block, ranks r0 + 8 half .. + 7
        float h[MT][8], up[MT];
        u32x4 fh[MT][kTerms];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[i][e] = 0.0f;
            if (id[i] >= 0) {
                const float *p = a.H + (int64_t)(row0 + 32 * i + l32) * a.rank_pad + r0 + 8 * half;
                for (int s = 0; s < a.slices; ++s, p += (int64_t)a.rows * a.rank_pad) {
                    const f32x4 lo = *(const f32x4 *)p, hi = *(const f32x4 *)(p + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[i][e] += lo[e];
                        h[i][4 + e] += hi[e];
                    }
                }
            }
        }
        if constexpr (DT != 0) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                float top = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = fmaxf(top, fabsf(h[i][e]));
                top = fmaxf(top, __shfl_xor(top, 32));
                int ex = (int)((bits_of(top) >> 23) & 255) - 137;  // top = 2^(ex + 10) * [1, 2)
                ex = top < __builtin_inff() ? (ex < -100 ? -100 : ex) : 0;
                const float down = __builtin_bit_cast(float, (uint32_t)(127 - ex) << 23);
                up[i] = __builtin_bit_cast(float, (uint32_t)(127 + ex) << 23);
                T t[kTerms][8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float rest = h[i][e] * down;
#pragma unroll
                    for (int s = 0; s < kTerms; ++s) {
                        t[s][e] = (T)rest;
                        // (an infinity or NaN leaves nothing for the later terms)
                        rest = fabsf(rest) < __builtin_inff() ? rest - (float)t[s][e] : 0.0f;
                    }
                }
#pragma unroll
                for (int s = 0; s < kTerms; ++s)
                    __builtin_memcpy(&fh[i][s], t[s], 16);
            }
        }
        uint64_t left[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
            left[i] = __builtin_amdgcn_ballot_w64(id[i] >= 0) & 0xffffffffull;
        for (int nth = 0;; ++nth) {
            // the first row still waiting names the adapter
            int mine = -1;
#pragma unroll
            for (int i = MT - 1; i >= 0; --i)
                if (left[i])
                    mine = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(left[i]));
            if (mine < 0)
                break;
            uint64_t here[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                here[i] = __builtin_amdgcn_ballot_w64(id[i] == mine) & 0xffffffffull;
                left[i] &= ~here[i];
            }
            if (nth % parts != part)
                continue;
            const T *B = (const T *)a.B + (int64_t)mine * a.N * a.rank;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int n = col0 + 32 * j + l32;
                if constexpr (DT != 0) {
                    const int k = r0 + 8 * half;
                    const u32x4 fb = load_some(B + (int64_t)n * a.rank + k, n < a.N ? a.rank - k : 0);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        if (!here[i])
                            continue;
                        f32x16 sum = f32x16{};
                        if constexpr (kTerms > 2)
                            if (a.terms > 2)
                                mfma16<DT>(sum, fb, fh[i][2]);
                        mfma16<DT>(sum, fb, fh[i][1]);
                        mfma16<DT>(sum, fb, fh[i][0]);
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            acc[i][j][v] = id[i] == mine ? __builtin_fmaf(sum[v], up[i], acc[i][j][v])
                                                         : acc[i][j][v];
                    }
                } else {
                    // ranks r0 + 8 half + e of both operands meet in instruction e
                    f32x16 sum[MT];
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        sum[i] = f32x16{};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int k = r0 + 8 * half + e;
                        const float fb = n < a.N && k < a.rank ? (float)B[(int64_t)n * a.rank + k] : 0.0f;
#pragma unroll
                        for (int i = 0; i < MT; ++i)
                            sum[i] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb, h[i][e], sum[i], 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            acc[i][j][v] = id[i] == mine ? acc[i][j][v] + sum[i][v] : acc[i][j][v];
                }
            }
        }
    }
}

__device__ __forceinline__ uint32_t c_row_bytes(const AdapterArgs &a)
{
    return (uint32_t)a.N * (a.c_dtype ? 2 : 4);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t c_rows(const AdapterArgs &a, int64_t row)
{
    return make_rsrc(a.C + row * c_row_bytes(a));
}

// Tile of workgroup hw: each die takes a run of consecutive tiles, row tiles
// outermost, so that it reads few rows of X and its columns of W once.
__device__ __forceinline__ bool find_tile(const AdapterArgs &a, int hw, int *tm, int *tn)
{
    const int total = a.tiles_m * a.tiles_n;
    const int share = (total + a.xcds - 1) / a.xcds;
    const int id = hw % a.xcds * share + hw / a.xcds;
    if (hw / a.xcds >= share || id >= total)
        return false;
    *tm = id / a.tiles_n;
    *tn = id - *tm * a.tiles_n;
    return true;
}

template <int LB>
__device__ __forceinline__ TileWork shared_work(const AdapterArgs &a, int m0, int n0, int k0, int k)
{
    TileWork w;
    w.a = a.X + ((int64_t)m0 * a.ldx + k0) * 2;
    w.b = a.W + (LB == LINES ? (int64_t)n0 * a.ldw + k0 : (int64_t)k0 * a.ldw + n0) * 2;
    w.lda = a.ldx;
    w.ldb = a.ldw;
    w.m = a.rows - m0;
    w.n = a.N - n0;
    w.k = k;
    return w;
}

template <int DT, int LB>
__global__ __launch_bounds__(512, 1) void adapter_big_kernel(AdapterArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[(ring_of(LINES) + ring_of(LB)) * kPiece];
    int tm, tn;
    if (!find_tile(a, (int)blockIdx.x, &tm, &tn))
        return;
    const int m0 = tm * kBig, n0 = tn * kBig;
    const TileWork w = shared_work<LB>(a, m0, n0, 0, a.K);
    const __amdgpu_buffer_rsrc_t c = c_rows(a, m0);
    const bool vec = a.c_vec || n0 + kBig <= a.N;
    big_tile<DT, LINES, LB>(w, lds, [&](f32x16 (&acc)[4][2], int row, int col) {
        // (a row block at a time: all four at once do not fit the registers)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x16 blk[1][2] = {{acc[i][0], acc[i][1]}};
            add_adapters<DT, 1, 2>(blk, a, m0 + row + 32 * i, n0 + col, 0, 1);
            acc[i][0] = blk[0][0];
            acc[i][1] = blk[0][1];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            store_block(acc[i >> 1][i & 1], c, c_row_bytes(a), row + (i >> 1) * 32, w.m,
                        n0 + col + (i & 1) * 32, a.N, vec, a.c_dtype);
    });
}

// Few rows: 32 MT x 128 tiles, the depth cut into parts (blockIdx.y) where
// there are too few tiles to fill the chip.  Each part parks its fp32 sums and
// counts itself in; the last one adds all parts in their order, whichever it
// is, so the result does not depend on who that was.
template <int DT, int LB, int MT>
__global__ __launch_bounds__(256, 2) void adapter_narrow_kernel(AdapterArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[narrow_lds(MT)];
    int tm, tn;
    if (!find_tile(a, (int)blockIdx.x, &tm, &tn))
        return;
    const int m0 = tm * 32 * MT, n0 = tn * kNarrow, part = (int)blockIdx.y;
    const int k0 = part * a.part_k;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const TileWork w =
        shared_work<LB>(a, m0, n0, k0, a.K - k0 < a.part_k ? a.K - k0 : a.part_k);
    f32x16 acc[MT][1];
    narrow_tile<DT, LB, MT>(acc, w, lds);
    add_adapters<DT, MT, 1>(acc, a, m0, n0 + wave * 32, part, a.parts);
    if (a.parts > 1) {
        // slot layout: wave, block, quad, lane: 16-byte vectors side by side.
        // The stores and loads are coherent across the dies (sc1).
        constexpr int kCoherent = 16, kSlot = MT * 32 * kNarrow;
        const int tiles = a.tiles_m * a.tiles_n, tile = tm * a.tiles_n + tn;
        const __amdgpu_buffer_rsrc_t slot = make_rsrc(a.partials + ((int64_t)part * tiles + tile) * kSlot);
        const int off = (wave * MT * 4 * 64 + lane) * 16;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const u32x4 u = u32x4{bits_of(acc[i][0][4 * g]), bits_of(acc[i][0][4 * g + 1]),
                                      bits_of(acc[i][0][4 * g + 2]), bits_of(acc[i][0][4 * g + 3])};
                __builtin_amdgcn_raw_buffer_store_b128(u, slot, off + (i * 4 + g) * 1024, 0, kCoherent);
            }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        int32_t *arrived = (int32_t *)lds;  // (nobody reads the ring any more)
        if (threadIdx.x == 0)
            *arrived = __hip_atomic_fetch_add(a.counters + tile, 1, __ATOMIC_ACQ_REL,
                                              __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (*arrived != a.parts - 1)
            return;
#pragma unroll
        for (int i = 0; i < MT; ++i)
            acc[i][0] = f32x16{};
        for (int p = 0; p < a.parts; ++p) {
            const __amdgpu_buffer_rsrc_t from = make_rsrc(a.partials + ((int64_t)p * tiles + tile) * kSlot);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 v = __builtin_bit_cast(
                        f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, off + (i * 4 + g) * 1024, 0,
                                                                     kCoherent));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][0][4 * g + e] += v[e];
                }
        }
    }
    const __amdgpu_buffer_rsrc_t c = c_rows(a, m0);
    const bool vec = a.c_vec || n0 + kNarrow <= a.N;
#pragma unroll
    for (int i = 0; i < MT; ++i)
        store_block(acc[i][0], c, c_row_bytes(a), i * 32, w.m, n0 + wave * 32, a.N, vec, a.c_dtype);
}

template <bool W_KC>
__global__ __launch_bounds__(kXThreads) void adapter_exact_kernel(AdapterArgs a)
{
    __shared__ __attribute__((aligned(16))) float lds[4 * kXDeep * kXPitch];
    int tm, tn;
    if (!find_tile(a, (int)blockIdx.x, &tm, &tn))
        return;
    const int m0 = tm * kXTile, n0 = tn * kXTile;
    const int m = a.rows - m0 < kXTile ? a.rows - m0 : kXTile;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    f32x16 acc[2][2];
    exact_tile<float, true, W_KC>(acc, lds, (const float *)a.X + (int64_t)m0 * a.ldx, a.ldx, m,
                                  (const float *)a.W + (W_KC ? (int64_t)n0 * a.ldw : n0), a.ldw,
                                  a.N - n0, a.K);
    add_adapters<0, 2, 2>(acc, a, m0 + (wave >> 1) * 64, n0 + (wave & 1) * 64, 0, 1);
    store_exact(acc, a.C + (int64_t)m0 * c_row_bytes(a), a.N, m, n0, a.N, a.c_dtype, a.c_vec);
}

// ------------------------------------------------------------------- the host

constexpr int kMaxRank = 128;
constexpr int kCus = 256;

int elem_bytes(int dtype)
{
    return dtype == GEMM_F32 ? 4 : (dtype == GEMM_F16 || dtype == GEMM_BF16 ? 2 : 0);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }

int check(const gemm_adapter *p)
{
    if (!p) {
        set_error("NULL problem");
        return -1;
    }
    if (!elem_bytes(p->dtype)) {
        set_error("adapters take fp32, fp16 or bf16; got dtype %d", p->dtype);
        return -1;
    }
    if (p->flags & ~(uint32_t)GEMM_FLAG_C_INPUT_DTYPE) {
        set_error("adapters take no flag but GEMM_FLAG_C_INPUT_DTYPE (flags 0x%x)", p->flags);
        return -1;
    }
    if (p->rows < 0 || p->K < 0 || p->N < 0 || p->adapters < 0) {
        set_error("rows, K, N and adapters must not be negative");
        return -1;
    }
    if (p->rank < 1 || p->rank > kMaxRank) {
        set_error("rank must be between 1 and %d, got %d", kMaxRank, p->rank);
        return -1;
    }
    const int64_t widest = (int64_t)1 << 20;
    if (p->rows >= (int64_t)1 << 24 || p->K >= widest || p->N >= widest) {
        set_error("rows must stay below 2^24, K and N below 2^20");
        return -1;
    }
    return 0;
}

// Tiles, splits and the workspace of one problem.
struct AdapterPlan {
    int mt;                  // few-rows tiles of 32 mt x 128; 0: 256x256 (fp32: 128x128)
    int64_t tiles_m, tiles_n;
    int parts, part_k, slices, slice_k, rank_pad;
    int64_t ldx, ldw, w_rows, w_cols;
    bool pack_x, pack_w;
    size_t off_h, off_counters, off_partials, off_x, off_w, bytes;
};

AdapterPlan plan(const gemm_adapter *p)
{
    AdapterPlan l{};
    const int E = elem_bytes(p->dtype);
    l.rank_pad = (int)cdiv(p->rank, 16) * 16;
    l.w_rows = p->w_transposed ? p->N : p->K;
    l.w_cols = p->w_transposed ? p->K : p->N;
    l.pack_x = E == 2 && p->K % 8 != 0;
    l.pack_w = E == 2 && l.w_cols % 8 != 0;
    l.ldx = l.pack_x ? cdiv(p->K, 8) * 8 : p->K;
    l.ldw = l.pack_w ? cdiv(l.w_cols, 8) * 8 : l.w_cols;
    int bm = kXTile, bn = kXTile;
    if (E == 2) {
        // 256x256 tiles once they can occupy half the chip
        const int64_t big = cdiv(p->rows, kBig) * cdiv(p->N, kBig);
        l.mt = big >= kCus / 2 ? 0 : (p->rows <= 32 ? 1 : (p->rows <= 64 ? 2 : 4));
        bm = l.mt ? 32 * l.mt : kBig;
        bn = l.mt ? kNarrow : kBig;
    }
    l.tiles_m = cdiv(p->rows, bm);
    l.tiles_n = cdiv(p->N, bn);
    l.parts = 1;
    if (l.mt) {
        // two workgroups per CU, each at least four slabs deep
        const int64_t want = 2 * kCus / (l.tiles_m * l.tiles_n > 0 ? l.tiles_m * l.tiles_n : 1);
        const int64_t most = p->K / 256 > 0 ? p->K / 256 : 1;
        l.parts = (int)(want < 1 ? 1 : (want < most ? want : most));
    }
    l.part_k = (int)(cdiv(cdiv(p->K, l.parts), 64) * 64);
    l.parts = l.part_k ? (int)cdiv(p->K, l.part_k) : 1;
    const int64_t blocks = cdiv(p->rows, kShrinkRows);
    int64_t slices = blocks ? 128 / blocks : 1;
    slices = slices < 1 ? 1 : (slices > 16 ? 16 : slices);
    const int64_t most = p->K / 256 > 0 ? p->K / 256 : 1;
    slices = slices < most ? slices : most;
    l.slice_k = (int)(cdiv(cdiv(p->K, slices), 32) * 32);
    l.slices = l.slice_k ? (int)cdiv(p->K, l.slice_k) : 1;
    size_t at = 0;
    l.off_h = at;
    at += align_up((size_t)l.slices * p->rows * l.rank_pad * 4);
    l.off_counters = at;
    if (l.parts > 1)
        at += align_up((size_t)(l.tiles_m * l.tiles_n) * 4);
    l.off_partials = at;
    if (l.parts > 1)
        at += (size_t)l.parts * l.tiles_m * l.tiles_n * bm * bn * 4;
    l.off_x = at;
    if (l.pack_x)
        at += align_up((size_t)p->rows * l.ldx * E);
    l.off_w = at;
    if (l.pack_w)
        at += align_up((size_t)l.w_rows * l.ldw * E);
    l.bytes = at;
    return l;
}

template <int DT>
void launch_shrink(const AdapterArgs &a, dim3 grid, hipStream_t s)
{
    const dim3 t(64 * kShrinkWaves);
    if (a.rank <= 16)
        hipLaunchKernelGGL((shrink_kernel<DT, 1>), grid, t, 0, s, a);
    else if (a.rank <= 32)
        hipLaunchKernelGGL((shrink_kernel<DT, 2>), grid, t, 0, s, a);
    else if (a.rank <= 64)
        hipLaunchKernelGGL((shrink_kernel<DT, 4>), grid, t, 0, s, a);
    else
        hipLaunchKernelGGL((shrink_kernel<DT, 8>), grid, t, 0, s, a);
}

template <int DT, int LB>
void launch_shared(const AdapterArgs &a, int mt, unsigned tiles, hipStream_t s)
{
    const dim3 grid(tiles, (unsigned)a.parts);
    if (mt == 1)
        hipLaunchKernelGGL((adapter_narrow_kernel<DT, LB, 1>), grid, dim3(256), 0, s, a);
    else if (mt == 2)
        hipLaunchKernelGGL((adapter_narrow_kernel<DT, LB, 2>), grid, dim3(256), 0, s, a);
    else if (mt == 4)
        hipLaunchKernelGGL((adapter_narrow_kernel<DT, LB, 4>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((adapter_big_kernel<DT, LB>), grid, dim3(512), 0, s, a);
}

}  // namespace
}  // namespace gsk

using namespace gsk;

extern "C" {

size_t gemm_adapter_workspace_size(const gemm_adapter *p) { return check(p) ? 0 : plan(p).bytes; }

int gemm_adapter_run(const gemm_adapter *p, const void *X, const void *W, const void *A,
                     const void *B, const int32_t *ids, const float *scales, void *C,
                     void *workspace, void *stream)
{
    if (check(p))
        return -1;
    if (p->rows == 0 || p->N == 0)
        return 0;
    const int c_dtype = (p->flags & GEMM_FLAG_C_INPUT_DTYPE) ? p->dtype : GEMM_F32;
    const int E = elem_bytes(p->dtype), CE = elem_bytes(c_dtype);
    if (!C || !ids || (p->K && (!X || !W)) || (p->adapters && (!B || (p->K && !A)))) {
        set_error("NULL argument");
        return -1;
    }
    if (((uintptr_t)X & 15) || ((uintptr_t)W & 15) || ((uintptr_t)A & (E - 1)) ||
        ((uintptr_t)B & (E - 1)) || ((uintptr_t)C & (CE - 1)) || ((uintptr_t)ids & 3) ||
        ((uintptr_t)scales & 3) || ((uintptr_t)workspace & 255)) {
        set_error("misaligned pointer: X and W take 16 bytes, the workspace 256, the others an "
                  "element");
        return -1;
    }
    const AdapterPlan l = plan(p);
    if (l.bytes && !workspace) {
        set_error("this product needs %zu bytes of workspace", l.bytes);
        return -2;
    }
    uint8_t *ws = (uint8_t *)workspace;
    const hipStream_t s = (hipStream_t)stream;
    AdapterArgs a{};
    a.X = (const uint8_t *)X;
    a.x_plain = (const uint8_t *)X;
    a.W = (const uint8_t *)W;
    a.A = (const uint8_t *)A;
    a.B = (const uint8_t *)B;
    a.ids = ids;
    a.scales = scales;
    a.C = (uint8_t *)C;
    a.H = (float *)(ws + l.off_h);
    a.counters = (int32_t *)(ws + l.off_counters);
    a.partials = (float *)(ws + l.off_partials);
    a.rows = (int32_t)p->rows;
    a.N = (int32_t)p->N;
    a.K = (int32_t)p->K;
    a.rank = p->rank;
    a.rank_pad = l.rank_pad;
    a.adapters = p->adapters;
    a.ldx = (int32_t)l.ldx;
    a.ldw = (int32_t)l.ldw;
    a.slices = l.slices;
    a.slice_k = l.slice_k;
    a.parts = l.parts;
    a.part_k = l.part_k;
    a.terms = p->dtype == GEMM_BF16 && c_dtype == GEMM_F32 ? 3 : 2;
    a.tiles_m = (int32_t)l.tiles_m;
    a.tiles_n = (int32_t)l.tiles_n;
    a.c_dtype = c_dtype;
    a.c_vec = p->N % 4 == 0 && ((uintptr_t)C & (4 * CE - 1)) == 0;
    a.xcds = 8;
    const int64_t tiles = cdiv(l.tiles_m * l.tiles_n, a.xcds) * a.xcds;
    if (tiles >= ((int64_t)1 << 32) / 512) {
        set_error("too many tiles for one launch (%lld)", (long long)tiles);
        return -1;
    }
    if (p->K && (l.pack_x || l.pack_w)) {
        if (launch_pack_pair(X, ws + l.off_x, l.pack_x ? p->rows : 0, p->K, p->K, l.ldx, W,
                             ws + l.off_w, l.pack_w ? l.w_rows : 0, l.w_cols, l.w_cols, l.ldw, E,
                             s)) {
            set_error("pack launch failed: %s", hipGetErrorString(hipGetLastError()));
            return -3;
        }
        if (l.pack_x)
            a.X = ws + l.off_x;
        if (l.pack_w)
            a.W = ws + l.off_w;
    }
    const dim3 shrink((unsigned)cdiv(p->rows, kShrinkRows), (unsigned)l.slices);
    if (p->dtype == GEMM_F32) {
        launch_shrink<0>(a, shrink, s);
        if (p->w_transposed)
            hipLaunchKernelGGL((adapter_exact_kernel<true>), dim3((unsigned)tiles), dim3(kXThreads),
                               0, s, a);
        else
            hipLaunchKernelGGL((adapter_exact_kernel<false>), dim3((unsigned)tiles), dim3(kXThreads),
                               0, s, a);
    } else if (p->dtype == GEMM_F16) {
        launch_shrink<1>(a, shrink, s);
        if (p->w_transposed)
            launch_shared<1, LINES>(a, l.mt, (unsigned)tiles, s);
        else
            launch_shared<1, KROWS>(a, l.mt, (unsigned)tiles, s);
    } else {
        launch_shrink<2>(a, shrink, s);
        if (p->w_transposed)
            launch_shared<2, LINES>(a, l.mt, (unsigned)tiles, s);
        else
            launch_shared<2, KROWS>(a, l.mt, (unsigned)tiles, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        set_error("adapter product launch failed: %s", hipGetErrorString(e));
        return -3;
    }
    return 0;
}

}  // extern "C"
