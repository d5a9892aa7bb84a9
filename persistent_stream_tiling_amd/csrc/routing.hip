// Rows to their groups and back: the stable sort of (token, choice) entries by
// group, the copy of the tokens' rows into that order, the weighted sum back,
// and the gradients of both.  gfx950.
//
// Every kernel here moves bytes and does next to no arithmetic, so each is
// written to touch each byte once: the row kernels walk tokens (not sorted
// rows), so a token's own row is read or written once however many choices it
// has, and the rows in sorted order, which are all distinct, are each touched
// once as well.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "errors.h"
#include "gemm_sk.h"

namespace gsk {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ the sort

constexpr int kRouteThreads = 1024;
constexpr int kRouteLds = 64 * 1024;      // counter rows of the sort's waves
constexpr int kRouteChunk = 4096;         // entries per workgroup, at least
constexpr int kRouteMaxBlocks = 256;
constexpr int kRouteMaxGroups = 16382;    // one wave's counters (groups + 1) fit kRouteLds

// Waves of a sorting workgroup: as many as have a row of groups + 1 counters.
int route_waves(int groups)
{
    const int fit = kRouteLds / 4 / (groups + 1);
    return fit < kRouteThreads / 64 ? fit : kRouteThreads / 64;
}

// Entries per workgroup: a multiple of 64 per wave.
int64_t route_chunk(int64_t entries)
{
    const int64_t even = (entries + kRouteMaxBlocks - 1) / kRouteMaxBlocks;
    const int64_t c = even > kRouteChunk ? even : kRouteChunk;
    return (c + kRouteThreads - 1) / kRouteThreads * kRouteThreads;
}

int route_blocks(int64_t entries)
{
    const int64_t c = route_chunk(entries);
    const int64_t b = (entries + c - 1) / c;
    return b < 1 ? 1 : (int)b;
}

template <typename Id>
__device__ __forceinline__ int key_of(const Id *ids, int64_t i, int groups)
{
    const Id g = ids[i];
    return g >= 0 && g < (Id)groups ? (int)g : groups;  // `groups`: dropped, sorts last
}

// hist[block][g]: how many of the block's entries have key g.
template <typename Id>
__global__ __launch_bounds__(kRouteThreads) void route_count_kernel(const Id *__restrict__ ids,
                                                                    int64_t entries, int groups,
                                                                    int64_t chunk,
                                                                    int32_t *__restrict__ hist)
{
    extern __shared__ int32_t count[];
    for (int g = threadIdx.x; g <= groups; g += kRouteThreads)
        count[g] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * chunk;
    const int64_t hi = lo + chunk < entries ? lo + chunk : entries;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kRouteThreads)
        atomicAdd(&count[key_of(ids, i, groups)], 1);  // integer: any order, same sums
    __syncthreads();
    for (int g = threadIdx.x; g <= groups; g += kRouteThreads)
        hist[(int64_t)blockIdx.x * (groups + 1) + g] = count[g];
}

// Places the block's entries.  Wave w owns the w-th run of the block's
// entries and a row of counters in LDS; three passes:
//   1. each wave counts its keys;
//   2. the counters become first rows: over groups (all blocks' totals), over
//      earlier blocks (hist) and over earlier waves;
//   3. each wave walks its entries 64 at a time.  Lanes with the same key are
//      found bit by bit with ballots, so an entry's row is its wave's counter
//      plus the number of lower lanes with its key: stable, no atomics.
// With one block hist is not read: its totals are the block's own.  Decoding
// steps (entries <= 4096) are that case: one launch, its time that of a few
// dependent memory round trips.
template <typename Id>
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(
    const Id *__restrict__ ids, int64_t entries, int groups, int64_t chunk, int waves,
    const int32_t *__restrict__ hist, int32_t *__restrict__ offsets, int32_t *__restrict__ order,
    int32_t *__restrict__ position)
{
    extern __shared__ int32_t first[];  // [waves][groups + 1]
    __shared__ int32_t wave_sum[kRouteThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int keys = groups + 1;
    for (int i = tid; i < waves * keys; i += kRouteThreads)
        first[i] = 0;
    __syncthreads();

    const int64_t lo = (int64_t)blockIdx.x * chunk;
    const int64_t hi = lo + chunk < entries ? lo + chunk : entries;
    const int64_t per = ((chunk + waves - 1) / waves + 63) / 64 * 64;
    const int64_t wlo = lo + wave * per;
    const int64_t whi = wave < waves ? (wlo + per < hi ? wlo + per : hi) : wlo;
    for (int64_t i = wlo + lane; i < whi; i += 64)
        atomicAdd(&first[wave * keys + key_of(ids, i, groups)], 1);
    __syncthreads();

    // Thread tid owns the keys [tid * each, tid * each + each): their totals
    // are scanned over the threads, then the thread turns its keys' counters
    // into first rows.
    const int each = (keys + kRouteThreads - 1) / kRouteThreads;
    const int g_lo = tid * each < keys ? tid * each : keys;
    const int g_hi = g_lo + each < keys ? g_lo + each : keys;
    const bool alone = gridDim.x == 1;
    int32_t mine = 0;
    for (int g = g_lo; g < g_hi; ++g) {
        if (alone) {
            for (int w = 0; w < waves; ++w)
                mine += first[w * keys + g];
        } else {
#pragma unroll 8
            for (int b = 0; b < (int)gridDim.x; ++b)
                mine += hist[(int64_t)b * keys + g];
        }
    }
    int32_t sum = mine;  // inclusive over the wave's lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t up = __shfl_up(sum, d);
        sum += lane >= d ? up : 0;
    }
    if (lane == 63)
        wave_sum[wave] = sum;
    __syncthreads();
    int32_t at = sum - mine;
    for (int w = 0; w < wave; ++w)
        at += wave_sum[w];
    for (int g = g_lo; g < g_hi; ++g) {
        if (blockIdx.x == 0)
            offsets[g] = at;  // g = groups: the number of entries kept
        int32_t before = 0, total = 0;
        if (!alone) {
#pragma unroll 8
            for (int b = 0; b < (int)gridDim.x; ++b) {
                const int32_t n = hist[(int64_t)b * keys + g];
                before += b < (int)blockIdx.x ? n : 0;
                total += n;
            }
        }
        int32_t row = at + before;
        for (int w = 0; w < waves; ++w) {
            const int32_t n = first[w * keys + g];
            first[w * keys + g] = row;
            row += n;
        }
        at = alone ? row : at + total;
    }
    __syncthreads();

    const int bits = 32 - __clz(groups);  // keys 0 .. groups
    for (int64_t i0 = wlo; i0 < whi; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool ok = i < whi;
        const int key = ok ? key_of(ids, i, groups) : 0;
        uint64_t same = __ballot(ok);
        for (int b = 0; b < bits; ++b) {
            const bool one = (key >> b) & 1;
            const uint64_t m = __ballot(one);
            same &= one ? m : ~m;
        }
        if (ok) {
            const int before = __popcll(same & ((1ull << lane) - 1));
            volatile int32_t *slot = &first[wave * keys + key];
            const int32_t row = *slot + before;
            // the lowest lane of a key moves its counter on; LDS accesses of
            // one wave complete in order, so every lane has read it by then
            __builtin_amdgcn_wave_barrier();
            if (before == 0)
                *slot = row + __popcll(same);
            __builtin_amdgcn_wave_barrier();
            order[row] = key < groups ? (int32_t)i : -1;
            position[i] = key < groups ? row : -1;
        }
    }
}

template <typename Id>
int launch_route(const Id *ids, int64_t entries, int groups, int32_t *offsets, int32_t *order,
                 int32_t *position, int32_t *hist, hipStream_t stream)
{
    const int blocks = route_blocks(entries), waves = route_waves(groups);
    const int64_t chunk = route_chunk(entries);
    const size_t keys = (size_t)groups + 1;
    if (blocks > 1)
        hipLaunchKernelGGL((route_count_kernel<Id>), dim3(blocks), dim3(kRouteThreads), keys * 4,
                           stream, ids, entries, groups, chunk, hist);
    hipLaunchKernelGGL((route_place_kernel<Id>), dim3(blocks), dim3(kRouteThreads),
                       (size_t)waves * keys * 4, stream, ids, entries, groups, chunk, waves, hist,
                       offsets, order, position);
    return hipGetLastError() == hipSuccess ? 0 : -3;
}

// ------------------------------------------------------------- the row copies

constexpr int kRowThreads = 256;
constexpr int kRowMaxBlocks = 1 << 16;  // further tokens go round again (a launch holds 2^32 threads)

// 16 bytes of a row.  Rows need not be whole 16-byte words, so they start at
// any element: gfx950 code runs with unaligned global access enabled, and a
// 16-byte copy to or from an element-aligned address is one access.  (The
// values stay whole vectors from load to store: as arrays of elements they
// were moved two bytes at a time.)
template <typename T>
struct Row16 {
    static constexpr int V = 16 / (int)sizeof(T);
    typedef T Elements __attribute__((ext_vector_type(16 / sizeof(T))));
};

// Sorted rows past the size of the caches are read and written with the
// non-temporal hint: their lines are used once.  Measured with and without, by
// the size of the sorted rows: 268 MB gather 65.0 / 72.3 us, 268 MB sum 52.5 /
// 60.6 us, 134 MB gradient of a sum 65.0 / 70.9 us; but 69 MB, which the last
// cache still held, 20.9 / 17.0 us.
constexpr int64_t kStreamBytes = (int64_t)100 << 20;

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// The elements of a row from column c, those past `cols` as zero.
template <bool STREAM = false, typename T>
__device__ __forceinline__ u32x4 load_vec(const T *row, int c, int cols)
{
    constexpr int V = Row16<T>::V;
    u32x4 w;
    if (c + V <= cols) {
        if constexpr (STREAM)
            w = __builtin_nontemporal_load((const u32x4_any *)(row + c));
        else
            __builtin_memcpy(&w, row + c, 16);
    } else {
        T x[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            x[e] = c + e < cols ? row[c + e] : (T)0.0f;
        __builtin_memcpy(&w, x, 16);
    }
    return w;
}

template <bool STREAM = false, typename T>
__device__ __forceinline__ void store_vec(T *row, int c, int cols, u32x4 w)
{
    constexpr int V = Row16<T>::V;
    if (c + V <= cols) {
        if constexpr (STREAM)
            __builtin_nontemporal_store(w, (u32x4_any *)(row + c));
        else
            __builtin_memcpy(row + c, &w, 16);
    } else {
        T x[V];
        __builtin_memcpy(x, &w, 16);
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c + e < cols)
                row[c + e] = x[e];
    }
}

template <typename T>
__device__ __forceinline__ void widen(float (&x)[Row16<T>::V], u32x4 w)
{
    const auto v = __builtin_bit_cast(typename Row16<T>::Elements, w);
#pragma unroll
    for (int e = 0; e < Row16<T>::V; ++e)
        x[e] = (float)v[e];
}

template <typename T>
__device__ __forceinline__ u32x4 narrow(const float (&x)[Row16<T>::V])
{
    typename Row16<T>::Elements v;
#pragma unroll
    for (int e = 0; e < Row16<T>::V; ++e)
        v[e] = (T)x[e];
    return __builtin_bit_cast(u32x4, v);
}

// How a workgroup covers rows: `lanes` threads (a power of two) per token and
// kRowThreads / lanes tokens per workgroup.
struct RowGrid {
    int64_t tokens;
    int32_t choices, cols;
    int32_t lanes_log2;
};

// The number of rows kept, read on the GPU; kept inside the buffer whatever it is.
__device__ __forceinline__ int64_t rows_kept(const int32_t *kept, int64_t entries)
{
    const int64_t n = *kept;
    return n < 0 ? 0 : (n < entries ? n : entries);
}

// Sorted rows of choices j0 .. j0 + J - 1 of token t (-1: dropped, or past the
// last choice).  All J loads are in flight at once.
template <int J>
__device__ __forceinline__ void load_rows(int32_t (&row)[J], const int32_t *position, int64_t e0,
                                          int j0, int choices, int64_t entries)
{
#pragma unroll
    for (int j = 0; j < J; ++j)
        row[j] = position[e0 + (j0 + j < choices ? j0 + j : 0)];
#pragma unroll
    for (int j = 0; j < J; ++j)
        row[j] = j0 + j < choices && row[j] < entries ? row[j] : -1;
}

// xs[position[t][j]] = x[t] for every choice j; rows past the kept ones are
// zeroed (row e = t * choices + j by token t: rows and entries count alike).
// J: choices per round.  Bound by the writes, choices rows for each row read:
// 8192 tokens x 8 choices of 2048 bf16 in about 50 us, 6 TB/s.  (Walking the
// sorted rows instead, each copying its token's row, took 72 us where this took
// 52: it reads x eight times over.)
template <typename T, int J, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void gather_kernel(const T *__restrict__ x,
                                                             const int32_t *__restrict__ position,
                                                             const int32_t *__restrict__ kept,
                                                             T *__restrict__ xs, RowGrid g)
{
    constexpr int V = Row16<T>::V;
    const int lanes = 1 << g.lanes_log2, per = kRowThreads >> g.lanes_log2;
    const int64_t entries = g.tokens * g.choices, live = rows_kept(kept, entries);
    const int c = ((int)blockIdx.y * lanes + (threadIdx.x & (lanes - 1))) * V;
    if (c >= g.cols)
        return;
    for (int64_t t = (int64_t)blockIdx.x * per + (threadIdx.x >> g.lanes_log2); t < g.tokens;
         t += (int64_t)gridDim.x * per) {
        const u32x4 v = load_vec(x + t * g.cols, c, g.cols);
        const int64_t e0 = t * g.choices;
        for (int j0 = 0; j0 < g.choices; j0 += J) {
            int32_t row[J];
            load_rows<J>(row, position, e0, j0, g.choices, entries);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (row[j] >= 0)
                    store_vec<STREAM>(xs + (int64_t)row[j] * g.cols, c, g.cols, v);
        }
        for (int64_t e = e0 > live ? e0 : live; e < e0 + g.choices; ++e)
            store_vec<STREAM>(xs + e * g.cols, c, g.cols, u32x4{});
    }
}

// y[t] = sum over j of w[t][j] * ys[position[t][j]], in fp32 in the order of
// j, rounded once.  A dropped choice adds nothing (its loads go to row 0, so
// that all J of a round are in flight together, and are then ignored).
// Without weights: the plain sum, which is the gradient of gather_kernel.
// Bound by the reads of the sorted rows: 8192 tokens x 8 choices of 2048 bf16 in
// 52 us, 5.8 TB/s.
template <typename T, bool WEIGHTS, int J, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(const T *__restrict__ ys,
                                                              const int32_t *__restrict__ position,
                                                              const float *__restrict__ weights,
                                                              T *__restrict__ y, RowGrid g)
{
    constexpr int V = Row16<T>::V;
    const int lanes = 1 << g.lanes_log2, per = kRowThreads >> g.lanes_log2;
    const int64_t entries = g.tokens * g.choices;
    const int c = ((int)blockIdx.y * lanes + (threadIdx.x & (lanes - 1))) * V;
    if (c >= g.cols)
        return;
    for (int64_t t = (int64_t)blockIdx.x * per + (threadIdx.x >> g.lanes_log2); t < g.tokens;
         t += (int64_t)gridDim.x * per) {
        const int64_t e0 = t * g.choices;
        float sum[V] = {};
        for (int j0 = 0; j0 < g.choices; j0 += J) {
            int32_t row[J];
            float w[J];
            u32x4 v[J];
            load_rows<J>(row, position, e0, j0, g.choices, entries);
#pragma unroll
            for (int j = 0; j < J; ++j)
                w[j] = WEIGHTS ? weights[e0 + (j0 + j < g.choices ? j0 + j : 0)] : 1.0f;
#pragma unroll
            for (int j = 0; j < J; ++j)
                v[j] = load_vec<STREAM>(ys + (int64_t)(row[j] >= 0 ? row[j] : 0) * g.cols, c, g.cols);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float x[V];
                widen<T>(x, v[j]);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float next = WEIGHTS ? __builtin_fmaf(w[j], x[e], sum[e]) : sum[e] + x[e];
                    sum[e] = row[j] >= 0 ? next : sum[e];
                }
            }
        }
        store_vec(y + t * g.cols, c, g.cols, narrow<T>(sum));
    }
}

// The gradient of combine_kernel: dys[position[t][j]] = w[t][j] * dy[t] and
// dw[t][j] = <dy[t], ys[position[t][j]]> (zero for a dropped choice), in one
// pass over ys; rows of dys past the kept ones are zeroed.  The dot products
// are summed per lane over its columns, then over the lanes in a fixed order.
// U: column steps whose loads are in flight together.  4096 tokens x 2 choices
// of 4096 fp32: 57 us, 5.8 TB/s.
template <typename T, int J, int U, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(
    const T *__restrict__ dy, const T *__restrict__ ys, const int32_t *__restrict__ position,
    const int32_t *__restrict__ kept, const float *__restrict__ weights, T *__restrict__ dys,
    float *__restrict__ dweights, RowGrid g)
{
    constexpr int V = Row16<T>::V;
    __shared__ float part[kRowThreads / 64][J];
    const int lanes = 1 << g.lanes_log2, per = kRowThreads >> g.lanes_log2;
    const int l = threadIdx.x & (lanes - 1), wave = threadIdx.x >> 6;
    const int64_t entries = g.tokens * g.choices, live = rows_kept(kept, entries);
    // (the workgroup's threads go round together: there are barriers inside)
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < g.tokens; t0 += (int64_t)gridDim.x * per) {
        const int64_t t = t0 + (threadIdx.x >> g.lanes_log2);
        const bool ok = t < g.tokens;
        const int64_t e0 = ok ? t * g.choices : 0;
        const T *dy_row = dy + (ok ? t : 0) * g.cols;
        const int cols = ok ? g.cols : 0;
        for (int j0 = 0; j0 < g.choices; j0 += J) {
            int32_t row[J];
            float w[J], dot[J];
            load_rows<J>(row, position, e0, j0, g.choices, entries);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                w[j] = weights[e0 + (j0 + j < g.choices ? j0 + j : 0)];
                dot[j] = 0.0f;
            }
            for (int c0 = l * V; c0 < cols; c0 += U * lanes * V) {
                u32x4 d[U], v[U][J];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * lanes * V;
                    if (c < cols) {
                        d[u] = load_vec(dy_row, c, cols);
#pragma unroll
                        for (int j = 0; j < J; ++j)
                            v[u][j] = load_vec<STREAM>(ys + (int64_t)(row[j] >= 0 ? row[j] : 0) * cols,
                                                       c, cols);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * lanes * V;
                    if (c < cols) {
                        float df[V];
                        widen<T>(df, d[u]);
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            float vf[V], out[V];
                            widen<T>(vf, v[u][j]);
#pragma unroll
                            for (int e = 0; e < V; ++e) {
                                dot[j] = __builtin_fmaf(df[e], vf[e], dot[j]);
                                out[e] = w[j] * df[e];
                            }
                            if (row[j] >= 0)
                                store_vec<STREAM>(dys + (int64_t)row[j] * cols, c, cols, narrow<T>(out));
                        }
                    }
                }
            }
            // over the token's lanes: within the wave, then over its waves
            const int width = lanes < 64 ? lanes : 64;
#pragma unroll
            for (int j = 0; j < J; ++j)
                for (int d = width >> 1; d; d >>= 1)
                    dot[j] += __shfl_xor(dot[j], d);
            if (lanes > 64) {
                __syncthreads();
                if ((threadIdx.x & 63) == 0)
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        part[wave][j] = dot[j];
                __syncthreads();
                const int w0 = (threadIdx.x >> g.lanes_log2) * (lanes >> 6);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    dot[j] = part[w0][j];
                    for (int i = 1; i < lanes >> 6; ++i)
                        dot[j] += part[w0 + i][j];
                }
            }
            if (ok && l == 0)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (j0 + j < g.choices)
                        dweights[e0 + j0 + j] = row[j] >= 0 ? dot[j] : 0.0f;
        }
        if (ok && e0 + g.choices > live) {
            for (int64_t e = e0 > live ? e0 : live; e < e0 + g.choices; ++e)
                for (int c = l * V; c < g.cols; c += lanes * V)
                    store_vec<STREAM>(dys + e * g.cols, c, g.cols, u32x4{});
        }
    }
}

RowGrid row_grid(int64_t tokens, int32_t choices, int32_t cols, int elem)
{
    RowGrid g{tokens, choices, cols, 0};
    const int vecs = (cols + 16 / elem - 1) / (16 / elem);
    while ((1 << g.lanes_log2) < vecs && (1 << g.lanes_log2) < kRowThreads)
        ++g.lanes_log2;
    return g;
}

dim3 row_blocks(const RowGrid &g, int elem, bool split_cols)
{
    const int per = kRowThreads >> g.lanes_log2;
    const int vecs = (g.cols + 16 / elem - 1) / (16 / elem);
    const int lanes = 1 << g.lanes_log2;
    const int64_t blocks = (g.tokens + per - 1) / per;
    return dim3((unsigned)(blocks < kRowMaxBlocks ? blocks : kRowMaxBlocks),
                split_cols ? (unsigned)((vecs + lanes - 1) / lanes) : 1);
}

int launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess)
        return 0;
    set_error("%s launch failed: %s", what, hipGetErrorString(e));
    return -3;
}

int elem_bytes(int dtype)
{
    return dtype == GEMM_F32 ? 4 : (dtype == GEMM_F16 || dtype == GEMM_BF16 ? 2 : 0);
}

// Common checks; 0 when there is work, 1 when there is none, -1 on an error.
int check_rows(int64_t tokens, int32_t choices, int64_t cols, int dtype)
{
    if (tokens < 0 || choices < 1 || cols < 0) {
        set_error("tokens %lld, choices %d and cols %lld must not be negative (choices >= 1)",
                  (long long)tokens, choices, (long long)cols);
        return -1;
    }
    if (tokens >= ((int64_t)1 << 31) / choices) {
        set_error("tokens * choices must stay below 2^31 (%lld * %d)", (long long)tokens, choices);
        return -1;
    }
    if (cols >= (int64_t)1 << 22) {
        set_error("cols must stay below 2^22, got %lld", (long long)cols);
        return -1;
    }
    if (!elem_bytes(dtype)) {
        set_error("rows are fp32, fp16 or bf16; got dtype %d", dtype);
        return -1;
    }
    return tokens == 0 || cols == 0 ? 1 : 0;
}

bool aligned(const void *p, int n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; }

// Sorted rows that the caches cannot hold: the first kernel, else the second.
#define GSK_LAUNCH_ROWS(STREAMS, KEEPS, ...)                                                     \
    do {                                                                                         \
        if (tokens * choices * cols * E >= kStreamBytes)                                         \
            hipLaunchKernelGGL(STREAMS, blocks, dim3(kRowThreads), 0, s, __VA_ARGS__);           \
        else                                                                                     \
            hipLaunchKernelGGL(KEEPS, blocks, dim3(kRowThreads), 0, s, __VA_ARGS__);             \
    } while (0)

// One of the kernels for 1, 2, 4 or 8 choices a round: LAUNCH(T, J).
#define GSK_BY_CHOICES(LAUNCH, T)                                                                \
    do {                                                                                         \
        if (choices == 1)                                                                        \
            LAUNCH(T, 1);                                                                        \
        else if (choices == 2)                                                                   \
            LAUNCH(T, 2);                                                                        \
        else if (choices <= 4)                                                                   \
            LAUNCH(T, 4);                                                                        \
        else                                                                                     \
            LAUNCH(T, 8);                                                                        \
    } while (0)

}  // namespace
}  // namespace gsk

using namespace gsk;

extern "C" {

size_t gemm_route_workspace_size(int64_t tokens, int32_t choices, int32_t groups)
{
    if (tokens <= 0 || choices < 1 || groups < 1 || groups > kRouteMaxGroups ||
        tokens >= ((int64_t)1 << 31) / choices)
        return 0;
    const int blocks = route_blocks(tokens * choices);
    return blocks > 1 ? (size_t)blocks * ((size_t)groups + 1) * 4 : 0;
}

int gemm_route(const void *ids, int32_t id_bytes, int64_t tokens, int32_t choices, int32_t groups,
               int32_t *offsets, int32_t *order, int32_t *position, void *workspace, void *stream)
{
    if (check_rows(tokens, choices, 0, GEMM_F32) < 0)
        return -1;
    if (groups < 1 || groups > kRouteMaxGroups) {
        set_error("groups must be between 1 and %d, got %d", kRouteMaxGroups, groups);
        return -1;
    }
    if (id_bytes != 4 && id_bytes != 8) {
        set_error("ids are int32 or int64 (4 or 8 bytes), got %d", id_bytes);
        return -1;
    }
    if (!offsets || (tokens && (!ids || !order || !position))) {
        set_error("NULL argument");
        return -1;
    }
    if (!aligned(ids, id_bytes) || !aligned(offsets, 4) || !aligned(order, 4) ||
        !aligned(position, 4) || !aligned(workspace, 4)) {
        set_error("misaligned pointer");
        return -1;
    }
    const size_t need = gemm_route_workspace_size(tokens, choices, groups);
    if (need && !workspace) {
        set_error("this sort needs %zu bytes of workspace", need);
        return -2;
    }
    const int64_t entries = tokens * choices;
    const int rc = id_bytes == 4
                       ? launch_route((const int32_t *)ids, entries, groups, offsets, order,
                                      position, (int32_t *)workspace, (hipStream_t)stream)
                       : launch_route((const int64_t *)ids, entries, groups, offsets, order,
                                      position, (int32_t *)workspace, (hipStream_t)stream);
    if (rc)
        set_error("route launch failed");
    return rc;
}

int gemm_gather_rows(const void *x, const int32_t *position, const int32_t *kept, void *xs,
                     int64_t tokens, int32_t choices, int64_t cols, gemm_dtype dtype, void *stream)
{
    const int c = check_rows(tokens, choices, cols, dtype);
    if (c)
        return c < 0 ? -1 : 0;
    const int E = elem_bytes(dtype);
    if (!x || !position || !kept || !xs) {
        set_error("NULL argument");
        return -1;
    }
    if (!aligned(x, E) || !aligned(xs, E) || !aligned(position, 4) || !aligned(kept, 4)) {
        set_error("misaligned pointer");
        return -1;
    }
    const RowGrid g = row_grid(tokens, choices, (int32_t)cols, E);
    const dim3 blocks = row_blocks(g, E, true);
    const hipStream_t s = (hipStream_t)stream;
    // a copy: only the element size matters
#define GSK_GATHER(T, J)                                                                         \
    GSK_LAUNCH_ROWS((gather_kernel<T, J, true>), (gather_kernel<T, J, false>), (const T *)x,     \
                    position, kept, (T *)xs, g)
    if (E == 4)
        GSK_BY_CHOICES(GSK_GATHER, float);
    else
        GSK_BY_CHOICES(GSK_GATHER, _Float16);
#undef GSK_GATHER
    return launched("gather");
}

int gemm_combine_rows(const void *ys, const int32_t *position, const float *weights, void *y,
                      int64_t tokens, int32_t choices, int64_t cols, gemm_dtype dtype, void *stream)
{
    const int c = check_rows(tokens, choices, cols, dtype);
    if (c)
        return c < 0 ? -1 : 0;
    const int E = elem_bytes(dtype);
    if (!ys || !position || !y) {
        set_error("NULL argument");
        return -1;
    }
    if (!aligned(ys, E) || !aligned(y, E) || !aligned(position, 4) || !aligned(weights, 4)) {
        set_error("misaligned pointer");
        return -1;
    }
    const RowGrid g = row_grid(tokens, choices, (int32_t)cols, E);
    const dim3 blocks = row_blocks(g, E, true);
    const hipStream_t s = (hipStream_t)stream;
#define GSK_COMBINE(T, W, J)                                                                     \
    GSK_LAUNCH_ROWS((combine_kernel<T, W, J, true>), (combine_kernel<T, W, J, false>),           \
                    (const T *)ys, position, weights, (T *)y, g)
#define GSK_WEIGHTED(T, J) GSK_COMBINE(T, true, J)
#define GSK_PLAIN(T, J) GSK_COMBINE(T, false, J)
#define GSK_BY_TYPE(T)                                                                           \
    if (weights)                                                                                 \
        GSK_BY_CHOICES(GSK_WEIGHTED, T);                                                         \
    else                                                                                         \
        GSK_BY_CHOICES(GSK_PLAIN, T)
    if (dtype == GEMM_F32) {
        GSK_BY_TYPE(float);
    } else if (dtype == GEMM_F16) {
        GSK_BY_TYPE(_Float16);
    } else {
        GSK_BY_TYPE(__bf16);
    }
#undef GSK_BY_TYPE
#undef GSK_WEIGHTED
#undef GSK_PLAIN
#undef GSK_COMBINE
    return launched("combine");
}

int gemm_combine_rows_backward(const void *dy, const void *ys, const int32_t *position,
                               const int32_t *kept, const float *weights, void *dys,
                               float *dweights, int64_t tokens, int32_t choices, int64_t cols,
                               gemm_dtype dtype, void *stream)
{
    const int c = check_rows(tokens, choices, cols, dtype);
    if (c < 0 || tokens == 0)
        return c < 0 ? -1 : 0;
    const int E = elem_bytes(dtype);
    // cols = 0 still writes dweights (empty sums)
    if (!position || !kept || !weights || !dweights || (cols && (!dy || !ys || !dys))) {
        set_error("NULL argument");
        return -1;
    }
    if (!aligned(dy, E) || !aligned(ys, E) || !aligned(dys, E) || !aligned(position, 4) ||
        !aligned(kept, 4) || !aligned(weights, 4) || !aligned(dweights, 4)) {
        set_error("misaligned pointer");
        return -1;
    }
    const RowGrid g = row_grid(tokens, choices, (int32_t)cols, E);
    const dim3 blocks = row_blocks(g, E, false);
    const hipStream_t s = (hipStream_t)stream;
#define GSK_BACK(T, J)                                                                           \
    GSK_LAUNCH_ROWS((combine_backward_kernel<T, J, (J > 2 ? 1 : 4 / J), true>),                  \
                    (combine_backward_kernel<T, J, (J > 2 ? 1 : 4 / J), false>), (const T *)dy,  \
                    (const T *)ys, position, kept, weights, (T *)dys, dweights, g)
    if (dtype == GEMM_F32)
        GSK_BY_CHOICES(GSK_BACK, float);
    else if (dtype == GEMM_F16)
        GSK_BY_CHOICES(GSK_BACK, _Float16);
    else
        GSK_BY_CHOICES(GSK_BACK, __bf16);
#undef GSK_BACK
    return launched("combine backward");
}

}  // extern "C"
