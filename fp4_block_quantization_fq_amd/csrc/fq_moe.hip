// fq_moe.hip -- tokens sorted by expert and back on gfx950.
//
// Token t is assigned to experts ids[t, 0 .. k-1]; assignment a = t * k + j.
// The sorted order holds expert e's assignments in ascending a in rows
// offsets[e] .. offsets[e] + count_e - 1, offsets[e] a multiple of `align`
// (the backward products of the quantized linears take whole multiples of 64
// or 128 rows); rows that hold no assignment are padding.  pos[a] is a's row
// (-1: no expert), src[row] the assignment of a row (-1: padding).
//
//   dispatch      y[pos[t, j]] = x[t], padding rows 0
//   combine       out[t] = sum_j w[t, j] * y[pos[t, j]]
//   combine_bwd   dy[pos[t, j]] = w[t, j] * dout[t], dw[t, j] = <dout[t], y[pos[t, j]]>
//
// The gradient of dispatch is combine without weights.  No step uses floating
// atomics: every output has one writer, and sums run over j in order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_internal.h"
#include "fq_rows.hpp"

using namespace fqdev;

namespace {

constexpr int kThreads = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxExperts = fqimpl::kMoeMaxExperts;

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
// A stable counting sort.  Workgroup b owns assignments [b * chunk, (b + 1) *
// chunk).  With more than one workgroup a first launch leaves every chunk's
// counts in the workspace; the second one has each workgroup add up those of
// all chunks (the experts' totals) and of the chunks before its own.
__device__ __forceinline__ uint32_t expert_of(const int32_t *__restrict__ ids, int64_t a,
                                              int64_t n, uint32_t E)
{
    const uint32_t e = a < n ? (uint32_t)ids[a] : E;
    return e < E ? e : E;                 // E: no expert
}

__global__ __launch_bounds__(kSortThreads) void k_moe_count(fqimpl::MoeSortArgs a)
{
    __shared__ uint32_t cnt[kMaxExperts];
    for (uint32_t e = threadIdx.x; e < a.E; e += kSortThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * a.chunk, hi = min(lo + a.chunk, a.n);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        const uint32_t e = expert_of(a.ids, i, a.n, a.E);
        if (e < a.E) atomicAdd(&cnt[e], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.E; e += kSortThreads)
        a.ws[(size_t)blockIdx.x * a.E + e] = cnt[e];
}

__global__ __launch_bounds__(kSortThreads) void k_moe_place(fqimpl::MoeSortArgs a)
{
    // next[e]: the row of the next assignment of e; before[w][e]: those of
    // the waves before w in the present step
    __shared__ uint32_t next[kMaxExperts], total[kMaxExperts], start[kMaxExperts + 1];
    __shared__ uint16_t before[kSortWaves][kMaxExperts];
    __shared__ uint32_t wave_sums[kSortWaves];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t lo = (int64_t)blockIdx.x * a.chunk, hi = min(lo + a.chunk, a.n);
    const uint32_t e = tid;                // kSortThreads == kMaxExperts: one expert a thread
    // totals, and the counts of the chunks before this one
    next[e] = 0;
    __syncthreads();
    uint32_t all = 0, mine = 0;
    if (gridDim.x == 1) {
        for (int64_t i = lo + tid; i < hi; i += kSortThreads) {
            const uint32_t x = expert_of(a.ids, i, a.n, a.E);
            if (x < a.E) atomicAdd(&next[x], 1u);
        }
        __syncthreads();
        all = next[e];
    } else if (e < a.E) {
        for (uint32_t b = 0; b < gridDim.x; ++b) {
            const uint32_t c = a.ws[(size_t)b * a.E + e];
            all += c;
            if (b < blockIdx.x) mine += c;
        }
    }
    // starts: exclusive sum of the padded totals over the experts
    const uint32_t padded = (all + a.align - 1) / a.align * a.align;
    uint32_t incl = padded;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = (uint32_t)__shfl_up((int)incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 63) wave_sums[wave] = incl;
    __syncthreads();
    uint32_t first = incl - padded;
    for (int w = 0; w < wave; ++w) first += wave_sums[w];
    next[e] = first + mine;
    total[e] = all;
    start[e] = first;
    if (e == kMaxExperts - 1) start[kMaxExperts] = first + padded;
    __syncthreads();
    // offsets (padded totals past E are 0, so start[E] is the rows' number)
    if (blockIdx.x == 0) {
        for (uint32_t i = tid; i <= a.E; i += kSortThreads) a.offsets[i] = (int32_t)start[i];
    }
    // src of the padding rows: the segments' ends and what follows the last one
    for (uint32_t i = blockIdx.x; i <= a.E; i += gridDim.x) {
        const uint32_t from = i < a.E ? start[i] + total[i] : start[a.E];
        const uint32_t to = i < a.E ? start[i + 1] : (uint32_t)a.rows;
        for (uint32_t r = from + tid; r < to; r += kSortThreads) a.src[r] = -1;
    }
    // places, 1024 assignments at a time in their order
    for (int64_t i0 = lo; i0 < hi; i0 += kSortThreads) {
        const int64_t i = i0 + tid;
        const uint32_t x = i < hi ? expert_of(a.ids, i, a.n, a.E) : a.E;
        // lanes of this wave with the same expert
        uint64_t same = ~0ull;
        for (uint32_t bit = 1; bit <= a.E; bit <<= 1) {
            const uint64_t m = __ballot((x & bit) != 0);
            same &= (x & bit) ? m : ~m;
        }
        const uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1));
        for (uint32_t j = tid; j < a.E; j += kSortThreads)
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) before[w][j] = 0;
        __syncthreads();
        if (x < a.E && rank == 0) before[wave][x] = (uint16_t)__popcll(same);
        __syncthreads();
        uint32_t sum = 0;
        if (e < a.E) {
            uint32_t c[kSortWaves];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) c[w] = before[w][e];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                before[w][e] = (uint16_t)sum;
                sum += c[w];
            }
        }
        __syncthreads();
        if (i < hi) {
            int32_t p = -1;
            if (x < a.E) {
                p = (int32_t)(next[x] + before[wave][x] + rank);
                a.src[p] = (int32_t)i;
            }
            a.pos[i] = p;
        }
        __syncthreads();
        if (e < a.E) next[e] += sum;
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
// A workgroup per token reads its row once and writes it to its k places; the
// workgroups after those look through src, 16 rows each, and clear the padding.
constexpr int kPadRows = 16;

__device__ __forceinline__ void clear_padding(const fqimpl::MoeRowsArgs &a, int64_t block,
                                              uint16_t *__restrict__ y)
{
    const uint32_t chunks = (uint32_t)(a.H / 8);
    const u32w4 zero = {0, 0, 0, 0};
    for (int i = 0; i < kPadRows; ++i) {
        const int64_t r = block * kPadRows + i;
        if (r >= a.rows) return;
        if ((uint64_t)(int64_t)a.src[r] < (uint64_t)(a.T * a.k)) continue;
        for (uint32_t c = threadIdx.x; c < chunks; c += kThreads)
            *(u32w4 *)(y + r * a.H + c * 8) = zero;
    }
}

template <int F8>
__global__ __launch_bounds__(kThreads) void k_moe_dispatch(fqimpl::MoeRowsArgs a)
{
    uint16_t *y = (uint16_t *)a.rows_out;
    if (blockIdx.x >= a.T) return clear_padding(a, (int64_t)blockIdx.x - a.T, y);
    const int64_t t = blockIdx.x;
    const uint32_t chunks = (uint32_t)(a.H / 8);
    for (uint32_t c = threadIdx.x; c < chunks; c += kThreads) {
        u32w4 v;
        if (F8 == fqimpl::F8_NONE) {
            v = *(const u32w4 *)((const uint16_t *)a.x + t * a.H + c * 8);
        } else {
            float f[8];
            e4m3_decode8(*(const u32w2 *)((const uint8_t *)a.x + t * a.H + c * 8), f);
            float s;
            if (F8 == fqimpl::F8_MX) {
                const uint32_t code = ((const uint8_t *)a.scales)[t * (a.H / 32) + c / 4];
                s = code == 255u ? as_f(0x7FC00000u) : e8m0_value(code);
            } else {
                s = ((const float *)a.scales)[t];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = bf16_pair_rne(f[2 * i] * s, f[2 * i + 1] * s);
        }
        for (int j = 0; j < a.k; ++j) {
            const int64_t p = a.pos[t * a.k + j];
            if ((uint64_t)p < (uint64_t)a.rows) *(u32w4 *)(y + p * a.H + c * 8) = v;
        }
    }
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void k_moe_combine(fqimpl::MoeRowsArgs a)
{
    const uint16_t *y = (const uint16_t *)a.y;
    const int64_t t = blockIdx.x;
    const uint32_t chunks = (uint32_t)(a.H / 8);
    for (uint32_t c = threadIdx.x; c < chunks; c += kThreads) {
        float acc[8] = {};
        for (int j = 0; j < a.k; ++j) {
            const int64_t p = a.pos[t * a.k + j];
            if ((uint64_t)p >= (uint64_t)a.rows) continue;
            const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
            float v[8];
            load8<false>(y + p * a.H + c * 8, 8, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += w * v[e];
        }
        store8<false>((uint16_t *)a.out + t * a.H + c * 8, 8, acc);
    }
}

// A wave per assignment; the waves of one token are neighbours, so dout's row
// comes from memory once.  The workgroups after those clear the padding.
__global__ __launch_bounds__(kThreads) void k_moe_combine_bwd(fqimpl::MoeRowsArgs a, uint32_t work)
{
    uint16_t *dy = (uint16_t *)a.rows_out;
    if (blockIdx.x >= work) return clear_padding(a, (int64_t)blockIdx.x - work, dy);
    const int64_t i = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (i >= a.T * a.k) return;
    const int64_t t = i / a.k, p = a.pos[i];
    const uint32_t lane = threadIdx.x & 63, chunks = (uint32_t)(a.H / 8);
    float dot = 0.0f;
    if ((uint64_t)p < (uint64_t)a.rows) {
        const float w = a.weights[i];
        for (uint32_t c = lane; c < chunks; c += 64) {
            float d[8], v[8];
            load8<false>((const uint16_t *)a.dout + t * a.H + c * 8, 8, d);
            load8<false>((const uint16_t *)a.y + p * a.H + c * 8, 8, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dot += d[e] * v[e];
                d[e] = w * d[e];
            }
            store8<false>(dy + p * a.H + c * 8, 8, d);
        }
        dot = wave_sum(dot);
    }
    if (lane == 0) a.dweights[i] = dot;
}

}  // namespace

namespace fqimpl {

uint32_t moe_sort_chunk(int64_t n)
{
    const int64_t c = (n + kMoeMaxChunks - 1) / kMoeMaxChunks;
    const int64_t least = 2 * kSortThreads;
    return (uint32_t)(c <= least ? least : (c + kSortThreads - 1) / kSortThreads * kSortThreads);
}

hipError_t launch_moe_sort(MoeSortArgs a, hipStream_t stream)
{
    a.chunk = moe_sort_chunk(a.n);
    const uint32_t grid = (uint32_t)((a.n + a.chunk - 1) / a.chunk);
    if (grid > 1) {
        k_moe_count<<<dim3(grid), dim3(kSortThreads), 0, stream>>>(a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    k_moe_place<<<dim3(grid), dim3(kSortThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch(int f8, const MoeRowsArgs &a, hipStream_t stream)
{
    const dim3 grid((uint32_t)(a.T + (a.rows + kPadRows - 1) / kPadRows)), block(kThreads);
    if (f8 == F8_MX) k_moe_dispatch<F8_MX><<<grid, block, 0, stream>>>(a);
    else if (f8 == F8_ROW) k_moe_dispatch<F8_ROW><<<grid, block, 0, stream>>>(a);
    else k_moe_dispatch<F8_NONE><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeRowsArgs &a, hipStream_t stream)
{
    k_moe_combine<<<dim3((uint32_t)a.T), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const MoeRowsArgs &a, hipStream_t stream)
{
    const uint32_t work = (uint32_t)((a.T * a.k + kThreads / 64 - 1) / (kThreads / 64));
    const uint32_t pads = (uint32_t)((a.rows + kPadRows - 1) / kPadRows);
    k_moe_combine_bwd<<<dim3(work + pads), dim3(kThreads), 0, stream>>>(a, work);
    return hipGetLastError();
}

}  // namespace fqimpl
