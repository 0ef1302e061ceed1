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
//
// The row operators are bound by memory (8192 tokens of 2880 over four of 32
// experts: dispatch from 8-bit rows 42 us, 5.7 TB/s, combine 42 us, 5.6 TB/s, its
// backward 76 us, 5.9 TB/s), the sort by latency: two launches of 3 and 5 us for
// 32768 assignments, one of 3.3 us for four.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fq_internal.h"
#include "fq_rows.hpp"

using namespace fqdev;

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxExperts = fqimpl::kMoeMaxExperts;

static_assert(kSortThreads == kMaxExperts, "one expert a thread");

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
// A stable counting sort.  Workgroup b owns assignments [b * chunk, (b + 1) *
// chunk) and needs the counts of all assignments (the experts' totals) and of
// those before its own.  Up to kCountAll of them every workgroup counts them all
// itself; beyond, a first launch leaves every chunk's counts in the workspace,
// and the workgroups add those up.
// 32 experts: 4096 assignments 4.7 us counted by all and 6.0 in two launches, 8192
// 5.3 and 6.3, 16384 6.4 and 6.4; all 8192 of one expert, whose counter then is
// the bound, 10.0 and 6.9.
constexpr int64_t kCountAll = int64_t(1) << 13;

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
    // next[e]: the row of the next assignment of e; before[e][w]: e's
    // assignments in wave w of the present step, then those in the waves before
    // w (one 32-byte row an expert, so its thread moves it in two accesses)
    __shared__ uint32_t total[kMaxExperts], next[kMaxExperts], start[kMaxExperts + 1];
    __shared__ __attribute__((aligned(16))) uint16_t before[kMaxExperts][kSortWaves];
    __shared__ uint32_t wave_sums[kSortWaves];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t lo = (int64_t)blockIdx.x * a.chunk, hi = min(lo + a.chunk, a.n);
    const uint32_t e = tid;                // one expert a thread
    u32w4 *mine_before = (u32w4 *)before[e];
    uint32_t x = expert_of(a.ids, lo + tid, hi, a.E);     // of the first step
    total[e] = next[e] = 0;
    if (e < a.E) mine_before[0] = mine_before[1] = (u32w4){0, 0, 0, 0};
    __syncthreads();
    // total[e]: assignments from this chunk on (all, from the workspace), next[e]:
    // those before it
    if (!a.ws) {
        constexpr int kBatch = kCountAll / kSortThreads;     // loads in flight together
        uint32_t o[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            o[u] = (uint32_t)a.ids[min((int64_t)(u * kSortThreads + tid), a.n - 1)];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = u * kSortThreads + tid;
            if (i < a.n && o[u] < a.E) atomicAdd(i < lo ? &next[o[u]] : &total[o[u]], 1u);
        }
    } else {
        for (uint32_t i = tid; i < gridDim.x * a.E; i += kSortThreads) {
            const uint32_t c = a.ws[i], b = i / a.E, o = i - b * a.E;
            if (!c) continue;
            atomicAdd(&total[o], c);
            if (b < blockIdx.x) atomicAdd(&next[o], c);
        }
    }
    // assignments a step of 1024 at a time, in their order
    bool first_step = true;
    for (int64_t i0 = lo; i0 < hi; i0 += kSortThreads) {
        const int64_t i = i0 + tid;
        // lanes of this wave with the same expert
        uint64_t same = ~0ull;
        for (uint32_t bit = 1; bit <= a.E; bit <<= 1) {
            const uint64_t m = __ballot((x & bit) != 0);
            same &= (x & bit) ? m : ~m;
        }
        const uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1));
        if (x < a.E && rank == 0) before[x][wave] = (uint16_t)__popcll(same);
        __syncthreads();
        uint32_t sum = 0;
        if (e < a.E) {
            u32w4 c[2] = {mine_before[0], mine_before[1]};
#pragma unroll
            for (int w = 0; w < kSortWaves; w += 2) {
                const uint32_t both = c[w / 8][w / 2 % 4], low = both & 0xFFFFu;
                c[w / 8][w / 2 % 4] = sum | (sum + low) << 16;
                sum += low + (both >> 16);
            }
            mine_before[0] = c[0];
            mine_before[1] = c[1];
        }
        if (first_step) {
            // starts: exclusive sum of the padded totals over the experts
            if (!a.ws) total[e] += next[e];
            const uint32_t all = total[e], padded = (all + a.align - 1) / a.align * a.align;
            uint32_t incl = padded;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const uint32_t o = (uint32_t)__shfl_up((int)incl, d);
                if (lane >= d) incl += o;
            }
            if (lane == 63) wave_sums[wave] = incl;
            __syncthreads();
            uint32_t first = incl - padded;
#pragma unroll
            for (int w = 0; w < kSortWaves - 1; ++w) first += w < wave ? wave_sums[w] : 0u;
            next[e] += first;
            start[e] = first;
            if (e == kMaxExperts - 1) start[kMaxExperts] = first + padded;
        }
        __syncthreads();
        if (i < hi) {
            int32_t p = -1;
            if (x < a.E) {
                p = (int32_t)(next[x] + before[x][wave] + rank);
                a.src[p] = (int32_t)i;
            }
            a.pos[i] = p;
        }
        first_step = false;
        if (i0 + kSortThreads >= hi) break;
        x = expert_of(a.ids, i + kSortThreads, hi, a.E);
        __syncthreads();
        if (e < a.E) {
            next[e] += sum;
            mine_before[0] = mine_before[1] = (u32w4){0, 0, 0, 0};
        }
        __syncthreads();
    }
    // offsets (padded totals past E are 0, so start[E] is the rows' number)
    if (blockIdx.x == 0)
        for (uint32_t i = tid; i <= a.E; i += kSortThreads) a.offsets[i] = (int32_t)start[i];
    // src of the padding rows: a wave an expert for the segments' ends, then all
    // threads for what follows the last one
    for (uint32_t i = blockIdx.x * kSortWaves + wave; i < a.E; i += gridDim.x * kSortWaves)
        for (uint32_t r = start[i] + total[i] + lane; r < start[i + 1]; r += 64) a.src[r] = -1;
    for (int64_t r = (int64_t)start[a.E] + blockIdx.x * kSortThreads + tid; r < a.rows;
         r += (int64_t)gridDim.x * kSortThreads)
        a.src[r] = -1;
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
// LANES lanes share a token: 8 for a row of 64 elements up to a wave, or, with
// LANES 0, a workgroup of as many waves as the row has 64 chunks of 8 elements
// (512 threads at most, which then walk over the row).  A lane has one chunk
// and moves it for up to four of the token's assignments at a time, all loads
// issued together: what bounds these kernels is the bytes a CU has in flight
// (a wave a token instead of 360 lanes: combine 46.2 us instead of 41.6 at 8192
// tokens of 2880, 7.6 instead of 3.2 at 16; 8 lanes instead of a wave for rows
// of 64: 8.5 instead of 25.7 at 65536 tokens).
constexpr int kThreads = 256;               // of a workgroup of several tokens
constexpr int kMostThreads = 512;
constexpr int kPadRows = 16;

// Four assignments from `first` on, those before `end`: rows (negative: none)
// and weights.
struct Four {
    int64_t p[4];
    float w[4];
};
template <int LANES>
__device__ __forceinline__ Four four_of(const fqimpl::MoeRowsArgs &a, int64_t first, int64_t end)
{
    Four f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = min(first + i, end - 1);
        int32_t p = a.pos[at];
        if (LANES == 0 || LANES == 64) p = __builtin_amdgcn_readfirstlane(p);    // a wave has one token
        f.p[i] = first + i < end && (uint32_t)p < (uint64_t)a.rows ? (int64_t)p : -1;
        f.w[i] = a.weights ? a.weights[at] : 1.0f;
    }
    return f;
}

// +0 into the rows of [block * 16, block * 16 + 16) that hold no assignment.
template <int LANES, bool NT>
__device__ __forceinline__ void clear_padding(const fqimpl::MoeRowsArgs &a, int64_t block,
                                              uint16_t *__restrict__ y)
{
    const uint32_t chunks = (uint32_t)(a.H / 8);
    const int64_t r0 = block * kPadRows;
    const u32w4 zero = {0, 0, 0, 0};
    if (LANES) {                           // a row for each group of lanes
        constexpr int kLanes = LANES ? LANES : 64;
        const uint32_t c = threadIdx.x % kLanes;
        for (int i = threadIdx.x / kLanes; i < kPadRows; i += kThreads / kLanes) {
            const int64_t r = r0 + i;
            if (r >= a.rows || (uint64_t)(int64_t)a.src[r] < (uint64_t)(a.T * a.k)) continue;
            if (c < chunks) store16<NT>((u32w4 *)(y + r * a.H + c * 8), zero);
        }
        return;
    }
    const uint32_t lane = threadIdx.x & 63;
    bool pad = false;
    if (lane < kPadRows && r0 + lane < a.rows)
        pad = (uint64_t)(int64_t)a.src[r0 + lane] >= (uint64_t)(a.T * a.k);
    for (uint64_t left = __ballot(pad); left; left &= left - 1) {
        uint16_t *row = y + (r0 + __builtin_ctzll(left)) * a.H;
        for (uint32_t c = threadIdx.x; c < chunks; c += blockDim.x)
            store16<NT>((u32w4 *)(row + c * 8), zero);
    }
}

// Token of this lane's group in unit `b` of the work (a workgroup's share), and
// its first chunk.
template <int LANES>
__device__ __forceinline__ int64_t token_of(uint32_t b)
{
    if (LANES == 0) return b;
    constexpr int kLanes = LANES ? LANES : 64;
    const int g = threadIdx.x / kLanes;
    return (int64_t)b * (kThreads / kLanes) + (LANES == 64 ? __builtin_amdgcn_readfirstlane(g) : g);
}
template <int LANES>
__device__ __forceinline__ uint32_t chunk_of()
{
    return LANES ? threadIdx.x % (LANES ? LANES : 64) : threadIdx.x;
}

template <int LANES, int F8, bool NT>
__device__ __forceinline__ void dispatch_unit(const fqimpl::MoeRowsArgs &a, uint32_t b,
                                              uint32_t chunks, uint16_t *__restrict__ y)
{
    const int64_t t = token_of<LANES>(b);
    if (t >= a.T) return;
    for (uint32_t c = chunk_of<LANES>(); c < chunks; c += LANES ? LANES : blockDim.x) {
        u32w4 v;
        if (F8 == fqimpl::F8_NONE) {
            v = *(const u32w4 *)((const uint16_t *)a.x + t * a.H + c * 8);
        } else {
            float f[8], s;
            e4m3_decode8(*(const u32w2 *)((const uint8_t *)a.x + t * a.H + c * 8), f);
            if (F8 == fqimpl::F8_MX) {
                const uint32_t code = ((const uint8_t *)a.scales)[t * (a.H / 32) + c / 4];
                s = code == 255u ? as_f(0x7FC00000u) : e8m0_value(code);
            } else {
                s = ((const float *)a.scales)[t];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = bf16_pair_rne(f[2 * i] * s, f[2 * i + 1] * s);
        }
        for (int64_t j = t * a.k; j < (t + 1) * a.k; j += 4) {
            const Four f = four_of<LANES>(a, j, (t + 1) * a.k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (f.p[i] >= 0) store16<NT>((u32w4 *)(y + f.p[i] * a.H + c * 8), v);
        }
    }
}

// y[pos[t, j]] = x[t]; the units from `work` on clear the padding.
template <int LANES, int F8, bool NT>
__global__ __launch_bounds__(LANES ? kThreads : kMostThreads) void k_moe_dispatch(
    fqimpl::MoeRowsArgs a, uint32_t work, uint32_t units)
{
    uint16_t *y = (uint16_t *)a.rows_out;
    const uint32_t chunks = (uint32_t)(a.H / 8);
    for (uint32_t b = blockIdx.x; b < units; b += gridDim.x) {
        if (b < work) dispatch_unit<LANES, F8, NT>(a, b, chunks, y);
        else clear_padding<LANES, NT>(a, (int64_t)b - work, y);
    }
}

// out[t] = sum_j w[t, j] * y[pos[t, j]].  K 0: any k, a token at a time.  K 1 or
// 2: that k, and a group takes the tokens of four assignments together.
template <int LANES, int K, bool NT>
__device__ __forceinline__ void combine_unit(const fqimpl::MoeRowsArgs &a, uint32_t b,
                                             uint32_t chunks)
{
    constexpr int kTokens = K ? 4 / K : 1, kEach = K ? K : 4;      // of four assignments
    const uint16_t *__restrict__ y = (const uint16_t *)a.y;
    const int64_t t = token_of<LANES>(b) * kTokens;
    if (t >= a.T) return;
    for (uint32_t c = chunk_of<LANES>(); c < chunks; c += LANES ? LANES : blockDim.x) {
        float acc[kTokens][8] = {};
        const int64_t end = K ? a.T * K : (t + 1) * a.k;
        for (int64_t j = t * a.k; j < end; j += 4) {
            const Four f = four_of<LANES>(a, j, end);
            Raw8<uint16_t> r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (f.p[i] >= 0) load_raw8<false, NT>(y + f.p[i] * a.H + c * 8, 8, r[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (f.p[i] < 0) continue;
                float v[8];
                unpack8(r[i], v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[i / kEach][e] = __builtin_fmaf(f.w[i], v[e], acc[i / kEach][e]);
            }
            if (K) break;
        }
#pragma unroll
        for (int i = 0; i < kTokens; ++i)
            if (i == 0 || t + i < a.T)
                store8<false, NT>((uint16_t *)a.out + (t + i) * a.H + c * 8, 8, acc[i]);
    }
}

template <int LANES, int K, bool NT>
__global__ __launch_bounds__(LANES ? kThreads : kMostThreads) void k_moe_combine(
    fqimpl::MoeRowsArgs a, uint32_t work)
{
    const uint32_t chunks = (uint32_t)(a.H / 8);
    for (uint32_t b = blockIdx.x; b < work; b += gridDim.x) combine_unit<LANES, K, NT>(a, b, chunks);
}

// Up to four assignments a group: those of 4 / K tokens, or with K 0 one of the
// ceil(k / 4) even parts of a token's, of which none is empty.  Parts read
// dout[t] again, from the caches, and have nothing to wait for: 64 tokens with
// k = 8 and rows of 2880 take 4.6 us, one part after the other 6.3, 2048 tokens
// 39 and 42; the wide rows of 8192 tokens, 4096, lose 1 to 4 % with k of 5, 7
// and 8 (219 and 216).
template <int LANES, int K, bool NT>
__device__ __forceinline__ void combine_bwd_unit(const fqimpl::MoeRowsArgs &a, uint32_t b,
                                                 uint32_t chunks, uint16_t *__restrict__ dy,
                                                 float (*part)[kMostThreads / 64])
{
    constexpr int kTokens = K ? 4 / K : 1, kEach = K ? K : 4;
    const uint16_t *__restrict__ y = (const uint16_t *)a.y;
    const int64_t group = token_of<LANES>(b);
    int64_t t = group * kTokens, first = group * 4, end = a.T * K;
    if (K == 0) {
        const uint32_t parts = (uint32_t)(a.k + 3) / 4, each = ((uint32_t)a.k + parts - 1) / parts;
        t = (uint32_t)group / parts;
        first = t * a.k + ((uint32_t)group - (uint32_t)t * parts) * each;
        end = min(first + each, (t + 1) * a.k);
    }
    if (t >= a.T) return;                       // not with LANES 0, which has barriers
    const uint32_t c0 = chunk_of<LANES>();
    const Four f = four_of<LANES>(a, first, end);
    float dot[4] = {};
    for (uint32_t c = c0; c < chunks; c += LANES ? LANES : blockDim.x) {
        Raw8<uint16_t> r[4], dr[kTokens];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (f.p[i] >= 0) load_raw8<false, NT>(y + f.p[i] * a.H + c * 8, 8, r[i]);
#pragma unroll
        for (int i = 0; i < kTokens; ++i)
            load_raw8<false>((const uint16_t *)a.dout + min(t + i, a.T - 1) * a.H + c * 8, 8, dr[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (f.p[i] < 0) continue;
            float v[8], d[8];
            unpack8(r[i], v);
            unpack8(dr[i / kEach], d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dot[i] = __builtin_fmaf(d[e], v[e], dot[i]);
                v[e] = f.w[i] * d[e];
            }
            store8<false, NT>(dy + f.p[i] * a.H + c * 8, 8, v);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) dot[i] = lanes_sum<LANES ? LANES : 64>(dot[i]);
    if (LANES) {
        if (c0 == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (first + i < end) a.dweights[first + i] = dot[i];
        return;
    }
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[i][threadIdx.x >> 6] = dot[i];
    __syncthreads();
    if (threadIdx.x < 4 && first + threadIdx.x < end) {
        float v = part[threadIdx.x][0];
        for (uint32_t w = 1; w < blockDim.x / 64; ++w) v += part[threadIdx.x][w];
        a.dweights[first + threadIdx.x] = v;
    }
    __syncthreads();
}

// dy[pos[t, j]] = w[t, j] * dout[t], dw[t, j] = <dout[t], y[pos[t, j]]>; the
// units from `work` on clear the padding.
template <int LANES, int K, bool NT>
__global__ __launch_bounds__(LANES ? kThreads : kMostThreads) void k_moe_combine_bwd(
    fqimpl::MoeRowsArgs a, uint32_t work, uint32_t units)
{
    __shared__ float part[4][kMostThreads / 64];
    uint16_t *dy = (uint16_t *)a.rows_out;
    const uint32_t chunks = (uint32_t)(a.H / 8);
    for (uint32_t b = blockIdx.x; b < units; b += gridDim.x) {
        if (b < work) combine_bwd_unit<LANES, K, NT>(a, b, chunks, dy, part);
        else clear_padding<LANES, NT>(a, (int64_t)b - work, dy);
    }
}

// ---- launch -------------------------------------------------------------------
// A grid holds fewer than 2^32 lanes; the kernels walk over what is left.
constexpr uint32_t kMaxGrid = 1u << 22;

// Lanes of a group from the width alone: launch(lanes, units of work, threads)
// for `groups` groups.
template <typename F>
hipError_t by_width(const fqimpl::MoeRowsArgs &a, int64_t groups, F launch)
{
    const int64_t chunks = a.H / 8;
    const auto shared = [&](auto lanes) {
        const int64_t per = kThreads / decltype(lanes)::value;
        return launch(lanes, (uint32_t)((groups + per - 1) / per), (uint32_t)kThreads);
    };
    if (chunks <= 8) return shared(std::integral_constant<int, 8>());
    if (chunks <= 16) return shared(std::integral_constant<int, 16>());
    if (chunks <= 32) return shared(std::integral_constant<int, 32>());
    if (chunks <= 64) return shared(std::integral_constant<int, 64>());
    const int64_t threads = (chunks + 63) / 64 * 64;
    return launch(std::integral_constant<int, 0>(), (uint32_t)groups,
                  (uint32_t)(threads < kMostThreads ? threads : kMostThreads));
}

// Four assignments a group, of several tokens where k is 1 or 2 and there are
// many tokens: launch(k or 0, groups).  Rows of 2880: 16384 tokens with k = 1
// 34.6 us, one at a time 64.3, with k = 2 50.3 and 67.1; 2048 tokens 6.5 and
// 8.2; of fewer there are too few groups (1024 with k = 2 5.3 and 5.5).
constexpr int64_t kManyTokens = 2048;
template <typename F>
hipError_t by_k(const fqimpl::MoeRowsArgs &a, F launch)
{
    if (a.k == 1 && a.T >= kManyTokens) return launch(std::integral_constant<int, 1>(), (a.T + 3) / 4);
    if (a.k == 2 && a.T >= kManyTokens) return launch(std::integral_constant<int, 2>(), (a.T + 1) / 2);
    return launch(std::integral_constant<int, 0>(), a.T);
}

// Streaming accesses from this many elements of assigned rows (T * k * H) on, where
// they leave the caches.  Padding, which dispatch and combine's backward write
// too, does not count: its share is not known without the ids, and a call that is
// mostly padding streams late.  Of 8192 tokens (94 M elements) and 2048 (24 M): combine
// 41.6 us streaming, 46.8 not, and 13.1, 12.1; dispatch (its stores) 41.3, 50.6
// and 15.6, 15.5; combine's backward 76, 90 and 25.5, 29.2, of 1024 tokens (12 M)
// 16.0, 14.5.
constexpr int64_t kStreamForward = int64_t(1) << 25, kStreamBwd = int64_t(1) << 24;

}  // namespace

namespace fqimpl {

// a step of a workgroup, as far as the number of workgroups allows
static uint32_t moe_sort_chunk(int64_t n)
{
    const int64_t c = (n + kMoeMaxChunks - 1) / kMoeMaxChunks;
    return (uint32_t)((c + kSortThreads - 1) / kSortThreads * kSortThreads);
}

size_t moe_sort_counts(int64_t n, int64_t E)
{
    const int64_t chunk = moe_sort_chunk(n);
    return n <= kCountAll ? 0 : (size_t)((n + chunk - 1) / chunk * E);
}

hipError_t launch_moe_sort(MoeSortArgs a, hipStream_t stream)
{
    a.chunk = moe_sort_chunk(a.n);
    const uint32_t grid = (uint32_t)((a.n + a.chunk - 1) / a.chunk);
    if (a.n <= kCountAll) a.ws = nullptr;
    if (a.ws) {
        k_moe_count<<<dim3(grid), dim3(kSortThreads), 0, stream>>>(a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    k_moe_place<<<dim3(grid), dim3(kSortThreads), 0, stream>>>(a);
    return hipGetLastError();
}

template <int F8>
static hipError_t dispatch(const MoeRowsArgs &a, hipStream_t stream)
{
    const uint32_t pads = (uint32_t)((a.rows + kPadRows - 1) / kPadRows);
    return by_width(a, a.T, [&](auto lanes, uint32_t work, uint32_t threads) {
        constexpr int kLanes = decltype(lanes)::value;
        const uint32_t units = work + pads;
        const dim3 grid(units < kMaxGrid ? units : kMaxGrid), block(threads);
        if (a.T * a.k * a.H < kStreamForward)
            k_moe_dispatch<kLanes, F8, false><<<grid, block, 0, stream>>>(a, work, units);
        else
            k_moe_dispatch<kLanes, F8, true><<<grid, block, 0, stream>>>(a, work, units);
        return hipGetLastError();
    });
}

hipError_t launch_moe_dispatch(int f8, const MoeRowsArgs &a, hipStream_t stream)
{
    if (f8 == F8_MX) return dispatch<F8_MX>(a, stream);
    if (f8 == F8_ROW) return dispatch<F8_ROW>(a, stream);
    return dispatch<F8_NONE>(a, stream);
}

hipError_t launch_moe_combine(const MoeRowsArgs &a, hipStream_t stream)
{
    return by_k(a, [&](auto k, int64_t groups) {
        return by_width(a, groups, [&](auto lanes, uint32_t work, uint32_t threads) {
            constexpr int kLanes = decltype(lanes)::value, K = decltype(k)::value;
            const dim3 grid(work < kMaxGrid ? work : kMaxGrid), block(threads);
            if (a.T * a.k * a.H < kStreamForward)
                k_moe_combine<kLanes, K, false><<<grid, block, 0, stream>>>(a, work);
            else
                k_moe_combine<kLanes, K, true><<<grid, block, 0, stream>>>(a, work);
            return hipGetLastError();
        });
    });
}

hipError_t launch_moe_combine_bwd(const MoeRowsArgs &a, hipStream_t stream)
{
    const uint32_t pads = (uint32_t)((a.rows + kPadRows - 1) / kPadRows);
    return by_k(a, [&](auto k, int64_t groups) {
        const int64_t parts = decltype(k)::value ? 1 : (a.k + 3) / 4;
        return by_width(a, groups * parts, [&](auto lanes, uint32_t work, uint32_t threads) {
            constexpr int kLanes = decltype(lanes)::value, K = decltype(k)::value;
            const uint32_t units = work + pads;
            const dim3 grid(units < kMaxGrid ? units : kMaxGrid), block(threads);
            if (a.T * a.k * a.H < kStreamBwd)
                k_moe_combine_bwd<kLanes, K, false><<<grid, block, 0, stream>>>(a, work, units);
            else
                k_moe_combine_bwd<kLanes, K, true><<<grid, block, 0, stream>>>(a, work, units);
            return hipGetLastError();
        });
    });
}

}  // namespace fqimpl
