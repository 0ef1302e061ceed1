// fq_norm.hip -- residual addition and root-mean-square norm on gfx950, with
// BF16 or 8-bit output, and its backward.
//
//   h = x + res (stored in the stream's type), r = 1 / sqrt(mean(h^2) + eps),
//   n = h * r * gamma;   y = BF16(n), or E4M3 codes of n under a power-of-two
//   scale per 32 elements or an FP32 scale per row.
//   Backward: xh = h * r, g = dy * gamma,
//   dh = r * (g - xh * mean(g * xh)) + dres,  dgamma = sum over rows of dy * xh.
//
// Both passes are bound by memory: one read of every input and one write of
// every output, a row staying in registers between the statistic and its use.
//  * LANES lanes share a row (8 for a row of 64 elements, up to a workgroup of
//    1024; powers of two, or 5/8 of one), each holding NCH chunks of 8
//    consecutive elements (16-byte BF16 accesses); chunk i of lane l is i * LANES
//    + l, so neighbouring lanes read neighbouring chunks.  One chunk a lane up to
//    8192 columns in the backward, and in the forward of few rows or of a large
//    call with a residual: many short waves keep the loads of some rows in flight
//    while others wait for their sum (16384x4096 with 8-bit output: 512 lanes 100
//    us, 256 lanes of two chunks 107, 64 of eight 113; backward 8192x2880: 37.1,
//    39.5 and 41.2).  Two chunks a lane in the other forwards from 512 rows on
//    (Fwd::go).
//  * An MX block of 32 is four neighbouring lanes (two DPP steps).
//  * dgamma: each group of lanes walks over rows and keeps its column sums in
//    registers; the groups of a workgroup are added through LDS, the
//    workgroups' sums go to the workspace, and a second kernel adds those, all
//    in a fixed order (no atomics, the same bits on every call).
// Forward 16384x4096 with 8-bit output 98 to 101 us (6.0 to 6.2 TB/s), backward
// 8192x2880 37 us (5.1 TB/s, 4 us of it the second kernel); one row 2.6 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_internal.h"
#include "fq_rows.hpp"

using namespace fqdev;

namespace {

// Threads of a workgroup, or one row's lanes.  The backward's are more, because
// each workgroup leaves a row of column sums (32768x1024: 512 workgroups
// of 512 threads 47.5 us, of 256 52.0).
constexpr int kFwdThreads = 256, kBwdThreads = 512;
template <int LANES, int LEAST>
constexpr int threads_of() { return LANES <= LEAST ? LEAST : LANES; }

// Which of the workgroup's rows this lane works on: the same one for a whole
// wave where a row has at least one, so that addresses are a scalar base and a
// 32-bit offset.
template <int LANES>
__device__ __forceinline__ int group_of()
{
    const int g = threadIdx.x / LANES;
    return LANES >= 64 ? __builtin_amdgcn_readfirstlane(g) : g;
}

// Sum / maximum over the lanes of a row.  Where a row has several waves, `slot`
// is another one than the previous reduction's, so that one barrier between
// writing and reading is enough.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int slot)
{
    if (LANES <= 64) return lanes_sum<LANES>(v);
    v = lanes_sum<64>(v);
    const int wave = threadIdx.x >> 6, first = group_of<LANES>() * (LANES / 64);
    if ((threadIdx.x & 63) == 0) red[slot][wave] = v;
    __syncthreads();
    v = red[slot][first];
#pragma unroll
    for (int w = 1; w < LANES / 64; ++w) v += red[slot][first + w];
    return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float (*red)[16], int slot)
{
    if (LANES <= 64) return lanes_max<LANES>(v);
    v = lanes_max<64>(v);
    const int wave = threadIdx.x >> 6, first = group_of<LANES>() * (LANES / 64);
    if ((threadIdx.x & 63) == 0) red[slot][wave] = as_f(v);
    __syncthreads();
    v = as_u(red[slot][first]);
#pragma unroll
    for (int w = 1; w < LANES / 64; ++w) v = max(v, as_u(red[slot][first + w]));
    return v;
}

// Rows whose length is no multiple of 8 (ANY) start at any element.  A lane's
// chunks lie where 8-element boundaries of the whole array are, so that all of
// them but a row's first and last are 16-byte accesses: `shift` elements of the
// first one belong to the row before, and element e of the chunk at `pos` is
// column pos - shift + e.
struct Span {
    int lo, hi;              // the row's elements of a chunk; hi 0: none
};
template <bool ANY>
__device__ __forceinline__ Span span_of(uint32_t pos, int shift, int64_t cols, bool live)
{
    if (!ANY) return {0, live && pos < cols ? 8 : 0};
    const int lo = max(0, shift - (int)pos), hi = min(8, (int)cols + shift - (int)pos);
    return live && hi > lo ? Span{lo, hi} : Span{0, 0};
}
__device__ __forceinline__ bool inside(int e, Span s) { return e >= s.lo && e < s.hi; }

__device__ __forceinline__ void clear_outside(Raw8<uint16_t> &r, Span s)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r.w[i] &= (inside(2 * i, s) ? 0xFFFFu : 0u) | (inside(2 * i + 1, s) ? 0xFFFF0000u : 0u);
}
__device__ __forceinline__ void clear_outside(Raw8<float> &r, Span s)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.a[i] = inside(i, s) ? r.a[i] : 0u;
        r.b[i] = inside(i + 4, s) ? r.b[i] : 0u;
    }
}
// The chunk of an array at p (a chunk boundary) + pos; `left` elements of the
// array are left from p on.  What is not the row's reads as 0.
template <bool ANY, bool NT, typename T>
__device__ __forceinline__ void load_span(const T *__restrict__ p, uint32_t pos, Span s, int left,
                                          Raw8<T> &r)
{
    if (!ANY) return load_raw8<false, NT>(p + pos, 8, r);
    if ((int)pos + 8 <= left) load_raw8<false, NT>(p + pos, 8, r);
    else load_raw8<true>(p + pos, left - (int)pos, r);
    if (s.lo > 0 || s.hi < 8) clear_outside(r, s);
}
template <bool ANY, bool NT, typename T>
__device__ __forceinline__ void store_span(T *__restrict__ p, uint32_t pos, Span s, const float (&v)[8])
{
    if (!ANY || (s.lo == 0 && s.hi == 8)) return store8<false, NT>(p + pos, 8, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (inside(e, s)) store1(p + pos + e, v[e]);
}
// gamma of a chunk's columns in either type, 0 outside the row
template <bool ANY, typename T>
__device__ __forceinline__ void load_columns(const T *__restrict__ gamma, uint32_t pos, int shift,
                                             Span s, float (&g)[8])
{
    const T *q = gamma + ((int)pos - shift);
    if (s.lo == 0 && s.hi == 8) return load8<ANY>(q, 8, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = 0.0f;
    if (!ANY || s.hi == 0) return;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = load1(q + min(max(e, s.lo), s.hi - 1));   // in flight together
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = inside(e, s) ? v[e] : 0.0f;
}
template <bool ANY>
__device__ __forceinline__ void load_gamma(const void *gamma, int f32, uint32_t pos, int shift,
                                           Span s, float (&g)[8])
{
    if (f32) load_columns<ANY>((const float *)gamma, pos, shift, s, g);
    else load_columns<ANY>((const uint16_t *)gamma, pos, shift, s, g);
}

template <int STREAM> struct StreamType { typedef uint16_t type; };
template <> struct StreamType<2> { typedef float type; };

// STREAM: 0 no residual (h = x), 1 BF16 residual, 2 FP32 residual.
template <int LANES, int NCH, int STREAM, int F8, bool ANY, bool NT>
__global__ __launch_bounds__((threads_of<LANES, kFwdThreads>())) void k_rmsnorm_fwd(fqimpl::NormFwdArgs a)
{
    typedef typename StreamType<STREAM>::type T;
    constexpr int kGroups = threads_of<LANES, kFwdThreads>() / LANES;      // rows per workgroup
    __shared__ float red[4][16];
    const uint32_t l = threadIdx.x % LANES;
    const int group = group_of<LANES>();
    int slot = 0;
    // every lane of a workgroup makes the same number of turns (the barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < a.rows; r0 += (int64_t)gridDim.x * kGroups) {
        const int64_t row = r0 + group;
        const bool live = row < a.rows;
        const int64_t base = (live ? row : 0) * a.cols;
        const int shift = ANY ? (int)(base & 7) : 0;
        const int64_t start = base - shift;
        const int left = (int)min(a.rows * a.cols - start, (int64_t)1 << 30);
        float h[NCH][8];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t pos = (i * LANES + l) * 8;
            const Span s = span_of<ANY>(pos, shift, a.cols, live);
            if (s.hi == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
                continue;
            }
            Raw8<uint16_t> x;
            load_span<ANY, NT>((const uint16_t *)a.x + start, pos, s, left, x);
            if (STREAM) {
                Raw8<T> res;
                float r[8];
                load_span<ANY, NT>((const T *)a.res + start, pos, s, left, res);
                unpack8(x, h[i]);
                unpack8(res, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    h[i][e] = h[i][e] + r[e];
                    // the norm sees the stream's stored value, as the backward will
                    if (STREAM == 1) h[i][e] = (float)(__bf16)h[i][e];
                }
                store_span<ANY, NT>((T *)a.h + start, pos, s, h[i]);
            } else {
                unpack8(x, h[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += h[i][e] * h[i][e];
        }
        const float rstd = 1.0f / __builtin_sqrtf(row_sum<LANES>(ss, red, slot) / (float)a.cols + a.eps);
        if (a.rstd && live && l == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t pos = (i * LANES + l) * 8;
            const Span s = span_of<ANY>(pos, shift, a.cols, live);
            if (s.hi == 0) continue;
            float g[8];
            load_gamma<ANY>(a.gamma, a.gamma_f32, pos, shift, s, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = (h[i][e] * rstd) * g[e];
        }
        uint32_t top = 0;
        float scale = 0.0f, inv = 0.0f;
        if (F8 == fqimpl::F8_ROW) {
#pragma unroll
            for (int i = 0; i < NCH; ++i) top = max(top, absmax(h[i]));
            top = row_max<LANES>(top, red, 2 + slot);
            scale = __builtin_fmaxf(as_f(top) * (1.0f / 448.0f), 0x1p-126f);
            inv = 1.0f / scale;
            if (top >= 0x7F800000u) scale = as_f(0x7FC00000u);
            if (a.scales && live && l == 0) ((float *)a.scales)[row] = scale;
        }
        slot ^= 1;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t pos = (i * LANES + l) * 8;
            const Span s = span_of<ANY>(pos, shift, a.cols, live);
            if (s.hi == 0) continue;
            if (F8 != fqimpl::F8_NONE) {          // not with ANY
                const int64_t at = base + pos;
                if (F8 == fqimpl::F8_MX) {
                    top = dpp_max_xor2(dpp_max_xor1(absmax(h[i])));
                    const uint32_t code = mx8_scale_code(top);
                    scale = e8m0_value(code);
                    inv = e8m0_recip(code);
                    if (top >= 0x7F800000u) scale = as_f(0x7FC00000u);
                    if (a.scales && (l & 3) == 0)
                        ((uint8_t *)a.scales)[at >> 5] = (uint8_t)(top >= 0x7F800000u ? 255u : code);
                }
                float q[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    q[e] = F8 == fqimpl::F8_MX ? h[i][e] * inv
                                               : __builtin_fminf(__builtin_fmaxf(h[i][e] * inv, -448.0f), 448.0f);
                u32w2 codes = e4m3_encode8(q);
                if (top >= 0x7F800000u) codes = (u32w2){0x7F7F7F7Fu, 0x7F7F7F7Fu};
                if (a.codes) {
                    u32w2 *p = (u32w2 *)((uint8_t *)a.codes + at);
                    if (NT) __builtin_nontemporal_store(codes, p);
                    else *p = codes;
                }
                if (a.y) {
                    e4m3_decode8(codes, q);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[i][e] = q[e] * scale;
                }
            }
            if (a.y) store_span<ANY, NT>((uint16_t *)a.y + start, pos, s, h[i]);
        }
    }
}

// ---- backward -----------------------------------------------------------------
// Stops the compiler from carrying values computed from r across this point:
// they are computed from it again.
__device__ __forceinline__ void renew(Raw8<uint16_t> &r) { asm volatile("" : "+v"(r.w)); }
__device__ __forceinline__ void renew(Raw8<float> &r)
{
    asm volatile("" : "+v"(r.a));
    asm volatile("" : "+v"(r.b));
}

// A group of LANES lanes walks over rows group, group + groups, ...; T is the
// stream's type (h, dres, dh).  What bounds the walk is the number of bytes a
// CU has in flight, so all of a row's loads are issued together, and the row
// stays as it was loaded (a BF16 element in half a register) and is unpacked
// twice, before and after the row's sum.  A lane's share of gamma stays in
// registers, or in LDS where it has several chunks.  A group's rows are
// `groups` apart, a multiple of 8 if it has more than one: they all have the
// same shift, so a lane's columns stay the same ones.
template <int LANES, int NCH, typename T, bool ANY, bool NT>
__device__ __forceinline__ void bwd_rows(const fqimpl::NormBwdArgs &a, uint32_t workgroups)
{
    constexpr int kWgThreads = threads_of<LANES, kBwdThreads>(), kGroups = kWgThreads / LANES;
    static_assert(NCH == 1 || kGroups == 1, "several chunks a lane only where a row fills the workgroup");
    // dres with the other loads, unless it is wide and a lane's share long
    constexpr bool kEarly = sizeof(T) == 2 || NCH <= 4;
    constexpr bool kGammaLds = NCH > 1;
    __shared__ float red[2][16];
    __shared__ float sums[kGroups > 1 ? kGroups : 1][kGroups > 1 ? LANES * 8 : 1];
    __shared__ u32w4 gamma_lds[kGammaLds ? NCH * 2 : 1][kGammaLds ? LANES : 1];
    const uint32_t l = threadIdx.x % LANES;
    const int group = group_of<LANES>();
    const int64_t groups = (int64_t)workgroups * kGroups;
    const float inv_cols = 1.0f / (float)a.cols;
    const auto shift_of = [&](int g) {
        return ANY ? (int)(((int64_t)blockIdx.x * kGroups + g) * a.cols & 7) : 0;
    };
    const int shift = shift_of(group);
    float gamma[8], acc[NCH][8];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
        const uint32_t pos = (i * LANES + l) * 8;
        load_gamma<ANY>(a.gamma, a.gamma_f32, pos, shift, span_of<ANY>(pos, shift, a.cols, true), gamma);
        if (kGammaLds) {             // each lane reads its own
            gamma_lds[2 * i][l] = (u32w4){as_u(gamma[0]), as_u(gamma[1]), as_u(gamma[2]), as_u(gamma[3])};
            gamma_lds[2 * i + 1][l] = (u32w4){as_u(gamma[4]), as_u(gamma[5]), as_u(gamma[6]), as_u(gamma[7])};
        }
    }
    const auto gamma_of = [&](int i, float (&g)[8]) {
        if (kGammaLds) {
            unpack8(Raw8<float>{gamma_lds[2 * i][l], gamma_lds[2 * i + 1][l]}, g);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = gamma[e];
        }
    };
    int slot = 0;
    // every lane of a workgroup makes the same number of turns (row_sum's barrier)
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < a.rows; r0 += groups) {
        const int64_t row = r0 + group;
        const bool live = row < a.rows;
        const int64_t start = live ? row * a.cols - shift : 0;
        const int left = (int)min(a.rows * a.cols - start, (int64_t)1 << 30);
        Raw8<uint16_t> dy[NCH] = {};
        Raw8<T> h[NCH] = {}, dres[kEarly ? NCH : 1] = {};
        const float r = live ? a.rstd[row] : 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t pos = (i * LANES + l) * 8;
            const Span s = span_of<ANY>(pos, shift, a.cols, live);
            if (s.hi == 0) continue;
            load_span<ANY, NT>((const T *)a.h + start, pos, s, left, h[i]);
            load_span<ANY, NT>((const uint16_t *)a.dy + start, pos, s, left, dy[i]);
            if (kEarly && a.dres) load_span<ANY, NT>((const T *)a.dres + start, pos, s, left, dres[kEarly ? i : 0]);
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            float xh[8], d[8], g[8];
            unpack8(h[i], xh);
            unpack8(dy[i], d);
            gamma_of(i, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[e] = xh[e] * r;
                acc[i][e] = __builtin_fmaf(d[e], xh[e], acc[i][e]);
                dot = __builtin_fmaf(d[e] * g[e], xh[e], dot);
                asm volatile("" : "+v"(acc[i][e]));      // added here, not at the turn's end
            }
            renew(h[i]);
            renew(dy[i]);
            __builtin_amdgcn_sched_barrier(0);   // one chunk's temporaries at a time
        }
        dot = row_sum<LANES>(dot, red, slot) * inv_cols;
        slot ^= 1;
        if (kGammaLds) asm volatile("" ::: "memory");    // gamma is read again
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t pos = (i * LANES + l) * 8;
            const Span s = span_of<ANY>(pos, shift, a.cols, live);
            if (s.hi == 0) continue;
            float xh[8], d[8], g[8], o[8];
            if (!kEarly && a.dres) load_span<ANY, NT>((const T *)a.dres + start, pos, s, left, dres[0]);
            unpack8(h[i], xh);
            unpack8(dy[i], d);
            gamma_of(i, g);
            unpack8(dres[kEarly ? i : 0], o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = __builtin_fmaf(r, __builtin_fmaf(-(xh[e] * r), dot, d[e] * g[e]), o[e]);
            store_span<ANY, NT>((T *)a.dh + start, pos, s, o);
            if (a.dx) store_span<ANY, NT>((uint16_t *)a.dx + start, pos, s, o);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (!a.partials) return;
    // the workgroup's column sums; its groups may have different shifts
    float *out = a.partials + (int64_t)blockIdx.x * a.cols;
    if (kGroups > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[group][l * 8 + e] = acc[0][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += kWgThreads) {
            float v = sums[0][c + shift_of(0)];
#pragma unroll 8
            for (int g = 1; g < kGroups; ++g) v += sums[g][c + shift_of(g)];
            out[c] = v;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const uint32_t pos = (i * LANES + l) * 8;
        const Span s = span_of<ANY>(pos, shift, a.cols, true);
        float *at = out + ((int)pos - shift);
        if (s.lo == 0 && s.hi == 8) store8<ANY>(at, 8, acc[i]);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (inside(e, s)) at[e] = acc[i][e];
    }
}

template <int LANES, int NCH, typename T, bool ANY, bool NT>
__global__ __launch_bounds__((threads_of<LANES, kBwdThreads>()), 2) void k_rmsnorm_bwd(fqimpl::NormBwdArgs a)
{
    bwd_rows<LANES, NCH, T, ANY, NT>(a, gridDim.x);
}

// dgamma of 64 columns (eight lanes of 8) over all rows, by one workgroup.
template <int THREADS, typename T, bool ANY>
__device__ __forceinline__ void column_sums(const fqimpl::NormBwdArgs &a, int64_t c0)
{
    constexpr int kWaves = THREADS / 64;
    __shared__ float sums[kWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // the last lane's eight columns end with the row; some are its neighbour's too
    const int64_t mine = c0 + (threadIdx.x % 8) * 8, c = max((int64_t)0, min(mine, a.cols - 8));
    const int n = mine < a.cols ? (int)min((int64_t)8, a.cols) : 0;
    constexpr int kBatch = 4, kStep = THREADS / 8;     // rows in flight together
    float acc[8] = {};
    for (int64_t row0 = threadIdx.x / 8; n > 0 && row0 < a.rows; row0 += kBatch * kStep) {
        Raw8<uint16_t> dy[kBatch];
        Raw8<T> hr[kBatch];
        float r[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int64_t row = min(row0 + b * kStep, a.rows - 1);
            load_raw8<ANY>((const uint16_t *)a.dy + row * a.cols + c, n, dy[b]);
            load_raw8<ANY>((const T *)a.h + row * a.cols + c, n, hr[b]);
            r[b] = a.rstd[row];
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (row0 + b * kStep >= a.rows) break;
            float d[8], h[8];
            unpack8(dy[b], d);
            unpack8(hr[b], h);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(d[e], h[e] * r[b], acc[e]);
        }
    }
    // lanes with the same columns are eight apart
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        acc[e] += dpp_f<0x128>(acc[e]);
        acc[e] = as_f(across_rows<1>(as_u(acc[e]), add_f32));
        acc[e] = as_f(across_rows<2>(as_u(acc[e]), add_f32));
    }
    if (lane < 8)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e >= mine && e < n) sums[wave][c + e - c0] = acc[e];
    __syncthreads();
    if (threadIdx.x >= 64 || c0 + threadIdx.x >= a.cols) return;
    float v = sums[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += sums[w][threadIdx.x];
    a.dgamma[c0 + threadIdx.x] = v;
}

// The backward of few rows in one launch: the workgroups from a.groups on do
// dgamma, which needs no row's sum, 64 columns each, reading dy and h again.
template <int LANES, int NCH, typename T, bool ANY>
__global__ __launch_bounds__((threads_of<LANES, kBwdThreads>())) void k_rmsnorm_bwd_few(fqimpl::NormBwdArgs a)
{
    constexpr int kWgThreads = threads_of<LANES, kBwdThreads>();
    if (blockIdx.x >= a.groups) column_sums<kWgThreads, T, ANY>(a, (blockIdx.x - a.groups) * 64);
    else bwd_rows<LANES, NCH, T, ANY, false>(a, (uint32_t)a.groups);
}

// dgamma[c] = sum over the workgroups' sums, in their order: a workgroup takes
// 16 columns (64-byte pieces of a row), 64 threads each every 64th row; a wave
// joins its four sums of a column and one thread the sixteen waves' (512x2880
// 2.4 us; one thread adding all 64 sums 2.8).
constexpr int kSumCols = 16, kSumThreads = 1024, kSumParts = kSumThreads / kSumCols;
__global__ __launch_bounds__(kSumThreads) void k_column_sum(const float *__restrict__ partials,
                                                            int64_t groups, int64_t cols,
                                                            float *__restrict__ out)
{
    __shared__ float s[kSumThreads / 64][kSumCols];
    const int k = threadIdx.x % kSumCols, part = threadIdx.x / kSumCols;
    const int64_t c = (int64_t)blockIdx.x * kSumCols + k;
    float v = 0.0f;
    if (c < cols)
#pragma unroll 8
        for (int64_t g = part; g < groups; g += kSumParts) v += partials[g * cols + c];
    // four parts of a wave, 16 lanes apart, then the waves
    v = as_f(across_rows<1>(as_u(v), add_f32));
    v = as_f(across_rows<2>(as_u(v), add_f32));
    if (part % 4 == 0) s[part / 4][k] = v;
    __syncthreads();
    if (part || c >= cols) return;
#pragma unroll
    for (int w = 1; w < kSumThreads / 64; ++w) v += s[w][k];
    out[c] = v;
}

// ---- launch -------------------------------------------------------------------
// Lanes of a row and chunks per lane from the width alone; rows that start at
// any element take up to 7 more than their own.
int64_t width_of(int64_t cols) { return cols % 8 ? cols + 7 : cols; }

template <template <int, int> class F, typename A>
hipError_t by_width(const A &a, hipStream_t st)
{
    const int64_t width = width_of(a.cols);
    if (width <= 64) return F<8, 1>::go(a, st);
    if (width <= 128) return F<16, 1>::go(a, st);
    if (width <= 256) return F<32, 1>::go(a, st);
    if (width <= 512) return F<64, 1>::go(a, st);
    if (width <= 1024) return F<128, 1>::go(a, st);
    if (width <= 2048) return F<256, 1>::go(a, st);
    if (width <= 4096) return F<512, 1>::go(a, st);
    if (width <= 8192) return F<1024, 1>::go(a, st);
    if (width <= 16384) return F<1024, 2>::go(a, st);
    constexpr int kLanes = F<1024, 1>::kLanesMost;
    if (width <= 32768) return F<kLanes, 4096 / kLanes>::go(a, st);
    return F<kLanes, 4096 / kLanes + 1>::go(a, st);
}

// A grid holds fewer than 2^32 lanes; the kernels walk over what is left.
constexpr int64_t kMaxGrid = int64_t(1) << 20;
// Streaming accesses from this many elements on: what a call reads and writes
// no longer stays in the caches for the next one (forward with 8-bit output
// 4096x4096: 27.1 us streaming, 32.0 not; 2048x4096: 15.4 and 14.2; backward
// 31.2 and 32.3, 21.6 and 18.1).
constexpr int64_t kStreamElems = int64_t(1) << 24;

// Two chunks a lane instead of one: without a residual, where a lane has only 16
// bytes to load (16384x2880 in BF16 37.0 us instead of 40.5, with 8-bit rows 47
// instead of 58; 8471x6304 with MX blocks 54 instead of 72), and with one up to
// this many elements, whose workgroups then fit the CUs at once (1777x4096 in
// BF16 10.1 us instead of 11.4, 3000x4096 18.8 and 19.0, with an FP32 stream 22.1
// and 20.7).  Not of few rows (16x4096 3.4 us instead of 3.2).
constexpr int64_t kHalfRows = 512, kHalfElems = int64_t(1) << 23;

// Widths just over a power of two would leave up to half of the lanes without
// work.  Up to 5 / 8 of the next one a row of a call of many takes five waves
// (of two chunks) instead of eight (or sixteen) in BF16, and ten in the backward:
// with a residual 16384x2336 53.3 us instead of 59.7, 9000x5120 63.7 instead of
// 68.8, 9000x4095, which starts at any element, 61.3 instead of 71.5, without one
// 37.3 instead of 41.8.  Not with an FP32 stream, whose lanes have as many bytes
// in flight as two chunks (9000x5120 96 us with ten waves and with sixteen, 102
// with five), and rows of 2336 without a residual take four waves of two chunks
// (9000x2337 23.1 us, five waves 25.9).
template <int LANES, int NCH>
bool five_eighths(int64_t cols) { return LANES >= 512 && NCH == 1 && width_of(cols) <= 5 * LANES; }

template <int LANES, int NCH>
struct Fwd {
    static constexpr int kLanesMost = 1024;
    template <int STREAM, int F8, bool ANY, bool NT>
    static hipError_t launch(const fqimpl::NormFwdArgs &a, hipStream_t st)
    {
        constexpr int kWgThreads = threads_of<LANES, kFwdThreads>(), kGroups = kWgThreads / LANES;
        const int64_t wgs = (a.rows + kGroups - 1) / kGroups;
        k_rmsnorm_fwd<LANES, NCH, STREAM, F8, ANY, NT>
            <<<dim3((uint32_t)(wgs < kMaxGrid ? wgs : kMaxGrid)), dim3(kWgThreads), 0, st>>>(a);
        return hipGetLastError();
    }
    template <int STREAM, int F8>
    static hipError_t by_size(const fqimpl::NormFwdArgs &a, hipStream_t st)
    {
        const bool nt = a.rows * a.cols >= kStreamElems;
        if constexpr (F8 == fqimpl::F8_NONE)
            if (a.cols % 8)
                return nt ? launch<STREAM, F8, true, true>(a, st) : launch<STREAM, F8, true, false>(a, st);
        if constexpr (LANES * NCH > 4096) return hipErrorInvalidValue;     // wider than any row
        else return nt ? launch<STREAM, F8, false, true>(a, st) : launch<STREAM, F8, false, false>(a, st);
    }
    template <int STREAM>
    static hipError_t by_output(const fqimpl::NormFwdArgs &a, hipStream_t st)
    {
        if (a.f8 == fqimpl::F8_MX) return by_size<STREAM, fqimpl::F8_MX>(a, st);
        if (a.f8 == fqimpl::F8_ROW) return by_size<STREAM, fqimpl::F8_ROW>(a, st);
        return by_size<STREAM, fqimpl::F8_NONE>(a, st);
    }
    static hipError_t by_stream(const fqimpl::NormFwdArgs &a, hipStream_t st)
    {
        if (!a.res) return by_output<0>(a, st);
        return a.stream_f32 ? by_output<2>(a, st) : by_output<1>(a, st);
    }
    static hipError_t go(const fqimpl::NormFwdArgs &a, hipStream_t st)
    {
        // half the lanes, two chunks each, where that keeps enough in flight
        constexpr int kHalf = LANES > 64 ? 2 : 1;
        const bool half = a.rows >= kHalfRows && (!a.res || a.rows * a.cols < kHalfElems);
        if (five_eighths<LANES, NCH>(a.cols) && a.rows >= kHalfRows && !(a.res && a.stream_f32)) {
            if constexpr (LANES == 512 && NCH == 1)
                if (!half) return Fwd<320, 1>::template by_output<1>(a, st);
            if constexpr (LANES == 1024 && NCH == 1)
                return a.res ? Fwd<320, 2>::template by_output<1>(a, st)
                             : Fwd<320, 2>::template by_output<0>(a, st);
        }
        if (half) return Fwd<LANES / kHalf, NCH * kHalf>::by_stream(a, st);
        return by_stream(a, st);
    }
};

// The gradients of the rows and of gamma in one launch while reading dy and h
// again, from the caches, takes less than a second launch and its column sums,
// which grows with the rows (one and two, on inputs of three calls in turn:
// 333x1000 FP32 4.3 and 5.7 us, 512x2880 7.7 and 10.4, 640x2880 9.1 and 10.9,
// 640x1000 7.0 and 6.2, 640x4096 9.6 and 13.1, 768x2880 10.5 and 10.9, 768x1000
// 8.6 and 6.5, 1024x2880 14.4 and 11.6; 640x6072 11.8 and 13.8, FP32 16.6 and
// 16.5; rows that start at any element 320x6073 9.6 and 14.2, 640x6073 17.1 and
// 15.3).  The crossing depends on the columns, the limit does not: at 1000 columns
// one launch still wins at 512 rows (5.4 and 5.9), at 640 it loses 0.8 us, and up
// to 1.1 in FP32 rows that start at any element (640x2047 13.8 and 12.7).
constexpr int64_t kFewRows = 640, kFewElems = int64_t(1) << 22, kFewElemsAny = int64_t(1) << 21;

template <int LANES, int NCH>
struct Bwd {
    static constexpr int kLanesMost = 512;      // 1024 lanes would have 128 registers each: too few
    template <typename T>
    static hipError_t launch(const fqimpl::NormBwdArgs &a, hipStream_t st)
    {
        if (a.cols % 8) return by_size<T, true>(a, st);
        if constexpr (LANES * NCH > 4096) return hipErrorInvalidValue;     // wider than any row
        else return by_size<T, false>(a, st);
    }
    template <typename T, bool ANY>
    static hipError_t by_size(const fqimpl::NormBwdArgs &a, hipStream_t st)
    {
        const dim3 block(threads_of<LANES, kBwdThreads>());
        const uint32_t grid = (uint32_t)a.groups;
        if (a.few)
            k_rmsnorm_bwd_few<LANES, NCH, T, ANY><<<dim3(grid + (uint32_t)((a.cols + 63) / 64)), block, 0, st>>>(a);
        else if (a.rows * a.cols >= kStreamElems)
            k_rmsnorm_bwd<LANES, NCH, T, ANY, true><<<dim3(grid), block, 0, st>>>(a);
        else
            k_rmsnorm_bwd<LANES, NCH, T, ANY, false><<<dim3(grid), block, 0, st>>>(a);
        return hipGetLastError();
    }
    static hipError_t go(const fqimpl::NormBwdArgs &a, hipStream_t st)
    {
        if constexpr (LANES == 1024 && NCH == 1)
            if (five_eighths<LANES, NCH>(a.cols)) return Bwd<640, 1>::go(a, st);
        return a.stream_f32 ? launch<float>(a, st) : launch<uint16_t>(a, st);
    }
};

}  // namespace

namespace fqimpl {

hipError_t launch_rmsnorm_fwd(const NormFwdArgs &a, hipStream_t stream)
{
    return by_width<Fwd>(a, stream);
}

// Workgroups that would take all rows at once.
static int64_t rows_workgroups(int64_t rows, int64_t cols)
{
    int64_t lanes = 8;
    while (lanes < kBwdThreads && lanes * 8 < width_of(cols)) lanes *= 2;
    const int64_t per_wg = kBwdThreads / lanes;
    return (rows + per_wg - 1) / per_wg;
}

// Workgroups that walk over the rows, each leaving a row of column sums, no more
// than there are rows for: two on each of 256 CUs, one where a row has 640 lanes
// or more (or 512 with many registers).  In streaming calls two also of 640
// lanes, except of FP32 rows of whole chunks (9000x5120 BF16 68.8 us, one 77.8,
// FP32 142 and 133; 9000x4095 64.2 and 83.5, FP32 118 and 131), and three of BF16
// rows that start at any element and fill more than a wave (12836x2337 55.5 us,
// two 63.3; 38560x778 50.4 and 54.2; 61224x490 51.7 and 48.0, 1711x2337 16.0 and
// 15.1, FP32 17355x2881 167 and 161).
static int64_t bwd_groups(int64_t rows, int64_t cols, bool f32)
{
    const int64_t wgs = rows_workgroups(rows, cols), width = width_of(cols);
    const bool any = cols % 8, large = rows * cols >= kStreamElems;
    int64_t most = width <= kBwdThreads * 8 ? 512 : 256;
    if (large && width > 512 && width <= 4096 && any && !f32) most = 768;
    if (large && width > 4096 && width <= 5120 && (any || !f32)) most = 512;
    return wgs < most ? wgs : most;
}
int64_t rmsnorm_bwd_groups(int64_t rows, int64_t cols)
{
    return bwd_groups(rows, cols, false);          // of FP32 rows there are no more
}

static bool few_rows(const NormBwdArgs &a)
{
    // a gradient written over dy or h would be read as one of them
    return a.dgamma && a.rows <= kFewRows &&
           a.rows * a.cols <= (a.cols % 8 ? kFewElemsAny : kFewElems) && a.dh != a.h && a.dh != a.dy && a.dx != a.h &&
           a.dx != a.dy;
}

hipError_t launch_rmsnorm_bwd(NormBwdArgs a, hipStream_t stream)
{
    a.few = few_rows(a);
    a.groups = a.few ? rows_workgroups(a.rows, a.cols)
                       : bwd_groups(a.rows, a.cols, a.stream_f32);
    if (!a.dgamma || a.few) a.partials = nullptr;
    const hipError_t e = by_width<Bwd>(a, stream);
    if (e != hipSuccess || !a.partials) return e;
    k_column_sum<<<dim3((uint32_t)((a.cols + kSumCols - 1) / kSumCols)), dim3(kSumThreads), 0, stream>>>(
        a.partials, a.groups, a.cols, a.dgamma);
    return hipGetLastError();
}

}  // namespace fqimpl
