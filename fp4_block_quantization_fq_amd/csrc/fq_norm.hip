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
//  * WPR waves share a row, each lane holding NCH chunks of 8 consecutive
//    elements (16-byte BF16 accesses); chunk i of lane l of the row's lanes is
//    i * 64 * WPR + l, so every access of a wave covers 1 KB.
//  * An MX block of 32 is four neighbouring lanes (two DPP steps).
//  * dgamma: each group of WPR waves walks over rows and keeps its column sums
//    in registers; they go to the workspace once, and a second kernel adds the
//    groups in a fixed order (no atomics, the same bits on every call).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_internal.h"
#include "fq_rows.hpp"

using namespace fqdev;

namespace {

// Sum / maximum over the WPR waves of a row.  `slot` alternates per use so
// that one barrier between writing and reading is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int slot)
{
    v = wave_sum(v);
    if (WPR == 1) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[slot][wave] = v;
    __syncthreads();
    const int first = wave / WPR * WPR;
    v = red[slot][first];
#pragma unroll
    for (int w = 1; w < WPR; ++w) v += red[slot][first + w];
    return v;
}
template <int WPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float (*red)[16], int slot)
{
    v = wave_max(v);
    if (WPR == 1) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[slot][wave] = as_f(v);
    __syncthreads();
    const int first = wave / WPR * WPR;
    v = as_u(red[slot][first]);
#pragma unroll
    for (int w = 1; w < WPR; ++w) v = max(v, as_u(red[slot][first + w]));
    return v;
}

template <int WPR>
constexpr int threads_of() { return WPR <= 4 ? 256 : WPR * 64; }

// gamma of eight columns in either type
template <bool ANY>
__device__ __forceinline__ void load_gamma(const void *gamma, int f32, int64_t c, int n,
                                           float (&g)[8])
{
    if (f32) load8<ANY>((const float *)gamma + c, n, g);
    else load8<ANY>((const uint16_t *)gamma + c, n, g);
}

template <int STREAM> struct StreamType { typedef uint16_t type; };
template <> struct StreamType<2> { typedef float type; };

// STREAM: 0 no residual (h = x), 1 BF16 residual, 2 FP32 residual.
template <int WPR, int NCH, int STREAM, int F8, bool ANY>
__global__ __launch_bounds__(threads_of<WPR>()) void k_rmsnorm_fwd(fqimpl::NormFwdArgs a)
{
    typedef typename StreamType<STREAM>::type T;
    constexpr int kGroups = threads_of<WPR>() / 64 / WPR;      // rows per workgroup
    __shared__ float red[2][16];
    const int wave = threadIdx.x >> 6, l = (wave % WPR) * 64 + (threadIdx.x & 63);
    const int64_t row = (int64_t)blockIdx.x * kGroups + wave / WPR;
    const bool live = row < a.rows;
    const int64_t base = (live ? row : 0) * a.cols;
    float h[NCH][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * WPR * 64 + l) * 8;
        const int n = live ? min(8, (int)a.cols - c) : 0;
        if (n <= 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
            continue;
        }
        load8<ANY>((const uint16_t *)a.x + base + c, n, h[i]);
        if (STREAM) {
            float r[8];
            load8<ANY>((const T *)a.res + base + c, n, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = h[i][e] + r[e];
                // the norm sees the stream's stored value, as the backward will
                if (STREAM == 1) h[i][e] = (float)(__bf16)h[i][e];
            }
            store8<ANY>((T *)a.h + base + c, n, h[i]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += h[i][e] * h[i][e];
    }
    const float rstd = 1.0f / __builtin_sqrtf(row_sum<WPR>(ss, red, 0) / (float)a.cols + a.eps);
    if (a.rstd && live && l == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * WPR * 64 + l) * 8;
        const int n = live ? min(8, (int)a.cols - c) : 0;
        if (n <= 0) continue;
        float g[8];
        load_gamma<ANY>(a.gamma, a.gamma_f32, c, n, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = (h[i][e] * rstd) * g[e];
    }
    uint32_t top = 0;
    float scale = 0.0f, inv = 0.0f;
    if (F8 == fqimpl::F8_ROW) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) top = max(top, absmax8(h[i]));
        top = row_max<WPR>(top, red, 1);
        scale = __builtin_fmaxf(as_f(top) * (1.0f / 448.0f), 0x1p-126f);
        inv = 1.0f / scale;
        if (top >= 0x7F800000u) scale = as_f(0x7FC00000u);
        if (a.scales && live && l == 0) ((float *)a.scales)[row] = scale;
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * WPR * 64 + l) * 8;
        const int n = live ? min(8, (int)a.cols - c) : 0;
        if (n <= 0) continue;
        if (F8 != fqimpl::F8_NONE) {
            if (F8 == fqimpl::F8_MX) {
                top = dpp_max_xor2(dpp_max_xor1(absmax8(h[i])));
                const uint32_t code = mx8_scale_code(top);
                scale = e8m0_value(code);
                inv = e8m0_recip(code);
                if (top >= 0x7F800000u) scale = as_f(0x7FC00000u);
                if (a.scales && (l & 3) == 0)
                    ((uint8_t *)a.scales)[(base + c) >> 5] = (uint8_t)(top >= 0x7F800000u ? 255u : code);
            }
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                q[e] = F8 == fqimpl::F8_MX ? h[i][e] * inv
                                           : __builtin_fminf(__builtin_fmaxf(h[i][e] * inv, -448.0f), 448.0f);
            u32w2 codes = e4m3_encode8(q);
            if (top >= 0x7F800000u) codes = (u32w2){0x7F7F7F7Fu, 0x7F7F7F7Fu};
            if (a.codes) *(u32w2 *)((uint8_t *)a.codes + base + c) = codes;
            if (a.y) {
                e4m3_decode8(codes, q);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] = q[e] * scale;
            }
        }
        if (a.y) store8<ANY>((uint16_t *)a.y + base + c, n, h[i]);
    }
}

// One group of WPR waves walks over rows group, group + groups, ...; T is the
// stream's type (h, dres, dh).
template <int WPR, int NCH, typename T, bool ANY>
__global__ __launch_bounds__(threads_of<WPR>()) void k_rmsnorm_bwd(fqimpl::NormBwdArgs a)
{
    constexpr int kGroups = threads_of<WPR>() / 64 / WPR;
    __shared__ float red[2][16];
    const int wave = threadIdx.x >> 6, l = (wave % WPR) * 64 + (threadIdx.x & 63);
    const int64_t group = (int64_t)blockIdx.x * kGroups + wave / WPR;
    const int64_t groups = (int64_t)gridDim.x * kGroups;
    const float inv_cols = 1.0f / (float)a.cols;
    float gamma[NCH][8], acc[NCH][8];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * WPR * 64 + l) * 8;
        const int n = min(8, (int)a.cols - c);
#pragma unroll
        for (int e = 0; e < 8; ++e) gamma[i][e] = acc[i][e] = 0.0f;
        if (n > 0) load_gamma<ANY>(a.gamma, a.gamma_f32, c, n, gamma[i]);
    }
    int slot = 0;
    // every wave of a workgroup makes the same number of turns (row_sum's barrier)
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < a.rows; r0 += groups) {
        const int64_t row = r0 + wave / WPR;
        const bool live = row < a.rows;
        const int64_t base = (live ? row : 0) * a.cols;
        const float r = live ? a.rstd[row] : 0.0f;
        float xh[NCH][8], g[NCH][8];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * WPR * 64 + l) * 8;
            const int n = live ? min(8, (int)a.cols - c) : 0;
            if (n <= 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) xh[i][e] = g[i][e] = 0.0f;
                continue;
            }
            load8<ANY>((const T *)a.h + base + c, n, xh[i]);
            load8<ANY>((const uint16_t *)a.dy + base + c, n, g[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[i][e] = xh[i][e] * r;
                acc[i][e] += g[i][e] * xh[i][e];
                g[i][e] = g[i][e] * gamma[i][e];
                dot += g[i][e] * xh[i][e];
            }
        }
        dot = row_sum<WPR>(dot, red, slot) * inv_cols;
        slot ^= 1;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * WPR * 64 + l) * 8;
            const int n = live ? min(8, (int)a.cols - c) : 0;
            if (n <= 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[i][e] = r * (g[i][e] - xh[i][e] * dot);
            if (a.dres) {
                load8<ANY>((const T *)a.dres + base + c, n, xh[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[i][e] += xh[i][e];
            }
            store8<ANY>((T *)a.dh + base + c, n, g[i]);
            if (a.dx) store8<ANY>((uint16_t *)a.dx + base + c, n, g[i]);
        }
    }
    if (!a.partials) return;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * WPR * 64 + l) * 8;
        const int n = min(8, (int)a.cols - c);
        if (n > 0) store8<ANY>(a.partials + group * a.cols + c, n, acc[i]);
    }
}

// dgamma[c] = sum over groups, in the groups' order: a workgroup takes 64
// columns, its waves every 16th group, and wave 0 adds the 16 sums.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void k_column_sum(const float *__restrict__ partials,
                                                            int64_t groups, int64_t cols,
                                                            float *__restrict__ out)
{
    __shared__ float s[kSumThreads / 64][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (c < cols)
#pragma unroll 8
        for (int64_t g = wave; g < groups; g += kSumThreads / 64) v += partials[g * cols + c];
    s[wave][lane] = v;
    __syncthreads();
    if (wave || c >= cols) return;
#pragma unroll
    for (int w = 1; w < kSumThreads / 64; ++w) v += s[w][lane];
    out[c] = v;
}

// ---- launch -------------------------------------------------------------------
// Waves per row and chunks per lane from the width alone.
template <template <int, int> class F, typename A>
hipError_t by_width(const A &a, hipStream_t st)
{
    if (a.cols <= 512) return F<1, 1>::go(a, st);
    if (a.cols <= 1024) return F<1, 2>::go(a, st);
    if (a.cols <= 2048) return F<1, 4>::go(a, st);
    if (a.cols <= 4096) return F<4, 2>::go(a, st);
    if (a.cols <= 8192) return F<4, 4>::go(a, st);
    if (a.cols <= 16384) return F<16, 2>::go(a, st);
    return F<16, 4>::go(a, st);
}

template <int WPR, int NCH>
struct Fwd {
    template <int STREAM, int F8, bool ANY>
    static hipError_t launch(const fqimpl::NormFwdArgs &a, hipStream_t st)
    {
        constexpr int kThreads = threads_of<WPR>(), kGroups = kThreads / 64 / WPR;
        k_rmsnorm_fwd<WPR, NCH, STREAM, F8, ANY>
            <<<dim3((uint32_t)((a.rows + kGroups - 1) / kGroups)), dim3(kThreads), 0, st>>>(a);
        return hipGetLastError();
    }
    template <int STREAM>
    static hipError_t by_output(const fqimpl::NormFwdArgs &a, hipStream_t st)
    {
        if (a.f8 == fqimpl::F8_MX) return launch<STREAM, fqimpl::F8_MX, false>(a, st);
        if (a.f8 == fqimpl::F8_ROW) return launch<STREAM, fqimpl::F8_ROW, false>(a, st);
        return a.cols % 8 ? launch<STREAM, fqimpl::F8_NONE, true>(a, st)
                          : launch<STREAM, fqimpl::F8_NONE, false>(a, st);
    }
    static hipError_t go(const fqimpl::NormFwdArgs &a, hipStream_t st)
    {
        if (!a.res) return by_output<0>(a, st);
        return a.stream_f32 ? by_output<2>(a, st) : by_output<1>(a, st);
    }
};

template <int WPR, int NCH>
struct Bwd {
    template <typename T>
    static hipError_t launch(const fqimpl::NormBwdArgs &a, hipStream_t st)
    {
        constexpr int kThreads = threads_of<WPR>(), kGroups = kThreads / 64 / WPR;
        const uint32_t grid = (uint32_t)(a.groups / kGroups);
        if (a.cols % 8) k_rmsnorm_bwd<WPR, NCH, T, true><<<dim3(grid), dim3(kThreads), 0, st>>>(a);
        else k_rmsnorm_bwd<WPR, NCH, T, false><<<dim3(grid), dim3(kThreads), 0, st>>>(a);
        return hipGetLastError();
    }
    static hipError_t go(const fqimpl::NormBwdArgs &a, hipStream_t st)
    {
        return a.stream_f32 ? launch<float>(a, st) : launch<uint16_t>(a, st);
    }
};

}  // namespace

namespace fqimpl {

hipError_t launch_rmsnorm_fwd(const NormFwdArgs &a, hipStream_t stream)
{
    return by_width<Fwd>(a, stream);
}

// Groups of waves that walk over the rows, a multiple of the groups of a
// workgroup: enough for two workgroups on each of 256 CUs, no more than rows.
int64_t rmsnorm_bwd_groups(int64_t rows, int64_t cols)
{
    const int64_t per_wg = cols <= 2048 ? 4 : 1;
    const int64_t wgs = (rows + per_wg - 1) / per_wg;
    return (wgs < 512 ? wgs : 512) * per_wg;
}

hipError_t launch_rmsnorm_bwd(NormBwdArgs a, float *dgamma, hipStream_t stream)
{
    a.groups = rmsnorm_bwd_groups(a.rows, a.cols);
    if (!dgamma) a.partials = nullptr;
    hipError_t e = by_width<Bwd>(a, stream);
    if (e != hipSuccess || !dgamma) return e;
    k_column_sum<<<dim3((uint32_t)((a.cols + 63) / 64)), dim3(kSumThreads), 0, stream>>>(
        a.partials, a.groups, a.cols, dgamma);
    return hipGetLastError();
}

}  // namespace fqimpl
