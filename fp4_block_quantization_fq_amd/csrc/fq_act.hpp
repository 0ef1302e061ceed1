// fq_act.hpp -- device code that the feed-forward products and the kernels
// around them share: activations and their derivatives, the gate, 8-bit blocks,
// and the experts' segments of rows.
//
// Activations are FP32, from the hardware's exp2 and reciprocal (1 ulp each).  The
// exponent is rounded: exp(-z) is off by |z| 2^-23 of itself, exp(-z^2 / 2) by z^2 2^-24.
// So are a sigmoid and a normal distribution where they fall to 0; where they are near 1
// the error falls as their distance to 1 does.  An infinite value before SiLU or GELU may
// give NaN (infinity times 0), as their formulas have it.
#pragma once

#include <type_traits>

#include "fq_internal.h"
#include "fq_rows.hpp"

namespace fqdev {

using fqimpl::Gate;

constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2E));
}
// The normal distribution function and *e = exp(-z^2 / 2).  With x = |z| / sqrt 2 its
// smaller side is erfc(x) / 2 = e erfcx(x) / 2, and erfcx(x) = t P(t) for
// t = 1 / (1 + 0.34 x), P of degree 9 fitted to erfcx for the least largest relative
// error: 2.5e-08 with its coefficients in FP32.  So the far side has a relative precision
// too: 4e-07 up to |z| = 1, 2e-06 at 6, 8e-06 at 12.6, nearly all of it the exponent's.
__device__ __forceinline__ float normal_cdf(float z, float *e)
{
    constexpr float P[] = {0.191816539f, 0.192037061f, 0.178268477f, 0.174870953f,
                           0.0593979955f, 0.275508434f, -0.278319448f, 0.401717603f,
                           -0.246014193f, 0.0507165603f};
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(z), 0.240416306f, 1.0f));
    float q = P[9];
#pragma unroll
    for (int i = 8; i >= 0; --i) q = __builtin_fmaf(q, t, P[i]);
    *e = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2E));
    q *= 0.5f * t * *e;
    return z < 0.0f ? q : 1.0f - q;
}

// a(z) and a'(z)
template <int ACT>
__device__ __forceinline__ float act_of(float alpha, float z)
{
    if (ACT == fqimpl::ACT_SILU) return z * sigmoid(alpha * z);
    if (ACT == fqimpl::ACT_GELU) {
        float e;
        return z * normal_cdf(z, &e);
    }
    if (ACT == fqimpl::ACT_RELU) return z <= 0.0f ? 0.0f : z;
    return z;
}
template <int ACT>
__device__ __forceinline__ float act_grad_of(float alpha, float z, float *value)
{
    if (ACT == fqimpl::ACT_SILU) {
        const float s = sigmoid(alpha * z);
        *value = z * s;
        return __builtin_fmaf(alpha, *value * (1.0f - s), s);          // in this order no finite z overflows
    }
    if (ACT == fqimpl::ACT_GELU) {
        float e;
        const float phi = normal_cdf(z, &e);
        *value = z * phi;
        return phi + z * (0.39894228040143268f * e);
    }
    if (ACT == fqimpl::ACT_RELU) {
        *value = z <= 0.0f ? 0.0f : z;
        return z <= 0.0f ? 0.0f : 1.0f;
    }
    *value = z;
    return 1.0f;
}

// The choice of the activation stands around the eight values, so that their chains
// of instructions interleave (inside, a branch before each of them cost 7 us in a
// call of 27).
template <typename F>
__device__ __forceinline__ void with_act(int act, F run)
{
    if (act == fqimpl::ACT_SILU) run(std::integral_constant<int, fqimpl::ACT_SILU>());
    else if (act == fqimpl::ACT_GELU) run(std::integral_constant<int, fqimpl::ACT_GELU>());
    else if (act == fqimpl::ACT_RELU) run(std::integral_constant<int, fqimpl::ACT_RELU>());
    else run(std::integral_constant<int, fqimpl::ACT_NONE>());
}
template <int N>
__device__ __forceinline__ void act_n(int act, float alpha, float (&z)[N])
{
    with_act(act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = act_of<decltype(kind)::value>(alpha, z[i]);
    });
}
// dy *= a'(z)
__device__ __forceinline__ void act8_grad(int act, const float (&z)[8], float (&dy)[8])
{
    with_act(act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float value;
            dy[i] *= act_grad_of<decltype(kind)::value>(1.0f, z[i], &value);
        }
    });
}

// g = a(min(g, limit)) (clamp(u, -limit, limit) + shift); NaN stays NaN
template <int N>
__device__ __forceinline__ void glu_n(const Gate &t, float (&g)[N], const float (&u)[N])
{
    with_act(t.act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float gate = g[i] > t.limit ? t.limit : g[i];
            const float up = u[i] > t.limit ? t.limit : u[i] < -t.limit ? -t.limit : u[i];
            g[i] = act_of<decltype(kind)::value>(t.alpha, gate) * (up + t.shift);
        }
    });
}
// Its backward for the gradient dh: dg and du into g and u, h's value into dh.
__device__ __forceinline__ void glu8_grad(const Gate &t, float (&g)[8], float (&u)[8], float (&dh)[8])
{
    with_act(t.act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool g_out = g[i] > t.limit, u_out = u[i] > t.limit || u[i] < -t.limit;
            const float gate = g_out ? t.limit : g[i];
            const float up = (u[i] > t.limit ? t.limit : u[i] < -t.limit ? -t.limit : u[i]) + t.shift;
            float a;
            const float da = act_grad_of<decltype(kind)::value>(t.alpha, gate, &a);
            // dh up first, whose underflow is the result's; where it overflows, dh da first
            float dg = dh[i] * up;
            dg = __builtin_fabsf(dg) == __builtin_inff() ? dh[i] * da * up : dg * da;
            g[i] = g_out ? 0.0f : dg;
            u[i] = u_out ? 0.0f : dh[i] * a;
            dh[i] = a * up;
        }
    });
}

// ---- 8-bit blocks ------------------------------------------------------------------
// Eight of a block's 32 values (four neighbouring lanes hold the block): E4M3
// codes under the smallest power of two that keeps them below 448; returns its
// E8M0 code (255 and codes 0x7F where the block has an infinity or NaN).
__device__ __forceinline__ uint32_t mx8_encode8(const float (&v)[8], u32w2 *codes)
{
    const uint32_t top = dpp_max_xor2(dpp_max_xor1(absmax(v)));
    const uint32_t code = mx8_scale_code(top);
    const float inv = e8m0_recip(code);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] * inv;
    *codes = e4m3_encode8(q);
    if (top < 0x7F800000u) return code;
    *codes = (u32w2){0x7F7F7F7Fu, 0x7F7F7F7Fu};
    return 255u;
}
// the value of an E8M0 code, NaN for 255
__device__ __forceinline__ float mx8_scale(uint32_t code)
{
    return code == 255u ? as_f(0x7FC00000u) : e8m0_value(code);
}
// An FP32 scale of a row (normal, or NaN) as a power of two and a mantissa.  Mantissas
// are from 1/2 to 1, so that a finite gradient times one is finite in BF16.  From 2^100
// on they are from 1 to 2: there twice the power could take a code's value out of range.
__device__ __forceinline__ bool row_scale_large(float s) { return !(s < 0x1p100f); }
__device__ __forceinline__ float row_scale_power(float s)
{
    const float p = as_f(as_u(s) & 0xFF800000u);
    return row_scale_large(s) ? p : 2.0f * p;
}
__device__ __forceinline__ float row_scale_mantissa(float s)
{
    return as_f((as_u(s) & 0x7FFFFFu) | (row_scale_large(s) ? 0x3F800000u : 0x3F000000u));
}

// ---- grids -----------------------------------------------------------------------------
// `n` workgroups of THREADS and one's number.  The threads along an axis of a grid have
// to stay below 2^32, which the largest calls' workgroups are not; the last row of such a
// grid has numbers from n on.  A row is a constant: gridDim would have to be loaded (0.2
// of 7 us in a call of one row).
constexpr int grid_row(int threads) { return (1 << 30) / threads; }       // a multiple of the XCDs
template <int THREADS>
dim3 grid_of(int64_t n)
{
    constexpr int row = grid_row(THREADS);
    if (n <= row) return dim3((uint32_t)n);
    return dim3((uint32_t)row, (uint32_t)((n + row - 1) / row));
}
template <int THREADS>
__device__ __forceinline__ int workgroup()
{
    return (int)(blockIdx.y * grid_row(THREADS) + blockIdx.x);
}

// ---- the experts' segments of rows ---------------------------------------------------
// offsets[e] .. offsets[e + 1], brought into 0 .. rows, so that no entry can lead
// outside the buffers.
__device__ __forceinline__ void segment_of(const int32_t *offsets, int e, int rows, int *begin, int *end)
{
    *begin = min(max(offsets[e], 0), rows);
    *end = max(*begin, min(offsets[e + 1], rows));
}
__device__ __forceinline__ int wave_total(int v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return __builtin_amdgcn_readfirstlane(v);
}
// Tiles of `size` rows that experts first .. last take, the same in all lanes.
__device__ __forceinline__ int segment_tiles(const int32_t *offsets, int experts, int rows, int size, int lane)
{
    int n = 0;
    for (int e = lane; e < experts; e += 64) {
        int a, b;
        segment_of(offsets, e, rows, &a, &b);
        n += (b - a + size - 1) / size;
    }
    return wave_total(n);
}
// The expert and the rows of tile number `tile`; whether there is one (there is below
// segment_tiles, unless offsets that do not ascend have made its sum wrap).
__device__ __forceinline__ bool find_segment(const int32_t *offsets, int experts, int rows, int size, int tile,
                                             int lane, int *expert, int *row0, int *row_end)
{
    int before = 0;
    for (int first = 0; first < experts; first += 64) {
        const int e = first + lane;
        int a = 0, b = 0;
        if (e < experts) segment_of(offsets, e, rows, &a, &b);
        const int n = (b - a + size - 1) / size;
        int sum = n;                                     // of this lane and those before it
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int s = __shfl_up(sum, d);
            if (lane >= d) sum += s;
        }
        const uint64_t found = __ballot(before + sum > tile);
        if (found) {
            const int at = __builtin_ctzll(found);
            *expert = first + at;
            *row0 = __builtin_amdgcn_readlane(a, at) +
                    (tile - before - __builtin_amdgcn_readlane(sum - n, at)) * size;
            *row_end = __builtin_amdgcn_readlane(b, at);
            return *row0 < *row_end;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    *expert = *row0 = *row_end = 0;
    return false;
}

}  // namespace fqdev
