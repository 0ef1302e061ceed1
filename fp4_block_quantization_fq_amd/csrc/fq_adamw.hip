// fq_adamw.hip -- one AdamW step over many tensors on gfx950, with the moments
// in FP32 or in 8-bit floats.
//
//   g' = g * grad_scale;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   w = w (1 - lr wd) - (lr / (1 - b1^t)) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//   w_bf16 = BF16_RNE(w)
//
// 8-bit moments: blocks of 128 elements of a tensor, an FP32 scale each, m in
// E4M3 and v in E5M2 (v is a square: 32 octaves of it are 16 octaves of |g|),
// both rounded stochastically from Philox draws.  Rounding to nearest would
// lose every change smaller than half a step: with b2 = 0.999 v moves by at
// most 0.1 % a step while half a step of an 8-bit float is 3 to 12 %.  A
// positive v never becomes 0, which would leave m over eps as the update.
//
// Bound by memory: 28 bytes an element with FP32 moments, BF16 gradients and
// the BF16 copy, 16.1 with 8-bit ones.  One launch takes up to kAdamWTensors
// tensors: their table travels in the kernel's arguments, and a workgroup
// finds its tensor by bisecting the first-workgroup numbers in scalar code.
// A lane owns 8 consecutive elements (16-byte accesses for every 4-byte and
// 2-byte array), so a state block is one 16-lane DPP row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_internal.h"
#include "fq_rows.hpp"

using namespace fqdev;

namespace {

constexpr int kThreads = 256;
constexpr int kTile = kThreads * 8;         // elements of a workgroup

// bits of the largest finite magnitude of eight values
__device__ __forceinline__ uint32_t finite_max8(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = as_u(v[i]) & 0x7FFFFFFFu;
        m = max(m, u < 0x7F800000u ? u : 0u);
    }
    return m;
}

// scale of a state block from the bits of its largest magnitude
__device__ __forceinline__ float state_scale(uint32_t top, float per_largest)
{
    return __builtin_fmaxf(as_f(top) * per_largest, 0x1p-126f);
}

__device__ __forceinline__ u32w2 load_codes(const uint8_t *__restrict__ p, int n)
{
    if (n == 8) return *(const u32w2 *)p;
    u32w2 c = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) c[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    return c;
}
__device__ __forceinline__ void store_codes(uint8_t *__restrict__ p, int n, u32w2 c)
{
    if (n == 8) {
        *(u32w2 *)p = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint8_t)(c[i / 4] >> (8 * (i % 4)));
}

template <bool F8>
__global__ __launch_bounds__(kThreads) void k_adamw(fqimpl::AdamWArgs a)
{
    // the tensor of this workgroup: the last one that starts at or before it
    uint32_t lo = 0, hi = a.count;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (a.first[mid] <= blockIdx.x) lo = mid;
        else hi = mid;
    }
    const fqimpl::AdamWTensor &t = a.t[lo];
    const int64_t i = (int64_t)(blockIdx.x - a.first[lo]) * kTile + threadIdx.x * 8;
    const int n = (int)min((int64_t)8, t.n - i);
    // lanes past the end stay for their block's maximum
    float w[8], g[8], m[8], v[8];
    const int64_t at = n > 0 ? i : 0;
    const int nn = max(n, 0);
    const bool whole = n == 8;
    if (whole) load8<false>(t.w + at, 8, w);
    else load8<true>(t.w + at, nn, w);
    if (t.g_f32) {
        if (whole) load8<false>((const float *)t.g + at, 8, g);
        else load8<true>((const float *)t.g + at, nn, g);
    } else {
        if (whole) load8<false>((const uint16_t *)t.g + at, 8, g);
        else load8<true>((const uint16_t *)t.g + at, nn, g);
    }
    if (F8) {
        const float ms = t.m_scale[at >> 7], vs = t.v_scale[at >> 7];
        e4m3_decode8(load_codes((const uint8_t *)t.m + at, nn), m);
        e5m2_decode8(load_codes((const uint8_t *)t.v + at, nn), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            m[e] = m[e] * ms;
            v[e] = v[e] * vs;
        }
    } else if (whole) {
        load8<false>((const float *)t.m + at, 8, m);
        load8<false>((const float *)t.v + at, 8, v);
    } else {
        load8<true>((const float *)t.m + at, nn, m);
        load8<true>((const float *)t.v + at, nn, v);
    }
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const float lr = a.lr * t.lr_mult;
    const float keep = 1.0f - lr * t.weight_decay, step = lr * a.inv_bc1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float gg = g[e] * gs;
        m[e] = m[e] * a.beta1 + gg * a.one_beta1;
        v[e] = v[e] * a.beta2 + (gg * a.one_beta2) * gg;
        w[e] = w[e] * keep - (m[e] / (__builtin_sqrtf(v[e]) * a.inv_sqrt_bc2 + a.eps)) * step;
    }
    if (whole) store8<false>(t.w + at, 8, w);
    else store8<true>(t.w + at, nn, w);
    if (t.w_bf16) {
        if (whole) store8<false>((uint16_t *)t.w_bf16 + at, 8, w);
        else store8<true>((uint16_t *)t.w_bf16 + at, nn, w);
    }
    if (!F8) {
        if (whole) {
            store8<false>((float *)t.m + at, 8, m);
            store8<false>((float *)t.v + at, 8, v);
        } else {
            store8<true>((float *)t.m + at, nn, m);
            store8<true>((float *)t.v + at, nn, v);
        }
        return;
    }
    // draws of elements i .. i + 7: Philox counters i / 4 and i / 4 + 1 of the
    // tensor at this step; word n mod 4, low half for m, high half for v
    uint32_t r[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t q = (uint64_t)(at >> 2) + h;
        const u32x4 o = philox4x32_10((uint32_t)q, (uint32_t)(q >> 32), a.index[lo], a.step,
                                      a.seed_lo, a.seed_hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) r[4 * h + e] = ~o.v[e];
    }
    // lanes past the end hold zeros
    uint32_t mt = absmax8(m), vt = absmax8(v);
    const bool finite = max(mt, vt) < 0x7F800000u;
    if (!finite) {
        mt = finite_max8(m);
        vt = finite_max8(v);
    }
    const float ms = state_scale(dpp_max_16lanes(mt), 1.0f / 448.0f);
    const float vs = state_scale(dpp_max_16lanes(vt), 1.0f / 57344.0f);
    const float mi = 1.0f / ms, vi = 1.0f / vs;
    // The converter adds its random operand, shifted down to the dropped bits,
    // and truncates: with 0xFFFF - r16 in the top 16 bits and zeros below, the
    // kept bits grow exactly when r16 < floor(2^16 * fraction).
    uint32_t mc[2] = {0, 0}, vc[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = 4 * h;
        const auto ma = [&](int k) { return __builtin_amdgcn_fmed3f(m[e + k] * mi, -448.0f, 448.0f); };
        // a positive v is at least the smallest code's value, 2^-16
        const auto va = [&](int k) {
            return __builtin_amdgcn_fmed3f(v[e + k] * vi, v[e + k] > 0.0f ? 0x1p-16f : 0.0f, 57344.0f);
        };
        mc[h] = __builtin_amdgcn_cvt_sr_fp8_f32(ma(0), r[e] << 16, mc[h], 0);
        mc[h] = __builtin_amdgcn_cvt_sr_fp8_f32(ma(1), r[e + 1] << 16, mc[h], 1);
        mc[h] = __builtin_amdgcn_cvt_sr_fp8_f32(ma(2), r[e + 2] << 16, mc[h], 2);
        mc[h] = __builtin_amdgcn_cvt_sr_fp8_f32(ma(3), r[e + 3] << 16, mc[h], 3);
        vc[h] = __builtin_amdgcn_cvt_sr_bf8_f32(va(0), r[e] & 0xFFFF0000u, vc[h], 0);
        vc[h] = __builtin_amdgcn_cvt_sr_bf8_f32(va(1), r[e + 1] & 0xFFFF0000u, vc[h], 1);
        vc[h] = __builtin_amdgcn_cvt_sr_bf8_f32(va(2), r[e + 2] & 0xFFFF0000u, vc[h], 2);
        vc[h] = __builtin_amdgcn_cvt_sr_bf8_f32(va(3), r[e + 3] & 0xFFFF0000u, vc[h], 3);
    }
    if (!finite) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int shift = 8 * (e % 4);
            const uint32_t mu = as_u(m[e]);
            if ((mu & 0x7FFFFFFFu) >= 0x7F800000u)
                mc[e / 4] = (mc[e / 4] & ~(0xFFu << shift)) | ((0x7Fu | (mu >> 31) << 7) << shift);
            if ((as_u(v[e]) & 0x7FFFFFFFu) >= 0x7F800000u)
                vc[e / 4] = (vc[e / 4] & ~(0xFFu << shift)) | (0x7Fu << shift);
        }
    }
    if (n <= 0) return;
    store_codes((uint8_t *)t.m + at, nn, (u32w2){mc[0], mc[1]});
    store_codes((uint8_t *)t.v + at, nn, (u32w2){vc[0], vc[1]});
    if ((threadIdx.x & 15) == 0) {
        t.m_scale[at >> 7] = ms;
        t.v_scale[at >> 7] = vs;
    }
}

}  // namespace

namespace fqimpl {

uint32_t adamw_workgroups(int64_t n) { return (uint32_t)((n + kTile - 1) / kTile); }

hipError_t launch_adamw(const AdamWArgs &a, bool f8, uint32_t grid, hipStream_t stream)
{
    if (f8) k_adamw<true><<<dim3(grid), dim3(kThreads), 0, stream>>>(a);
    else k_adamw<false><<<dim3(grid), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace fqimpl
