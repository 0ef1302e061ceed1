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
// the BF16 copy, 16.1 with 8-bit ones.  With FP32 moments a lane owns 4
// consecutive elements, so that each access of a wave is one contiguous kilobyte
// of an FP32 array, which streaming accesses need (100 M elements: 466 to 476 us,
// 5.9 to 6.0 TB/s; with 8 elements a lane 515, and 532 streaming).  With 8-bit moments it owns 8, so
// that a state block is one 16-lane DPP row and the work for its scale is done
// once for 8 elements; the master weight's two half-used kilobytes go through
// the caches, the rest streams (134 M elements: 378 us; two times 4 elements a
// lane 416, the weight streaming too 396).  One launch takes a whole plan,
// whose table of tensors lies in device memory, or up to kAdamWTensors tensors,
// whose table travels in the kernel's arguments.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_internal.h"
#include "fq_rows.hpp"

using namespace fqdev;

namespace {

template <bool F8>
constexpr int threads_of() { return F8 ? 256 : 1024; }
template <bool F8>
constexpr int tile_of() { return threads_of<F8>() * (F8 ? 8 : 4); }    // elements of a workgroup

// Bits of the largest finite magnitude of eight values.
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

// Elements at .. at + n - 1 of an array (n <= 4, or 8 codes); missing ones
// read as 0 and are not written.  A tail's loads repeat its last element rather
// than branch, so that they are in flight together.
template <bool NT>
__device__ __forceinline__ void get4(const float *p, int64_t at, int n, float (&v)[4])
{
    u32w4 r = {0, 0, 0, 0};
    if (n == 4) {
        r = load16<NT>((const u32w4 *)(p + at));
    } else if (n) {
        float e[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) e[i] = p[at + min(i, n - 1)];
#pragma unroll
        for (int i = 0; i < 3; ++i) r[i] = i < n ? as_u(e[i]) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = as_f(r[i]);
}
template <bool NT>
__device__ __forceinline__ void get4(const uint16_t *p, int64_t at, int n, float (&v)[4])
{
    u32w2 r = {0, 0};
    if (n == 4) {
        r = NT ? __builtin_nontemporal_load((const u32w2 *)(p + at)) : *(const u32w2 *)(p + at);
    } else if (n) {
        uint16_t e[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) e[i] = p[at + min(i, n - 1)];
#pragma unroll
        for (int i = 0; i < 3; ++i) r[i / 2] |= i < n ? (uint32_t)e[i] << (16 * (i % 2)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = as_f(i % 2 ? hi_bits(r[i / 2]) : lo_bits(r[i / 2]));
}
template <bool NT>
__device__ __forceinline__ void put4(float *p, int64_t at, int n, const float (&v)[4])
{
    if (n == 4) {
        store16<NT>((u32w4 *)(p + at), (u32w4){as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3])});
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < n) p[at + i] = v[i];
}
template <bool NT>
__device__ __forceinline__ void put4(uint16_t *p, int64_t at, int n, const float (&v)[4])
{
    const u32w2 w = {bf16_pair_rne(v[0], v[1]), bf16_pair_rne(v[2], v[3])};
    if (n == 4) {
        if (NT) __builtin_nontemporal_store(w, (u32w2 *)(p + at));
        else *(u32w2 *)(p + at) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < n) p[at + i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
}
template <bool NT>
__device__ __forceinline__ u32w2 get_codes(const uint8_t *p, int n)
{
    if (n == 8) return NT ? __builtin_nontemporal_load((const u32w2 *)p) : *(const u32w2 *)p;
    u32w2 c = {0, 0};
    if (n == 0) return c;
    uint8_t e[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) e[i] = p[min(i, n - 1)];
#pragma unroll
    for (int i = 0; i < 7; ++i) c[i / 4] |= i < n ? (uint32_t)e[i] << (8 * (i % 4)) : 0u;
    return c;
}
template <bool NT>
__device__ __forceinline__ void put_codes(uint8_t *p, int n, u32w2 c)
{
    if (n == 8) {
        if (NT) __builtin_nontemporal_store(c, (u32w2 *)p);
        else *(u32w2 *)p = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) p[i] = (uint8_t)(c[i / 4] >> (8 * (i % 4)));
}

// The tensor that tile `tile` belongs to: the last one that starts at or before
// it.  In a plan the wave looks at 64 starts at once, first at those of 64 parts
// of the list; the arguments' short table is bisected in scalar code.
__device__ __forceinline__ uint32_t tensor_of(const uint32_t *__restrict__ first, uint32_t count,
                                              uint32_t tile)
{
    const uint32_t lane = threadIdx.x & 63, part = (count + 63) / 64;
    const auto starts = [&](uint32_t at, uint32_t end) {
        return (uint32_t)__popcll(__ballot(at < end && first[at] <= tile));
    };
    uint32_t n = 0;
    if (part > 1) n = (starts(lane * part, count) - 1) * part;
    for (const uint32_t end = part > 1 ? min(n + part, count) : count; n < end;) {
        const uint32_t m = starts(n + lane, end);
        n += m;
        if (m < 64) break;
    }
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)n) - 1;
}

// One element's moments and weight after another: m and v from the gradient,
// then w from m / (sqrt(v) * c + eps).  Up to v = 2^79 by the hardware's square
// root and reciprocal, each within one unit in the last place, of v * 2^48,
// which lifts subnormal v into the range they take (c2 = c * 2^-24); above, and
// for infinities and NaN, by the correctly rounded operations.  With the latter
// alone calls that the caches hold are slower (8-bit moments, 2^22 elements 15.7
// us instead of 13.8, 2^20 6.1 and 5.5; FP32 2^21 9.1 and 8.6); from 2^25 on
// memory hides them.  They also take every v (divide_from 0) where a positive
// eps is outside 2^-100 .. 2^100: alone, as for v = 0, it may have no normal
// reciprocal, while a positive root is between 2^-75 and 2^67 (c is at most 2^27).
template <int N>
__device__ __forceinline__ void update(const fqimpl::AdamWStep &a, const fqimpl::AdamWTensor &t,
                                       const float (&g)[N], float (&w)[N], float (&m)[N],
                                       float (&v)[N])
{
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const float lr = a.lr * t.lr_mult;
    const float keep = 1.0f - lr * t.weight_decay, step = lr * a.inv_bc1;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float gg = g[e] * gs;
        m[e] = m[e] * a.beta1 + gg * a.one_beta1;
        v[e] = v[e] * a.beta2 + (gg * a.one_beta2) * gg;
    }
    const float c = a.inv_sqrt_bc2, c2 = c * 0x1p-24f;
    if (__any(absmax(v) >= a.divide_from)) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            w[e] = w[e] * keep - (m[e] / (__builtin_sqrtf(v[e]) * c + a.eps)) * step;
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            w[e] = w[e] * keep - (m[e] * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v[e] * 0x1p48f) * c2 + a.eps)) * step;
    }
}

template <bool NT>
__device__ __forceinline__ void tile_f32(const fqimpl::AdamWStep &a, const fqimpl::AdamWTensor &t,
                                         uint32_t tile)
{
    const int64_t i = (int64_t)tile * tile_of<false>() + threadIdx.x * 4;
    const int n = (int)max((int64_t)0, min((int64_t)4, t.n - i));
    const int64_t at = n ? i : 0;
    float w[4], g[4], m[4], v[4];
    get4<NT>(t.w, at, n, w);
    get4<NT>((const float *)t.m, at, n, m);
    get4<NT>((const float *)t.v, at, n, v);
    if (t.g_f32) get4<NT>((const float *)t.g, at, n, g);
    else get4<NT>((const uint16_t *)t.g, at, n, g);
    update(a, t, g, w, m, v);
    put4<NT>(t.w, at, n, w);
    if (t.w_bf16) put4<NT>((uint16_t *)t.w_bf16, at, n, w);
    put4<NT>((float *)t.m, at, n, m);
    put4<NT>((float *)t.v, at, n, v);
}

// Element i's draw is word i mod 4 of Philox counter i / 4 of the tensor at this
// step, low half for m, high half for v.  The converter adds its random operand,
// shifted down to the dropped bits, and truncates: with 0xFFFF - r16 in the top
// 16 bits and zeros below, the kept bits grow exactly when r16 < floor(2^16 *
// fraction).
__device__ __forceinline__ void encode_quad(const float *m, const float *v, u32x4 draws, float mi,
                                            float vi, uint32_t &mc, uint32_t &vc)
{
    const auto ma = [&](int e) { return __builtin_amdgcn_fmed3f(m[e] * mi, -448.0f, 448.0f); };
    const auto mr = [&](int e) { return ~draws.v[e] << 16; };
    // a positive v is at least the smallest code's value, 2^-16
    const auto va = [&](int e) {
        return __builtin_amdgcn_fmed3f(v[e] * vi, v[e] > 0.0f ? 0x1p-16f : 0.0f, 57344.0f);
    };
    const auto vr = [&](int e) { return ~draws.v[e] & 0xFFFF0000u; };
    mc = __builtin_amdgcn_cvt_sr_fp8_f32(ma(0), mr(0), 0, 0);
    mc = __builtin_amdgcn_cvt_sr_fp8_f32(ma(1), mr(1), mc, 1);
    mc = __builtin_amdgcn_cvt_sr_fp8_f32(ma(2), mr(2), mc, 2);
    mc = __builtin_amdgcn_cvt_sr_fp8_f32(ma(3), mr(3), mc, 3);
    vc = __builtin_amdgcn_cvt_sr_bf8_f32(va(0), vr(0), 0, 0);
    vc = __builtin_amdgcn_cvt_sr_bf8_f32(va(1), vr(1), vc, 1);
    vc = __builtin_amdgcn_cvt_sr_bf8_f32(va(2), vr(2), vc, 2);
    vc = __builtin_amdgcn_cvt_sr_bf8_f32(va(3), vr(3), vc, 3);
}

template <bool NT>
__device__ __forceinline__ void tile_f8(const fqimpl::AdamWStep &a, const fqimpl::AdamWTensor &t,
                                        uint32_t tile, uint32_t number)
{
    // lanes past the end stay for their block's maximum, with zeros
    const int64_t i = (int64_t)tile * tile_of<true>() + threadIdx.x * 8;
    const int n = (int)max((int64_t)0, min((int64_t)8, t.n - i));
    const int64_t at = n ? i : 0;
    float w[8], g[8], m[8], v[8];
    if (n == 8) load8<false>(t.w + at, 8, w);
    else load8<true>(t.w + at, n, w);
    u32w2 mc = get_codes<NT>((const uint8_t *)t.m + at, n);
    u32w2 vc = get_codes<NT>((const uint8_t *)t.v + at, n);
    float ms = t.m_scale[at >> 7], vs = t.v_scale[at >> 7];
    if (t.g_f32) {
        if (n == 8) load8<false>((const float *)t.g + at, 8, g);
        else load8<true>((const float *)t.g + at, n, g);
    } else {
        if (n == 8) load8<false, NT>((const uint16_t *)t.g + at, 8, g);
        else load8<true>((const uint16_t *)t.g + at, n, g);
    }
    e4m3_decode8(mc, m);
    e5m2_decode8(vc, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m[e] = m[e] * ms;
        v[e] = v[e] * vs;
    }
    update(a, t, g, w, m, v);
    if (n == 8) store8<false>(t.w + at, 8, w);
    else store8<true>(t.w + at, n, w);
    if (t.w_bf16) {
        if (n == 8) store8<false, NT>((uint16_t *)t.w_bf16 + at, 8, w);
        else store8<true>((uint16_t *)t.w_bf16 + at, n, w);
    }
    uint32_t mt = absmax(m), vt = absmax(v);
    const bool finite = max(mt, vt) < 0x7F800000u;
    if (!finite) {
        mt = finite_max8(m);
        vt = finite_max8(v);
    }
    ms = state_scale(lanes_max<16>(mt), 1.0f / 448.0f);
    vs = state_scale(lanes_max<16>(vt), 1.0f / 57344.0f);
    const float mi = 1.0f / ms, vi = 1.0f / vs;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t c = ((uint64_t)at >> 2) + h;
        const u32x4 draws = philox4x32_10((uint32_t)c, (uint32_t)(c >> 32), number, a.step,
                                          a.seed_lo, a.seed_hi);
        uint32_t mq, vq;
        encode_quad(m + 4 * h, v + 4 * h, draws, mi, vi, mq, vq);
        mc[h] = mq;
        vc[h] = vq;
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
    if (n == 0) return;
    put_codes<NT>((uint8_t *)t.m + at, n, mc);
    put_codes<NT>((uint8_t *)t.v + at, n, vc);
    if ((threadIdx.x & 15) == 0) {
        t.m_scale[at >> 7] = ms;
        t.v_scale[at >> 7] = vs;
    }
}

template <bool F8, bool NT>
__device__ __forceinline__ void adamw_tile(const fqimpl::AdamWStep &a, const fqimpl::AdamWTensor &t,
                                           uint32_t tile, uint32_t number)
{
    if (F8) tile_f8<NT>(a, t, tile, number);
    else tile_f32<NT>(a, t, tile);
}

template <bool F8, bool NT>
__global__ __launch_bounds__(threads_of<F8>()) void k_adamw(fqimpl::AdamWArgs a)
{
    for (uint32_t tile = blockIdx.x; tile < a.step.tiles; tile += gridDim.x) {
        uint32_t lo = 0, hi = a.step.count;
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) / 2;
            if (a.first[mid] <= tile) lo = mid;
            else hi = mid;
        }
        adamw_tile<F8, NT>(a.step, a.t[lo], tile - a.first[lo], a.index[lo]);
    }
}

template <bool F8, bool NT>
__global__ __launch_bounds__(threads_of<F8>()) void k_adamw_plan(
    fqimpl::AdamWStep a, const fqimpl::AdamWTensor *__restrict__ t,
    const uint32_t *__restrict__ first, const uint32_t *__restrict__ index)
{
    for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const uint32_t k = tensor_of(first, a.count, tile);
        adamw_tile<F8, NT>(a, t[k], tile - first[k], index[k]);
    }
}

// Streaming accesses from this many elements on.  2^24 elements: FP32 moments 79
// us streaming, 90 not, 8-bit ones 45.5 and 54.1; 2^23: 40.5, 45.9 and 26.5, 24.8;
// 2^22: 21.0, 19.9 and 16.3, 14.7.  One limit for both kinds: it is the 8-bit
// moments', FP32 ones cross near 2^22.5 and lose up to 5 us below the limit.
constexpr int64_t kStreamElems = int64_t(1) << 24;
// A grid holds fewer than 2^32 lanes; the kernels walk over what is left, and a
// tile's number with the grid added stays below 2^32.  A list of kAdamWTensors
// has few enough tiles by itself.
constexpr uint32_t kMaxGrid = 1u << 20;
static_assert(fqimpl::kAdamWMaxTiles + kMaxGrid <= UINT32_MAX, "a walk's tile numbers");
static_assert(fqimpl::kAdamWTensors * ((uint64_t(1) << 34) / tile_of<true>()) <= fqimpl::kAdamWMaxTiles,
              "tiles of a list");

bool streams(uint32_t tiles, bool f8)
{
    return tiles >= kStreamElems / (f8 ? tile_of<true>() : tile_of<false>());
}

}  // namespace

namespace fqimpl {

uint32_t adamw_tile(bool f8) { return f8 ? tile_of<true>() : tile_of<false>(); }
uint32_t adamw_tiles(int64_t n, bool f8)
{
    const int64_t tile = adamw_tile(f8);
    return (uint32_t)((n + tile - 1) / tile);
}

hipError_t launch_adamw(const AdamWArgs &a, bool f8, hipStream_t stream)
{
    const dim3 grid(a.step.tiles < kMaxGrid ? a.step.tiles : kMaxGrid);
    const dim3 block(f8 ? threads_of<true>() : threads_of<false>());
    const bool nt = streams(a.step.tiles, f8);
    if (f8 && nt) k_adamw<true, true><<<grid, block, 0, stream>>>(a);
    else if (f8) k_adamw<true, false><<<grid, block, 0, stream>>>(a);
    else if (nt) k_adamw<false, true><<<grid, block, 0, stream>>>(a);
    else k_adamw<false, false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_adamw_plan(const AdamWStep &a, const AdamWTensor *t, const uint32_t *first,
                             const uint32_t *index, bool f8, hipStream_t stream)
{
    const dim3 grid(a.tiles < kMaxGrid ? a.tiles : kMaxGrid);
    const dim3 block(f8 ? threads_of<true>() : threads_of<false>());
    const bool nt = streams(a.tiles, f8);
    if (f8 && nt) k_adamw_plan<true, true><<<grid, block, 0, stream>>>(a, t, first, index);
    else if (f8) k_adamw_plan<true, false><<<grid, block, 0, stream>>>(a, t, first, index);
    else if (nt) k_adamw_plan<false, true><<<grid, block, 0, stream>>>(a, t, first, index);
    else k_adamw_plan<false, false><<<grid, block, 0, stream>>>(a, t, first, index);
    return hipGetLastError();
}

}  // namespace fqimpl
