// fq_rows.hpp -- device-side building blocks of the row operators around the
// quantized linears (norm, expert sorting, optimizer): eight-element chunks
// of BF16 or FP32 rows at any alignment, sums and maxima across a wave, and
// the 8-bit float encodings.
//
// 8-bit formats (OCP OFP8 v1.0): E4M3 (4 exponent bits, bias 7, largest 448,
// NaN 0x7F) and E5M2 (5 exponent bits, bias 15, largest 57344, NaN 0x7F used
// here).  gfx950's converters decode both exactly.
#pragma once

#include "fq_device.hpp"

namespace fqdev {

typedef uint32_t u32w4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32w2 __attribute__((ext_vector_type(2)));
typedef u32w4 u32w4_any __attribute__((aligned(2)));   // unaligned global access
typedef u32w4 u32w4_any4 __attribute__((aligned(4)));

// ---- eight consecutive elements of a row ------------------------------------
// `n` of them exist (8, or fewer in the last chunk of a row whose length is
// no multiple of 8); missing ones read as 0 and are not written.  ANY: the
// row may start at any element; gfx950 serves the 16-byte access at element
// alignment, so only the last chunk goes element by element.  NT: streaming
// accesses, for calls whose data is larger than the caches; not for FP32, whose
// two accesses use half of each line and have to meet in the cache.
template <bool NT, typename V>
__device__ __forceinline__ u32w4 load16(const V *p)
{
    if (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32w4 *>(p));
    return *p;
}
template <bool NT, typename V>
__device__ __forceinline__ void store16(V *p, u32w4 v)
{
    if (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32w4 *>(p));
    else *p = v;
}

// as loaded: 4 registers of BF16 pairs, or 8 of FP32
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { u32w4 w; };
template <> struct Raw8<float> { u32w4 a, b; };

template <bool ANY, bool NT = false>
__device__ __forceinline__ void load_raw8(const uint16_t *__restrict__ p, int n, Raw8<uint16_t> &r)
{
    if (!ANY) {
        r.w = load16<NT>(reinterpret_cast<const u32w4 *>(p));
    } else if (n >= 8) {
        r.w = *reinterpret_cast<const u32w4_any *>(p);
    } else {
        r.w = (u32w4){0, 0, 0, 0};
        if (n <= 0) return;
        uint16_t v[7];
#pragma unroll
        for (int i = 0; i < 7; ++i) v[i] = p[min(i, n - 1)];     // in flight together
#pragma unroll
        for (int i = 0; i < 7; ++i) r.w[i / 2] |= i < n ? (uint32_t)v[i] << (16 * (i & 1)) : 0u;
    }
}
template <bool ANY, bool NT = false>
__device__ __forceinline__ void load_raw8(const float *__restrict__ p, int n, Raw8<float> &r)
{
    if (!ANY) {
        r.a = reinterpret_cast<const u32w4 *>(p)[0];
        r.b = reinterpret_cast<const u32w4 *>(p)[1];
    } else if (n >= 8) {
        r.a = reinterpret_cast<const u32w4_any4 *>(p)[0];
        r.b = reinterpret_cast<const u32w4_any4 *>(p)[1];
    } else {
        r.a = r.b = (u32w4){0, 0, 0, 0};
        if (n <= 0) return;
        float v[7];
#pragma unroll
        for (int i = 0; i < 7; ++i) v[i] = p[min(i, n - 1)];     // in flight together
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.a[i] = i < n ? as_u(v[i]) : 0u;
            if (i < 3) r.b[i] = i + 4 < n ? as_u(v[i + 4]) : 0u;
        }
    }
}
__device__ __forceinline__ void unpack8(const Raw8<uint16_t> &r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = as_f(lo_bits(r.w[i]));
        v[2 * i + 1] = as_f(hi_bits(r.w[i]));
    }
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = as_f(r.a[i]);
        v[4 + i] = as_f(r.b[i]);
    }
}
__device__ __forceinline__ float load1(const uint16_t *p) { return as_f((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = (uint16_t)bf16_pair_rne(v, v); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

template <bool ANY, bool NT = false, typename T>
__device__ __forceinline__ void load8(const T *__restrict__ p, int n, float (&v)[8])
{
    Raw8<T> r;
    load_raw8<ANY, NT>(p, n, r);
    unpack8(r, v);
}
// BF16: each value rounded once, to nearest even.
template <bool ANY, bool NT = false>
__device__ __forceinline__ void store8(uint16_t *__restrict__ p, int n, const float (&v)[8])
{
    u32w4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_pair_rne(v[2 * i], v[2 * i + 1]);
    if (!ANY) {
        store16<NT>(reinterpret_cast<u32w4 *>(p), w);
    } else if (n >= 8) {
        *reinterpret_cast<u32w4_any *>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    }
}
template <bool ANY, bool NT = false>
__device__ __forceinline__ void store8(float *__restrict__ p, int n, const float (&v)[8])
{
    const u32w4 a = {as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3])};
    const u32w4 b = {as_u(v[4]), as_u(v[5]), as_u(v[6]), as_u(v[7])};
    if (!ANY) {
        reinterpret_cast<u32w4 *>(p)[0] = a;
        reinterpret_cast<u32w4 *>(p)[1] = b;
    } else if (n >= 8) {
        reinterpret_cast<u32w4_any4 *>(p)[0] = a;
        reinterpret_cast<u32w4_any4 *>(p)[1] = b;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}

// ---- across the wave ----------------------------------------------------------
// DPP inside a 16-lane row (quad permutes, then the row's halves and the row
// mirrored, each pairing lanes that hold equal partial results), and swaps of
// rows with a copy of the same value across the four rows: the two results hold
// one row's value and its neighbour's in both rows' lanes.  Every lane of a
// group gets the same value.
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int ROWS, typename F>
__device__ __forceinline__ uint32_t across_rows(uint32_t v, F join)
{
    const auto r = ROWS == 1 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                             : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return join(r[0], r[1]);
}
__device__ __forceinline__ uint32_t add_f32(uint32_t a, uint32_t b) { return as_u(as_f(a) + as_f(b)); }
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return max(a, b); }

// Sum over groups of LANES neighbouring lanes.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
    v += dpp_f<0xB1>(v);
    v += dpp_f<0x4E>(v);
    v += dpp_f<0x141>(v);
    if (LANES >= 16) v += dpp_f<0x140>(v);
    if (LANES >= 32) v = as_f(across_rows<1>(as_u(v), add_f32));
    if (LANES >= 64) v = as_f(across_rows<2>(as_u(v), add_f32));
    return v;
}
// Maximum over groups of LANES neighbouring lanes (values >= 0, or their bits).
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    v = dpp_max_8lanes(v);
    if (LANES >= 16) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
    if (LANES >= 32) v = across_rows<1>(v, max_u32);
    if (LANES >= 64) v = across_rows<2>(v, max_u32);
    return v;
}

// bits of the largest magnitude of N values; a NaN's bits exceed infinity's,
// which exceed every finite value's
template <int N>
__device__ __forceinline__ uint32_t absmax(const float (&v)[N])
{
    uint32_t m = as_u(v[0]) & 0x7FFFFFFFu;
#pragma unroll
    for (int i = 1; i < N; ++i) m = max(m, as_u(v[i]) & 0x7FFFFFFFu);
    return m;
}

// ---- E4M3 with a scale ---------------------------------------------------------
// E8M0 code of the smallest power of two 2^e with amax <= 448 * 2^e = 1.75 *
// 2^(e + 8) (amax as FP32 bits, finite): one more than the exponent's own
// where the significand exceeds 1.75.  Codes 0 .. 247.
__device__ __forceinline__ uint32_t mx8_scale_code(uint32_t amax_bits)
{
    const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(e, 0);
}
// eight values (|v| <= 448) -> eight E4M3 codes, nearest even
__device__ __forceinline__ u32w2 e4m3_encode8(const float (&v)[8])
{
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
    return (u32w2){(uint32_t)a, (uint32_t)b};
}
__device__ __forceinline__ void e4m3_decode8(u32w2 c, float (&v)[8])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], true);
        v[4 * h] = lo[0];
        v[4 * h + 1] = lo[1];
        v[4 * h + 2] = hi[0];
        v[4 * h + 3] = hi[1];
    }
}
__device__ __forceinline__ void e5m2_decode8(u32w2 c, float (&v)[8])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)c[h], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)c[h], true);
        v[4 * h] = lo[0];
        v[4 * h + 1] = lo[1];
        v[4 * h + 2] = hi[0];
        v[4 * h + 3] = hi[1];
    }
}

}  // namespace fqdev
