// fq_product.hpp -- the tile kernel of the feed-forward products, on BF16 matrix
// cores: y = a(x w + b) + res, the gated h = a(x wg + bg) (x wu + bu), and the two
// products of their backward, dx = dz w^T and dw = x^T dz.  One product, or one
// per expert over the segments of rows that fq_moe_sort made.
//
// A product is C[M, N] = sum over k of A(m, k) B(k, n), FP32 sums on
// v_mfma_f32_32x32x16_bf16.  Weights lie [K, N] and activations [rows, K], so
// an operand is either contiguous along the contraction (x in the forward, dz
// and w in dx) or across it (w in the forward, x and dz in dw).  Both go from
// global memory straight to LDS as they lie, 16 bytes a lane; the second kind
// is transposed on the way into registers by gfx950's ds_read_b64_tr_b16: in a
// group of 16 lanes, lane s reads four columns of row s / 4 and receives the
// four rows of column s.  Those reads run at 124 B a clock and CU, ds_read_b128
// at 240 (measured), which is enough for either (below).
//
// LDS tiles: contraction-contiguous, a 128-byte row (64 k) per tile row, 16-byte
// chunks XORed with (row & 7) ^ (row >> 3 & 1); otherwise a row per k of all the
// tile's columns, its 64-byte units moved by the row's number so that the four
// rows that a transposing read touches lie in different banks (no conflicts,
// measured).
//
// Schedule: two stages of 64 k (more where a workgroup is alone on its CU).  A substep of 16 k has its fragments in registers
// when it begins and reads the next one's between its products.  The stage's one
// barrier lies in front of its last substep, whose fragments are in registers by
// then: the other stage has landed, this one is free, and the loads that refill it
// go out between the products of the next two substeps.  What that took:
//  - The direct loads are written as assembly (they have no result register) and
//    waited for by hand.  The compiler cannot tell which LDS bytes a load in flight
//    writes from those that a transposing read asks for: it waited for all loads
//    behind the barrier, a memory latency a stage (1.77 us a stage of 256 x 256,
//    with these loads 1.46).
//  - Order is pinned product by product.  Loads issued together at the barrier keep
//    the waves from issuing products while the address unit works through them.
// At 1.46 us a stage the chip runs at 1.8 GHz of its 2.4: power is what is left
// (products alone, fragments in registers, 1.16 us at 1.8 GHz; with the LDS reads
// 1.31).
//
// Past the end of the contraction both operands are read as zeros (from an
// array of zeros, chosen by address), so neither infinities nor NaN of other
// rows reach a sum.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_act.hpp"
#include "fq_internal.h"

namespace {

using namespace fqdev;
using fqimpl::ProductArgs;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

enum { ALONG = 0, ACROSS = 1 };                  // operand against the contraction
// what becomes of the sums: stored; bias and residual added; all of the linear's
// epilogue; the gated block's
enum { EPI_STORE = 0, EPI_RES = 1, EPI_LINEAR = 2, EPI_GLU = 3 };

constexpr int BK = 64;
constexpr int kXcds = 8;

__device__ const u32w4 kZeros = {0, 0, 0, 0};

// 16 bytes a lane from base + off (or src) to LDS at `lds` (uniform) + 16 * lane.
// The instruction takes its LDS address from m0.
__device__ __forceinline__ void direct_load(const uint8_t *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 : : "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds)) : "m0");
}
__device__ __forceinline__ void direct_load(const uint8_t *src, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 : : "v"(src), "s"(__builtin_amdgcn_readfirstlane(lds)) : "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void *p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

__device__ __forceinline__ int swz(int row, int chunk)
{
    return chunk ^ (row & 7) ^ ((row >> 3) & 1);
}

// ---- operand tiles ---------------------------------------------------------------
// 64 k of ROWS rows (ALONG) or columns (ACROSS): ROWS * 128 bytes, 1 KB a wave
// instruction.  Lane offsets are fixed; the base moves on by a step of 64 k.
template <int L, int ROWS, int WAVES>
struct Tile {
    static constexpr int NI = ROWS / 8 / WAVES;            // instructions a wave
    static constexpr int CHUNKS = ROWS / 8;                // of 16 bytes of a k's row (ACROSS)
    static constexpr int UNITS = ROWS / 32;                // and of 64 bytes
    static_assert(NI * WAVES * 8 == ROWS && ROWS % 64 == 0, "whole instructions");
    const uint8_t *base;
    uint32_t off[NI];
    int64_t step;

    // Where unit `unit` of k's row lies.  A row is a multiple of the banks' 256
    // bytes, or (192 columns) one and a half of it: then rows k and k + 2 would meet.
    static __device__ __forceinline__ int place(int k, int unit)
    {
        if (UNITS % 4 == 0) return unit ^ (k & 3);
        unit += (k >> 1) & 1;
        return unit >= UNITS ? unit - UNITS : unit;
    }
    static __device__ __forceinline__ int unit_at(int k, int place)
    {
        if (UNITS % 4 == 0) return place ^ (k & 3);
        place -= (k >> 1) & 1;
        return place < 0 ? place + UNITS : place;
    }

    // `first` of `count` rows or columns; pitch in elements.  SPLIT: the columns
    // are 32 of the first half, 32 of the second half (`half` columns on), ...
    template <bool SPLIT>
    __device__ __forceinline__ void init(const uint16_t *p, int64_t pitch, int first, int count,
                                         int half, int wave, int lane)
    {
        if (L == ALONG) {
            base = (const uint8_t *)(p + (int64_t)first * pitch);
            step = BK * 2;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int r = (wave * NI + i) * 8 + (lane >> 3);
                const int row = min(r, count - first - 1);          // never stored
                off[i] = (uint32_t)row * (uint32_t)(pitch * 2) + swz(r, lane & 7) * 16;
            }
        } else {
            base = (const uint8_t *)p;
            step = BK * 2 * pitch;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int id = (wave * NI + i) * 64 + lane, k = id / CHUNKS, slot = id % CHUNKS;
                const int t = unit_at(k, slot >> 2) * 32 + (slot & 3) * 8;
                int col = first + t, more = 0;
                if (SPLIT) {
                    col = first + (t >> 6) * 32 + (t & 31);
                    more = (t & 32) ? half : 0;
                }
                if (col >= count) col = first;                      // never stored
                off[i] = (uint32_t)k * (uint32_t)(pitch * 2) + (uint32_t)(col + more) * 2;
            }
        }
    }
    // k of instruction i's chunk within the step
    __device__ __forceinline__ int k_of(int i, int wave, int lane) const
    {
        if (L == ALONG) return swz((wave * NI + i) * 8 + (lane >> 3), lane & 7) * 8;
        return ((wave * NI + i) * 64 + lane) / CHUNKS;
    }
    // Instruction i of a step; `left` k of it exist (64 or more: all).
    __device__ __forceinline__ void issue(uint32_t lds, int i) const
    {
        direct_load(base, off[i], lds + i * 1024);
    }
    __device__ __forceinline__ void issue(uint32_t lds, int i, int left, int wave, int lane) const
    {
        if (left >= BK) return issue(lds, i);
        direct_load(k_of(i, wave, lane) < left ? base + off[i] : (const uint8_t *)&kZeros, lds + i * 1024);
    }
    // eight k of row (column) 32 * t + lane % 32 for substep ks of 16 k
    static __device__ __forceinline__ bf16x8 read(const uint8_t *lds, int t, int ks, int lane)
    {
        if (L == ALONG) {
            const int r = t * 32 + (lane & 31);
            return *reinterpret_cast<const bf16x8 *>(lds + r * 128 + swz(r, ks * 2 + (lane >> 5)) * 16);
        }
        const int k = ks * 16 + (lane >> 5) * 8 + ((lane & 15) >> 2);
        const uint8_t *p = lds + k * (ROWS * 2) + place((lane & 15) >> 2, t) * 64 + (lane & 16) * 2 + (lane & 3) * 8;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * ROWS * 2));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// ---- epilogues ---------------------------------------------------------------------
__device__ __forceinline__ void load_bias(const ProductArgs &p, int64_t at, float (&b)[8])
{
    if (!p.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = 0.0f;
    } else if (p.bias_f32) {
        load8<false>((const float *)p.bias + at, 8, b);
    } else {
        load8<false>((const uint16_t *)p.bias + at, 8, b);
    }
}

// Eight values before the activation, kept for the backward: rounded to BF16, or
// to E4M3 under a power of two per 32 columns, which four neighbouring lanes hold
// (from FP32: a rounding to BF16 before would move a block's maximum across a
// border of its scale now and then).
__device__ __forceinline__ void keep_pre(const ProductArgs &p, int64_t at, const float (&z)[8])
{
    if (p.pre_kind == fqimpl::PRE_BF16) {
        store8<false>((uint16_t *)p.pre + at, 8, z);
        return;
    }
    u32w2 codes;
    const uint32_t scale = mx8_encode8(z, &codes);
    *(u32w2 *)((uint8_t *)p.pre + at) = codes;
    if ((at & 31) == 0) ((uint8_t *)p.pre_scales)[at >> 5] = (uint8_t)scale;
}

__device__ __forceinline__ void load_res(const ProductArgs &p, int64_t at, float (&r)[8])
{
    if (p.y_f32) load8<false>((const float *)p.res + at, 8, r);
    else load8<false>((const uint16_t *)p.res + at, 8, r);
}
// STREAM: past the L2s where the output would fill them (4 MB each), whose lines the
// operands' tiles need (8192 x 5760 -> 2880 222 -> 211 us, dw 2880 x 5760 264 -> 247, of
// 32 experts 402 -> 325; a gated block's h and codes gain nothing).  Smaller ones gain little
// (1024 x 2880 -> 1440 18.0 and 17.7) and are left to the next kernel.  FP32 outputs are not
// streamed: 8192 x 2880 -> 2880 with its residual 174 plain, 181 streamed, 4096 rows 93 and
// 90, dw of 2880 x 2880 152 and 151, of 32 experts 270 and 269.
template <bool STREAM = false>
__device__ __forceinline__ void store_y(const ProductArgs &p, int64_t at, const float (&v)[8])
{
    if (p.y_f32) store8<false>((float *)p.y + at, 8, v);
    else store8<false, STREAM>((uint16_t *)p.y + at, 8, v);
}

// What becomes of eight sums (column `col` of row `row`, of N columns) and the
// residual's values.
__device__ __forceinline__ void finish_linear(const ProductArgs &p, int64_t row, int col, int N,
                                              float (&z)[8], const float (&bias)[8], const float (&res)[8])
{
    const int64_t at = row * N + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += bias[i];
    if (p.pre_kind) keep_pre(p, at, z);
    act_n(p.act, 1.0f, z);
    if (p.res) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += res[i];
    }
    store_y(p, at, z);
}
// and of eight pairs of the gated block
__device__ __forceinline__ void finish_glu(const ProductArgs &p, int64_t row, int col, int n,
                                           float (&g)[8], float (&u)[8], const float (&bg)[8],
                                           const float (&bu)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        g[i] += bg[i];
        u[i] += bu[i];
    }
    if (p.pre_kind) {
        keep_pre(p, row * 2 * n + col, g);
        keep_pre(p, row * 2 * n + n + col, u);
    }
    glu_n(p.gate, g, u);
    store8<false>((uint16_t *)p.y + row * n + col, 8, g);
}

// ---- the kernel ----------------------------------------------------------------------
// WM x WN waves of TM x TN accumulator tiles of 32 x 32, STAGES buffers of 64 k.
// SEGK: the experts' segments are of the contraction (dw), else of C's rows.
template <int LA, int LB, int TM, int TN, int WM, int WN, int STAGES, int EPI, bool SEGK>
__device__ __forceinline__ void product_tile(const ProductArgs &p, uint8_t *lds, const int block)
{
    constexpr int BM = WM * TM * 32, BN = WN * TN * 32, WAVES = WM * WN;
    constexpr int BNC = EPI == EPI_GLU ? BN / 2 : BN;      // columns of the output
    constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 128;
    static_assert(EPI != EPI_GLU || TN % 2 == 0, "32 columns of either half next to each other");

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int wm = wave / WN, wn = wave % WN;

    // this workgroup's tile
    const int tiles_n = (p.N + BNC - 1) / BNC;
    int tiles_m = (p.M + BM - 1) / BM;
    if (p.offsets) tiles_m = SEGK ? tiles_m * p.experts : segment_tiles(p.offsets, p.experts, p.rows, BM, lane);
    const int total = tiles_m * tiles_n;
    // part of the contraction (of one product, stored as FP32 partial sums)
    const int split = EPI == EPI_STORE && p.splits > 1 && total ? block / total : 0;
    const int b = block - split * total;
    if (b >= total || split >= max(p.splits, 1)) return;
    // the hardware deals workgroups round-robin to eight XCDs, each with its own
    // L2: a contiguous run of tiles each
    const int each = total / kXcds, rest = total % kXcds, xcd = b % kXcds;
    const int logical = xcd * each + min(xcd, rest) + b / kXcds;
    const int in_group = p.group * tiles_n, g = logical / in_group, first_m = g * p.group;
    const int gm = min(tiles_m - first_m, p.group);
    const int tm = first_m + logical % in_group % gm, tn = logical % in_group / gm;

    int row0, row_end, expert = 0, k_begin = 0, k_end = p.K;
    if (!p.offsets) {
        row0 = tm * BM;
        row_end = p.M;
    } else if (SEGK) {
        const int per = (p.M + BM - 1) / BM;
        expert = tm / per;
        row0 = tm % per * BM;
        row_end = p.M;
        segment_of(p.offsets, expert, p.rows, &k_begin, &k_end);
        k_begin = __builtin_amdgcn_readfirstlane(k_begin);
        k_end = __builtin_amdgcn_readfirstlane(k_end);
    } else {
        if (!find_segment(p.offsets, p.experts, p.rows, BM, tm, lane, &expert, &row0, &row_end)) return;
    }
    const int col0 = tn * BNC;
    if (EPI == EPI_STORE && p.splits > 1) {
        k_begin = split * p.split_k;
        k_end = min(k_begin + p.split_k, p.K);
    }

    Tile<LA, BM, WAVES> ta;
    Tile<LB, BN, WAVES> tb;
    const uint16_t *pa = p.a, *pb = p.b + (SEGK ? 0 : expert * p.b_stride);
    if (SEGK || EPI == EPI_STORE) {
        pa += k_begin * (LA == ACROSS ? p.lda : 1);
        pb += k_begin * (LB == ACROSS ? p.ldb : 1);
    }
    ta.template init<false>(pa, p.lda, row0, row_end, 0, wave, lane);
    tb.template init<EPI == EPI_GLU>(pb, p.ldb, col0, p.N, p.N, wave, lane);

    floatx16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    constexpr int NA = decltype(ta)::NI, LOADS = NA + decltype(tb)::NI;
    constexpr int READS = TM + TN, MFMAS = TM * TN, HALF = LOADS / 2;
    static_assert(MFMAS >= READS, "a product in front of every read");
    bf16x8 fa[2][TM], fb[2][TN];
    const uint32_t to_a = lds_address(lds) + wave * NA * 1024;
    const uint32_t to_b = lds_address(lds) + A_BYTES + wave * (LOADS - NA) * 1024;
    // a wave all of whose rows or columns lie behind the end only loads: the other
    // wave of its SIMD then has the matrix cores for itself
    const bool idle = row0 + wm * TM * 32 >= row_end ||
                      col0 + wn * (EPI == EPI_GLU ? TN * 16 : TN * 32) >= p.N;
    int left = k_end - k_begin;                // of the contraction

    // fragment n of a substep, in the order of their first use: b0 a0 b1 b2 .. a1 a2 ..
    auto read = [&](const uint8_t *from, int ks, int to, int n) {
        if (n == 0 || (n > 1 && n <= TN)) {
            const int j = n ? n - 1 : 0;
            fb[to][j] = tb.read(from + A_BYTES, wn * TN + j, ks, lane);
        } else {
            const int i = n == 1 ? 0 : n - TN;
            fa[to][i] = ta.read(from, wm * TM + i, ks, lane);
        }
    };
    // load n of a stage into buffer `buf`; `have` k of it exist (not looked at if FULL)
    auto load = [&](int buf, int n, int have, bool full) {
        if (n < NA) {
            if (full) ta.issue(to_a + buf * STAGE, n);
            else if (have > 0) ta.issue(to_a + buf * STAGE, n, have, wave, lane);
        } else {
            if (full) tb.issue(to_b + buf * STAGE, n - NA);
            else if (have > 0) tb.issue(to_b + buf * STAGE, n - NA, have, wave, lane);
        }
    };
    // One substep: its products from fragments `from`; between them the reads of
    // the next one's from `at` and `count` loads from number `first` on.
    auto substep = [&](int from, bool reads, const uint8_t *at, int ks, int buf, int first, int count,
                       int have, bool full) {
#pragma unroll
        for (int q = 0; q < MFMAS; ++q) {
            const int i = q / TN, j = q % TN;
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[from][i], fb[from][j], acc[i][j], 0, 0, 0);
            if (reads && q < READS) read(at, ks, 1 - from, q);
#pragma unroll
            for (int n = 0; n < LOADS; ++n)
                if (n < count && n * MFMAS / count == q) load(buf, first + n, have, full);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // the next stage has landed (of the loads in flight, `behind` are of later ones),
    // and this wave has read all of this one
    auto turn = [&](bool behind) {
        if (behind) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"((STAGES - 2) * LOADS) : "memory");
        else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // Stage in buffer `cur`; FULL: STAGES more of 64 k follow it at least.
    auto stage = [&](int cur, bool full) {
        const uint8_t *here = lds + cur * STAGE, *there = lds + (cur + 1) % STAGES * STAGE;
        const int next = left - BK;                                // k of the next stage
        const int rest = left - (STAGES - 1) * BK, after = left - STAGES * BK;
        substep(0, true, here, 1, (cur + STAGES - 1) % STAGES, HALF, LOADS - HALF, rest, full);
        substep(1, true, here, 2, 0, 0, 0, 0, true);
        substep(0, true, here, 3, 0, 0, 0, 0, true);
        ta.base += ta.step;
        tb.base += tb.step;
        if (full || next > 0) turn(full);
        substep(1, full || next > 0, there, 0, cur, 0, HALF, after, full);
        left -= BK;
    };
    auto stage_idle = [&](int cur) {
        const int rest = left - (STAGES - 1) * BK, after = left - STAGES * BK;
#pragma unroll
        for (int n = HALF; n < LOADS; ++n) load((cur + STAGES - 1) % STAGES, n, rest, false);
        ta.base += ta.step;
        tb.base += tb.step;
        if (left > BK) turn(false);
#pragma unroll
        for (int n = 0; n < HALF; ++n) load(cur, n, after, false);
        left -= BK;
    };
    if (left > 0) {
        // the first STAGES - 1 stages and the first half of the next one's loads
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
#pragma unroll
            for (int n = 0; n < LOADS; ++n) load(s, n, left - s * BK, false);
            ta.base += ta.step;
            tb.base += tb.step;
        }
        if (left >= (STAGES - 1) * BK) asm volatile("s_waitcnt vmcnt(%0)" : : "n"((STAGES - 2) * LOADS) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int n = 0; n < HALF; ++n) load(STAGES - 1, n, left - (STAGES - 1) * BK, false);
        if (idle) {
            while (left > 0) {
#pragma unroll
                for (int s = 0; s < STAGES; ++s)
                    if (left > 0) stage_idle(s);
            }
        } else {
#pragma unroll
            for (int n = 0; n < READS; ++n) read(lds, 0, 0, n);
            while (left >= 2 * STAGES * BK) {  // all loads of these stages are whole
#pragma unroll
                for (int s = 0; s < STAGES; ++s) stage(s, true);
            }
            while (left > 0) {
#pragma unroll
                for (int s = 0; s < STAGES; ++s)
                    if (left > 0) stage(s, false);
            }
        }
        __syncthreads();
    }
    if (idle) return;                          // no barrier follows

    // Epilogue: 32 rows at a time through this wave's part of the idle stages, so
    // that a lane gets eight neighbouring columns.  Element v of lane l of an
    // accumulator is row v / 4 * 8 + l / 32 * 4 + v % 4, column l % 32.
    constexpr int WCOLS = TN * 32, CHUNKS = EPI == EPI_GLU ? WCOLS / 16 : WCOLS / 8;
    constexpr int STEP = 64 / CHUNKS, PASSES = (32 + STEP - 1) / STEP;      // whole rows a pass: a lane keeps its columns
    constexpr int SLAB = 32 * WCOLS * 4;
    static_assert(WAVES * SLAB <= STAGES * STAGE, "a slab for every wave");
    float *slab = reinterpret_cast<float *>(lds + wave * SLAB);
    const int c = lane % CHUNKS * 8, r0 = lane / CHUNKS;
    const int col = col0 + wn * (EPI == EPI_GLU ? WCOLS / 2 : WCOLS) + c;
    const bool mine = col < p.N && r0 < STEP;
    auto inside = [&](int i, int k) {
        const int r = k * STEP + r0;
        return mine && r < 32 && row0 + (wm * TM + i) * 32 + r < row_end;
    };
    auto row_of = [&](int i, int k) { return (int64_t)row0 + (wm * TM + i) * 32 + k * STEP + r0; };
    auto slab_at = [&](int k) { return slab + min(k * STEP + r0, 31) * WCOLS; };
    float bias[8] = {}, bias_up[8] = {};
    if (EPI != EPI_STORE && mine) {
        const int64_t at = (int64_t)expert * (EPI == EPI_GLU ? 2 : 1) * p.N + col;
        load_bias(p, at, bias);
        if (EPI == EPI_GLU) load_bias(p, at + p.N, bias_up);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        // residuals first, so that their loads overlap
        Raw8<uint16_t> res16[EPI == EPI_RES ? PASSES : 1];
        if (EPI == EPI_RES && p.res && !p.y_f32) {
#pragma unroll
            for (int k = 0; k < PASSES; ++k)
                if (inside(i, k)) load_raw8<false>((const uint16_t *)p.res + row_of(i, k) * p.N + col, 8, res16[k]);
        }
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                slab[((v >> 2) * 8 + (lane >> 5) * 4 + (v & 3)) * WCOLS + j * 32 + (lane & 31)] = acc[i][j][v];
        // the wave reads what it wrote itself: LDS keeps a wave's order
        __builtin_amdgcn_wave_barrier();
        if (EPI == EPI_STORE || EPI == EPI_RES) {
            auto store_rows = [&](auto streamed) {
#pragma unroll
                for (int k = 0; k < PASSES; ++k) {
                    float z[8];
                    load8<false>(slab_at(k) + c, 8, z);
                    if (!inside(i, k)) continue;
                    const int64_t at = (EPI == EPI_STORE ? (int64_t)(expert * SEGK + split) * p.M * p.N : 0) +
                                       row_of(i, k) * p.N + col;
                    if (EPI == EPI_RES) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[e] += bias[e];
                        if (p.res) {
                            float v[8];
                            if (p.y_f32) load_res(p, at, v);
                            else unpack8(res16[k], v);
#pragma unroll
                            for (int e = 0; e < 8; ++e) z[e] += v[e];
                        }
                    }
                    store_y<decltype(streamed)::value>(p, at, z);
                }
            };
            if (p.stream) {
                // marked, so that the two branches are not merged, without the hint
                asm volatile("; streamed rows");
                store_rows(std::true_type());
                asm volatile("; end of streamed rows");
            } else {
                store_rows(std::false_type());
            }
        } else {
            // two rows a turn, not unrolled further: the activations' code is long
#pragma unroll 1
            for (int k = 0; k < PASSES; k += 2) {
                float z[2][8], u[2][8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float *at = slab_at(k + h);
                    if (EPI == EPI_GLU) {
                        at += (c >> 5) * 64 + (c & 31);
                        load8<false>(at, 8, z[h]);
                        load8<false>(at + 32, 8, u[h]);
                    } else {
                        load8<false>(at + c, 8, z[h]);
                        if (p.res && inside(i, k + h)) load_res(p, row_of(i, k + h) * p.N + col, u[h]);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!inside(i, k + h)) continue;
                    if (EPI == EPI_GLU) finish_glu(p, row_of(i, k + h), col, p.N, z[h], u[h], bias, bias_up);
                    else finish_linear(p, row_of(i, k + h), col, p.N, z[h], bias, u[h]);
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <int LA_, int LB_, int TM, int TN, int WM, int WN, int STAGES, int EPI, bool SEGK>
struct Shape {
    static constexpr int kThreads = 64 * WM * WN, kRows = WM * TM * 32, kCols = WN * TN * 32;
    static constexpr int kOutCols = EPI == EPI_GLU ? kCols / 2 : kCols, kLds = STAGES * (kRows + kCols) * 128;
    static constexpr bool kSegK = SEGK;
    static __device__ __forceinline__ void run(const ProductArgs &p, uint8_t *lds, int block)
    {
        product_tile<LA_, LB_, TM, TN, WM, WN, STAGES, EPI, SEGK>(p, lds, block);
    }
};

template <typename S>
__global__ __launch_bounds__(S::kThreads, 1) void k_product(const ProductArgs p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
    S::run(p, lds, workgroup<S::kThreads>());
}
// Two products in one launch: the second one's tiles fill the CUs that the first one's
// last ones leave.
template <typename S0, typename S1>
__global__ __launch_bounds__(S0::kThreads, 1) void k_product_pair(const ProductArgs p0, const ProductArgs p1, int n0)
{
    static_assert(S0::kThreads == S1::kThreads, "one size of workgroups");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S0::kLds > S1::kLds ? S0::kLds : S1::kLds];
    const int block = workgroup<S0::kThreads>();
    if (block < n0) S0::run(p0, lds, block);
    else S1::run(p1, lds, block - n0);
}

// ---- launches ------------------------------------------------------------------------
// Tiles of `bm` rows and `bn` columns (of the output), for the grid at most.
template <bool SEGK>
int64_t product_tiles(const ProductArgs &p, int bm, int bn)
{
    const int64_t n = ((int64_t)p.N + bn - 1) / bn;
    int64_t m = ((int64_t)p.M + bm - 1) / bm;
    if (p.offsets) {
        const int64_t used = p.experts < p.rows ? p.experts : p.rows;
        m = SEGK ? m * p.experts : p.rows / bm + used;          // segments end inside tiles
    }
    return m * n;
}

// Time of a call in one shape of tiles, to compare the shapes: rounds of 256 CUs
// times a round's, of `step` per 64 k and `fixed` around them (us, measured on
// 8192 x 2880 and 2880 x 5760 outputs).  Segments are taken to end in the middle of a tile;
// where they are shorter than a tile that counts too few.  32 even experts, 2880 -> 2880, us
// in tiles of 128 x 128, 256 x 192, 256 x 256, the one taken last: dx of 512 rows 112, 126,
// 138 (128 x 128), 1024 114, 128, 139 (256 x 256), 2048 118, 129, 140 (128 x 128), 4099 137,
// 135, 142 (256 x 192), 8192 193, 163, 164 (256 x 192), 16384 334, 268, 256 (256 x 256);
// forward of 4099 138, 139, 146 (256 x 192), 8192 194, 165, 166 (256 x 192), 16384 336, 280,
// 258 (256 x 192).
template <bool SEGK>
float product_time(const ProductArgs &p, int bm, int bn, int per_cu, float step, float fixed)
{
    const int64_t n = ((int64_t)p.N + bn - 1) / bn;
    float m = (float)(((int64_t)p.M + bm - 1) / bm), k = (float)p.K;
    if (p.offsets) {
        const float used = (float)(p.experts < p.rows ? p.experts : p.rows);
        if (SEGK) {
            m *= (float)p.experts;
            k /= (float)p.experts;
        } else {
            m = (float)p.rows / bm + 0.5f * used;              // on average
        }
    }
    const float rounds = ceilf(m * n / (256.0f * per_cu));
    return rounds * (ceilf(k / 64) * step + fixed);
}

// Workgroups of a product in tiles of shape S, and its arguments for them.
template <typename S>
int64_t shape_grid(const ProductArgs &p)
{
    return product_tiles<S::kSegK>(p, S::kRows, S::kOutCols) * (p.splits > 1 ? p.splits : 1);
}
template <typename S>
ProductArgs shape_args(ProductArgs p)
{
    const int64_t n = (int64_t)p.M * p.N * (S::kSegK && p.experts ? p.experts : 1);
    p.stream = n >= int64_t(1) << 22;                              // 8 MB of BF16
    return p;
}
template <typename S>
hipError_t launch_shape(const ProductArgs &p, hipStream_t stream)
{
    hipLaunchKernelGGL((k_product<S>), grid_of<S::kThreads>(shape_grid<S>(p)), dim3(S::kThreads), 0, stream, shape_args<S>(p));
    return hipGetLastError();
}
template <typename S0, typename S1>
hipError_t launch_pair(const ProductArgs &p0, const ProductArgs &p1, hipStream_t stream)
{
    const int64_t n0 = (shape_grid<S0>(p0) + kXcds - 1) / kXcds * kXcds;       // the second one's XCDs stay in step
    hipLaunchKernelGGL((k_product_pair<S0, S1>), grid_of<S0::kThreads>(n0 + shape_grid<S1>(p1)), dim3(S0::kThreads), 0,
                       stream, shape_args<S0>(p0), shape_args<S1>(p1), (int)n0);
    return hipGetLastError();
}
template <int LA, int LB, int TM, int TN, int WM, int WN, int STAGES, int EPI, bool SEGK>
hipError_t launch_tiles(const ProductArgs &p, hipStream_t stream)
{
    return launch_shape<Shape<LA, LB, TM, TN, WM, WN, STAGES, EPI, SEGK>>(p, stream);
}

// Tiles of 128 x 128: two workgroups a CU, or one with four stages where there is no
// second one to fill its waits.
template <int LA, int LB, int EPI, bool SEGK>
hipError_t launch_small(const ProductArgs &p, hipStream_t stream)
{
    const int64_t n = product_tiles<SEGK>(p, 128, EPI == EPI_GLU ? 64 : 128) * (p.splits > 1 ? p.splits : 1);
    if (n <= 256) return launch_tiles<LA, LB, 2, 2, 2, 2, 4, EPI, SEGK>(p, stream);
    return launch_tiles<LA, LB, 2, 2, 2, 2, 2, EPI, SEGK>(p, stream);
}

// The arguments of a product whose parts go to the workspace (`columns` of B).
inline ProductArgs split_args(ProductArgs p, int columns)
{
    p.N = columns;
    p.res = nullptr;
    p.y = p.partial;
    p.y_f32 = 1;
    p.split_k = (p.K / 64 + (p.K % 64 ? 1 : 0) + p.splits - 1) / p.splits * 64;
    return p;
}
// One product of few tiles: its parts to the workspace, then joined as `epilogue` says.
template <int LA, int LB, bool SEGK>
hipError_t launch_split(const ProductArgs &p, int columns, int epilogue, hipStream_t stream)
{
    const hipError_t e = launch_small<LA, LB, EPI_STORE, SEGK>(split_args(p, columns), stream);
    return e != hipSuccess ? e : fqimpl::launch_product_join(p, epilogue, p.partial, stream);
}

}  // namespace
