// fq_product.hip -- the feed-forward products of a training step on BF16
// matrix cores: y = a(x w + b) + res, the gated h = a(x wg + bg) (x wu + bu),
// and the two products of their backward, dx = dz w^T and dw = x^T dz.  One
// product, or one per expert over the segments of rows that fq_moe_sort made.
//
// A product is C[M, N] = sum over k of A(m, k) B(k, n), FP32 sums on
// v_mfma_f32_32x32x16_bf16.  Weights lie [K, N] and activations [rows, K], so
// an operand is either contiguous along the contraction (x in the forward, dz
// and w in dx) or across it (w in the forward, x and dz in dw).  Both go from
// global memory straight to LDS as they lie, 16 bytes a lane; the second kind
// is transposed on the way into registers by gfx950's ds_read_b64_tr_b16: in a
// group of 16 lanes, lane s reads four columns of row s / 4 and receives the
// four rows of column s.
//
// LDS tiles: contraction-contiguous, a 128-byte row (64 k) per tile row, 16-byte
// chunks XORed with (row & 7) ^ (row >> 3 & 1); otherwise a row per k of all the
// tile's columns, chunks XORed with (k & 3) << 2, so the four rows that a
// transposing read touches lie in different banks.
//
// Past the end of the contraction both operands are read as zeros (from an
// array of zeros, chosen by address), so neither infinities nor NaN of other
// rows reach a sum.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_internal.h"
#include "fq_act.hpp"

namespace {

using namespace fqdev;
using fqimpl::ProductArgs;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

enum { ALONG = 0, ACROSS = 1 };                  // operand against the contraction
enum { EPI_STORE = 0, EPI_LINEAR = 1, EPI_GLU = 2 };

constexpr int BK = 64;
constexpr int kXcds = 8;

__device__ const u32w4 kZeros = {0, 0, 0, 0};

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
    static constexpr int CHUNKS = ROWS / 8;                // of a row (ACROSS)
    static constexpr int PER = 64 / CHUNKS;                // rows an instruction (ACROSS)
    const uint8_t *base;
    uint32_t off[NI];
    int64_t step;

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
                const int row = min(r, count - first - 1);
                off[i] = (uint32_t)row * (uint32_t)(pitch * 2) + swz(r, lane & 7) * 16;
            }
        } else {
            base = (const uint8_t *)p;
            step = BK * 2 * pitch;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int k = (wave * NI + i) * PER + lane / CHUNKS;
                const int t = (((lane % CHUNKS) ^ ((k & 3) << 2))) * 8;
                int col = first + t, more = 0;
                if (SPLIT) {
                    col = first + (t >> 6) * 32 + (t & 31);
                    more = (t & 32) ? half : 0;
                }
                if (col >= count) col = first;          // never stored
                off[i] = (uint32_t)k * (uint32_t)(pitch * 2) + (uint32_t)(col + more) * 2;
            }
        }
    }
    // k of instruction i's chunk within the step
    __device__ __forceinline__ int k_of(int i, int wave, int lane) const
    {
        if (L == ALONG) return swz((wave * NI + i) * 8 + (lane >> 3), lane & 7) * 8;
        return (wave * NI + i) * PER + lane / CHUNKS;
    }
    __device__ __forceinline__ void load(uint8_t *lds, int left, int wave, int lane)
    {
        if (left >= BK) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                __builtin_amdgcn_global_load_lds((const void *)(base + off[i]),
                                                 (lds_void *)(lds + (wave * NI + i) * 1024), 16, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const uint8_t *src = k_of(i, wave, lane) < left ? base + off[i] : (const uint8_t *)&kZeros;
                __builtin_amdgcn_global_load_lds((const void *)src,
                                                 (lds_void *)(lds + (wave * NI + i) * 1024), 16, 0, 0);
            }
        }
        base += step;
    }
    // eight k of row (column) `r` + lane % 32 for substep ks of 16 k
    static __device__ __forceinline__ bf16x8 read(const uint8_t *lds, int r0, int ks, int lane)
    {
        if (L == ALONG) {
            const int r = r0 + (lane & 31);
            return *reinterpret_cast<const bf16x8 *>(lds + r * 128 + swz(r, ks * 2 + (lane >> 5)) * 16);
        }
        const int row = ks * 16 + (lane >> 5) * 8 + ((lane & 15) >> 2);
        const int col = r0 + (lane & 16) + (lane & 3) * 4;
        const uint8_t *p = lds + row * (ROWS * 2) + (((col >> 3) ^ (((lane & 15) >> 2) << 2)) << 4) +
                           (col & 4) * 2;
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

__device__ __forceinline__ void store_y(const ProductArgs &p, int64_t at, float (&v)[8])
{
    if (p.y_f32) {
        if (p.res) {
            float r[8];
            load8<false>((const float *)p.res + at, 8, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
        }
        store8<false>((float *)p.y + at, 8, v);
    } else {
        if (p.res) {
            float r[8];
            load8<false>((const uint16_t *)p.res + at, 8, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
        }
        store8<false>((uint16_t *)p.y + at, 8, v);
    }
}

// What becomes of eight sums (column `col` of row `row`, of N columns).
__device__ __forceinline__ void finish_linear(const ProductArgs &p, int64_t row, int col, int N,
                                              float (&z)[8], const float (&bias)[8])
{
    const int64_t at = row * N + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += bias[i];
    if (p.pre_kind) keep_pre(p, at, z);
    act8(p.act, 1.0f, z);
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
    glu8(p.gate, g, u);
    store8<false>((uint16_t *)p.y + row * n + col, 8, g);
}

// ---- the kernel ----------------------------------------------------------------------
// WM x WN waves of TM 32-row and two 32-column accumulator tiles.  SEGK: the
// experts' segments are of the contraction (dw), else of C's rows.
template <int LA, int LB, int TM, int WM, int WN, int EPI, bool SEGK>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_product(const ProductArgs p)
{
    constexpr int BM = WM * TM * 32, BN = WN * 64, WAVES = WM * WN, TN = 2;
    constexpr int BNC = EPI == EPI_GLU ? BN / 2 : BN;      // columns of the output
    constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 128;
    // two stages as two variables, each access naming its own: the compiler
    // then does not wait for the loads in flight into the other one
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[STAGE];

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int wm = wave / WN, wn = wave % WN;

    // this workgroup's tile
    const int tiles_n = (p.N + BNC - 1) / BNC;
    int tiles_m = (p.M + BM - 1) / BM;
    if (p.offsets) tiles_m = SEGK ? tiles_m * p.experts : segment_tiles(p.offsets, p.experts, p.rows, BM, lane);
    const int total = tiles_m * tiles_n, b = (int)blockIdx.x;
    if (b >= total) return;
    // the hardware deals workgroups round-robin to eight XCDs, each with its own
    // L2: a contiguous run of tiles each
    const int each = total / kXcds, rest = total % kXcds, xcd = b % kXcds;
    const int logical = xcd * each + min(xcd, rest) + b / kXcds;
    const int in_group = p.group * tiles_n, g = logical / in_group, first_m = g * p.group;
    const int gm = min(tiles_m - first_m, p.group);
    int tm = first_m + logical % in_group % gm;
    const int tn = logical % in_group / gm;

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
    } else {
        find_segment(p.offsets, p.experts, p.rows, BM, tm, lane, &expert, &row0, &row_end);
    }
    const int col0 = tn * BNC;

    Tile<LA, BM, WAVES> ta;
    Tile<LB, BN, WAVES> tb;
    const uint16_t *pa = p.a, *pb = p.b + (SEGK ? 0 : expert * p.b_stride);
    if (SEGK) {
        pa += (int64_t)k_begin * p.lda;
        pb += (int64_t)k_begin * p.ldb;
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

    int left = k_end - k_begin;                // of the contraction
    auto stage = [&](const uint8_t *cur, uint8_t *nxt) {
        if (left > BK) {
            ta.load(nxt, left - BK, wave, lane);
            tb.load(nxt + A_BYTES, left - BK, wave, lane);
        }
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks) {
            bf16x8 fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[i] = ta.read(cur, (wm * TM + i) * 32, ks, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[j] = tb.read(cur + A_BYTES, (wn * TN + j) * 32, ks, lane);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_iglp_opt(1);
        }
        __builtin_amdgcn_s_waitcnt(0);         // this wave's loads of the next stage have landed
        __syncthreads();
        left -= BK;
    };
    if (left > 0) {
        ta.load(lds0, left, wave, lane);
        tb.load(lds0 + A_BYTES, left, wave, lane);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        while (left > 0) {
            stage(lds0, lds1);
            if (left > 0) stage(lds1, lds0);
        }
    }

    // Epilogue: 32 rows at a time through 8 KB of the idle stage, of this wave
    // alone, so that a lane gets eight neighbouring columns.  Element v of lane l
    // of an accumulator is row v / 4 * 8 + l / 32 * 4 + v % 4, column l % 32.
    static_assert(WAVES * 8192 <= STAGE, "a slab for every wave");
    float *slab = reinterpret_cast<float *>(lds0) + wave * 2048;
    const int lanes_row = EPI == EPI_GLU ? 4 : 8;          // lanes of a row
    const int c8 = (lane % lanes_row) * 8;
    const int col = col0 + wn * (EPI == EPI_GLU ? 32 : 64) + c8;
    const bool col_ok = col < p.N;
    float bias[8], bias_up[8];
    if (EPI != EPI_STORE) {
        const int64_t at = (int64_t)expert * (EPI == EPI_GLU ? 2 : 1) * p.N + min(col, p.N - 8);
        load_bias(p, at, bias);
        if (EPI == EPI_GLU) load_bias(p, at + p.N, bias_up);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                slab[((v >> 2) * 8 + (lane >> 5) * 4 + (v & 3)) * 64 + j * 32 + (lane & 31)] = acc[i][j][v];
        // the wave reads what it wrote itself: LDS keeps a wave's order
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < 32 * lanes_row / 64; ++k) {
            const int r = k * (64 / lanes_row) + lane / lanes_row;
            const int64_t row = (int64_t)row0 + (wm * TM + i) * 32 + r;
            float z[8], u[8];
            load8<false>(slab + r * 64 + c8, 8, z);
            if (EPI == EPI_GLU) load8<false>(slab + r * 64 + 32 + c8, 8, u);
            if (row >= row_end || !col_ok) continue;
            if (EPI == EPI_GLU) {
                finish_glu(p, row, col, p.N, z, u, bias, bias_up);
            } else if (EPI == EPI_LINEAR) {
                finish_linear(p, row, col, p.N, z, bias);
            } else {
                const int64_t at = (SEGK ? (int64_t)expert * p.M * p.N : 0) + row * p.N + col;
                if (p.y_f32) store8<false>((float *)p.y + at, 8, z);
                else store8<false>((uint16_t *)p.y + at, 8, z);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <int LA, int LB, int EPI, bool SEGK>
hipError_t launch(ProductArgs p, hipStream_t stream)
{
    const int64_t cols = p.N;
    auto tiles = [&](int bm, int bnc) {
        const int64_t n = (cols + bnc - 1) / bnc;
        int64_t m = (p.M + bm - 1) / bm;
        if (p.offsets) {
            const int64_t used = p.experts < p.rows ? p.experts : p.rows;
            m = SEGK ? m * p.experts : p.rows / bm + used;      // segments end inside tiles
        }
        return m * n;
    };
    const int64_t big = tiles(256, EPI == EPI_GLU ? 128 : 256);
    p.group = p.offsets && !SEGK ? 2 : 8;
    if (big >= 256 && !(p.offsets && !SEGK && p.rows / p.experts < 256)) {
        hipLaunchKernelGGL((k_product<LA, LB, 4, 2, 4, EPI, SEGK>), dim3((uint32_t)big), dim3(512), 0,
                           stream, p);
    } else {
        hipLaunchKernelGGL((k_product<LA, LB, 2, 2, 2, EPI, SEGK>),
                           dim3((uint32_t)tiles(128, EPI == EPI_GLU ? 64 : 128)), dim3(256), 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace

namespace fqimpl {

hipError_t launch_product_linear(const ProductArgs &p, hipStream_t stream)
{
    return launch<ALONG, ACROSS, EPI_LINEAR, false>(p, stream);
}
hipError_t launch_product_glu(const ProductArgs &p, hipStream_t stream)
{
    return launch<ALONG, ACROSS, EPI_GLU, false>(p, stream);
}
hipError_t launch_product_dx(const ProductArgs &p, hipStream_t stream)
{
    return launch<ALONG, ALONG, EPI_STORE, false>(p, stream);
}
hipError_t launch_product_dw(const ProductArgs &p, hipStream_t stream)
{
    return launch<ACROSS, ACROSS, EPI_STORE, true>(p, stream);
}

}  // namespace fqimpl
