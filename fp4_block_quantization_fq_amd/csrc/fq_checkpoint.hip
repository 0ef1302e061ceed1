// fq_checkpoint.hip -- activations kept in 8 bits between the forward and the
// backward, and what the backward of the feed-forward products computes from
// them element by element: the gradient before the activation, the block's
// output once more, and the bias gradient's column sums.
//
// All of it is bound by memory: 16 bytes of BF16 (8 of codes) a lane and access,
// one pass over the data.  Column sums are FP32 in a fixed order: rows of a lane,
// lanes of a workgroup, then the tiles of an expert by a second kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_internal.h"
#include "fq_act.hpp"

namespace {

using namespace fqdev;
using fqimpl::RowArgs8;
using fqimpl::DzArgs;

constexpr int kBlock = 256;

// ---- 8-bit rows --------------------------------------------------------------------
// MX blocks know nothing of rows: chunk after chunk of eight elements.  NT: streaming
// accesses, where the call's data exceeds the caches.
template <bool NT>
__global__ __launch_bounds__(kBlock) void k_encode_mx(RowArgs8 a, int64_t chunks)
{
    const int64_t step = (int64_t)gridDim.x * kBlock;
    for (int64_t c = (int64_t)blockIdx.x * kBlock + threadIdx.x; c < chunks; c += step) {
        float v[8];
        load8<false, NT>((const uint16_t *)a.x + c * 8, 8, v);
        u32w2 codes;
        const uint32_t scale = mx8_encode8(v, &codes);
        if (NT) __builtin_nontemporal_store(codes, (u32w2 *)a.codes + c);
        else ((u32w2 *)a.codes)[c] = codes;
        if ((c & 3) == 0) ((uint8_t *)a.scales)[c >> 2] = (uint8_t)scale;
    }
}

// FP32 scale per row: LANES lanes hold a row of at most LANES * NCH chunks.
template <int LANES, int NCH>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void k_encode_row(RowArgs8 a)
{
    constexpr int THREADS = LANES < 256 ? 256 : LANES, WAVES = LANES / 64;
    __shared__ uint32_t tops[WAVES > 0 ? WAVES : 1];
    const int l = threadIdx.x % LANES;
    const int64_t row = (int64_t)workgroup<THREADS>() * (THREADS / LANES) + threadIdx.x / LANES;
    if (row >= a.rows) return;                   // of whole waves or workgroups, where those share rows
    const uint16_t *x = (const uint16_t *)a.x + row * a.cols;
    Raw8<uint16_t> raw[NCH];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        raw[i].w = (u32w4){0, 0, 0, 0};
        const int at = (i * LANES + l) * 8;
        if (at < a.cols) load_raw8<false>(x + at, 8, raw[i]);
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        float v[8];
        unpack8(raw[i], v);
        top = max(top, absmax(v));
    }
    top = lanes_max<(LANES < 64 ? LANES : 64)>(top);
    if (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i) top = max(top, tops[i]);
    }
    const bool bad = top >= 0x7F800000u;
    const float s = __builtin_fmaxf(as_f(top) * (1.0f / 448.0f), as_f(0x00800000u));
    const float inv = 1.0f / s;
    if (l == 0) ((float *)a.scales)[row] = bad ? as_f(0x7FC00000u) : s;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int at = (i * LANES + l) * 8;
        if (at >= a.cols) continue;
        float v[8];
        unpack8(raw[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_fminf(__builtin_fmaxf(v[e] * inv, -448.0f), 448.0f);
        *(u32w2 *)((uint8_t *)a.codes + row * a.cols + at) = bad ? (u32w2){0x7F7F7F7Fu, 0x7F7F7F7Fu} : e4m3_encode8(v);
    }
}

template <bool ROW, bool NT>
__global__ __launch_bounds__(kBlock) void k_decode(RowArgs8 a, int64_t chunks)
{
    const int64_t step = (int64_t)gridDim.x * kBlock;
    const uint32_t per_row = (uint32_t)(a.cols / 8);
    for (int64_t c = (int64_t)blockIdx.x * kBlock + threadIdx.x; c < chunks; c += step) {
        const u32w2 codes = NT ? __builtin_nontemporal_load((const u32w2 *)a.codes + c) : ((const u32w2 *)a.codes)[c];
        float s = ROW ? ((const float *)a.scales)[(uint32_t)c / per_row]            // chunks are below 2^31
                      : mx8_scale(((const uint8_t *)a.scales)[c >> 2]);
        if (ROW && a.power) s = row_scale_power(s);
        float v[8];
        e4m3_decode8(codes, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= s;
        store8<false, NT>((uint16_t *)a.y + c * 8, 8, v);
    }
}

// ---- gradient before the activation ----------------------------------------------------
// A workgroup: a tile of a segment's rows, 256 columns of the output (32 lanes of
// eight columns, eight rows at a time).  Tiles have 64 rows; where that leaves CUs
// without work (fewer than 512 workgroups), 8: 333 x 776 with GELU takes 4 us
// so, 29 in tiles of 64.  More than 2^28 rows have tiles of 512, for the grid's sake.

template <bool MX>
__device__ __forceinline__ void load_pre(const DzArgs &a, int64_t at, float (&v)[8])
{
    if (!MX) {
        load8<false>((const uint16_t *)a.pre + at, 8, v);
        return;
    }
    const float s = mx8_scale(((const uint8_t *)a.pre_scales)[at >> 5]);
    e4m3_decode8(*(const u32w2 *)((const uint8_t *)a.pre + at), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= s;
}

// Eight values of dz, rounded to BF16, which is what the matrix cores take: the products
// of this backward are then off by 0.0023 of their norm with outputs in BF16, whose own
// rounding is 0.0017 of it.  Two BF16 parts would hold 16 bits of dz and cost both products
// again (460 to 500 of 530 us at 8192 x 2880 -> 2 x 2880).  Column sums take the FP32 values.
// Where x comes with a scale per row, dw = x^T dz takes the codes
// times the scale's power of two, which BF16 holds exactly, and the scale's mantissa
// here: one rounding to BF16 (0.0017 of dw in the mean) instead of x's and dz's (0.0024).
__device__ __forceinline__ void store_dz(const DzArgs &a, int64_t at, float mantissa, const float (&v)[8])
{
    if (a.dz) store8<false>((uint16_t *)a.dz + at, 8, v);
    if (!a.dz_scaled) return;
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = v[e] * mantissa;
    store8<false>((uint16_t *)a.dz_scaled + at, 8, t);
}

// GLU: two halves of pre and dz; else pre may be missing (no activation), then
// only the column sums are made.
template <bool GLU, bool MX>
__global__ __launch_bounds__(kBlock) void k_dz(DzArgs a)
{
    __shared__ float sums[GLU ? 2 : 1][8][256 + 8];
    const int lane = threadIdx.x & 63;
    const int tile = blockIdx.x;
    int row0 = tile * a.tile, row_end = (int)a.rows, expert;
    if (a.offsets) {
        if (tile >= segment_tiles(a.offsets, a.experts, (int)a.rows, a.tile, lane)) return;
        if (!find_segment(a.offsets, a.experts, (int)a.rows, a.tile, tile, lane, &expert, &row0, &row_end)) return;
    }
    row_end = row_end - row0 < a.tile ? row_end : row0 + a.tile;
    const int c = threadIdx.x & 31, r0 = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.y * 256 + c * 8;
    const int64_t cols = GLU ? 2 * a.n : a.n;
    float s0[8] = {}, s1[8] = {};
    if (col < a.n) {
        for (int64_t r = row0 + r0; r < row_end; r += 8) {
            float d[8], g[8], u[8];
            load8<false>((const uint16_t *)a.dy + r * a.n + col, 8, d);
            const int64_t at = r * cols + col;
            const float mantissa = a.dz_scaled ? row_scale_mantissa(a.row_scales[r]) : 1.0f;
            if (GLU) {
                load_pre<MX>(a, at, g);
                load_pre<MX>(a, at + a.n, u);
                glu8_grad(a.gate, g, u, d);
                store_dz(a, at, mantissa, g);
                store_dz(a, at + a.n, mantissa, u);
                if (a.h) store8<false>((uint16_t *)a.h + r * a.n + col, 8, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s0[e] += g[e];
                    s1[e] += u[e];
                }
            } else {
                if (a.pre) {
                    load_pre<MX>(a, at, g);
                    act8_grad(a.gate.act, g, d);
                    store_dz(a, at, mantissa, d);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) s0[e] += d[e];
            }
        }
    }
    if (!a.partials) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sums[0][r0][c * 8 + e] = s0[e];
        if (GLU) sums[GLU ? 1 : 0][r0][c * 8 + e] = s1[e];
    }
    __syncthreads();
    const int64_t to = (int64_t)blockIdx.y * 256 + threadIdx.x;
    if (to >= a.n) return;
#pragma unroll
    for (int half = 0; half < (GLU ? 2 : 1); ++half) {
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r) t += sums[half][r][threadIdx.x];
        a.partials[(int64_t)tile * cols + half * a.n + to] = t;
    }
}

// dbias of one expert and COLS columns: its tiles' sums, 256 / COLS lanes a column,
// joined in the order of the tiles' numbers modulo those.
template <int COLS>
__global__ __launch_bounds__(kBlock) void k_dbias(DzArgs a, int64_t cols)
{
    constexpr int SLICES = kBlock / COLS;
    __shared__ float part[SLICES][COLS + 1];
    const int lane = threadIdx.x & 63, c = threadIdx.x % COLS, slice = threadIdx.x / COLS, expert = blockIdx.y;
    int first = 0, count = (int)((a.rows + a.tile - 1) / a.tile);
    if (a.offsets) {
        int s, e;
        first = segment_tiles(a.offsets, expert, (int)a.rows, a.tile, lane);
        segment_of(a.offsets, expert, (int)a.rows, &s, &e);
        count = (e - s + a.tile - 1) / a.tile;
        // offsets that do not ascend may name more tiles than there are
        if (first < 0 || first >= a.tiles) count = 0;
        else count = min(count, a.tiles - first);
    }
    const int64_t col = (int64_t)blockIdx.x * COLS + c;
    float t = 0.0f;
    if (col < cols) {
        const float *p = a.partials + first * cols + col;
#pragma unroll 4
        for (int i = slice; i < count; i += SLICES) t += p[i * cols];
    }
    part[slice][c] = t;
    __syncthreads();
    if (slice == 0 && col < cols) {
        t = 0.0f;
#pragma unroll
        for (int i = 0; i < SLICES; ++i) t += part[i][c];
        a.dbias[expert * cols + col] = t;
    }
}

// Chunks from which a call streams: 192 MB of values and codes, of the 256 MB that the
// memory-side cache holds.  What is better below depends on who uses the data next (widths
// of 4096, plain / streamed, us).  Encoding and decoding again: 4096 rows 22 / 21, 8192 40 /
// 38, 16384 75 / 70, 32768 142 / 134.  Encoding what was just made: 20 / 17, 42 / 36, 78 /
// 70, 160 / 136.  Decoding for a pass over the values: 21 / 23, 39 / 42, 77 / 82, 157 / 157,
// and in a product's backward 8192 x 2880 247 / 266, 16384 468 / 497, 32768 1021 / 1014.  So
// smaller calls leave their values where a backward finds them.
constexpr int64_t kStreamChunks = int64_t(1) << 23;

uint32_t flat_grid(int64_t chunks)
{
    const int64_t n = (chunks + kBlock - 1) / kBlock;
    return (uint32_t)(n < 65536 ? n : 65536);
}

}  // namespace

namespace fqimpl {

hipError_t launch_f8_encode(int f8, const RowArgs8 &a, hipStream_t stream)
{
    const int64_t chunks = a.rows * a.cols / 8;
    if (f8 == F8_MX) {
        hipLaunchKernelGGL((chunks >= kStreamChunks ? k_encode_mx<true> : k_encode_mx<false>), dim3(flat_grid(chunks)),
                           dim3(kBlock), 0, stream, a, chunks);
        return hipGetLastError();
    }
    const int64_t need = a.cols / 8;         // chunks of a row
#define FQ_ENCODE_ROW(LANES, NCH)                                                                        \
    hipLaunchKernelGGL((k_encode_row<LANES, NCH>),                                                       \
                       grid_of<(LANES < 256 ? 256 : LANES)>(                                            \
                           LANES < 256 ? (a.rows + 256 / LANES - 1) / (256 / LANES) : a.rows),          \
                       dim3(LANES < 256 ? 256 : LANES), 0, stream, a)
    if (need <= 16) FQ_ENCODE_ROW(16, 1);
    else if (need <= 64) FQ_ENCODE_ROW(64, 1);
    else if (need <= 256) FQ_ENCODE_ROW(256, 1);
    else if (need <= 512) FQ_ENCODE_ROW(256, 2);
    else if (need <= 1024) FQ_ENCODE_ROW(512, 2);
    else FQ_ENCODE_ROW(1024, 4);
#undef FQ_ENCODE_ROW
    return hipGetLastError();
}

hipError_t launch_f8_decode(int f8, const RowArgs8 &a, hipStream_t stream)
{
    const int64_t chunks = a.rows * a.cols / 8;
    const bool nt = chunks >= kStreamChunks;
    const auto kernel = f8 == F8_MX ? (nt ? k_decode<false, true> : k_decode<false, false>)
                                    : (nt ? k_decode<true, true> : k_decode<true, false>);
    hipLaunchKernelGGL(kernel, dim3(flat_grid(chunks)), dim3(kBlock), 0, stream, a, chunks);
    return hipGetLastError();
}

int dz_tile(int64_t rows, int64_t n)
{
    if (rows > int64_t(1) << 28) return 512;
    return (rows + 63) / 64 * ((n + 255) / 256) >= 512 ? 64 : 8;
}

int64_t dz_tiles(int64_t rows, int64_t n, int64_t experts)
{
    const int64_t tile = dz_tile(rows, n);
    if (!experts) return (rows + tile - 1) / tile;
    return rows / tile + (experts < rows ? experts : rows);
}

hipError_t launch_dz(DzArgs a, hipStream_t stream)
{
    a.tile = dz_tile(a.rows, a.n);
    a.tiles = (int)dz_tiles(a.rows, a.n, a.offsets ? a.experts : 0);
    const dim3 grid((uint32_t)a.tiles, (uint32_t)((a.n + 255) / 256));
    const int64_t cols = a.glu ? 2 * a.n : a.n;
    if (a.glu && a.pre_kind == PRE_MX) hipLaunchKernelGGL((k_dz<true, true>), grid, dim3(kBlock), 0, stream, a);
    else if (a.glu) hipLaunchKernelGGL((k_dz<true, false>), grid, dim3(kBlock), 0, stream, a);
    else if (a.pre_kind == PRE_MX) hipLaunchKernelGGL((k_dz<false, true>), grid, dim3(kBlock), 0, stream, a);
    else hipLaunchKernelGGL((k_dz<false, false>), grid, dim3(kBlock), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dbias) return e;
    // one long list of tiles, or an expert's short ones
    if (!a.offsets)
        hipLaunchKernelGGL((k_dbias<16>), dim3((uint32_t)((cols + 15) / 16)), dim3(kBlock), 0, stream, a, cols);
    else
        hipLaunchKernelGGL((k_dbias<64>), dim3((uint32_t)((cols + 63) / 64), (uint32_t)a.experts), dim3(kBlock), 0,
                           stream, a, cols);
    return hipGetLastError();
}

}  // namespace fqimpl
