// fq_product_few.hip -- the forward products of few rows (one token and a few
// dozen), which are bound by reading the weight once.
//
// A workgroup has COLS columns of the weight (a gated block's: half of them gate,
// half up); its waves split the contraction, wave w taking the steps w, w + WAVES,
// ... of 32 k, and join their sums at the end.  A wave streams its steps through
// LDS of its own, DEPTH of them in flight, with no barrier until the end: 16 bytes
// a lane straight from global memory (loads of 4 or 8 bytes a lane, which as many
// columns in registers would take, are bound by their addresses at 16 or 32 bytes
// a clock and CU), transposed on the way into registers (fq_product.hpp) for
// v_mfma_f32_16x16x32_bf16.  The activations of a step come the same way, so that
// the waits, written by hand, count them too.
#include "fq_product.hpp"

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bias1(const ProductArgs &p, int64_t at)
{
    return !p.bias ? 0.0f : p.bias_f32 ? ((const float *)p.bias)[at] : load1((const uint16_t *)p.bias + at);
}

// all but the last N loads of this wave have landed
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// RT: tiles of 16 rows.
template <int COLS, int RT, int WAVES, int DEPTH, int EPI>
__global__ __launch_bounds__(64 * WAVES) void k_product_few(const ProductArgs p)
{
    constexpr int ROWS = 16 * RT, TILES = COLS / 16;       // MFMA tiles of columns
    constexpr int BNC = EPI == EPI_GLU ? COLS / 2 : COLS;
    constexpr int W_LOADS = COLS / 16, LOADS = W_LOADS + RT, SLOT = LOADS * 1024;
    constexpr int CHUNKS_K = COLS / 8;                     // 16-byte chunks of a k's row
    constexpr int ZC = EPI == EPI_GLU ? 2 * BNC : BNC;
    struct Join {
        float part[WAVES][16][COLS], z[16][ZC + 4], y[16][BNC + 4];
    };
    constexpr int RING = WAVES * DEPTH * SLOT;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[RING > (int)sizeof(Join) ? RING : (int)sizeof(Join)];

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int tiles_n = (p.N + BNC - 1) / BNC;
    const int tiles_m = p.offsets ? segment_tiles(p.offsets, p.experts, p.rows, ROWS, lane) : (p.M + ROWS - 1) / ROWS;
    const int total = tiles_m * tiles_n, b = workgroup<64 * WAVES>();
    if (b >= total) return;
    // neighbours in one XCD share lines of the weight's rows
    const int each = total / kXcds, rest = total % kXcds, xcd = b % kXcds;
    const int logical = xcd * each + min(xcd, rest) + b / kXcds;
    const int tm = logical / tiles_n, tn = logical % tiles_n;
    int row0 = tm * ROWS, row_end = p.M, expert = 0;
    if (p.offsets && !find_segment(p.offsets, p.experts, p.rows, ROWS, tm, lane, &expert, &row0, &row_end)) return;
    const int rows = min(row_end - row0, ROWS), col0 = tn * BNC;

    // this lane's chunk of the weight's rows: its first k in a step and its columns
    const int chunk = lane % CHUNKS_K, lane_k = lane / CHUNKS_K;
    int col = col0 + chunk * 8, more = 0;
    if (EPI == EPI_GLU) {
        col = col0 + chunk % (CHUNKS_K / 2) * 8;
        more = chunk >= CHUNKS_K / 2 ? p.N : 0;
    }
    if (col >= p.N) col = col0;                            // never stored
    const uint16_t *w = p.b + expert * p.b_stride + (int64_t)lane_k * p.ldb + col + more;
    const uint16_t *x[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        x[i] = p.a + (int64_t)(row0 + min(i * 16 + (lane >> 2), rows - 1)) * p.lda + (lane & 3) * 8;

    const uint32_t ring = lds_address(lds) + wave * DEPTH * SLOT;
    auto issue = [&](int slot, int s) {
        const int k0 = s * 32;
        const uint32_t to = ring + slot * SLOT;
#pragma unroll
        for (int i = 0; i < W_LOADS; ++i) {
            const int k = i * (64 / CHUNKS_K);
            const uint16_t *src = k0 + k + lane_k < p.K ? w + (int64_t)(k0 + k) * p.ldb : (const uint16_t *)&kZeros;
            direct_load((const uint8_t *)src, to + i * 1024);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const uint16_t *src = k0 + (lane & 3) * 8 < p.K ? x[i] + k0 : (const uint16_t *)&kZeros;
            direct_load((const uint8_t *)src, to + (W_LOADS + i) * 1024);
        }
    };

    floatx4 acc[RT][TILES];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TILES; ++j) acc[i][j] = (floatx4){0, 0, 0, 0};

    const int steps = (p.K + 31) / 32;
    const int mine = wave < steps ? (steps - wave + WAVES - 1) / WAVES : 0;      // steps of this wave
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (d < mine) issue(d, wave + d * WAVES);
    for (int n = 0, slot = 0; n < mine; ++n) {
        const int behind = min(mine - n, DEPTH) - 1;       // steps in flight behind this one
        if (behind >= 3 && DEPTH > 3) wait_loads<3 * LOADS>();
        else if (behind == 2) wait_loads<2 * LOADS>();
        else if (behind == 1) wait_loads<LOADS>();
        else wait_loads<0>();
        const uint8_t *at = lds + (wave * DEPTH + slot) * SLOT;
        bf16x8 fx[RT], fw[TILES];
#pragma unroll
        for (int i = 0; i < RT; ++i)
            fx[i] = *reinterpret_cast<const bf16x8 *>(at + (W_LOADS + i) * 1024 + (lane & 15) * 64 + (lane >> 4) * 16);
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
            const uint8_t *q = at + ((lane >> 4) * 8 + ((lane & 15) >> 2)) * (COLS * 2) + j * 32 + (lane & 3) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)q);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(q + 4 * COLS * 2));
            fw[j] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");         // the slot has been read
        if (n + DEPTH < mine) issue(slot, wave + (n + DEPTH) * WAVES);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < TILES; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[i], fw[j], acc[i][j], 0, 0, 0);
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
    }

    // Joined 16 rows at a time, in the order of the waves: each thread some outputs
    // (so that the activation's code stands once, which a call this short notices),
    // then eight neighbouring ones to a lane.  Element v of lane l is row
    // l / 16 * 4 + v, column l % 16.
    Join &join = *reinterpret_cast<Join *>(lds);
    constexpr int CHUNKS = BNC / 8;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        if (i * 16 >= rows) break;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < TILES; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) join.part[wave][(lane >> 4) * 4 + v][j * 16 + (lane & 15)] = acc[i][j][v];
        __syncthreads();
        for (int e = tid; e < 16 * BNC; e += 64 * WAVES) {
            const int r = e / BNC, c = e % BNC;
            if (i * 16 + r >= rows || col0 + c >= p.N) continue;
            const int64_t at = (int64_t)expert * (EPI == EPI_GLU ? 2 : 1) * p.N + col0 + c;
            float z[1] = {0.0f}, u[1] = {0.0f};
#pragma unroll
            for (int q = 0; q < WAVES; ++q) {
                z[0] += join.part[q][r][c];
                if (EPI == EPI_GLU) u[0] += join.part[q][r][BNC + c];
            }
            z[0] += bias1(p, at);
            join.z[r][c] = z[0];
            if (EPI == EPI_GLU) {
                u[0] += bias1(p, at + p.N);
                join.z[r][BNC + c] = u[0];
                glu_n(p.gate, z, u);
            } else {
                act_n(p.act, 1.0f, z);
            }
            join.y[r][c] = z[0];
        }
        __syncthreads();
        for (int e = tid; e < 16 * CHUNKS; e += 64 * WAVES) {
            const int r = e / CHUNKS, c = e % CHUNKS * 8;
            const int64_t row = (int64_t)row0 + i * 16 + r;
            if (i * 16 + r >= rows || col0 + c >= p.N) continue;
            float v[8];
            if (p.pre_kind) {
                const int64_t at = row * (EPI == EPI_GLU ? 2 : 1) * p.N + col0 + c;
                load8<false>(&join.z[r][c], 8, v);
                keep_pre(p, at, v);
                if (EPI == EPI_GLU) {
                    load8<false>(&join.z[r][BNC + c], 8, v);
                    keep_pre(p, at + p.N, v);
                }
            }
            load8<false>(&join.y[r][c], 8, v);
            if (p.res) {
                float res[8];
                load_res(p, row * p.N + col0 + c, res);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] += res[q];
            }
            store_y(p, row * p.N + col0 + c, v);
        }
    }
}

template <int COLS, int RT, int WAVES, int DEPTH, int EPI>
hipError_t launch_few(const ProductArgs &p, hipStream_t stream)
{
    const int64_t tiles = product_tiles<false>(p, 16 * RT, COLS / (EPI == EPI_GLU ? 2 : 1));
    hipLaunchKernelGGL((k_product_few<COLS, RT, WAVES, DEPTH, EPI>), grid_of<64 * WAVES>(tiles), dim3(64 * WAVES), 0, stream, p);
    return hipGetLastError();
}

template <int EPI>
hipError_t few(const ProductArgs &p, hipStream_t stream)
{
    // rows that share a weight: with experts twice their average, so that most
    // segments fit one tile
    const int rows = p.offsets ? 2 * p.M / p.experts : p.M;
    // 32 columns of the weight a workgroup until 64 are enough for half of the CUs;
    // a gated block in 8 bits needs 32 columns of a half in one workgroup
    const int cols = EPI == EPI_GLU ? 2 * p.N : p.N;
    const bool narrow = cols < 64 * 128 && !(EPI == EPI_GLU && p.pre_kind == fqimpl::PRE_MX);
    if (rows <= 16) return narrow ? launch_few<32, 1, 16, 3, EPI>(p, stream) : launch_few<64, 1, 8, 4, EPI>(p, stream);
    if (rows <= 32) return narrow ? launch_few<32, 2, 8, 4, EPI>(p, stream) : launch_few<64, 2, 8, 3, EPI>(p, stream);
    return narrow ? launch_few<32, 4, 8, 3, EPI>(p, stream) : launch_few<64, 4, 8, 2, EPI>(p, stream);
}

}  // namespace

namespace fqimpl {

hipError_t launch_product_few_linear(const ProductArgs &p, hipStream_t stream) { return few<EPI_LINEAR>(p, stream); }
hipError_t launch_product_few_glu(const ProductArgs &p, hipStream_t stream) { return few<EPI_GLU>(p, stream); }

}  // namespace fqimpl
