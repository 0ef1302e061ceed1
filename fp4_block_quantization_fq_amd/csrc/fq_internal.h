// fq_internal.h -- launchers shared between the C-ABI layer and the kernels.
// Arguments are validated by the caller (fq_api.cpp); launchers only map the
// problem onto a grid and enqueue on `stream`.  Each returns hipSuccess or
// the launch error.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fqimpl {

enum { FMT_MX = 0, FMT_NVT = 1, FMT_NV128 = 2 };

// Number of partial maxima the per-tensor reduction writes (4 bytes each).
constexpr uint32_t kAbsmaxPartials = 1024;

struct QuantArgs {
    int fmt;              // FMT_*
    int sr;               // 0 = round to nearest even, 1 = stochastic
    int col;              // 0 = groups along rows of x, 1 = along columns
    uint64_t seed;
    const void *x;        // BF16 [R, C]
    int64_t R, C;
    void *y;              // BF16 [R, C] or null
    void *yt;             // column axis only: BF16 [C, R] (y transposed) or null
    void *codes;          // or null
    void *scales;         // or null
    float *outer;         // or null
    void *keep = nullptr; // uint8 [R, C/8] STE keep mask in the layout of x, or null
    int rht_n = 0;        // 16 / 128: quantize the random Hadamard rotation of x along
    uint64_t rht_seed = 0; //  the quantization axis (not with the per-tensor format)
    uint32_t *partials;   // kAbsmaxPartials words (NV per-tensor only)
    bool cached_outputs;  // ordinary stores (outputs re-read right away) instead of streaming
    // column axis only: retained FP8 channels (columns of x; bit mask [C/8])
    // and their FP32 scales [C], or null
    const void *retain = nullptr;
    const float *chan_scale = nullptr;
};

// Partial maxima of |x| for the per-tensor NVFP4 scale; with retain (bit
// c mod 8 of byte c / 8 for column c of a row of `cols` elements) the
// retained columns are left out.
hipError_t launch_absmax(const void *x, int64_t n_elems, uint32_t *partials,
                         uint32_t *npart_out, hipStream_t stream,
                         const void *retain = nullptr, int64_t cols = 0);
// The partial maxima of two tensors in one launch (no retained columns).
hipError_t launch_absmax_pair(const void *x0, int64_t n0, uint32_t *partials0, uint32_t *npart0,
                              const void *x1, int64_t n1, uint32_t *partials1, uint32_t *npart1,
                              hipStream_t stream);
hipError_t launch_quant(const QuantArgs &a, uint32_t npart, hipStream_t stream);
hipError_t launch_dequant(int fmt, int col, const void *codes, const void *scales,
                          const float *outer, int64_t R, int64_t C, void *y,
                          hipStream_t stream);
// dx = dy where the keep bit (bit c mod 8 of byte (r, c / 8)) is set, else +0.
hipError_t launch_ste_mask(const void *keep, const void *dy, int64_t R, int64_t C, void *dx,
                           hipStream_t stream);
hipError_t launch_ste(int fmt, int col, const void *x, const void *scales,
                      const float *outer, const void *dy, int64_t R, int64_t C,
                      void *dx, hipStream_t stream);
// MXFP4 product on the scaled FP4 matrix cores: C [M, N] BF16 = A . B^T with
// A given as E2M1 codes [M, K/2] and E8M0 scales [M, K/32], B as codes
// [N, K/2] and scales [N, K/32]; K a multiple of 64.
struct Fp4Operands {
    const void *a_codes, *a_scales, *b_codes, *b_scales;
    void *c;
    int64_t M, N, K;
    const void *keep = nullptr;   // optional STE keep mask of c (elements zeroed where clear)
};
hipError_t launch_gemm_mxfp4_nt_pair(const Fp4Operands &o0, const Fp4Operands &o1, int count,
                                     hipStream_t stream);

// Random Hadamard transform of x [R, C] in blocks of n (16 or 128) along the
// rows (col = 0) or the columns (col = 1) into y (same layout).
hipError_t launch_hadamard(const void *x, int64_t R, int64_t C, int col, int n, uint64_t seed,
                           void *y, bool cached, hipStream_t stream);
hipError_t launch_gemm_bf16_nt(const void *a, const void *bt, void *c, int64_t M,
                               int64_t N, int64_t K, hipStream_t stream);
// Two independent products C0 = A0 * Bt0^T and C1 = A1 * Bt1^T in one launch.
// keep0 / keep1: optional STE keep masks of c0 / c1 (bit n mod 8 of byte n / 8
// for element n of C in row-major order); clear bits store +0.
hipError_t launch_gemm_bf16_nt_pair(const void *a0, const void *bt0, void *c0, int64_t M0,
                                    int64_t N0, int64_t K0, const void *a1, const void *bt1,
                                    void *c1, int64_t M1, int64_t N1, int64_t K1,
                                    hipStream_t stream, const void *keep0 = nullptr,
                                    const void *keep1 = nullptr);

// TetraJet-v2 sec. 2.B / 2.C (fq_outcontrol.hip).  n is a multiple of 4.
hipError_t launch_osci_track(const float *w, const void *q, float *w_prev, void *q_prev,
                             float *dist_m, float *dist_q, int64_t n, int first,
                             hipStream_t stream);
struct OsciResetArgs {
    float *w;                // FP32 [R, C] master weight (n = R * C elements)
    const void *q;           // BF16 [R, C] quantized weight
    float *w_prev;
    void *q_prev;
    float *dist_m, *dist_q;
    int64_t n, R, C;
    float tau;
    bool grid_target;        // reset to q instead of the bin centre
    int fmt;                 // FMT_* of the quantization that gave q (bin-centre target)
    bool col;                // its axis
    const void *codes, *scales;
    const float *outer;
};
hipError_t launch_osci_reset(const OsciResetArgs &a, hipStream_t stream);
hipError_t launch_channel_absmax(const void *x, int64_t R, int64_t C, uint32_t *amax,
                                 hipStream_t stream);
hipError_t launch_select_channels(const uint32_t *amax, int64_t C, int64_t k, void *retain,
                                  float *chan_scale, hipStream_t stream);
// Row-axis fake quantization with retained FP8 channels (any format; the
// per-tensor one takes `npart` partial maxima over the other channels).
struct RetainArgs {
    int fmt;                 // FMT_*
    int sr;
    uint64_t seed;
    const void *x;           // BF16 [R, C]
    int64_t R, C;
    const void *retain;      // uint8 [C/8] channel bit mask
    const float *chan_scale; // FP32 [C]
    void *y, *codes, *scales;
    float *outer;
    void *keep = nullptr;          // STE keep mask [R, C/8] or null
    const uint32_t *partials = nullptr;
    uint32_t npart = 0;
    bool cached_outputs = false;
};
hipError_t launch_quant_retain(const RetainArgs &a, hipStream_t stream);

// ---- row operators around the quantized linears ------------------------------
enum { F8_NONE = 0, F8_MX = 1, F8_ROW = 2 };       // FQ_F8_* of fq.h

// fq_norm.hip
constexpr int64_t kNormMaxCols = 32768;
struct NormFwdArgs {
    const void *x;           // BF16 [rows, cols]
    const void *res;         // the stream, BF16 or FP32 [rows, cols], or null
    int stream_f32;
    const void *gamma;       // BF16 or FP32 [cols]
    int gamma_f32;
    float eps;
    int64_t rows, cols;
    int f8;                  // F8_*
    void *h;                 // x + res in the stream's type (may be res), with res only
    void *y;                 // BF16 or null
    void *codes;             // E4M3 or null
    void *scales;            // E8M0 [rows, cols / 32] or FP32 [rows], or null
    float *rstd;             // FP32 [rows] or null
};
hipError_t launch_rmsnorm_fwd(const NormFwdArgs &a, hipStream_t stream);
struct NormBwdArgs {
    const void *dy;          // BF16
    const void *h;           // the normalized values, BF16 or FP32
    int stream_f32;
    const void *gamma;
    int gamma_f32;
    const float *rstd;
    const void *dres;        // gradient of h from elsewhere, in h's type, or null
    int64_t rows, cols;
    void *dh;                // in h's type (may be dres)
    void *dx;                // BF16 copy of dh, or null
    float *dgamma;           // FP32 [cols] or null
    float *partials;         // groups * cols column sums (workspace)
    int64_t groups;          // set by the launcher, as the next
    bool few;                // rows and dgamma in one launch
};
// groups of column sums the backward leaves (its workspace holds as many rows)
int64_t rmsnorm_bwd_groups(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_bwd(NormBwdArgs a, hipStream_t stream);

// fq_moe.hip
constexpr int kMoeMaxExperts = 1024;
constexpr int64_t kMoeMaxChunks = 256;      // workgroups of the sort
struct MoeSortArgs {
    const int32_t *ids;      // [n] expert of each assignment
    int64_t n;
    uint32_t E, align;
    int64_t rows;            // of the sorted order, padding included
    int32_t *offsets;        // [E + 1]
    int32_t *pos;            // [n]
    int32_t *src;            // [rows]
    uint32_t *ws;            // counts of every chunk and expert (not for few assignments)
    uint32_t chunk;
};
size_t moe_sort_counts(int64_t n, int64_t E);   // counts that the workspace holds
hipError_t launch_moe_sort(MoeSortArgs a, hipStream_t stream);
struct MoeRowsArgs {
    int64_t T, k, H, rows;
    const int32_t *pos;      // [T, k]
    const int32_t *src;      // [rows]
    const float *weights;    // [T, k] or null
    const void *x;           // dispatch: BF16 or E4M3 [T, H]
    const void *scales;      // dispatch: E8M0 [T, H / 32] or FP32 [T]
    const void *y;           // BF16 [rows, H]
    const void *dout;        // BF16 [T, H]
    void *rows_out;          // dispatch's y, combine_bwd's dy: BF16 [rows, H]
    void *out;               // combine's BF16 [T, H]
    float *dweights;         // [T, k]
};
hipError_t launch_moe_dispatch(int f8, const MoeRowsArgs &a, hipStream_t stream);
hipError_t launch_moe_combine(const MoeRowsArgs &a, hipStream_t stream);
hipError_t launch_moe_combine_bwd(const MoeRowsArgs &a, hipStream_t stream);

// fq_adamw.hip
constexpr uint32_t kAdamWTensors = 32;      // of one launch whose table is its arguments
struct AdamWTensor {
    float *w;
    void *w_bf16;            // or null
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
    float lr_mult, weight_decay;
    int g_f32;
};
constexpr uint32_t kAdamWDivideFrom = 0x67000001u;      // the next FP32 above 2^79
struct AdamWStep {           // what all tensors of a launch share
    uint32_t count;          // tensors of this launch, all with n > 0
    uint32_t tiles;          // of all of them
    float lr, beta1, one_beta1, beta2, one_beta2, eps, inv_bc1, inv_sqrt_bc2;
    const float *grad_scale; // device scalar or null
    uint32_t step, seed_lo, seed_hi;
    uint32_t divide_from;    // bits of the smallest v of a correctly rounded update
};
struct AdamWArgs {
    AdamWStep step;
    uint32_t first[kAdamWTensors];          // first tile of each tensor
    uint32_t index[kAdamWTensors];          // number of each tensor in the whole list
    AdamWTensor t[kAdamWTensors];
};
static_assert(sizeof(AdamWTensor) == 80 && sizeof(AdamWArgs) <= 2880, "of 4 KB of arguments");
uint32_t adamw_tile(bool f8);               // elements of a workgroup
uint32_t adamw_tiles(int64_t n, bool f8);   // tiles that n elements take
constexpr uint64_t kAdamWMaxTiles = uint64_t(1) << 31;      // of one launch
hipError_t launch_adamw(const AdamWArgs &a, bool f8, hipStream_t stream);
// The same with the table in device memory.
hipError_t launch_adamw_plan(const AdamWStep &a, const AdamWTensor *t, const uint32_t *first,
                             const uint32_t *index, bool f8, hipStream_t stream);

}  // namespace fqimpl
