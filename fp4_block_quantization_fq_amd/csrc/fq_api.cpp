// fq_api.cpp -- the C ABI of libfq.so (declared in include/fq.h).
//
// Every entry point validates its arguments completely before touching the
// device: a rejected call enqueues nothing and writes nothing.  Accepted calls
// enqueue kernels on the caller's stream and return; launch failures are
// reported as FQ_ERR_DEVICE.  No exception crosses the boundary.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "fq.h"
#include "fq_internal.h"

namespace {

thread_local char g_err[512] = "";

fq_status fail(fq_status s, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return s;
}

fq_status ok()
{
    g_err[0] = '\0';
    return FQ_OK;
}

constexpr int64_t kMaxElems = int64_t(1) << 34;
// every dimension fits the kernels' 32-bit row/column arguments and the
// products' int tile arithmetic
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

struct Fmt {
    int fmt;   // fqimpl::FMT_*
    int B;     // block size
};

fq_status check_desc(const fq_desc *d, Fmt *out, const char *name)
{
    if (!d) return fail(FQ_ERR_NULL, "%s is NULL", name);
    if (d->reserved != 0) return fail(FQ_ERR_DESC, "%s->reserved must be 0", name);
    if (d->rounding != FQ_ROUND_RNE && d->rounding != FQ_ROUND_SR)
        return fail(FQ_ERR_DESC, "%s->rounding=%d is not FQ_ROUND_RNE/SR", name, d->rounding);
    if (d->axis != FQ_AXIS_ROW && d->axis != FQ_AXIS_COL)
        return fail(FQ_ERR_DESC, "%s->axis=%d is not FQ_AXIS_ROW/COL", name, d->axis);
    if (d->block_size == 32 && d->scale_type == FQ_SCALE_E8M0 && d->outer == FQ_OUTER_NONE) {
        *out = {fqimpl::FMT_MX, 32};
        return FQ_OK;
    }
    if (d->block_size == 16 && d->scale_type == FQ_SCALE_E4M3) {
        if (d->outer == FQ_OUTER_TENSOR) {
            *out = {fqimpl::FMT_NVT, 16};
            return FQ_OK;
        }
        if (d->outer == FQ_OUTER_BLOCK128) {
            *out = {fqimpl::FMT_NV128, 16};
            return FQ_OK;
        }
    }
    return fail(FQ_ERR_DESC,
                "%s: unsupported format {block_size=%d, scale_type=%d, outer=%d}; valid: "
                "MXFP4 {32, E8M0, NONE}, NVFP4 {16, E4M3, TENSOR|BLOCK128}",
                name, d->block_size, d->scale_type, d->outer);
}

fq_status check_shape(const Fmt &f, int axis, int64_t R, int64_t C)
{
    if (R < 1 || C < 1) return fail(FQ_ERR_SHAPE, "rows=%lld cols=%lld must be >= 1",
                                    (long long)R, (long long)C);
    if (R > kMaxDim || C > kMaxDim || R * C > kMaxElems)
        return fail(FQ_ERR_SHAPE, "rows=%lld cols=%lld: each must be below 2^31 and rows*cols at most 2^34", (long long)R,
                    (long long)C);
    const int64_t q = (axis == FQ_AXIS_ROW) ? C : R;    // quantized axis length
    const char *qn = (axis == FQ_AXIS_ROW) ? "cols" : "rows";
    if (q % f.B != 0)
        return fail(FQ_ERR_SHAPE, "%s=%lld must be a multiple of the block size %d", qn,
                    (long long)q, f.B);
    if (f.fmt == fqimpl::FMT_NV128 && q % 128 != 0)
        return fail(FQ_ERR_SHAPE, "%s=%lld must be a multiple of the 128-element outer block",
                    qn, (long long)q);
    if (axis == FQ_AXIS_COL && C % 8 != 0)
        return fail(FQ_ERR_SHAPE, "cols=%lld must be a multiple of 8 for FQ_AXIS_COL",
                    (long long)C);
    return FQ_OK;
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

fq_status check_ptr(const void *p, const char *name, bool required, uintptr_t align = 16)
{
    if (!p) {
        if (required) return fail(FQ_ERR_NULL, "%s is NULL", name);
        return FQ_OK;
    }
    if (!aligned(p, align))
        return fail(FQ_ERR_ALIGN, "%s=%p is not %u-byte aligned", name, p, (unsigned)align);
    return FQ_OK;
}

size_t quant_ws(const Fmt &f)
{
    return f.fmt == fqimpl::FMT_NVT ? fqimpl::kAbsmaxPartials * sizeof(uint32_t) : 0;
}

fq_status device_status(hipError_t e, const char *what)
{
    if (e != hipSuccess)
        return fail(FQ_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
    return ok();
}

#define FQ_TRY(expr)                       \
    do {                                   \
        fq_status _s = (expr);             \
        if (_s != FQ_OK) return _s;        \
    } while (0)

// Shared body of fq_quantize / fq_fake_quant once arguments are checked.
fq_status run_quant(const Fmt &f, const fq_desc *d, const void *x, int64_t R, int64_t C,
                    void *y, void *codes, void *scales, float *outer, void *ws,
                    hipStream_t st, bool cached = false, void *keep = nullptr, int rht_n = 0,
                    uint64_t rht_seed = 0, int64_t npart_given = -1)
{
    fqimpl::QuantArgs a;
    a.fmt = f.fmt;
    a.sr = d->rounding == FQ_ROUND_SR;
    a.col = d->axis == FQ_AXIS_COL;
    a.seed = d->seed;
    a.x = x;
    a.R = R;
    a.C = C;
    a.y = y;
    a.codes = codes;
    a.scales = scales;
    a.outer = (f.fmt == fqimpl::FMT_MX) ? nullptr : outer;
    a.yt = nullptr;
    a.partials = (uint32_t *)ws;
    a.keep = keep;
    a.rht_n = rht_n;
    a.rht_seed = rht_seed;
    a.cached_outputs = cached;
    // npart_given >= 0: the per-tensor partial maxima are already in ws
    uint32_t npart = npart_given >= 0 ? (uint32_t)npart_given : 0u;
    if (f.fmt == fqimpl::FMT_NVT && npart_given < 0) {
        hipError_t e = fqimpl::launch_absmax(x, R * C, a.partials, &npart, st);
        if (e != hipSuccess) return device_status(e, "tensor absmax launch");
    }
    return device_status(fqimpl::launch_quant(a, npart, st), "quantize launch");
}

}  // namespace

extern "C" {

fq_desc fq_desc_mxfp4(void)
{
    fq_desc d;
    std::memset(&d, 0, sizeof(d));
    d.block_size = 32;
    d.scale_type = FQ_SCALE_E8M0;
    d.outer = FQ_OUTER_NONE;
    d.rounding = FQ_ROUND_RNE;
    d.axis = FQ_AXIS_ROW;
    return d;
}

fq_desc fq_desc_nvfp4(void)
{
    fq_desc d;
    std::memset(&d, 0, sizeof(d));
    d.block_size = 16;
    d.scale_type = FQ_SCALE_E4M3;
    d.outer = FQ_OUTER_TENSOR;
    d.rounding = FQ_ROUND_RNE;
    d.axis = FQ_AXIS_ROW;
    return d;
}

size_t fq_workspace_size(const fq_desc *desc, int64_t rows, int64_t cols)
{
    (void)rows;
    (void)cols;
    Fmt f;
    if (check_desc(desc, &f, "desc") != FQ_OK) return 0;
    return quant_ws(f);
}

fq_status fq_quantize(const fq_desc *desc, const void *x_bf16, int64_t rows, int64_t cols,
                      void *codes, void *scales, float *outer, void *ws, size_t ws_bytes,
                      void *stream)
{
    Fmt f;
    FQ_TRY(check_desc(desc, &f, "desc"));
    FQ_TRY(check_shape(f, desc->axis, rows, cols));
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(codes, "codes", true));
    FQ_TRY(check_ptr(scales, "scales", true));
    if (f.fmt != fqimpl::FMT_MX) FQ_TRY(check_ptr(outer, "outer", true, 4));
    const size_t need = quant_ws(f);
    if (need) {
        FQ_TRY(check_ptr(ws, "ws", true));
        if (ws_bytes < need)
            return fail(FQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
    }
    return run_quant(f, desc, x_bf16, rows, cols, nullptr, codes, scales, outer, ws,
                     (hipStream_t)stream);
}

fq_status fq_dequantize(const fq_desc *desc, const void *codes, const void *scales,
                        const float *outer, int64_t rows, int64_t cols, void *y_bf16,
                        void *stream)
{
    Fmt f;
    FQ_TRY(check_desc(desc, &f, "desc"));
    FQ_TRY(check_shape(f, desc->axis, rows, cols));
    FQ_TRY(check_ptr(codes, "codes", true));
    FQ_TRY(check_ptr(scales, "scales", true));
    if (f.fmt != fqimpl::FMT_MX) FQ_TRY(check_ptr(outer, "outer", true, 4));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    return device_status(
        fqimpl::launch_dequant(f.fmt, desc->axis == FQ_AXIS_COL, codes, scales,
                               f.fmt == fqimpl::FMT_MX ? nullptr : outer, rows, cols, y_bf16,
                               (hipStream_t)stream),
        "dequantize launch");
}

fq_status fq_fake_quant(const fq_desc *desc, const void *x_bf16, int64_t rows, int64_t cols,
                        void *y_bf16, void *codes, void *scales, float *outer, void *ws,
                        size_t ws_bytes, void *stream)
{
    Fmt f;
    FQ_TRY(check_desc(desc, &f, "desc"));
    FQ_TRY(check_shape(f, desc->axis, rows, cols));
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    FQ_TRY(check_ptr(codes, "codes", false));
    FQ_TRY(check_ptr(scales, "scales", false));
    FQ_TRY(check_ptr(outer, "outer", false, 4));
    const size_t need = quant_ws(f);
    if (need) {
        FQ_TRY(check_ptr(ws, "ws", true));
        if (ws_bytes < need)
            return fail(FQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
    }
    return run_quant(f, desc, x_bf16, rows, cols, y_bf16, codes, scales, outer, ws,
                     (hipStream_t)stream);
}

}  // extern "C"

// ---- the entry point that allocates nothing --------------------------------
// The per-tensor maximum's partials live in this library-owned device array
// instead of a caller workspace.  Each GPU holds its own copy (allocated with
// the code object, kept until the process ends); its address on a device is
// looked up once, with that device current, and only that address is ever
// handed to kernels.  Nothing in it needs clearing: the maximum pass writes
// every partial the quantizer then reads.  Calls that overlap on one GPU share
// it and race.
namespace {

constexpr size_t kStaticScratchBytes = fqimpl::kAbsmaxPartials * sizeof(uint32_t);   // 4 KB
static __device__ __align__(256) uint32_t scratch[fqimpl::kAbsmaxPartials];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices];          // per device, null until looked up

fq_status device_scratch(void **out)
{
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return device_status(e, "hipGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(FQ_ERR_DEVICE, "device %d beyond the %d this library tracks", dev, kMaxDevices);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || !p) return device_status(e, "scratch symbol lookup");
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return FQ_OK;
}

}  // namespace

extern "C" {

fq_status fq_fake_quant_noalloc(const fq_desc *desc, const void *x_bf16, int64_t rows,
                                int64_t cols, void *y_bf16, void *codes, void *scales,
                                float *outer, void *stream)
{
    Fmt f;
    FQ_TRY(check_desc(desc, &f, "desc"));
    FQ_TRY(check_shape(f, desc->axis, rows, cols));
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    FQ_TRY(check_ptr(codes, "codes", false));
    FQ_TRY(check_ptr(scales, "scales", false));
    FQ_TRY(check_ptr(outer, "outer", false, 4));
    const size_t need = quant_ws(f);
    if (need > kStaticScratchBytes)
        return fail(FQ_ERR_WORKSPACE, "needs %zu bytes of scratch, the static array holds %zu",
                    need, kStaticScratchBytes);
    void *ws = nullptr;
    if (need) FQ_TRY(device_scratch(&ws));
    return run_quant(f, desc, x_bf16, rows, cols, y_bf16, codes, scales, outer, ws,
                     (hipStream_t)stream);
}

fq_status fq_fake_quant_mask(const fq_desc *desc, const void *x_bf16, int64_t rows,
                             int64_t cols, void *y_bf16, void *codes, void *scales,
                             float *outer, void *keep, void *ws, size_t ws_bytes, void *stream)
{
    Fmt f;
    FQ_TRY(check_desc(desc, &f, "desc"));
    FQ_TRY(check_shape(f, desc->axis, rows, cols));
    if (cols % 8 != 0)
        return fail(FQ_ERR_SHAPE, "cols=%lld must be a multiple of 8 for the keep mask",
                    (long long)cols);
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    FQ_TRY(check_ptr(codes, "codes", false));
    FQ_TRY(check_ptr(scales, "scales", false));
    FQ_TRY(check_ptr(outer, "outer", false, 4));
    FQ_TRY(check_ptr(keep, "keep", true));
    const size_t need = quant_ws(f);
    if (need) {
        FQ_TRY(check_ptr(ws, "ws", true));
        if (ws_bytes < need)
            return fail(FQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
    }
    return run_quant(f, desc, x_bf16, rows, cols, y_bf16, codes, scales, outer, ws,
                     (hipStream_t)stream, false, keep);
}

fq_status fq_fake_quant_rht(const fq_desc *desc, const void *x_bf16, int64_t rows, int64_t cols,
                            int32_t rht_block, uint64_t rht_seed, void *y_bf16, void *codes,
                            void *scales, float *outer, void *stream)
{
    Fmt f;
    FQ_TRY(check_desc(desc, &f, "desc"));
    if (f.fmt == fqimpl::FMT_NVT)
        return fail(FQ_ERR_DESC, "the rotated quantizer takes MXFP4 or NVFP4 FQ_OUTER_BLOCK128");
    if (rht_block != 16 && rht_block != 128)
        return fail(FQ_ERR_DESC, "rht_block=%d is not 16 or 128", rht_block);
    FQ_TRY(check_shape(f, desc->axis, rows, cols));
    const int64_t q = desc->axis == FQ_AXIS_ROW ? cols : rows;
    if (q % rht_block != 0)
        return fail(FQ_ERR_SHAPE, "%s=%lld must be a multiple of rht_block=%d",
                    desc->axis == FQ_AXIS_ROW ? "cols" : "rows", (long long)q, rht_block);
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    FQ_TRY(check_ptr(codes, "codes", false));
    FQ_TRY(check_ptr(scales, "scales", false));
    FQ_TRY(check_ptr(outer, "outer", false, 4));
    return run_quant(f, desc, x_bf16, rows, cols, y_bf16, codes, scales, outer, nullptr,
                     (hipStream_t)stream, false, nullptr, rht_block, rht_seed);
}

fq_status fq_ste_backward_mask(const void *keep, const void *dy_bf16, int64_t rows,
                               int64_t cols, void *dx_bf16, void *stream)
{
    if (rows < 1 || cols < 8 || cols % 8 != 0)
        return fail(FQ_ERR_SHAPE, "rows=%lld must be >= 1 and cols=%lld a positive multiple of 8",
                    (long long)rows, (long long)cols);
    if (rows > kMaxDim || cols > kMaxDim || rows * cols > kMaxElems)
        return fail(FQ_ERR_SHAPE, "rows=%lld cols=%lld: each must be below 2^31 and rows*cols at most 2^34", (long long)rows,
                    (long long)cols);
    FQ_TRY(check_ptr(keep, "keep", true));
    FQ_TRY(check_ptr(dy_bf16, "dy", true));
    FQ_TRY(check_ptr(dx_bf16, "dx", true));
    return device_status(fqimpl::launch_ste_mask(keep, dy_bf16, rows, cols, dx_bf16,
                                                 (hipStream_t)stream),
                         "ste mask launch");
}

fq_status fq_ste_backward(const fq_desc *desc, const void *x_bf16, const void *scales,
                          const float *outer, const void *dy_bf16, int64_t rows,
                          int64_t cols, void *dx_bf16, void *stream)
{
    Fmt f;
    FQ_TRY(check_desc(desc, &f, "desc"));
    FQ_TRY(check_shape(f, desc->axis, rows, cols));
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(scales, "scales", true));
    if (f.fmt != fqimpl::FMT_MX) FQ_TRY(check_ptr(outer, "outer", true, 4));
    FQ_TRY(check_ptr(dy_bf16, "dy", true));
    FQ_TRY(check_ptr(dx_bf16, "dx", true));
    return device_status(
        fqimpl::launch_ste(f.fmt, desc->axis == FQ_AXIS_COL, x_bf16, scales,
                           f.fmt == fqimpl::FMT_MX ? nullptr : outer, dy_bf16, rows, cols,
                           dx_bf16, (hipStream_t)stream),
        "ste launch");
}

// qlinear workspace: X_hat [M, K], W_hat^T [N, K] (BF16), reduction scratch.
static size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// The MXFP4 x MXFP4 linear keeps codes and scales instead of BF16 operands,
// inside the same workspace: X codes [M, K/2], X scales [M, K/32], W codes
// and scales in the transposed layout [N, K/2], [N, K/32].
struct MxLinLayout {
    size_t xc, xs, wc, wsc;
};
static MxLinLayout mx_lin_layout(int64_t M, int64_t K, int64_t N)
{
    MxLinLayout L;
    L.xc = 0;
    L.xs = round256((size_t)M * K / 2);
    L.wc = L.xs + round256((size_t)M * K / 32);
    L.wsc = L.wc + round256((size_t)N * K / 2);
    return L;
}

size_t fq_qlinear_workspace_size(const fq_desc *desc_x, const fq_desc *desc_w, int64_t M,
                                 int64_t K, int64_t N)
{
    (void)desc_x;
    (void)desc_w;
    if (M < 1 || K < 1 || N < 1 || M > kMaxDim || K > kMaxDim || N > kMaxDim) return 0;
    if (M * K > kMaxElems || K * N > kMaxElems) return 0;
    return round256((size_t)M * K * 2) + round256((size_t)N * K * 2) +
           2 * fqimpl::kAbsmaxPartials * sizeof(uint32_t);
}

// Retained-channel fake quantization along either axis (shared by
// fq_fake_quant_retain and the linear's retained paths): the per-tensor
// format's maximum pass leaves the retained columns out.
static fq_status run_quant_retain(const Fmt &f, const fq_desc *d, uint64_t seed, const void *x,
                                  int64_t R, int64_t C, void *y, void *yt, void *codes,
                                  void *scales, float *outer, void *keep, const void *retain,
                                  const float *chan_scale, uint32_t *parts, hipStream_t st,
                                  bool cached)
{
    uint32_t npart = 0;
    if (f.fmt == fqimpl::FMT_NVT) {
        hipError_t e = fqimpl::launch_absmax(x, R * C, parts, &npart, st, retain, C);
        if (e != hipSuccess) return device_status(e, "masked tensor absmax launch");
    }
    if (d->axis == FQ_AXIS_ROW) {
        fqimpl::RetainArgs a;
        a.fmt = f.fmt;
        a.sr = d->rounding == FQ_ROUND_SR;
        a.seed = seed;
        a.x = x;
        a.R = R;
        a.C = C;
        a.retain = retain;
        a.chan_scale = chan_scale;
        a.y = y;
        a.codes = codes;
        a.scales = scales;
        a.outer = f.fmt == fqimpl::FMT_MX ? nullptr : outer;
        a.keep = keep;
        a.partials = parts;
        a.npart = npart;
        a.cached_outputs = cached;
        return device_status(fqimpl::launch_quant_retain(a, st), "retain quantize launch");
    }
    fqimpl::QuantArgs a;
    a.fmt = f.fmt;
    a.sr = d->rounding == FQ_ROUND_SR;
    a.col = 1;
    a.seed = seed;
    a.x = x;
    a.R = R;
    a.C = C;
    a.y = y;
    a.yt = yt;
    a.codes = codes;
    a.scales = scales;
    a.outer = f.fmt == fqimpl::FMT_MX ? nullptr : outer;
    a.keep = keep;
    a.partials = parts;
    a.cached_outputs = cached;
    a.retain = retain;
    a.chan_scale = chan_scale;
    return device_status(fqimpl::launch_quant(a, npart, st), "retain quantize launch");
}

// The forward; retain / chan_scale (or null) keep the activation's retained
// channels (columns of X) in FP8.
static fq_status qlinear_fwd_impl(const fq_desc *desc_x, const fq_desc *desc_w,
                                  const void *x_bf16, const void *w_bf16, int64_t M, int64_t K,
                                  int64_t N, void *y_bf16, void *ws, size_t ws_bytes,
                                  void *stream, const void *retain, const float *chan_scale)
{
    Fmt fx, fw;
    FQ_TRY(check_desc(desc_x, &fx, "desc_x"));
    FQ_TRY(check_desc(desc_w, &fw, "desc_w"));
    if (desc_x->axis != FQ_AXIS_ROW)
        return fail(FQ_ERR_DESC, "desc_x->axis must be FQ_AXIS_ROW (groups along K)");
    if (desc_w->axis != FQ_AXIS_COL)
        return fail(FQ_ERR_DESC, "desc_w->axis must be FQ_AXIS_COL (groups along K)");
    if (M < 1 || K < 1 || N < 1)
        return fail(FQ_ERR_SHAPE, "M=%lld K=%lld N=%lld must be >= 1", (long long)M,
                    (long long)K, (long long)N);
    FQ_TRY(check_shape(fx, FQ_AXIS_ROW, M, K));
    FQ_TRY(check_shape(fw, FQ_AXIS_COL, K, N));
    if (K % 64 != 0)
        return fail(FQ_ERR_SHAPE, "K=%lld must be a multiple of 64", (long long)K);
    if (M * N > kMaxElems)
        return fail(FQ_ERR_SHAPE, "M*N exceeds 2^34 elements");
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(w_bf16, "w", true));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    FQ_TRY(check_ptr(ws, "ws", true));
    const size_t need = fq_qlinear_workspace_size(desc_x, desc_w, M, K, N);
    if (ws_bytes < need)
        return fail(FQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);

    char *base = (char *)ws;
    hipStream_t st = (hipStream_t)stream;
    uint32_t *parts = (uint32_t *)(base + round256((size_t)M * K * 2) + round256((size_t)N * K * 2));

    if (retain) {
        FQ_TRY(check_ptr(retain, "retain", true, 1));
        FQ_TRY(check_ptr(chan_scale, "chan_scale", true));
    }
    if (fx.fmt == fqimpl::FMT_MX && fw.fmt == fqimpl::FMT_MX && K % 64 == 0 && !retain) {
        // MXFP4 x MXFP4: the codes and E8M0 scales go straight to the scaled
        // FP4 matrix cores, nothing is dequantized
        const MxLinLayout L = mx_lin_layout(M, K, N);
        FQ_TRY(run_quant(fx, desc_x, x_bf16, M, K, nullptr, base + L.xc, base + L.xs, nullptr,
                         parts, st, /*cached=*/true));
        fqimpl::QuantArgs a;
        a.fmt = fw.fmt;
        a.sr = desc_w->rounding == FQ_ROUND_SR;
        a.col = 1;
        a.seed = desc_w->seed;
        a.x = w_bf16;
        a.R = K;
        a.C = N;
        a.y = nullptr;
        a.yt = nullptr;
        a.codes = base + L.wc;
        a.scales = base + L.wsc;
        a.outer = nullptr;
        a.partials = parts;
        a.cached_outputs = true;
        hipError_t e = fqimpl::launch_quant(a, 0, st);
        if (e != hipSuccess) return device_status(e, "transposed quantize launch");
        fqimpl::Fp4Operands o;
        o.a_codes = base + L.xc;
        o.a_scales = base + L.xs;
        o.b_codes = base + L.wc;
        o.b_scales = base + L.wsc;
        o.c = y_bf16;
        o.M = M;
        o.N = N;
        o.K = K;
        return device_status(fqimpl::launch_gemm_mxfp4_nt_pair(o, o, 1, st), "fp4 gemm launch");
    }

    void *xhat = base;
    char *what_t = base + round256((size_t)M * K * 2);
    uint32_t *parts_w = parts + fqimpl::kAbsmaxPartials;

    // both per-tensor: the two maximum passes in one launch
    int64_t npart_x = -1, npart_w = -1;
    if (fx.fmt == fqimpl::FMT_NVT && fw.fmt == fqimpl::FMT_NVT && !retain) {
        uint32_t nx = 0, nw = 0;
        hipError_t e = fqimpl::launch_absmax_pair(x_bf16, M * K, parts, &nx, w_bf16, K * N,
                                                  parts_w, &nw, st);
        if (e != hipSuccess) return device_status(e, "tensor absmax launch");
        npart_x = nx;
        npart_w = nw;
    }
    // X_hat = FQ(X) along K (rows of X), the retained channels in FP8
    if (retain)
        FQ_TRY(run_quant_retain(fx, desc_x, desc_x->seed, x_bf16, M, K, xhat, nullptr, nullptr,
                                nullptr, nullptr, nullptr, retain, chan_scale, parts, st, true));
    else
        FQ_TRY(run_quant(fx, desc_x, x_bf16, M, K, xhat, nullptr, nullptr, nullptr, parts, st,
                         /*cached=*/true, nullptr, 0, 0, npart_x));
    // W_hat^T: FQ(W) along K (columns of W), written transposed [N, K]
    {
        fqimpl::QuantArgs a;
        a.fmt = fw.fmt;
        a.sr = desc_w->rounding == FQ_ROUND_SR;
        a.col = 1;
        a.seed = desc_w->seed;
        a.x = w_bf16;
        a.R = K;
        a.C = N;
        a.y = nullptr;
        a.codes = nullptr;
        a.scales = nullptr;
        a.outer = nullptr;
        a.partials = parts_w;
        a.cached_outputs = true;
        uint32_t npart = npart_w >= 0 ? (uint32_t)npart_w : 0u;
        if (fw.fmt == fqimpl::FMT_NVT && npart_w < 0) {
            hipError_t e = fqimpl::launch_absmax(w_bf16, K * N, a.partials, &npart, st);
            if (e != hipSuccess) return device_status(e, "tensor absmax launch");
        }
        a.yt = what_t;
        hipError_t e = fqimpl::launch_quant(a, npart, st);
        if (e != hipSuccess) return device_status(e, "transposed quantize launch");
    }
    return device_status(fqimpl::launch_gemm_bf16_nt(xhat, what_t, y_bf16, M, N, K, st),
                         "gemm launch");
}

fq_status fq_qlinear_fwd(const fq_desc *desc_x, const fq_desc *desc_w, const void *x_bf16,
                         const void *w_bf16, int64_t M, int64_t K, int64_t N, void *y_bf16,
                         void *ws, size_t ws_bytes, void *stream)
{
    return qlinear_fwd_impl(desc_x, desc_w, x_bf16, w_bf16, M, K, N, y_bf16, ws, ws_bytes,
                            stream, nullptr, nullptr);
}

fq_status fq_qlinear_fwd_retain(const fq_desc *desc_x, const fq_desc *desc_w, const void *x_bf16,
                                const void *w_bf16, int64_t M, int64_t K, int64_t N,
                                const void *retain, const float *chan_scale, void *y_bf16,
                                void *ws, size_t ws_bytes, void *stream)
{
    if (!retain) return fail(FQ_ERR_NULL, "retain is NULL");
    if (!chan_scale) return fail(FQ_ERR_NULL, "chan_scale is NULL");
    if (K % 8 != 0) return fail(FQ_ERR_SHAPE, "K=%lld must be a multiple of 8", (long long)K);
    return qlinear_fwd_impl(desc_x, desc_w, x_bf16, w_bf16, M, K, N, y_bf16, ws, ws_bytes,
                            stream, retain, chan_scale);
}

// qlinear backward workspace regions, in order (each rounded up to 256 B).
struct BwdLayout {
    size_t xhat, xkeep, what, wkeep, dyq_n, wq_n, xq_mt, dyq_mt, parts, rdy_n, rw_n, rx_m, rdy_m,
        total;
};

// Backward workspace.  X_hat and W_hat are the forward's operands (BF16),
// xkeep / wkeep their STE keep masks (1 bit per element, layout of X and W);
// dyq_n, wq_n, xq_mt, dyq_mt hold the four quantized gradient-product
// operands: BF16 [M, N], [K, N], [K, M], [N, M] (transposed for the last
// two), or, for MXFP4 gradient operands, their codes followed by their E8M0
// scales in the same place (0.53 B instead of 2 B per element).
static BwdLayout bwd_layout(bool rht, int64_t M, int64_t K, int64_t N)
{
    BwdLayout L;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += round256(bytes);
        return at;
    };
    const size_t mk = (size_t)M * K, kn = (size_t)K * N, mn = (size_t)M * N;
    L.xhat = take(mk * 2);
    L.xkeep = take(mk / 8);
    L.what = take(kn * 2);
    L.wkeep = take(kn / 8);
    L.dyq_n = take(mn * 2);
    L.wq_n = take(kn * 2);
    L.xq_mt = take(mk * 2);
    L.dyq_mt = take(mn * 2);
    L.parts = take(2 * fqimpl::kAbsmaxPartials * sizeof(uint32_t));   // X, W
    // rotated operands (random Hadamard transform), only when requested
    L.rdy_n = take(rht ? mn * 2 : 0);
    L.rw_n = take(rht ? kn * 2 : 0);
    L.rx_m = take(rht ? mk * 2 : 0);
    L.rdy_m = take(rht ? mn * 2 : 0);
    L.total = off;
    return L;
}

size_t fq_qlinear_bwd_workspace_size(const fq_desc *desc_x, const fq_desc *desc_w,
                                     const fq_desc *desc_g, int32_t rht_block, int64_t M,
                                     int64_t K, int64_t N)
{
    Fmt fx, fw, fg;
    if (check_desc(desc_x, &fx, "desc_x") != FQ_OK || check_desc(desc_w, &fw, "desc_w") != FQ_OK ||
        check_desc(desc_g, &fg, "desc_g") != FQ_OK)
        return 0;
    if (rht_block != 0 && rht_block != 16 && rht_block != 128) return 0;
    if (M < 1 || K < 1 || N < 1 || M > kMaxDim || K > kMaxDim || N > kMaxDim) return 0;
    // rotated operand buffers only where the rotation cannot be fused into
    // the quantizer (per-tensor gradient format: its maximum needs a pass)
    return bwd_layout(rht_block != 0 && fg.fmt == fqimpl::FMT_NVT, M, K, N).total;
}

fq_status fq_hadamard(const void *x_bf16, int64_t rows, int64_t cols, int32_t axis,
                      int32_t block, uint64_t seed, void *y_bf16, void *stream)
{
    if (axis != FQ_AXIS_ROW && axis != FQ_AXIS_COL)
        return fail(FQ_ERR_DESC, "axis=%d is not FQ_AXIS_ROW/COL", axis);
    if (block != 16 && block != 128) return fail(FQ_ERR_DESC, "block=%d is not 16 or 128", block);
    if (rows < 1 || cols < 1) return fail(FQ_ERR_SHAPE, "rows=%lld cols=%lld must be >= 1",
                                          (long long)rows, (long long)cols);
    if (rows > kMaxDim || cols > kMaxDim || rows * cols > kMaxElems)
        return fail(FQ_ERR_SHAPE, "rows, cols must be below 2^31 and rows*cols at most 2^34");
    const int64_t q = axis == FQ_AXIS_ROW ? cols : rows;
    if (q % block != 0)
        return fail(FQ_ERR_SHAPE, "%s=%lld must be a multiple of the block %d",
                    axis == FQ_AXIS_ROW ? "cols" : "rows", (long long)q, block);
    if (axis == FQ_AXIS_COL && cols % 8 != 0)
        return fail(FQ_ERR_SHAPE, "cols=%lld must be a multiple of 8 for FQ_AXIS_COL",
                    (long long)cols);
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    const char *xb = (const char *)x_bf16, *yb = (const char *)y_bf16;
    const size_t bytes = (size_t)rows * cols * 2;
    if (xb < yb + bytes && yb < xb + bytes) return fail(FQ_ERR_SHAPE, "x and y overlap");
    return device_status(fqimpl::launch_hadamard(x_bf16, rows, cols, axis == FQ_AXIS_COL, block,
                                                 seed, y_bf16, false, (hipStream_t)stream),
                         "hadamard launch");
}

// One quantizer pass of the backward: src [R, C] along rows (col = false,
// output y [R, C]) or along columns (col = true, output the transpose
// yt [C, R]); optional codes/scales in the pass's own layout and an optional
// keep mask in the layout of src.
static fq_status bwd_quant(const Fmt &f, const fq_desc *d, uint64_t seed, bool col,
                           const void *src, int64_t R, int64_t C, void *y, void *yt,
                           void *codes, void *scales, void *keep, uint32_t *parts,
                           hipStream_t st, int rht_n = 0, uint64_t rht_seed = 0,
                           int64_t npart_given = -1)
{
    fqimpl::QuantArgs a;
    a.fmt = f.fmt;
    a.sr = d->rounding == FQ_ROUND_SR;
    a.col = col ? 1 : 0;
    a.seed = seed;
    a.x = src;
    a.R = R;
    a.C = C;
    a.y = y;
    a.yt = yt;
    a.codes = codes;
    a.scales = scales;
    a.outer = nullptr;
    a.keep = keep;
    a.rht_n = rht_n;
    a.rht_seed = rht_seed;
    a.partials = parts;
    a.cached_outputs = true;
    // npart_given >= 0: the per-tensor partial maxima are already in parts
    uint32_t npart = npart_given >= 0 ? (uint32_t)npart_given : 0u;
    if (f.fmt == fqimpl::FMT_NVT && npart_given < 0) {
        hipError_t e = fqimpl::launch_absmax(src, R * C, parts, &npart, st);
        if (e != hipSuccess) return device_status(e, "tensor absmax launch");
    }
    return device_status(fqimpl::launch_quant(a, npart, st), "quantize launch");
}

// The backward; retain / chan_scale (or null): the activation's retained
// channels stay FP8 in X_hat and in X_hat's quantization along M, and their
// STE keep bits follow the FP8 test.
static fq_status qlinear_bwd_impl(const fq_desc *desc_x, const fq_desc *desc_w,
                                  const fq_desc *desc_g, int32_t rht_block, uint64_t rht_seed,
                                  const void *x_bf16, const void *w_bf16, const void *dy_bf16,
                                  int64_t M, int64_t K, int64_t N, void *dx_bf16, void *dw_bf16,
                                  void *ws, size_t ws_bytes, void *stream, const void *retain,
                                  const float *chan_scale)
{
    Fmt fx, fw, fg;
    FQ_TRY(check_desc(desc_x, &fx, "desc_x"));
    FQ_TRY(check_desc(desc_w, &fw, "desc_w"));
    FQ_TRY(check_desc(desc_g, &fg, "desc_g"));
    if (desc_x->axis != FQ_AXIS_ROW)
        return fail(FQ_ERR_DESC, "desc_x->axis must be FQ_AXIS_ROW (groups along K)");
    if (desc_w->axis != FQ_AXIS_COL)
        return fail(FQ_ERR_DESC, "desc_w->axis must be FQ_AXIS_COL (groups along K)");
    if (M < 1 || K < 1 || N < 1)
        return fail(FQ_ERR_SHAPE, "M=%lld K=%lld N=%lld must be >= 1", (long long)M,
                    (long long)K, (long long)N);
    // forward quantizations (X along K, W along K) and the four backward ones
    FQ_TRY(check_shape(fx, FQ_AXIS_ROW, M, K));
    FQ_TRY(check_shape(fw, FQ_AXIS_COL, K, N));
    FQ_TRY(check_shape(fg, FQ_AXIS_ROW, M, N));     // dY along N
    FQ_TRY(check_shape(fg, FQ_AXIS_ROW, K, N));     // W_hat along N
    FQ_TRY(check_shape(fg, FQ_AXIS_COL, M, K));     // X_hat along M
    FQ_TRY(check_shape(fg, FQ_AXIS_COL, M, N));     // dY along M
    if (M % 64 != 0 || N % 64 != 0)
        return fail(FQ_ERR_SHAPE, "M=%lld and N=%lld must be multiples of 64 (contractions)",
                    (long long)M, (long long)N);
    if (rht_block != 0 && rht_block != 16 && rht_block != 128)
        return fail(FQ_ERR_DESC, "rht_block=%d is not 0, 16 or 128", rht_block);
    if (rht_block != 0 && (M % rht_block != 0 || N % rht_block != 0))
        return fail(FQ_ERR_SHAPE, "M=%lld and N=%lld must be multiples of rht_block=%d",
                    (long long)M, (long long)N, rht_block);
    if (M * N > kMaxElems)
        return fail(FQ_ERR_SHAPE, "M*N exceeds 2^34 elements");
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(w_bf16, "w", true));
    FQ_TRY(check_ptr(dy_bf16, "dy", true));
    FQ_TRY(check_ptr(dx_bf16, "dx", true));
    FQ_TRY(check_ptr(dw_bf16, "dw", true));
    FQ_TRY(check_ptr(ws, "ws", true));
    const bool rht = rht_block != 0;
    // MXFP4 and double-block gradient quantizers rotate their segments in
    // registers; the per-tensor format rotates in separate passes first
    const bool rht_fused = rht && fg.fmt != fqimpl::FMT_NVT;
    const BwdLayout L = bwd_layout(rht && !rht_fused, M, K, N);
    if (ws_bytes < L.total)
        return fail(FQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, L.total);

    char *b = (char *)ws;
    uint32_t *parts = (uint32_t *)(b + L.parts);
    hipStream_t st = (hipStream_t)stream;
    const uint64_t sg = desc_g->seed;

    // the forward's operands and their STE keep masks: X_hat [M, K], W_hat [K, N]
    // (both per-tensor: the two maximum passes in one launch)
    uint32_t *parts_w = parts + fqimpl::kAbsmaxPartials;
    int64_t npart_x = -1, npart_w = -1;
    if (fx.fmt == fqimpl::FMT_NVT && fw.fmt == fqimpl::FMT_NVT && !retain) {
        uint32_t nx = 0, nw = 0;
        hipError_t e = fqimpl::launch_absmax_pair(x_bf16, M * K, parts, &nx, w_bf16, K * N,
                                                  parts_w, &nw, st);
        if (e != hipSuccess) return device_status(e, "tensor absmax launch");
        npart_x = nx;
        npart_w = nw;
    }
    if (retain)
        FQ_TRY(run_quant_retain(fx, desc_x, desc_x->seed, x_bf16, M, K, b + L.xhat, nullptr,
                                nullptr, nullptr, nullptr, b + L.xkeep, retain, chan_scale, parts,
                                st, true));
    else
        FQ_TRY(bwd_quant(fx, desc_x, desc_x->seed, false, x_bf16, M, K, b + L.xhat, nullptr,
                         nullptr, nullptr, b + L.xkeep, parts, st, 0, 0, npart_x));
    FQ_TRY(bwd_quant(fw, desc_w, desc_w->seed, true, w_bf16, K, N, b + L.what, nullptr,
                     nullptr, nullptr, b + L.wkeep, npart_w >= 0 ? parts_w : parts, st, 0, 0,
                     npart_w));
    // the operands before quantization, rotated along each contraction axis
    const void *op_dy_n = dy_bf16, *op_w_n = b + L.what, *op_x_m = b + L.xhat, *op_dy_m = dy_bf16;
    if (rht && !rht_fused) {
        struct { const void *src; int64_t R, C; int col; size_t dst; } rot[4] = {
            {dy_bf16, M, N, 0, L.rdy_n}, {b + L.what, K, N, 0, L.rw_n},
            {b + L.xhat, M, K, 1, L.rx_m}, {dy_bf16, M, N, 1, L.rdy_m}};
        for (const auto &r : rot) {
            hipError_t e = fqimpl::launch_hadamard(r.src, r.R, r.C, r.col, rht_block, rht_seed,
                                                   b + r.dst, true, st);
            if (e != hipSuccess) return device_status(e, "hadamard launch");
        }
        op_dy_n = b + L.rdy_n;
        op_w_n = b + L.rw_n;
        op_x_m = b + L.rx_m;
        op_dy_m = b + L.rdy_m;
    }
    // The four gradient-product operands: dY and W_hat along N (dX = Q(dY) .
    // Q(W_hat)^T), X_hat and dY along M (dW = Q(X_hat)^T . Q(dY)), Philox keys
    // seed + 0 .. 3.  Both products run in one grouped launch whose epilogue
    // applies the STE keep masks (clipped entries of dX and dW are +0).
    struct Op { const void *src; int64_t R, C; bool col; size_t at; };
    const Op ops[4] = {{op_dy_n, M, N, false, L.dyq_n}, {op_w_n, K, N, false, L.wq_n},
                       {op_x_m, M, K, true, L.xq_mt}, {op_dy_m, M, N, true, L.dyq_mt}};
    hipError_t e;
    if (fg.fmt == fqimpl::FMT_MX && !retain) {
        // MXFP4 operands go to the scaled FP4 matrix cores as codes + scales
        // (quantized along the contraction axis, which is what the product
        // needs): [rows, red/2] codes then [rows, red/32] scales
        fqimpl::Fp4Operands o[2];
        const void *cd[4], *sc[4];
        for (int i = 0; i < 4; ++i) {
            const Op &p = ops[i];
            const size_t elems = (size_t)p.R * p.C;
            void *codes = b + p.at, *scales = b + p.at + round256(elems / 2);
            FQ_TRY(bwd_quant(fg, desc_g, sg + i, p.col, p.src, p.R, p.C, nullptr, nullptr, codes,
                             scales, nullptr, parts, st, rht_fused ? rht_block : 0, rht_seed));
            cd[i] = codes;
            sc[i] = scales;
        }
        o[0] = {cd[0], sc[0], cd[1], sc[1], dx_bf16, M, K, N, b + L.xkeep};
        o[1] = {cd[2], sc[2], cd[3], sc[3], dw_bf16, K, N, M, b + L.wkeep};
        e = fqimpl::launch_gemm_mxfp4_nt_pair(o[0], o[1], 2, st);
    } else {
        // BF16 operands: row passes write y, column passes write y transposed
        // (with retained channels, X_hat along M keeps them in FP8 and the
        // products run here whatever the gradient format)
        for (int i = 0; i < 4; ++i) {
            const Op &p = ops[i];
            if (retain && i == 2) {
                fq_desc dg = *desc_g;
                dg.axis = FQ_AXIS_COL;
                FQ_TRY(run_quant_retain(fg, &dg, sg + i, p.src, p.R, p.C, nullptr, b + p.at,
                                        nullptr, nullptr, nullptr, nullptr, retain, chan_scale,
                                        parts, st, true));
                continue;
            }
            FQ_TRY(bwd_quant(fg, desc_g, sg + i, p.col, p.src, p.R, p.C, p.col ? nullptr : b + p.at,
                             p.col ? b + p.at : nullptr, nullptr, nullptr, nullptr, parts, st,
                             rht_fused ? rht_block : 0, rht_seed));
        }
        e = fqimpl::launch_gemm_bf16_nt_pair(b + L.dyq_n, b + L.wq_n, dx_bf16, M, K, N,
                                             b + L.xq_mt, b + L.dyq_mt, dw_bf16, K, N, M, st,
                                             b + L.xkeep, b + L.wkeep);
    }
    return device_status(e, "gemm launch");
}

fq_status fq_qlinear_bwd(const fq_desc *desc_x, const fq_desc *desc_w, const fq_desc *desc_g,
                         int32_t rht_block, uint64_t rht_seed, const void *x_bf16,
                         const void *w_bf16, const void *dy_bf16, int64_t M, int64_t K, int64_t N,
                         void *dx_bf16, void *dw_bf16, void *ws, size_t ws_bytes, void *stream)
{
    return qlinear_bwd_impl(desc_x, desc_w, desc_g, rht_block, rht_seed, x_bf16, w_bf16,
                            dy_bf16, M, K, N, dx_bf16, dw_bf16, ws, ws_bytes, stream, nullptr,
                            nullptr);
}

fq_status fq_qlinear_bwd_retain(const fq_desc *desc_x, const fq_desc *desc_w,
                                const fq_desc *desc_g, const void *x_bf16, const void *w_bf16,
                                const void *dy_bf16, int64_t M, int64_t K, int64_t N,
                                const void *retain, const float *chan_scale, void *dx_bf16,
                                void *dw_bf16, void *ws, size_t ws_bytes, void *stream)
{
    if (!retain) return fail(FQ_ERR_NULL, "retain is NULL");
    if (!chan_scale) return fail(FQ_ERR_NULL, "chan_scale is NULL");
    FQ_TRY(check_ptr(retain, "retain", true, 1));
    FQ_TRY(check_ptr(chan_scale, "chan_scale", true));
    if (K % 8 != 0) return fail(FQ_ERR_SHAPE, "K=%lld must be a multiple of 8", (long long)K);
    return qlinear_bwd_impl(desc_x, desc_w, desc_g, 0, 0, x_bf16, w_bf16, dy_bf16, M, K, N,
                            dx_bf16, dw_bf16, ws, ws_bytes, stream, retain, chan_scale);
}

static fq_status check_osci(const float *w, const void *q, const float *w_prev,
                            const void *q_prev, const float *dm, const float *dq, int64_t n)
{
    if (n < 4 || n % 4 != 0 || n > kMaxElems)
        return fail(FQ_ERR_SHAPE, "n=%lld must be a positive multiple of 4 up to 2^34",
                    (long long)n);
    FQ_TRY(check_ptr(w, "w", true));
    FQ_TRY(check_ptr(q, "q", true, 8));
    FQ_TRY(check_ptr(w_prev, "w_prev", true));
    FQ_TRY(check_ptr(q_prev, "q_prev", true, 8));
    FQ_TRY(check_ptr(dm, "dist_m", true));
    FQ_TRY(check_ptr(dq, "dist_q", true));
    return FQ_OK;
}

fq_status fq_osci_track(const float *w, const void *q_bf16, float *w_prev, void *q_prev_bf16,
                        float *dist_m, float *dist_q, int64_t n, int32_t first, void *stream)
{
    FQ_TRY(check_osci(w, q_bf16, w_prev, q_prev_bf16, dist_m, dist_q, n));
    return device_status(fqimpl::launch_osci_track(w, q_bf16, w_prev, q_prev_bf16, dist_m,
                                                   dist_q, n, first ? 1 : 0,
                                                   (hipStream_t)stream),
                         "osci track launch");
}

fq_status fq_osci_reset(const fq_desc *desc, float *w, const void *q_bf16, const void *codes,
                        const void *scales, const float *outer, int64_t rows, int64_t cols,
                        float *w_prev, void *q_prev_bf16, float *dist_m, float *dist_q,
                        float tau, int32_t target, void *stream)
{
    if (target != FQ_OSCI_BIN_CENTRE && target != FQ_OSCI_GRID_VALUE)
        return fail(FQ_ERR_DESC, "target=%d is not FQ_OSCI_BIN_CENTRE/GRID_VALUE", target);
    if (rows < 1 || cols < 1 || rows > kMaxDim || cols > kMaxDim ||
        rows * cols > kMaxElems)
        return fail(FQ_ERR_SHAPE, "rows=%lld cols=%lld out of range", (long long)rows,
                    (long long)cols);
    if (cols % 4 != 0)
        return fail(FQ_ERR_SHAPE, "cols=%lld must be a multiple of 4", (long long)cols);
    const int64_t n = rows * cols;
    FQ_TRY(check_osci(w, q_bf16, w_prev, q_prev_bf16, dist_m, dist_q, n));
    if (!(tau >= 0.0f) || tau > 3.4e38f)
        return fail(FQ_ERR_DESC, "tau=%g must be finite and >= 0", (double)tau);
    fqimpl::OsciResetArgs a;
    a.w = w;
    a.q = q_bf16;
    a.w_prev = w_prev;
    a.q_prev = q_prev_bf16;
    a.dist_m = dist_m;
    a.dist_q = dist_q;
    a.n = n;
    a.R = rows;
    a.C = cols;
    a.tau = tau;
    a.grid_target = target == FQ_OSCI_GRID_VALUE;
    a.fmt = fqimpl::FMT_MX;
    a.col = false;
    a.codes = a.scales = nullptr;
    a.outer = nullptr;
    if (!a.grid_target) {
        Fmt f;
        FQ_TRY(check_desc(desc, &f, "desc"));
        FQ_TRY(check_shape(f, desc->axis, rows, cols));
        FQ_TRY(check_ptr(codes, "codes", true));
        FQ_TRY(check_ptr(scales, "scales", true));
        FQ_TRY(check_ptr(outer, "outer", f.fmt != fqimpl::FMT_MX, 4));
        a.fmt = f.fmt;
        a.col = desc->axis == FQ_AXIS_COL;
        a.codes = codes;
        a.scales = scales;
        a.outer = f.fmt == fqimpl::FMT_MX ? nullptr : outer;
    }
    return device_status(fqimpl::launch_osci_reset(a, (hipStream_t)stream), "osci reset launch");
}

fq_status fq_channel_absmax(const void *x_bf16, int64_t rows, int64_t cols, uint32_t *amax,
                            void *stream)
{
    if (rows < 1 || cols < 8 || cols % 8 != 0)
        return fail(FQ_ERR_SHAPE, "rows=%lld must be >= 1 and cols=%lld a positive multiple of 8",
                    (long long)rows, (long long)cols);
    if (rows > kMaxDim || cols > kMaxDim || rows * cols > kMaxElems)
        return fail(FQ_ERR_SHAPE, "rows, cols must be below 2^31 and rows*cols at most 2^34");
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(amax, "amax", true, 4));
    return device_status(fqimpl::launch_channel_absmax(x_bf16, rows, cols, amax,
                                                       (hipStream_t)stream),
                         "channel absmax launch");
}

fq_status fq_select_channels(const uint32_t *amax, int64_t cols, int64_t k, void *retain,
                             float *chan_scale, void *stream)
{
    if (cols < 8 || cols % 8 != 0 || cols > (int64_t(1) << 24))
        return fail(FQ_ERR_SHAPE, "cols=%lld must be a positive multiple of 8 up to 2^24",
                    (long long)cols);
    if (k < 0 || k > cols)
        return fail(FQ_ERR_SHAPE, "k=%lld must be in [0, cols=%lld]", (long long)k,
                    (long long)cols);
    FQ_TRY(check_ptr(amax, "amax", true, 4));
    FQ_TRY(check_ptr(retain, "retain", true, 1));
    FQ_TRY(check_ptr(chan_scale, "chan_scale", true, 4));
    return device_status(fqimpl::launch_select_channels(amax, cols, k, retain, chan_scale,
                                                        (hipStream_t)stream),
                         "select channels launch");
}

fq_status fq_fake_quant_retain(const fq_desc *desc, const void *x_bf16, int64_t rows,
                               int64_t cols, void *y_bf16, void *codes, void *scales,
                               float *outer, const void *retain, const float *chan_scale,
                               void *ws, size_t ws_bytes, void *stream)
{
    Fmt f;
    FQ_TRY(check_desc(desc, &f, "desc"));
    FQ_TRY(check_shape(f, desc->axis, rows, cols));
    if (cols % 8 != 0)
        return fail(FQ_ERR_SHAPE, "cols=%lld must be a multiple of 8 (channel mask bytes)",
                    (long long)cols);
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    FQ_TRY(check_ptr(codes, "codes", false));
    FQ_TRY(check_ptr(scales, "scales", false));
    FQ_TRY(check_ptr(outer, "outer", false, 4));
    FQ_TRY(check_ptr(retain, "retain", true, 1));
    FQ_TRY(check_ptr(chan_scale, "chan_scale", true));
    const size_t need = quant_ws(f);
    if (need) {
        FQ_TRY(check_ptr(ws, "ws", true));
        if (ws_bytes < need)
            return fail(FQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
    }
    return run_quant_retain(f, desc, desc->seed, x_bf16, rows, cols, y_bf16, nullptr, codes,
                            scales, outer, nullptr, retain, chan_scale, (uint32_t *)ws,
                            (hipStream_t)stream, false);
}

}  // extern "C"

// ---- row operators around the quantized linears ------------------------------
namespace {

fq_status check_type(int32_t type, const char *name)
{
    if (type != FQ_TYPE_BF16 && type != FQ_TYPE_F32)
        return fail(FQ_ERR_DESC, "%s=%d is not FQ_TYPE_BF16/F32", name, type);
    return FQ_OK;
}

fq_status check_f8(int32_t f8)
{
    if (f8 != FQ_F8_NONE && f8 != FQ_F8_MX && f8 != FQ_F8_ROW)
        return fail(FQ_ERR_DESC, "f8=%d is not FQ_F8_NONE/MX/ROW", f8);
    return FQ_OK;
}

fq_status check_norm_shape(int64_t rows, int64_t cols)
{
    if (rows < 1 || cols < 1)
        return fail(FQ_ERR_SHAPE, "rows=%lld cols=%lld must be >= 1", (long long)rows,
                    (long long)cols);
    if (cols > fqimpl::kNormMaxCols)
        return fail(FQ_ERR_SHAPE, "cols=%lld must be at most %lld", (long long)cols,
                    (long long)fqimpl::kNormMaxCols);
    if (rows > kMaxDim || rows * cols > kMaxElems)
        return fail(FQ_ERR_SHAPE, "rows=%lld must be below 2^31 and rows*cols at most 2^34",
                    (long long)rows);
    return FQ_OK;
}

// T, k, E of the expert sort
fq_status check_moe(int64_t T, int64_t k, int64_t E)
{
    if (T < 1 || k < 1 || E < 1)
        return fail(FQ_ERR_SHAPE, "tokens=%lld k=%lld experts=%lld must be >= 1", (long long)T,
                    (long long)k, (long long)E);
    if (k > FQ_MOE_MAX_K || E > fqimpl::kMoeMaxExperts)
        return fail(FQ_ERR_SHAPE, "k=%lld must be at most %d, experts=%lld at most %d",
                    (long long)k, FQ_MOE_MAX_K, (long long)E, fqimpl::kMoeMaxExperts);
    if (T > (int64_t(1) << 30) / k)
        return fail(FQ_ERR_SHAPE, "tokens*k=%lld*%lld must be at most 2^30", (long long)T,
                    (long long)k);
    return FQ_OK;
}

fq_status check_moe_rows(int64_t T, int64_t k, int64_t H, int64_t rows, int64_t unit)
{
    FQ_TRY(check_moe(T, k, 1));
    if (H < unit || H % unit != 0)
        return fail(FQ_ERR_SHAPE, "cols=%lld must be a positive multiple of %lld", (long long)H,
                    (long long)unit);
    if (rows < 1 || rows > kMaxDim)
        return fail(FQ_ERR_SHAPE, "rows=%lld must be >= 1 and below 2^31", (long long)rows);
    // the kernels number a row's elements in 32 bits
    if (H > kMaxDim || H > kMaxElems / (rows > T ? rows : T))
        return fail(FQ_ERR_SHAPE,
                    "cols=%lld must be below 2^31, rows*cols and tokens*cols at most 2^34",
                    (long long)H);
    return FQ_OK;
}

fq_status check_adamw_hyper(const fq_adamw_hyper *hyper)
{
    if (!hyper) return fail(FQ_ERR_NULL, "hyper is NULL");
    const fq_adamw_hyper &h = *hyper;
    if (h.reserved != 0) return fail(FQ_ERR_DESC, "hyper->reserved must be 0");
    if (h.state_type != FQ_STATE_F32 && h.state_type != FQ_STATE_F8)
        return fail(FQ_ERR_DESC, "hyper->state_type=%d is not FQ_STATE_F32/F8", h.state_type);
    if (!(h.beta1 >= 0 && h.beta1 < 1 && h.beta2 >= 0 && h.beta2 < 1))
        return fail(FQ_ERR_DESC, "beta1 and beta2 must be in [0, 1)");
    // as the kernels use them
    if (!(h.eps >= 0) || !std::isfinite((float)h.lr) || !std::isfinite((float)h.eps) ||
        (h.eps > 0 && (float)h.eps == 0))
        return fail(FQ_ERR_DESC, "lr must be finite, eps 0 or positive and finite, in FP32");
    if (h.step < 1 || h.step > 0xFFFFFFFFll)
        return fail(FQ_ERR_DESC, "step=%lld must be in [1, 2^32)", (long long)h.step);
    FQ_TRY(check_ptr(h.grad_scale, "hyper->grad_scale", false, 4));
    return FQ_OK;
}

fq_status check_adamw_tensors(const fq_adamw_tensor *tensors, int64_t count, bool f8)
{
    if (count < 0 || count > kMaxDim)
        return fail(FQ_ERR_SHAPE, "count=%lld must be >= 0 and below 2^31", (long long)count);
    if (count && !tensors) return fail(FQ_ERR_NULL, "tensors is NULL");
    for (int64_t i = 0; i < count; ++i) {
        const fq_adamw_tensor &t = tensors[i];
        if (t.reserved != 0)
            return fail(FQ_ERR_DESC, "tensors[%lld].reserved must be 0", (long long)i);
        if (t.g_type != FQ_TYPE_BF16 && t.g_type != FQ_TYPE_F32)
            return fail(FQ_ERR_DESC, "tensors[%lld].g_type=%d is not FQ_TYPE_BF16/F32",
                        (long long)i, t.g_type);
        if (t.n < 0 || t.n > kMaxElems)
            return fail(FQ_ERR_SHAPE, "tensors[%lld].n=%lld must be in [0, 2^34]", (long long)i,
                        (long long)t.n);
        if (!std::isfinite(t.lr_mult) || !std::isfinite(t.weight_decay))
            return fail(FQ_ERR_DESC, "tensors[%lld]: lr_mult and weight_decay must be finite",
                        (long long)i);
        if (t.n == 0) continue;
        const void *need[] = {t.w, t.g, t.m, t.v};
        for (const void *p : need) {
            if (!p) return fail(FQ_ERR_NULL, "tensors[%lld]: w, g, m or v is NULL", (long long)i);
            if (!aligned(p, 16))
                return fail(FQ_ERR_ALIGN, "tensors[%lld]: w, g, m or v is not 16-byte aligned",
                            (long long)i);
        }
        if (!aligned(t.w_bf16, 16))
            return fail(FQ_ERR_ALIGN, "tensors[%lld].w_bf16 is not 16-byte aligned", (long long)i);
        if (f8 && (!t.m_scale || !t.v_scale))
            return fail(FQ_ERR_NULL, "tensors[%lld]: m_scale or v_scale is NULL", (long long)i);
        if (f8 && !(aligned(t.m_scale, 4) && aligned(t.v_scale, 4)))
            return fail(FQ_ERR_ALIGN, "tensors[%lld]: m_scale or v_scale is not 4-byte aligned",
                        (long long)i);
    }
    return FQ_OK;
}

fqimpl::AdamWStep adamw_step_of(const fq_adamw_hyper &h)
{
    fqimpl::AdamWStep a = {};
    a.lr = (float)h.lr;
    a.beta1 = (float)h.beta1;
    a.one_beta1 = (float)(1.0 - h.beta1);
    a.beta2 = (float)h.beta2;
    a.one_beta2 = (float)(1.0 - h.beta2);
    a.eps = (float)h.eps;
    a.inv_bc1 = (float)(1.0 / (1.0 - std::pow(h.beta1, (double)h.step)));
    a.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(h.beta2, (double)h.step)));
    a.grad_scale = h.grad_scale;
    a.step = (uint32_t)h.step;
    a.seed_lo = (uint32_t)h.seed;
    a.seed_hi = (uint32_t)(h.seed >> 32);
    a.divide_from = a.eps == 0 || (a.eps >= 0x1p-100f && a.eps <= 0x1p100f)
                        ? fqimpl::kAdamWDivideFrom : 0;
    return a;
}

fqimpl::AdamWTensor adamw_entry(const fq_adamw_tensor &t)
{
    return {t.w, t.w_bf16, t.g, t.m, t.v, t.m_scale, t.v_scale, t.n,
            t.lr_mult, t.weight_decay, t.g_type == FQ_TYPE_F32};
}

// The image of a plan: this header, then for each tensor that has elements its
// entry, and after all entries their first tiles and their numbers in the list.
struct AdamWPlan {
    uint64_t magic;
    uint32_t count, tiles;
    int32_t state_type, reserved;
    int64_t padding[5];      // entries at a multiple of 64 bytes
};
constexpr uint64_t kPlanMagic = 0x4E4C50574D414441ull;
static_assert(sizeof(AdamWPlan) == 64, "plan header");

}  // namespace

extern "C" {

fq_status fq_rmsnorm_fwd(const void *x_bf16, const void *res, int32_t stream_type,
                         const void *gamma, int32_t gamma_type, float eps, int64_t rows,
                         int64_t cols, int32_t f8, void *h, void *y_bf16, void *codes,
                         void *scales, float *rstd, void *stream)
{
    FQ_TRY(check_type(stream_type, "stream_type"));
    FQ_TRY(check_type(gamma_type, "gamma_type"));
    FQ_TRY(check_f8(f8));
    if (!(eps >= 0.0f)) return fail(FQ_ERR_DESC, "eps must be >= 0");
    FQ_TRY(check_norm_shape(rows, cols));
    if (f8 != FQ_F8_NONE && cols % 32 != 0)
        return fail(FQ_ERR_SHAPE, "cols=%lld must be a multiple of 32 for an 8-bit output",
                    (long long)cols);
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(gamma, "gamma", true));
    FQ_TRY(check_ptr(res, "res", false));
    FQ_TRY(check_ptr(h, "h", res != nullptr));
    if (!res && h) return fail(FQ_ERR_DESC, "h is written only with a residual");
    FQ_TRY(check_ptr(y_bf16, "y", f8 == FQ_F8_NONE));
    FQ_TRY(check_ptr(codes, "codes", f8 != FQ_F8_NONE && !y_bf16));
    if (f8 == FQ_F8_NONE && (codes || scales))
        return fail(FQ_ERR_DESC, "codes and scales are written only for an 8-bit output");
    FQ_TRY(check_ptr(scales, "scales", codes != nullptr));
    FQ_TRY(check_ptr(rstd, "rstd", false, 4));
    fqimpl::NormFwdArgs a;
    a.x = x_bf16;
    a.res = res;
    a.stream_f32 = stream_type == FQ_TYPE_F32;
    a.gamma = gamma;
    a.gamma_f32 = gamma_type == FQ_TYPE_F32;
    a.eps = eps;
    a.rows = rows;
    a.cols = cols;
    a.f8 = f8;
    a.h = h;
    a.y = y_bf16;
    a.codes = codes;
    a.scales = scales;
    a.rstd = rstd;
    return device_status(fqimpl::launch_rmsnorm_fwd(a, (hipStream_t)stream), "norm launch");
}

size_t fq_rmsnorm_bwd_workspace_size(int64_t rows, int64_t cols)
{
    if (check_norm_shape(rows, cols) != FQ_OK) return 0;
    return (size_t)fqimpl::rmsnorm_bwd_groups(rows, cols) * cols * sizeof(float);
}

fq_status fq_rmsnorm_bwd(const void *dy_bf16, const void *h, int32_t stream_type,
                         const void *gamma, int32_t gamma_type, const float *rstd,
                         const void *dres, int64_t rows, int64_t cols, void *dh, void *dx_bf16,
                         float *dgamma, void *ws, size_t ws_bytes, void *stream)
{
    FQ_TRY(check_type(stream_type, "stream_type"));
    FQ_TRY(check_type(gamma_type, "gamma_type"));
    FQ_TRY(check_norm_shape(rows, cols));
    FQ_TRY(check_ptr(dy_bf16, "dy", true));
    FQ_TRY(check_ptr(h, "h", true));
    FQ_TRY(check_ptr(gamma, "gamma", true));
    FQ_TRY(check_ptr(rstd, "rstd", true, 4));
    FQ_TRY(check_ptr(dres, "dres", false));
    FQ_TRY(check_ptr(dh, "dh", true));
    FQ_TRY(check_ptr(dx_bf16, "dx", false));
    FQ_TRY(check_ptr(dgamma, "dgamma", false, 4));
    if (dgamma) {
        FQ_TRY(check_ptr(ws, "ws", true));
        const size_t need = fq_rmsnorm_bwd_workspace_size(rows, cols);
        if (ws_bytes < need)
            return fail(FQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
    }
    fqimpl::NormBwdArgs a;
    a.dy = dy_bf16;
    a.h = h;
    a.stream_f32 = stream_type == FQ_TYPE_F32;
    a.gamma = gamma;
    a.gamma_f32 = gamma_type == FQ_TYPE_F32;
    a.rstd = rstd;
    a.dres = dres;
    a.rows = rows;
    a.cols = cols;
    a.dh = dh;
    a.dx = dx_bf16;
    a.dgamma = dgamma;
    a.partials = (float *)ws;
    a.groups = 0;
    a.few = false;
    return device_status(fqimpl::launch_rmsnorm_bwd(a, (hipStream_t)stream),
                         "norm backward launch");
}

int64_t fq_moe_rows(int64_t tokens, int64_t k, int64_t experts, int64_t align)
{
    if (check_moe(tokens, k, experts) != FQ_OK) return 0;
    if (align < 1 || align > FQ_MOE_MAX_ALIGN) {
        fail(FQ_ERR_SHAPE, "align=%lld must be in [1, %d]", (long long)align, FQ_MOE_MAX_ALIGN);
        return 0;
    }
    const int64_t n = tokens * k, used = experts < n ? experts : n;
    return (n + used * (align - 1)) / align * align;
}

size_t fq_moe_sort_workspace_size(int64_t tokens, int64_t k, int64_t experts)
{
    if (check_moe(tokens, k, experts) != FQ_OK) return 0;
    return fqimpl::moe_sort_counts(tokens * k, experts) * sizeof(uint32_t);
}

fq_status fq_moe_sort(const int32_t *experts_of, int64_t tokens, int64_t k, int64_t experts,
                      int64_t align, int64_t rows, int32_t *offsets, int32_t *pos, int32_t *src,
                      void *ws, size_t ws_bytes, void *stream)
{
    const int64_t want = fq_moe_rows(tokens, k, experts, align);
    if (!want) return FQ_ERR_SHAPE;
    if (rows < want || rows > kMaxDim)
        return fail(FQ_ERR_SHAPE, "rows=%lld must be at least fq_moe_rows = %lld and below 2^31",
                    (long long)rows, (long long)want);
    FQ_TRY(check_ptr(experts_of, "experts_of", true, 4));
    FQ_TRY(check_ptr(offsets, "offsets", true, 4));
    FQ_TRY(check_ptr(pos, "pos", true, 4));
    FQ_TRY(check_ptr(src, "src", true, 4));
    const size_t need = fq_moe_sort_workspace_size(tokens, k, experts);
    if (need) {
        FQ_TRY(check_ptr(ws, "ws", true));
        if (ws_bytes < need)
            return fail(FQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
    }
    fqimpl::MoeSortArgs a;
    a.ids = experts_of;
    a.n = tokens * k;
    a.E = (uint32_t)experts;
    a.align = (uint32_t)align;
    a.rows = rows;
    a.offsets = offsets;
    a.pos = pos;
    a.src = src;
    a.ws = (uint32_t *)ws;
    a.chunk = 0;
    return device_status(fqimpl::launch_moe_sort(a, (hipStream_t)stream), "expert sort launch");
}

fq_status fq_moe_dispatch(const void *x, int32_t f8, const void *scales, int64_t tokens,
                          int64_t k, int64_t cols, int64_t rows, const int32_t *pos,
                          const int32_t *src, void *y_bf16, void *stream)
{
    FQ_TRY(check_f8(f8));
    FQ_TRY(check_moe_rows(tokens, k, cols, rows, f8 == FQ_F8_NONE ? 8 : 32));
    FQ_TRY(check_ptr(x, "x", true));
    if (f8 == FQ_F8_NONE && scales)
        return fail(FQ_ERR_DESC, "scales are read only with 8-bit rows");
    FQ_TRY(check_ptr(scales, "scales", f8 != FQ_F8_NONE));
    FQ_TRY(check_ptr(pos, "pos", true, 4));
    FQ_TRY(check_ptr(src, "src", true, 4));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    fqimpl::MoeRowsArgs a = {};
    a.T = tokens;
    a.k = k;
    a.H = cols;
    a.rows = rows;
    a.pos = pos;
    a.src = src;
    a.x = x;
    a.scales = scales;
    a.rows_out = y_bf16;
    return device_status(fqimpl::launch_moe_dispatch(f8, a, (hipStream_t)stream),
                         "dispatch launch");
}

fq_status fq_moe_combine(const void *y_bf16, const float *weights, int64_t tokens, int64_t k,
                         int64_t cols, int64_t rows, const int32_t *pos, void *out_bf16,
                         void *stream)
{
    FQ_TRY(check_moe_rows(tokens, k, cols, rows, 8));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    FQ_TRY(check_ptr(weights, "weights", false, 4));
    FQ_TRY(check_ptr(pos, "pos", true, 4));
    FQ_TRY(check_ptr(out_bf16, "out", true));
    fqimpl::MoeRowsArgs a = {};
    a.T = tokens;
    a.k = k;
    a.H = cols;
    a.rows = rows;
    a.pos = pos;
    a.weights = weights;
    a.y = y_bf16;
    a.out = out_bf16;
    return device_status(fqimpl::launch_moe_combine(a, (hipStream_t)stream), "combine launch");
}

fq_status fq_moe_combine_bwd(const void *dout_bf16, const void *y_bf16, const float *weights,
                             int64_t tokens, int64_t k, int64_t cols, int64_t rows,
                             const int32_t *pos, const int32_t *src, void *dy_bf16,
                             float *dweights, void *stream)
{
    FQ_TRY(check_moe_rows(tokens, k, cols, rows, 8));
    FQ_TRY(check_ptr(dout_bf16, "dout", true));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    FQ_TRY(check_ptr(weights, "weights", true, 4));
    FQ_TRY(check_ptr(pos, "pos", true, 4));
    FQ_TRY(check_ptr(src, "src", true, 4));
    FQ_TRY(check_ptr(dy_bf16, "dy", true));
    FQ_TRY(check_ptr(dweights, "dweights", true, 4));
    fqimpl::MoeRowsArgs a = {};
    a.T = tokens;
    a.k = k;
    a.H = cols;
    a.rows = rows;
    a.pos = pos;
    a.src = src;
    a.weights = weights;
    a.y = y_bf16;
    a.dout = dout_bf16;
    a.rows_out = dy_bf16;
    a.dweights = dweights;
    return device_status(fqimpl::launch_moe_combine_bwd(a, (hipStream_t)stream),
                         "combine backward launch");
}

fq_status fq_adamw_step(const fq_adamw_hyper *hyper, const fq_adamw_tensor *tensors,
                        int64_t count, void *stream)
{
    FQ_TRY(check_adamw_hyper(hyper));
    const bool f8 = hyper->state_type == FQ_STATE_F8;
    FQ_TRY(check_adamw_tensors(tensors, count, f8));
    fqimpl::AdamWArgs a;
    a.step = adamw_step_of(*hyper);
    for (int64_t i = 0; i < count; ++i) {
        const fq_adamw_tensor &t = tensors[i];
        if (!t.n) continue;
        const uint32_t tiles = fqimpl::adamw_tiles(t.n, f8);
        uint32_t &n = a.step.count;
        if (n == fqimpl::kAdamWTensors) {
            FQ_TRY(device_status(fqimpl::launch_adamw(a, f8, (hipStream_t)stream), "AdamW launch"));
            n = a.step.tiles = 0;
        }
        a.first[n] = a.step.tiles;
        a.index[n] = (uint32_t)i;
        a.t[n++] = adamw_entry(t);
        a.step.tiles += tiles;
    }
    if (!a.step.count) return ok();
    return device_status(fqimpl::launch_adamw(a, f8, (hipStream_t)stream), "AdamW launch");
}

size_t fq_adamw_plan_size(int64_t count)
{
    if (count < 0 || count > kMaxDim) {
        fail(FQ_ERR_SHAPE, "count=%lld must be >= 0 and below 2^31", (long long)count);
        return 0;
    }
    return sizeof(AdamWPlan) + (size_t)count * (sizeof(fqimpl::AdamWTensor) + 2 * sizeof(uint32_t));
}

fq_status fq_adamw_plan(const fq_adamw_tensor *tensors, int64_t count, int32_t state_type,
                        void *plan, size_t plan_bytes)
{
    if (state_type != FQ_STATE_F32 && state_type != FQ_STATE_F8)
        return fail(FQ_ERR_DESC, "state_type=%d is not FQ_STATE_F32/F8", state_type);
    const bool f8 = state_type == FQ_STATE_F8;
    FQ_TRY(check_adamw_tensors(tensors, count, f8));
    FQ_TRY(check_ptr(plan, "plan", true));
    const size_t need = fq_adamw_plan_size(count);
    if (plan_bytes < need)
        return fail(FQ_ERR_WORKSPACE, "plan %zu bytes < %zu required", plan_bytes, need);
    uint64_t live = 0, tiles = 0;
    for (int64_t i = 0; i < count; ++i) {
        live += tensors[i].n > 0;
        tiles += fqimpl::adamw_tiles(tensors[i].n, f8);
    }
    if (tiles > fqimpl::kAdamWMaxTiles)
        return fail(FQ_ERR_SHAPE, "a plan's tensors take %llu tiles of %d elements, at most 2^31",
                    (unsigned long long)tiles, (int)fqimpl::adamw_tile(f8));
    memset(plan, 0, need);
    AdamWPlan *p = (AdamWPlan *)plan;
    p->magic = kPlanMagic;
    p->count = (uint32_t)live;
    p->tiles = (uint32_t)tiles;
    p->state_type = state_type;
    auto *entries = (fqimpl::AdamWTensor *)(p + 1);
    auto *first = (uint32_t *)(entries + live), *index = first + live;
    uint32_t n = 0, at = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (!tensors[i].n) continue;
        entries[n] = adamw_entry(tensors[i]);
        first[n] = at;
        index[n++] = (uint32_t)i;
        at += fqimpl::adamw_tiles(tensors[i].n, f8);
    }
    return ok();
}

fq_status fq_adamw_step_plan(const fq_adamw_hyper *hyper, const void *plan,
                             const void *plan_device, void *stream)
{
    FQ_TRY(check_adamw_hyper(hyper));
    FQ_TRY(check_ptr(plan, "plan", true));
    const AdamWPlan &p = *(const AdamWPlan *)plan;
    if (p.magic != kPlanMagic) return fail(FQ_ERR_DESC, "plan was not made by fq_adamw_plan");
    if (p.state_type != hyper->state_type)
        return fail(FQ_ERR_DESC, "hyper->state_type=%d is not the plan's %d", hyper->state_type,
                    p.state_type);
    if (!p.count) return ok();
    FQ_TRY(check_ptr(plan_device, "plan_device", true));
    fqimpl::AdamWStep a = adamw_step_of(*hyper);
    a.count = p.count;
    a.tiles = p.tiles;
    const auto *entries = (const fqimpl::AdamWTensor *)((const AdamWPlan *)plan_device + 1);
    const auto *first = (const uint32_t *)(entries + p.count);
    return device_status(fqimpl::launch_adamw_plan(a, entries, first, first + p.count,
                                                   p.state_type == FQ_STATE_F8,
                                                   (hipStream_t)stream),
                         "AdamW launch");
}

}  // extern "C"

// ---- the feed-forward products of a training step ----------------------------
namespace {

constexpr int64_t kTensorMax = kMaxElems;

fq_status check_act(int32_t act)
{
    if (act < FQ_ACT_NONE || act > FQ_ACT_GELU)
        return fail(FQ_ERR_DESC, "act=%d is not FQ_ACT_NONE/RELU/SILU/GELU", act);
    return FQ_OK;
}

fq_status check_gate(const fq_gate *gate, fqimpl::Gate *out)
{
    if (!gate) return fail(FQ_ERR_NULL, "gate is NULL");
    FQ_TRY(check_act(gate->act));
    if (!std::isfinite(gate->alpha) || (gate->act != FQ_ACT_SILU && gate->alpha != 1.0f))
        return fail(FQ_ERR_DESC, "gate->alpha must be finite, and 1 unless act is FQ_ACT_SILU");
    if (!(gate->limit > 0.0f)) return fail(FQ_ERR_DESC, "gate->limit must be > 0");
    if (!std::isfinite(gate->shift)) return fail(FQ_ERR_DESC, "gate->shift must be finite");
    *out = {gate->act, gate->alpha, gate->limit, gate->shift};
    return FQ_OK;
}

// Sizes of a product: rows, k, and `halves` times n columns, per expert.
struct Product {
    int64_t rows, k, n, experts, halves;
    int64_t cols() const { return n * halves; }
    int64_t groups() const { return experts ? experts : 1; }
};

fq_status check_product(const Product &d)
{
    if (d.rows < 1 || d.rows > fqimpl::kProductMaxRows)
        return fail(FQ_ERR_SHAPE, "rows=%lld must be in [1, 2^30]", (long long)d.rows);
    if (d.k < 8 || d.n < 8 || d.k % 8 || d.n % 8 || d.k > fqimpl::kProductMaxDim ||
        d.n > fqimpl::kProductMaxDim)
        return fail(FQ_ERR_SHAPE, "k=%lld and n=%lld must be multiples of 8 from 8 to 2^20",
                    (long long)d.k, (long long)d.n);
    if (d.experts < 0 || d.experts > fqimpl::kProductMaxExperts)
        return fail(FQ_ERR_SHAPE, "experts=%lld must be in [0, %lld]", (long long)d.experts,
                    (long long)fqimpl::kProductMaxExperts);
    if (d.rows > kTensorMax / d.k || d.rows > kTensorMax / d.cols() ||
        d.groups() > kTensorMax / d.k / d.cols())
        return fail(FQ_ERR_SHAPE,
                    "rows*k, rows*columns and experts*k*columns must be at most 2^34 (rows=%lld k=%lld "
                    "columns=%lld experts=%lld)", (long long)d.rows, (long long)d.k,
                    (long long)d.cols(), (long long)d.experts);
    return FQ_OK;
}

fq_status check_offsets(const Product &d, const int32_t *offsets)
{
    if ((d.experts > 0) != (offsets != nullptr))
        return fail(FQ_ERR_NULL, offsets ? "offsets are given without experts"
                                         : "offsets is NULL with experts");
    return check_ptr(offsets, "offsets", false, 4);
}

// the values before the activation: *kind is set to a PRE_*
fq_status check_pre(const Product &d, const void *pre, int32_t f8, const void *scales, bool required,
                    int *kind)
{
    FQ_TRY(check_ptr(pre, "pre", required));
    if (f8 != FQ_F8_NONE && f8 != FQ_F8_MX)
        return fail(FQ_ERR_DESC, "pre_f8=%d is not FQ_F8_NONE/MX", f8);
    *kind = !pre ? fqimpl::PRE_NONE : f8 == FQ_F8_MX ? fqimpl::PRE_MX : fqimpl::PRE_BF16;
    const bool mx = *kind == fqimpl::PRE_MX;
    if (scales && !mx) return fail(FQ_ERR_DESC, "pre_scales belong to a pre in FQ_F8_MX");
    FQ_TRY(check_ptr(scales, "pre_scales", mx));
    if (mx && d.n % 32 != 0)
        return fail(FQ_ERR_SHAPE, "n=%lld must be a multiple of 32 for a pre in 8 bits", (long long)d.n);
    return FQ_OK;
}

// Parts of the contraction of one product [M, columns] over K, and their bytes.
int splits_of(const Product &d, int64_t M, int64_t columns, int64_t K)
{
    return d.experts ? 1 : fqimpl::product_splits(M, columns, K);
}
size_t split_bytes(const Product &d, int64_t M, int64_t columns, int64_t K)
{
    const int n = splits_of(d, M, columns, K);
    return n > 1 ? (size_t)n * M * columns * sizeof(float) : 0;
}

int fwd_splits(const Product &d)
{
    return fqimpl::product_few_rows(d.rows, d.experts) ? 1 : splits_of(d, d.rows, d.cols(), d.k);
}
size_t product_fwd_ws(const Product &d)
{
    return fwd_splits(d) > 1 ? split_bytes(d, d.rows, d.cols(), d.k) : 0;
}

// Workspace of a backward: dz, dz with the row scales' mantissas, x decoded, the tiles'
// column sums, the parts of a split dx and of a split dw.
struct ProductBwdLayout {
    size_t scaled, x, partials, dx_parts, dw_parts, total;
};
ProductBwdLayout product_bwd_layout(const Product &d, int32_t x_f8)
{
    ProductBwdLayout l;
    const size_t dz = round256((size_t)d.rows * d.cols() * 2);
    l.scaled = dz;
    l.x = l.scaled + (x_f8 == FQ_F8_ROW ? dz : 0);
    l.partials = l.x + (x_f8 != FQ_F8_NONE ? round256((size_t)d.rows * d.k * 2) : 0);
    l.dx_parts = l.partials +
                 round256((size_t)fqimpl::dz_tiles(d.rows, d.n, d.experts) * d.cols() * sizeof(float));
    l.dw_parts = l.dx_parts + round256(split_bytes(d, d.rows, d.k, d.cols()));
    l.total = l.dw_parts + split_bytes(d, d.k, d.cols(), d.rows);
    return l;
}

size_t product_bwd_ws(const Product &d, int32_t x_f8)
{
    if (check_product(d) != FQ_OK || check_f8(x_f8) != FQ_OK) return 0;
    return product_bwd_layout(d, x_f8).total;
}

fq_status check_ws(const void *ws, size_t ws_bytes, size_t need)
{
    if (!need) return FQ_OK;
    FQ_TRY(check_ptr(ws, "ws", true));
    if (ws_bytes < need)
        return fail(FQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
    return FQ_OK;
}

fqimpl::ProductArgs product_args(const Product &d, const int32_t *offsets)
{
    fqimpl::ProductArgs p = {};
    p.rows = (int)d.rows;
    p.experts = (int)d.experts;
    p.offsets = offsets;
    return p;
}

// The forward's operands that both products share.
fq_status product_fwd(fqimpl::ProductArgs *p, const Product &d, const void *x, const void *w,
                      const void *bias, int32_t bias_type, const int32_t *offsets, void *pre,
                      int32_t pre_f8, void *pre_scales)
{
    FQ_TRY(check_type(bias_type, "bias_type"));
    FQ_TRY(check_product(d));
    FQ_TRY(check_ptr(x, "x", true));
    FQ_TRY(check_ptr(w, "w", true));
    FQ_TRY(check_ptr(bias, "bias", false));
    FQ_TRY(check_offsets(d, offsets));
    *p = product_args(d, offsets);
    FQ_TRY(check_pre(d, pre, pre_f8, pre_scales, false, &p->pre_kind));
    p->a = (const uint16_t *)x;
    p->b = (const uint16_t *)w;
    p->lda = d.k;
    p->ldb = d.cols();
    p->b_stride = d.k * d.cols();
    p->M = (int)d.rows;
    p->N = (int)d.n;
    p->K = (int)d.k;
    p->bias = bias;
    p->bias_f32 = bias_type == FQ_TYPE_F32;
    p->pre = pre;
    p->pre_scales = pre_scales;
    return FQ_OK;
}

struct ProductBwd {
    const void *dy, *x;
    int32_t x_f8;
    const void *x_scales, *w, *pre;
    int32_t pre_f8;
    const void *pre_scales;
    const int32_t *offsets;
    fqimpl::Gate gate;
    void *dx, *dw;
    int32_t dw_type;
    float *dbias;
    void *h, *ws;
    size_t ws_bytes;
    hipStream_t stream;
};

fq_status product_bwd(const Product &d, const ProductBwd &a)
{
    const bool glu = d.halves == 2, plain = !glu && a.gate.act == FQ_ACT_NONE;
    FQ_TRY(check_f8(a.x_f8));
    FQ_TRY(check_type(a.dw_type, "dw_type"));
    FQ_TRY(check_product(d));
    if (!a.dx && !a.dw && !a.dbias && !a.h) return fail(FQ_ERR_NULL, "no output is given");
    FQ_TRY(check_ptr(a.dy, glu ? "dh" : "dy", true));
    FQ_TRY(check_ptr(a.x, "x", a.dw != nullptr));
    const bool x8 = a.x && a.x_f8 != FQ_F8_NONE;
    if (a.x_scales && !x8) return fail(FQ_ERR_DESC, "x_scales belong to an x in 8 bits");
    FQ_TRY(check_ptr(a.x_scales, "x_scales", x8));
    if (x8 && d.k % 32 != 0)
        return fail(FQ_ERR_SHAPE, "k=%lld must be a multiple of 32 for an x in 8 bits", (long long)d.k);
    FQ_TRY(check_ptr(a.w, "w", a.dx != nullptr));
    FQ_TRY(check_offsets(d, a.offsets));
    int pre_kind;
    FQ_TRY(check_pre(d, a.pre, a.pre_f8, a.pre_scales, !plain, &pre_kind));
    FQ_TRY(check_ptr(a.dx, "dx", false));
    FQ_TRY(check_ptr(a.dw, "dw", false));
    FQ_TRY(check_ptr(a.dbias, "dbias", false));
    FQ_TRY(check_ptr(a.h, "h", false));
    const ProductBwdLayout l = product_bwd_layout(d, a.x_f8);
    FQ_TRY(check_ws(a.ws, a.ws_bytes, l.total));

    uint8_t *ws = (uint8_t *)a.ws;
    const void *dz = plain ? a.dy : a.ws;
    // x's row scales go into dz where that is rounded anyway
    const bool scaled = x8 && a.dw && !plain && a.x_f8 == FQ_F8_ROW;
    if (!plain || a.dbias) {
        fqimpl::DzArgs z = {};
        z.glu = glu;
        z.dy = a.dy;
        z.pre = plain ? nullptr : a.pre;
        z.pre_scales = a.pre_scales;
        z.pre_kind = pre_kind;
        z.gate = a.gate;
        z.rows = d.rows;
        z.n = d.n;
        z.experts = (int)d.experts;
        z.offsets = a.offsets;
        z.dz = a.dx || (a.dw && !scaled) ? ws : nullptr;
        z.dz_scaled = scaled ? ws + l.scaled : nullptr;
        z.row_scales = (const float *)a.x_scales;
        z.h = a.h;
        z.partials = a.dbias ? (float *)(ws + l.partials) : nullptr;
        z.dbias = a.dbias;
        const hipError_t e = fqimpl::launch_dz(z, a.stream);
        if (e != hipSuccess) return device_status(e, "gradient before the activation launch");
    }
    fqimpl::ProductArgs dx = product_args(d, a.offsets), dw = dx;
    if (a.dx) {
        dx.a = (const uint16_t *)dz;
        dx.b = (const uint16_t *)a.w;
        dx.lda = dx.ldb = d.cols();
        dx.b_stride = d.k * d.cols();
        dx.M = (int)d.rows;
        dx.N = (int)d.k;
        dx.K = (int)d.cols();
        dx.y = a.dx;
        dx.splits = splits_of(d, d.rows, d.k, d.cols());
        dx.partial = (float *)(ws + l.dx_parts);
    }
    if (a.dw) {
        const void *x = a.x;
        if (x8) {
            fqimpl::RowArgs8 r = {};
            r.codes = const_cast<void *>(a.x);
            r.scales = const_cast<void *>(a.x_scales);
            r.y = ws + l.x;
            r.rows = d.rows;
            r.cols = d.k;
            r.power = scaled;
            const hipError_t e = fqimpl::launch_f8_decode(a.x_f8, r, a.stream);
            if (e != hipSuccess) return device_status(e, "decode launch");
            x = r.y;
        }
        dw.a = (const uint16_t *)x;
        dw.b = scaled ? (const uint16_t *)(ws + l.scaled) : (const uint16_t *)dz;
        dw.lda = d.k;
        dw.ldb = d.cols();
        dw.M = (int)d.k;
        dw.N = (int)d.cols();
        dw.K = (int)d.rows;
        dw.y = a.dw;
        dw.y_f32 = a.dw_type == FQ_TYPE_F32;
        dw.splits = splits_of(d, d.k, d.cols(), d.rows);
        dw.partial = (float *)(ws + l.dw_parts);
    }
    if (a.dx || a.dw) {
        const hipError_t e = fqimpl::launch_product_bwd(a.dx ? &dx : nullptr, a.dw ? &dw : nullptr, a.stream);
        if (e != hipSuccess) return device_status(e, "dx and dw launch");
    }
    return ok();
}

fq_status check_f8_rows(int32_t f8, int64_t rows, int64_t cols)
{
    FQ_TRY(check_f8(f8));
    if (f8 == FQ_F8_NONE) return fail(FQ_ERR_DESC, "f8 must be FQ_F8_MX or FQ_F8_ROW");
    if (rows < 1 || cols < 32 || cols % 32 != 0)
        return fail(FQ_ERR_SHAPE, "rows=%lld must be >= 1, cols=%lld a positive multiple of 32",
                    (long long)rows, (long long)cols);
    if (rows > kMaxDim || cols > kMaxDim || rows > kMaxElems / cols)
        return fail(FQ_ERR_SHAPE, "rows=%lld cols=%lld: each must be below 2^31 and rows*cols at most 2^34",
                    (long long)rows, (long long)cols);
    return FQ_OK;
}

}  // namespace

extern "C" {

fq_status fq_f8_encode(const void *x_bf16, int32_t f8, int64_t rows, int64_t cols, void *codes,
                       void *scales, void *stream)
{
    FQ_TRY(check_f8_rows(f8, rows, cols));
    if (f8 == FQ_F8_ROW && cols > fqimpl::kF8RowMaxCols)
        return fail(FQ_ERR_SHAPE, "cols=%lld must be at most %lld for FQ_F8_ROW", (long long)cols,
                    (long long)fqimpl::kF8RowMaxCols);
    FQ_TRY(check_ptr(x_bf16, "x", true));
    FQ_TRY(check_ptr(codes, "codes", true));
    FQ_TRY(check_ptr(scales, "scales", true));
    fqimpl::RowArgs8 a = {};
    a.x = x_bf16;
    a.codes = codes;
    a.scales = scales;
    a.rows = rows;
    a.cols = cols;
    return device_status(fqimpl::launch_f8_encode(f8, a, (hipStream_t)stream), "encode launch");
}

fq_status fq_f8_decode(const void *codes, const void *scales, int32_t f8, int64_t rows,
                       int64_t cols, void *y_bf16, void *stream)
{
    FQ_TRY(check_f8_rows(f8, rows, cols));
    FQ_TRY(check_ptr(codes, "codes", true));
    FQ_TRY(check_ptr(scales, "scales", true));
    FQ_TRY(check_ptr(y_bf16, "y", true));
    fqimpl::RowArgs8 a = {};
    a.codes = const_cast<void *>(codes);
    a.scales = const_cast<void *>(scales);
    a.y = y_bf16;
    a.rows = rows;
    a.cols = cols;
    return device_status(fqimpl::launch_f8_decode(f8, a, (hipStream_t)stream), "decode launch");
}

size_t fq_linear_fwd_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts)
{
    const Product d = {rows, k, n, experts, 1};
    return check_product(d) == FQ_OK ? product_fwd_ws(d) : 0;
}

fq_status fq_linear_fwd(const void *x_bf16, const void *w_bf16, const void *bias,
                        int32_t bias_type, const void *res, int64_t rows, int64_t k, int64_t n,
                        int64_t experts, const int32_t *offsets, int32_t act, void *pre,
                        int32_t pre_f8, void *pre_scales, void *y, int32_t y_type, void *ws,
                        size_t ws_bytes, void *stream)
{
    const Product d = {rows, k, n, experts, 1};
    fqimpl::ProductArgs p;
    FQ_TRY(check_act(act));
    FQ_TRY(check_type(y_type, "y_type"));
    FQ_TRY(product_fwd(&p, d, x_bf16, w_bf16, bias, bias_type, offsets, pre, pre_f8, pre_scales));
    FQ_TRY(check_ptr(res, "res", false));
    FQ_TRY(check_ptr(y, "y", true));
    FQ_TRY(check_ws(ws, ws_bytes, product_fwd_ws(d)));
    p.act = act;
    p.res = res;
    p.y = y;
    p.splits = fwd_splits(d);
    p.partial = (float *)ws;
    p.y_f32 = y_type == FQ_TYPE_F32;
    return device_status(fqimpl::launch_product_linear(p, (hipStream_t)stream), "linear launch");
}

size_t fq_linear_bwd_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts,
                                    int32_t x_f8)
{
    return product_bwd_ws({rows, k, n, experts, 1}, x_f8);
}

fq_status fq_linear_bwd(const void *dy_bf16, const void *x, int32_t x_f8, const void *x_scales,
                        const void *w_bf16, const void *pre, int32_t pre_f8,
                        const void *pre_scales, int64_t rows, int64_t k, int64_t n,
                        int64_t experts, const int32_t *offsets, int32_t act, void *dx_bf16,
                        void *dw, int32_t dw_type, float *dbias, void *ws, size_t ws_bytes,
                        void *stream)
{
    FQ_TRY(check_act(act));
    return product_bwd({rows, k, n, experts, 1},
                       {dy_bf16, x, x_f8, x_scales, w_bf16, pre, pre_f8, pre_scales, offsets,
                        {act, 1.0f, INFINITY, 0.0f}, dx_bf16, dw, dw_type, dbias, nullptr, ws,
                        ws_bytes, (hipStream_t)stream});
}

size_t fq_glu_fwd_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts)
{
    const Product d = {rows, k, n, experts, 2};
    return check_product(d) == FQ_OK ? product_fwd_ws(d) : 0;
}

fq_status fq_glu_fwd(const fq_gate *gate, const void *x_bf16, const void *w_bf16,
                     const void *bias, int32_t bias_type, int64_t rows, int64_t k, int64_t n,
                     int64_t experts, const int32_t *offsets, void *pre, int32_t pre_f8,
                     void *pre_scales, void *h_bf16, void *ws, size_t ws_bytes, void *stream)
{
    const Product d = {rows, k, n, experts, 2};
    fqimpl::ProductArgs p;
    fqimpl::Gate g;
    FQ_TRY(check_gate(gate, &g));
    FQ_TRY(product_fwd(&p, d, x_bf16, w_bf16, bias, bias_type, offsets, pre, pre_f8, pre_scales));
    FQ_TRY(check_ptr(h_bf16, "h", true));
    FQ_TRY(check_ws(ws, ws_bytes, product_fwd_ws(d)));
    p.gate = g;
    p.y = h_bf16;
    p.splits = fwd_splits(d);
    p.partial = (float *)ws;
    return device_status(fqimpl::launch_product_glu(p, (hipStream_t)stream), "gated block launch");
}

size_t fq_glu_bwd_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts, int32_t x_f8)
{
    return product_bwd_ws({rows, k, n, experts, 2}, x_f8);
}

fq_status fq_glu_bwd(const fq_gate *gate, const void *dh_bf16, const void *x, int32_t x_f8,
                     const void *x_scales, const void *w_bf16, const void *pre, int32_t pre_f8,
                     const void *pre_scales, int64_t rows, int64_t k, int64_t n, int64_t experts,
                     const int32_t *offsets, void *dx_bf16, void *dw, int32_t dw_type,
                     float *dbias, void *h_bf16, void *ws, size_t ws_bytes, void *stream)
{
    fqimpl::Gate g;
    FQ_TRY(check_gate(gate, &g));
    return product_bwd({rows, k, n, experts, 2},
                       {dh_bf16, x, x_f8, x_scales, w_bf16, pre, pre_f8, pre_scales, offsets, g,
                        dx_bf16, dw, dw_type, dbias, h_bf16, ws, ws_bytes, (hipStream_t)stream});
}

}  // extern "C"

extern "C" {

const char *fq_status_string(fq_status s)
{
    switch (s) {
    case FQ_OK: return "FQ_OK";
    case FQ_ERR_NULL: return "FQ_ERR_NULL: a required pointer is NULL";
    case FQ_ERR_DESC: return "FQ_ERR_DESC: unsupported descriptor";
    case FQ_ERR_SHAPE: return "FQ_ERR_SHAPE: unsupported shape";
    case FQ_ERR_ALIGN: return "FQ_ERR_ALIGN: misaligned pointer";
    case FQ_ERR_WORKSPACE: return "FQ_ERR_WORKSPACE: workspace too small";
    case FQ_ERR_DEVICE: return "FQ_ERR_DEVICE: HIP launch failed";
    }
    return "unknown fq_status";
}

const char *fq_last_error(void) { return g_err; }

const char *fq_version(void) { return "0.1.0"; }

}  // extern "C"
