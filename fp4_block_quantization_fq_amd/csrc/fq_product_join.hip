// fq_product_join.hip -- the second half of products whose contraction is split over
// workgroups: the parts, FP32 [splits, M, columns] in the workspace, are added in
// their order and go through the epilogue that the tile kernel would have applied.
//
// Where a product has fewer tiles than the chip has room for, its time is the
// latency of its steps: 128 x 2880 -> 2880 took 30 us on 23 workgroups, 15 with its
// contraction in four parts and this kernel.
#include "fq_product.hpp"

namespace {

template <int EPI>
__global__ __launch_bounds__(256) void k_join(const ProductArgs p, const float *part, int64_t chunks)
{
    const int64_t step = (int64_t)gridDim.x * 256;
    const int per_row = p.N / 8;
    const int64_t cols = EPI == EPI_GLU ? 2 * (int64_t)p.N : p.N, size = p.M * cols;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < chunks; id += step) {
        const int64_t row = (uint32_t)id / (uint32_t)per_row;      // chunks are below 2^31
        const int col = (int)(id - row * per_row) * 8;
        const float *from = part + row * cols + col;
        float z[8] = {}, u[8] = {};
        for (int s = 0; s < p.splits; ++s) {
            float v[8];
            load8<false>(from + s * size, 8, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += v[e];
            if (EPI == EPI_GLU) {
                load8<false>(from + s * size + p.N, 8, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] += v[e];
            }
        }
        if (EPI == EPI_STORE) {
            store_y(p, row * p.N + col, z);
            continue;
        }
        float bias[8], bias_up[8];
        load_bias(p, col, bias);
        if (EPI == EPI_GLU) {
            load_bias(p, col + p.N, bias_up);
            finish_glu(p, row, col, p.N, z, u, bias, bias_up);
        } else {
            if (p.res) load_res(p, row * p.N + col, u);
            finish_linear(p, row, col, p.N, z, bias, u);
        }
    }
}

}  // namespace

namespace fqimpl {

// Parts of the contraction for one product of 128 x 128 tiles: the fewest that are
// worth their join.  Steps of 64 k take 0.55 us alone on a CU, 0.9 where two
// workgroups share it; a join some 4 us and its bytes.
int product_splits(int64_t M, int64_t N, int64_t K)
{
    const int64_t tiles = (M + 127) / 128 * ((N + 127) / 128), steps = (K + 63) / 64;
    if (tiles >= 256) return 1;
    int best = 1;
    float least = 0;
    for (int s = 1; s <= kProductMaxSplits && steps / s >= 4; s *= 2) {
        const int64_t n = tiles * s;
        const float step = n <= 256 ? 0.55f : 0.9f, rounds = (float)((n + 511) / 512);
        const float time = rounds * ((steps + s - 1) / s * step + 5.0f) +
                           (s > 1 ? 4.0f + (float)(s * M * N) * 8.0f / 4e6f : 0.0f);
        if (s == 1 || time < 0.9f * least) {
            least = time;
            best = s;
        }
    }
    return best;
}

hipError_t launch_product_join(ProductArgs p, int epilogue, const float *part, hipStream_t stream)
{
    const int64_t chunks = (int64_t)p.M * p.N / 8;
    const int64_t n = (chunks + 255) / 256;
    const dim3 grid((uint32_t)(n < 4096 ? n : 4096)), block(256);
    if (epilogue == EPI_GLU) hipLaunchKernelGGL((k_join<EPI_GLU>), grid, block, 0, stream, p, part, chunks);
    else if (epilogue == EPI_STORE) hipLaunchKernelGGL((k_join<EPI_STORE>), grid, block, 0, stream, p, part, chunks);
    else hipLaunchKernelGGL((k_join<EPI_LINEAR>), grid, block, 0, stream, p, part, chunks);
    return hipGetLastError();
}

}  // namespace fqimpl
