// fq_product_fwd.hip -- the forward products: x w, w across the contraction.
#include "fq_product.hpp"

namespace {

using fqimpl::product_few_rows;

bool few_rows(const ProductArgs &p) { return product_few_rows(p.M, p.offsets ? p.experts : 0); }

template <int EPI>
hipError_t launch_linear(const ProductArgs &p, hipStream_t stream)
{
    const float big = product_time<false>(p, 256, 256, 1, 1.46f, 12.0f);
    const float wide = product_time<false>(p, 256, 192, 1, 1.15f, 10.0f);
    const float small = product_time<false>(p, 128, 128, 2, 0.90f, 8.0f);
    if (small <= big && small <= wide) return launch_small<ALONG, ACROSS, EPI, false>(p, stream);
    if (big <= wide) return launch_tiles<ALONG, ACROSS, 4, 2, 2, 4, 2, EPI, false>(p, stream);
    return launch_tiles<ALONG, ACROSS, 4, 3, 2, 2, 2, EPI, false>(p, stream);
}

}  // namespace

namespace fqimpl {

hipError_t launch_product_linear(ProductArgs p, hipStream_t stream)
{
    p.group = p.offsets ? 2 : 8;
    if (few_rows(p)) return launch_product_few_linear(p, stream);
    if (p.splits > 1) return launch_split<ALONG, ACROSS, false>(p, p.N, EPI_LINEAR, stream);
    if (p.act == ACT_NONE && p.pre_kind == PRE_NONE) return launch_linear<EPI_RES>(p, stream);
    return launch_linear<EPI_LINEAR>(p, stream);
}
hipError_t launch_product_glu(ProductArgs p, hipStream_t stream)
{
    p.group = 8;
    if (few_rows(p)) return launch_product_few_glu(p, stream);
    if (p.splits > 1) return launch_split<ALONG, ACROSS, false>(p, 2 * p.N, EPI_GLU, stream);
    // Experts of few rows each are bound by their weights, which more and smaller
    // workgroups read faster.  32 experts, 2880 -> 2 x 2880, us in tiles of 128 x 64 / 256 x
    // 128, segments of even and of uneven lengths: 65 rows each 206 / 236 and 220 / 237, 96
    // 221 / 241 and 266 / 255, 128 235 / 250 and 307 / 263, 160 330 / 276 and 336 / 320, 192
    // 339 / 286 and 365 / 333, 256 382 / 305 and 455 / 404, 512 679 / 519 and 733 / 641.  The
    // border is late for these: they cross between 96 and 160 rows.
    const bool short_segments = p.offsets && p.M < 192 * (int64_t)p.experts;
    const float big = product_time<false>(p, 256, 128, 1, 1.46f, 15.0f);
    const float small = product_time<false>(p, 128, 64, 2, p.offsets ? 1.13f : 0.90f, 10.0f);
    if (short_segments || small <= big) return launch_small<ALONG, ACROSS, EPI_GLU, false>(p, stream);
    return launch_tiles<ALONG, ACROSS, 4, 2, 2, 4, 2, EPI_GLU, false>(p, stream);
}

}  // namespace fqimpl
