// fq_product_bwd.hip -- the backward's products: dx = dz w^T, both operands along
// the contraction, and dw = x^T dz, both across it.
#include "fq_product.hpp"

namespace fqimpl {

hipError_t launch_product_dx(ProductArgs p, hipStream_t stream)
{
    p.group = p.offsets ? 2 : 8;
    if (p.splits > 1) return launch_split<ALONG, ALONG, false>(p, p.N, EPI_STORE, stream);
    const float big = product_time<false>(p, 256, 256, 1, 1.44f, 10.0f);
    const float wide = product_time<false>(p, 256, 192, 1, 1.13f, 10.0f);
    const float small = product_time<false>(p, 128, 128, 2, 0.90f, 7.0f);
    if (small <= big && small <= wide) return launch_small<ALONG, ALONG, EPI_STORE, false>(p, stream);
    if (big <= wide) return launch_tiles<ALONG, ALONG, 4, 2, 2, 4, 2, EPI_STORE, false>(p, stream);
    return launch_tiles<ALONG, ALONG, 4, 3, 2, 2, 2, EPI_STORE, false>(p, stream);
}
hipError_t launch_product_dw(ProductArgs p, hipStream_t stream)
{
    p.group = p.offsets ? 2 : 8;
    if (p.splits > 1) return launch_split<ACROSS, ACROSS, true>(p, p.N, EPI_STORE, stream);
    const float big = product_time<true>(p, 256, 256, 1, 1.44f, 10.0f);
    const float mid = product_time<true>(p, 192, 192, 1, 0.96f, 9.0f);
    const float small = product_time<true>(p, 128, 128, 2, 0.95f, 7.0f);
    if (small <= big && small <= mid) return launch_small<ACROSS, ACROSS, EPI_STORE, true>(p, stream);
    if (big <= mid) return launch_tiles<ACROSS, ACROSS, 4, 2, 2, 4, 2, EPI_STORE, true>(p, stream);
    return launch_tiles<ACROSS, ACROSS, 3, 3, 2, 2, 2, EPI_STORE, true>(p, stream);
}

}  // namespace fqimpl
