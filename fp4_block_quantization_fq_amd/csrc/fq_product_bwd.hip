// fq_product_bwd.hip -- the backward's products: dx = dz w^T, both operands along
// the contraction, and dw = x^T dz, both across it.
#include "fq_product.hpp"

namespace {

enum { SMALL, WIDE, BIG };         // 128 x 128; 256 x 192 or 192 x 192, four waves; 256 x 256, eight

template <int TM, int TN, int WM, int WN, int STAGES>
using Dx = Shape<ALONG, ALONG, TM, TN, WM, WN, STAGES, EPI_STORE, false>;
template <int TM, int TN, int WM, int WN, int STAGES>
using Dw = Shape<ACROSS, ACROSS, TM, TN, WM, WN, STAGES, EPI_STORE, true>;

int dx_shape(const ProductArgs &p)
{
    if (p.splits > 1) return SMALL;
    const float big = product_time<false>(p, 256, 256, 1, 1.44f, 10.0f);
    const float wide = product_time<false>(p, 256, 192, 1, 1.13f, 10.0f);
    const float small = product_time<false>(p, 128, 128, 2, 0.90f, 7.0f);
    return small <= big && small <= wide ? SMALL : big <= wide ? BIG : WIDE;
}
int dw_shape(const ProductArgs &p)
{
    if (p.splits > 1) return SMALL;
    const float big = product_time<true>(p, 256, 256, 1, 1.44f, 10.0f);
    const float mid = product_time<true>(p, 192, 192, 1, 0.96f, 9.0f);
    const float small = product_time<true>(p, 128, 128, 2, 0.95f, 7.0f);
    return small <= big && small <= mid ? SMALL : big <= mid ? BIG : WIDE;
}
ProductArgs parts_of(const ProductArgs &p) { return p.splits > 1 ? split_args(p, p.N) : p; }

}  // namespace

namespace fqimpl {

// Where dx has small tiles the two share a launch: such products are bound by their
// latency, which then runs side by side (333 x 1000 -> 776 26.7 -> 18.9 us).  Two large
// ones gain nothing from it.
hipError_t launch_product_bwd(const ProductArgs *dx, const ProductArgs *dw, hipStream_t stream)
{
    ProductArgs x = {}, w = {};
    int xs = 0, ws = 0;
    if (dx) {
        x = parts_of(*dx);
        x.group = x.offsets ? 2 : 8;
        xs = dx_shape(*dx);
    }
    if (dw) {
        w = parts_of(*dw);
        w.group = w.offsets ? 2 : 8;
        ws = dw_shape(*dw);
    }
    hipError_t e = hipSuccess;
    if (dx && dw && xs == SMALL && ws == SMALL) {
        const bool few = shape_grid<Dx<2, 2, 2, 2, 4>>(x) + shape_grid<Dw<2, 2, 2, 2, 4>>(w) <= 256;
        if (few) e = launch_pair<Dx<2, 2, 2, 2, 4>, Dw<2, 2, 2, 2, 4>>(x, w, stream);
        else e = launch_pair<Dx<2, 2, 2, 2, 2>, Dw<2, 2, 2, 2, 2>>(x, w, stream);
    } else if (dx && dw && xs == SMALL && ws == WIDE) {
        e = launch_pair<Dx<2, 2, 2, 2, 3>, Dw<3, 3, 2, 2, 2>>(x, w, stream);
    } else {
        if (dx)
            e = xs == SMALL ? launch_small<ALONG, ALONG, EPI_STORE, false>(x, stream)
                : xs == BIG ? launch_shape<Dx<4, 2, 2, 4, 2>>(x, stream)
                            : launch_shape<Dx<4, 3, 2, 2, 2>>(x, stream);
        if (e == hipSuccess && dw)
            e = ws == SMALL ? launch_small<ACROSS, ACROSS, EPI_STORE, true>(w, stream)
                : ws == BIG ? launch_shape<Dw<4, 2, 2, 4, 2>>(w, stream)
                            : launch_shape<Dw<3, 3, 2, 2, 2>>(w, stream);
    }
    if (e == hipSuccess && dx && dx->splits > 1) e = launch_product_join(*dx, EPI_STORE, dx->partial, stream);
    if (e == hipSuccess && dw && dw->splits > 1) e = launch_product_join(*dw, EPI_STORE, dw->partial, stream);
    return e;
}

}  // namespace fqimpl
