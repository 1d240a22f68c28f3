// fp4q_matmul_mx.hip -- the products with MXFP4 weights, launched.
#include "fp4q_matmul_kernels.h"

namespace fp4q {

namespace {

template <int NW>
hipError_t launch_weights(const MatmulArgs& a, const MatmulPlan& p)
{
    if (p.prepared) {
        const int64_t all = (a.m * (a.k / 32) + 255) / 256;
        const dim3 cover((uint32_t)(all < 1 ? 1 : (all < 65536 ? all : 65536)));
        if (p.parts == 2)
            matmul_parts<2><<<cover, 256, 0, a.stream>>>(a);
        else
            matmul_parts<3><<<cover, 256, 0, a.stream>>>(a);
    }
    if (p.many) {
        many_form<kMxBf16, NW>(a, p);
    } else {
        switch (p.parts) {
        case 1:
            if (p.tokens == 32)
                few_form<kMxBf16, NW, 1, false, 2>(a, p);
            else
                few_form<kMxBf16, NW, 1, false>(a, p);
            break;
        case 2:
            if (p.prepared)
                few_form<kMxBf16, NW, 2, false>(a, p);
            else
                few_form<kMxBf16, NW, 2, true>(a, p);
            break;
        default:
            if (p.prepared)
                few_form<kMxBf16, NW, 3, false>(a, p);
            else
                few_form<kMxBf16, NW, 3, true>(a, p);
            break;
        }
    }
    return hipGetLastError();
}

} // namespace

hipError_t launch_matmul_mx(const MatmulArgs& a, const MatmulPlan& p)
{
    return a.weights == 2 ? launch_weights<2>(a, p) : launch_weights<1>(a, p);
}

} // namespace fp4q
