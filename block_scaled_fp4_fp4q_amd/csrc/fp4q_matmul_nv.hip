// fp4q_matmul_nv.hip -- the products with NVFP4 weights, launched.
#include "fp4q_matmul_kernels.h"

namespace fp4q {

namespace {

template <int NW>
hipError_t launch_weights(const MatmulArgs& a, const MatmulPlan& p)
{
    if (p.prepared) {
        const dim3 rows((uint32_t)(a.m < 65536 ? a.m : 65536), (uint32_t)((a.m + 65535) / 65536));
        if (p.parts == 1)
            matmul_halves<1><<<rows, 256, 0, a.stream>>>(a, p);
        else
            matmul_halves<2><<<rows, 256, 0, a.stream>>>(a, p);
    }
    if (p.many) {
        if (p.prepared)
            many_form<kNvF16, NW>(a, p);
        else
            many_form<kNvBf16, NW>(a, p);
    } else if (p.prepared) {
        if (p.parts == 1 && p.tokens == 32)
            few_form<kNvF16, NW, 1, false, 2>(a, p);
        else if (p.parts == 1)
            few_form<kNvF16, NW, 1, false>(a, p);
        else
            few_form<kNvF16, NW, 2, false>(a, p);
    } else {
        switch (p.parts) {
        case 1:
            if (p.tokens == 32)
                few_form<kNvBf16, NW, 1, false, 2>(a, p);
            else
                few_form<kNvBf16, NW, 1, false>(a, p);
            break;
        case 2: few_form<kNvBf16, NW, 2, true>(a, p); break;
        default: few_form<kNvBf16, NW, 3, true>(a, p); break;
        }
    }
    return hipGetLastError();
}

} // namespace

hipError_t launch_matmul_nv(const MatmulArgs& a, const MatmulPlan& p)
{
    return a.weights == 2 ? launch_weights<2>(a, p) : launch_weights<1>(a, p);
}

} // namespace fp4q
