// fp4q_matmul_mx.hip -- the products with MXFP4 weights, launched.
#include "fp4q_matmul_kernels.h"

namespace fp4q {

hipError_t launch_matmul_mx(const MatmulArgs& a, const MatmulPlan& p)
{
    return a.weights == 2 ? launch_weights<kMx, 2>(a, p) : launch_weights<kMx, 1>(a, p);
}

} // namespace fp4q
