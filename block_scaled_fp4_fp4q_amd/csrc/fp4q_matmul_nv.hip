// fp4q_matmul_nv.hip -- the products with NVFP4 weights, launched.
#include "fp4q_matmul_kernels.h"

namespace fp4q {

hipError_t launch_matmul_nv(const MatmulArgs& a, const MatmulPlan& p)
{
    return a.weights == 2 ? launch_weights<kNv, 2>(a, p) : launch_weights<kNv, 1>(a, p);
}

} // namespace fp4q
