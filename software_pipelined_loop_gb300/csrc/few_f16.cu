// few_f16.cu -- the kernels for a few rows, fp16.
#include "few_kernel.cuh"

namespace gp {

cudaError_t launch_few_f16(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    return l.four ? launch_few_type<false, true>(l, p, s) : launch_few_type<false, false>(l, p, s);
}

}  // namespace gp
