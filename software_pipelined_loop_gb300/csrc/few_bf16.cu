// few_bf16.cu -- the kernels for a few rows, bf16.
#include "few_kernel.cuh"

namespace gp {

cudaError_t launch_few_bf16(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    return l.four ? launch_few_type<true, true>(l, p, s) : launch_few_type<true, false>(l, p, s);
}

}  // namespace gp
