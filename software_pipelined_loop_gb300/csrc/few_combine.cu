// few_combine.cu -- the tokens' sums of the rows that kFewParts left, one for
// each choice.  A thread takes one column of a token and adds its choices in
// order; the rows were written just before and are read from the L2 cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "few.h"
#include "ptx.cuh"

namespace gp {
namespace {

constexpr int kThreads = 128;

template <bool BF16>
__global__ void __launch_bounds__(kThreads) few_combine_kernel(int top_k, int experts, int64_t width,
                                                               const int32_t *ids, const float *parts, uint16_t *Y,
                                                               int64_t ldy)
{
    __shared__ int chosen[64];  // choices whose rows count
    __shared__ int count;
    pdl_launch_dependents();
    const int token = blockIdx.y;
    ids += static_cast<int64_t>(token) * top_k;
    if (threadIdx.x < 32) {  // top_k is at most 64: two choices a lane
        int n = 0;
        for (int j0 = 0; j0 < top_k; j0 += 32) {
            const int j = j0 + static_cast<int>(threadIdx.x);
            bool on = j < top_k;
            if (on) {
                const uint32_t e = static_cast<uint32_t>(ids[j]);
                on = e < static_cast<uint32_t>(experts);
                for (int i = 0; i < j && on; ++i) on = static_cast<uint32_t>(ids[i]) != e;
            }
            const uint32_t mask = __ballot_sync(0xffffffffu, on);
            if (on) chosen[n + __popc(mask & ((1u << threadIdx.x) - 1u))] = j;
            n += __popc(mask);
        }
        if (threadIdx.x == 0) count = n;
    }
    pdl_wait();  // the rows come from the launch before (the choices were there before both)
    __syncthreads();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (c >= width) return;
    const float *row = parts + static_cast<int64_t>(token) * top_k * width + c;
    float sum = 0.0f;
#pragma unroll 8
    for (int i = 0; i < count; ++i) sum += row[chosen[i] * width];
    uint16_t v;
    if constexpr (BF16) v = __bfloat16_as_ushort(__float2bfloat16_rn(sum));
    else v = __half_as_ushort(__float2half_rn(sum));
    Y[token * ldy + c] = v;
}

}  // namespace

cudaError_t launch_few_combine(bool bf16, int tokens, int top_k, int experts, int64_t width, const int32_t *ids,
                               const float *parts, uint16_t *Y, int64_t ldy, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((width + kThreads - 1) / kThreads), tokens, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, bf16 ? few_combine_kernel<true> : few_combine_kernel<false>, top_k,
                                             experts, width, ids, parts, Y, ldy);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gp
