// pack4.cu -- weights into 4 bits with group scales, and back.
//
// A group is `group` rows k of one column.  Its scale is the largest magnitude
// over 7, rounded to the weights' type; a value is w / scale, rounded to the
// nearest whole number (ties to even), held between -8 and 7, plus 8.  A
// thread takes a group of one column, neighbours the next columns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "few.h"

namespace gp {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t v)
{
    if constexpr (BF16)
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else
        return __half2float(__ushort_as_half(v));
}

template <bool BF16>
__device__ __forceinline__ uint16_t to_bits(float v)
{
    if constexpr (BF16)
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        return __half_as_ushort(__float2half_rn(v));
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) pack4_kernel(int64_t experts, int64_t K, int64_t N, int group,
                                                         const uint16_t *W, uint32_t *Q, uint16_t *S)
{
    const int64_t n4 = (N + 3) / 4 * 4, groups = (K + group - 1) / group, words = (K + 7) / 8;
    const int64_t total = experts * groups * n4;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t n = i % n4, eg = i / n4, gr = eg % groups, e = eg / groups;
        const int64_t k0 = gr * group;
        const int rows = static_cast<int>(K - k0 < group ? K - k0 : group);
        const uint16_t *w = W + (e * K + k0) * N + n;
        float top = 0.0f;
        bool finite = true;
        if (n < N)
            for (int r = 0; r < rows; ++r) {
                const float v = fabsf(to_float<BF16>(w[r * N]));
                finite &= v <= 3.402823466e38f;
                top = fmaxf(top, v);
            }
        // (Past the last column: scale 0, values 0.)
        const uint16_t bits = finite ? to_bits<BF16>(__fdiv_rn(top, 7.0f)) : to_bits<BF16>(__int_as_float(0x7fffffff));
        const float scale = to_float<BF16>(bits);
        S[eg * n4 + n] = bits;
        for (int b = 0; b < rows; b += 8) {
            uint32_t word = 0;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float q = 0.0f;
                if (b + r < rows && scale > 0.0f)
                    q = fminf(fmaxf(rintf(__fdiv_rn(to_float<BF16>(w[(b + r) * N]), scale)), -8.0f), 7.0f);
                word |= static_cast<uint32_t>(static_cast<int>(q) + 8) << (4 * ((r >> 1) + 4 * (r & 1)));
            }
            Q[(e * words + (k0 + b) / 8) * n4 + n] = word;
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) unpack4_kernel(int64_t experts, int64_t K, int64_t N, int group,
                                                           const uint32_t *Q, const uint16_t *S, uint16_t *W)
{
    const int64_t n4 = (N + 3) / 4 * 4, groups = (K + group - 1) / group, words = (K + 7) / 8;
    const int64_t total = experts * words * N;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t n = i % N, ew = i / N, b = ew % words, e = ew / words;
        const uint32_t word = Q[ew * n4 + n];
        const float scale = to_float<BF16>(S[(e * groups + 8 * b / group) * n4 + n]);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int q = static_cast<int>(word >> (4 * ((r >> 1) + 4 * (r & 1))) & 15u) - 8;
            if (8 * b + r < K) W[(e * K + 8 * b + r) * N + n] = to_bits<BF16>(static_cast<float>(q) * scale);
        }
    }
}

unsigned blocks_of(int64_t total)
{
    const int64_t n = (total + kThreads - 1) / kThreads;
    return static_cast<unsigned>(n < (1 << 20) ? n : (1 << 20));
}

}  // namespace

cudaError_t launch_pack4(bool bf16, int64_t experts, int64_t K, int64_t N, int group, const uint16_t *W, uint32_t *Q,
                         uint16_t *S, cudaStream_t s)
{
    const unsigned grid = blocks_of(experts * ((K + group - 1) / group) * ((N + 3) / 4 * 4));
    if (bf16)
        pack4_kernel<true><<<grid, kThreads, 0, s>>>(experts, K, N, group, W, Q, S);
    else
        pack4_kernel<false><<<grid, kThreads, 0, s>>>(experts, K, N, group, W, Q, S);
    return cudaGetLastError();
}

cudaError_t launch_unpack4(bool bf16, int64_t experts, int64_t K, int64_t N, int group, const uint32_t *Q,
                           const uint16_t *S, uint16_t *W, cudaStream_t s)
{
    const unsigned grid = blocks_of(experts * ((K + 7) / 8) * N);
    if (bf16)
        unpack4_kernel<true><<<grid, kThreads, 0, s>>>(experts, K, N, group, Q, S, W);
    else
        unpack4_kernel<false><<<grid, kThreads, 0, s>>>(experts, K, N, group, Q, S, W);
    return cudaGetLastError();
}

}  // namespace gp
