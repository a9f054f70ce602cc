// keep8.cu -- rows of activations kept in 8 bits, and brought back.
//
// 32 neighbouring values of a row share one power of two, step = 2^(m - 6)
// with m the exponent of the group's largest magnitude: that value becomes 64
// to 127 steps.  A value is stored as q = x / step rounded to the nearest
// whole number (ties to even), clamped to [-127, 127]; the step as the byte
// m - 6 + 127.  Powers of two keep the arithmetic exact: x / step has no
// rounding of its own, and q * step fits 16-bit floating point exactly (q has
// 7 bits), so the tensor cores multiply exactly the values that are stored.
// The exponent is held at or above that of the type's finest step (-24 for
// fp16, where the copy is then exact) or the byte's range (-127).  A group
// with an infinity or NaN has the byte 255 and comes back as NaN.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts.h"
#include "ptx.cuh"

namespace gp {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kNanStep = 255;

template <bool BF16>
__device__ __forceinline__ float value_of(uint32_t bits)
{
    if constexpr (BF16)
        return __uint_as_float(bits << 16);
    else
        return __half2float(__ushort_as_half(static_cast<uint16_t>(bits)));
}

template <bool BF16>
__device__ __forceinline__ uint32_t bits_of(float v)
{
    if constexpr (BF16)
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        return __half_as_ushort(__float2half_rn(v));
}

// Step byte of a group whose largest magnitude has these bits.
template <bool BF16>
__device__ __forceinline__ uint32_t step_byte(uint32_t top)
{
    if (top >= (BF16 ? 0x7f80u : 0x7c00u)) return kNanStep;
    const int m = static_cast<int>(__float_as_uint(value_of<BF16>(top)) >> 23) - 127;
    const int least = BF16 ? -127 : -24;
    const int e = m - 6 < least ? least : m - 6;
    return static_cast<uint32_t>(e + 127);
}

// 1 / step; the byte is at most 248, so this is a normal number.
__device__ __forceinline__ float per_step(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ float step_of(uint32_t byte)
{
    return byte == kNanStep ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

template <bool BF16>
__device__ __forceinline__ uint32_t quantise(uint32_t bits, float inv)
{
    const float q = fminf(fmaxf(rintf(value_of<BF16>(bits) * inv), -127.f), 127.f);
    return static_cast<uint32_t>(static_cast<int>(q)) & 255u;
}

// Four lanes hold a group, 8 values each.
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    keep8_wide_kernel(const uint16_t *X, int64_t rows, int64_t pieces, int64_t ldx, int8_t *Q, uint8_t *S)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t n = rows * pieces;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i - threadIdx.x % 32 < n;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const bool has = i < n;
        const int64_t r = has ? i / pieces : 0, c = has ? i - r * pieces : 0;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (has) x = ldg_nc_v4(X + r * ldx + 8 * c);
        const uint32_t a = 0x7fff7fffu;
        const uint32_t m2 = __vmaxu2(__vmaxu2(x.x & a, x.y & a), __vmaxu2(x.z & a, x.w & a));
        uint32_t top = (m2 & 0xffffu) > (m2 >> 16) ? (m2 & 0xffffu) : (m2 >> 16);
        uint32_t o = __shfl_xor_sync(0xffffffffu, top, 1);
        top = o > top ? o : top;
        o = __shfl_xor_sync(0xffffffffu, top, 2);
        top = o > top ? o : top;
        const uint32_t byte = step_byte<BF16>(top);
        const float inv = byte == kNanStep ? 0.f : per_step(byte);
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t q[2] = {0, 0};
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t b = (w[u >> 1] >> (16 * (u & 1))) & 0xffffu;
            q[u >> 2] |= (byte == kNanStep ? 0u : quantise<BF16>(b, inv)) << (8 * (u & 3));
        }
        if (has) {
            *reinterpret_cast<uint2 *>(Q + 8 * i) = make_uint2(q[0], q[1]);
            if ((i & 3) == 0) S[i >> 2] = static_cast<uint8_t>(byte);
        }
    }
}

// Any width, pitch and alignment: a warp per group, a value per lane.
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    keep8_kernel(const uint16_t *X, int64_t rows, int64_t width, int64_t ldx, int8_t *Q, uint8_t *S)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t groups = (width + 31) / 32, n = rows * groups;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; g < n; g += warps) {
        const int64_t r = g / groups, c = (g - r * groups) * 32 + lane;
        const uint32_t b = c < width ? X[r * ldx + c] : 0u;
        const uint32_t byte = step_byte<BF16>(__reduce_max_sync(0xffffffffu, b & 0x7fffu));
        if (c < width) Q[r * width + c] = byte == kNanStep ? 0 : static_cast<int8_t>(quantise<BF16>(b, per_step(byte)));
        if (lane == 0) S[g] = static_cast<uint8_t>(byte);
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    restore8_wide_kernel(const int8_t *Q, const uint8_t *S, int64_t rows, int64_t pieces, uint16_t *X, int64_t ldx)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t n = rows * pieces;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / pieces, c = i - r * pieces;
        const uint2 q = *reinterpret_cast<const uint2 *>(Q + 8 * i);
        const float step = step_of(S[i >> 2]);
        uint32_t o[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t w = u < 2 ? q.x : q.y;
            const int lo = static_cast<int8_t>(w >> (16 * (u & 1))), hi = static_cast<int8_t>(w >> (16 * (u & 1) + 8));
            o[u] = bits_of<BF16>(lo * step) | (bits_of<BF16>(hi * step) << 16);
        }
        *reinterpret_cast<uint4 *>(X + r * ldx + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    restore8_kernel(const int8_t *Q, const uint8_t *S, int64_t rows, int64_t width, uint16_t *X, int64_t ldx)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t groups = (width + 31) / 32, n = rows * groups;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; g < n; g += warps) {
        const int64_t r = g / groups, c = (g - r * groups) * 32 + lane;
        const float step = step_of(S[g]);
        if (c < width) X[r * ldx + c] = static_cast<uint16_t>(bits_of<BF16>(Q[r * width + c] * step));
    }
}

__global__ void __launch_bounds__(kThreads)
    repitch_kernel(const uint16_t *src, int64_t rows, int64_t width, int64_t lds, uint16_t *dst, int64_t ldd)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t pieces = ldd / 8, n = rows * pieces;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / pieces, c = (i - r * pieces) * 8;
        uint32_t o[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t lo = c + 2 * u < width ? src[r * lds + c + 2 * u] : 0u;
            const uint32_t hi = c + 2 * u + 1 < width ? src[r * lds + c + 2 * u + 1] : 0u;
            o[u] = lo | (hi << 16);
        }
        *reinterpret_cast<uint4 *>(dst + r * ldd + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <class... P, class... A>
cudaError_t launch(void (*k)(P...), int64_t work, int sms, cudaStream_t s, A... args)
{
    const int64_t blocks = (work + kThreads - 1) / kThreads, most = static_cast<int64_t>(sms) * 8;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most), 1, 1);
    c.blockDim = dim3(kThreads, 1, 1);
    c.stream = s;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = a;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k, static_cast<P>(args)...);
}

bool wide(const void *X, int64_t ldx, const void *Q, int64_t width)
{
    return width % 32 == 0 && ldx % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0 &&
           reinterpret_cast<uintptr_t>(Q) % 8 == 0;
}

}  // namespace

cudaError_t launch_keep8(bool bf16, int64_t rows, int64_t width, const uint16_t *X, int64_t ldx, int8_t *Q,
                         uint8_t *S, int sms, cudaStream_t s)
{
    if (wide(X, ldx, Q, width))
        return launch(bf16 ? keep8_wide_kernel<true> : keep8_wide_kernel<false>, rows * (width / 8), sms, s, X, rows,
                      width / 8, ldx, Q, S);
    return launch(bf16 ? keep8_kernel<true> : keep8_kernel<false>, rows * ((width + 31) / 32) * 32, sms, s, X, rows,
                  width, ldx, Q, S);
}

cudaError_t launch_restore8(bool bf16, int64_t rows, int64_t width, const int8_t *Q, const uint8_t *S, uint16_t *X,
                            int64_t ldx, int sms, cudaStream_t s)
{
    if (wide(X, ldx, Q, width))
        return launch(bf16 ? restore8_wide_kernel<true> : restore8_wide_kernel<false>, rows * (width / 8), sms, s, Q,
                      S, rows, width / 8, X, ldx);
    return launch(bf16 ? restore8_kernel<true> : restore8_kernel<false>, rows * ((width + 31) / 32) * 32, sms, s, Q,
                  S, rows, width, X, ldx);
}

cudaError_t launch_repitch(const uint16_t *src, int64_t rows, int64_t width, int64_t lds, uint16_t *dst, int64_t ldd,
                           int sms, cudaStream_t s)
{
    return launch(repitch_kernel, rows * (ldd / 8), sms, s, src, rows, width, lds, dst, ldd);
}

}  // namespace gp
