// pack4.cu -- weights into 4 bits with group scales, and back.
//
// A group is `group` rows k of one column.  Its scale s is the largest
// magnitude over 7, rounded to the weights' type; a value is w / s, rounded to
// the nearest whole number (ties to even), held between -8 and 7, plus 8.
//
// A lane takes 8 neighbouring columns of the 8 rows of a word, 16 bytes of each
// row, and makes or takes apart its 8 words in registers.  Memory (2 bytes of a
// weight on one side, half a byte and its share of a scale on the other) bounds
// unpacking; packing and rows off 16-byte boundaries are bound by instructions:
// places come by shifts and grid dimensions, as a lane has 64 weights only and a
// division is as long as the work on ten.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "few.h"
#include "ptx.cuh"

namespace gp {
namespace {

constexpr int kThreads = 128;  // four warps: 128 rows of 64 columns (pack)

template <bool BF16>
__device__ __forceinline__ float to_float(uint32_t bits)
{
    if constexpr (BF16)
        return __uint_as_float(bits << 16);
    else
        return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

template <bool BF16>
__device__ __forceinline__ uint16_t to_bits(float v)
{
    if constexpr (BF16)
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        return __half_as_ushort(__float2half_rn(v));
}

// Eight 16-bit elements at p, the first `count` of them (others: whatever is
// there, or zeros).  Only aligned words that hold one of those are read.
template <bool ANY>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int count)
{
    if constexpr (!ANY) return ld_global_v4_if(p, count > 0);
    const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
    const char *a = reinterpret_cast<const char *>(p) - s;
    const uint4 lo = ld_global_v4_if(a, count > 0);
    const uint4 hi = ld_global_v4_if(a + 16, count > 0 && static_cast<int>(s) + 2 * count > 16);
    uint32_t o[4];
    realign16_steps(lo, hi, s, o);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i)
{
    return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// Larger of two pairs of 16-bit numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// About 1 / s, off by an ulp or two.
__device__ __forceinline__ float about_inverse(float s)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}

// m / 7 for a 16-bit value m: the product with about 1 / 7, corrected by its exact
// remainder.  Rounded to 16 bits it is what the quotient gives (checked for all values).
__device__ __forceinline__ float seventh(float m)
{
    const float t = m * (1.0f / 7.0f);
    return fmaf(fmaf(-7.0f, t, m), 1.0f / 7.0f, t);
}

constexpr float kRound = 12582912.0f;            // 1.5 * 2^23: a sum with it ends in the nearest whole number
constexpr uint32_t kRoundBits = 0x4b400000u;

// The word of a column's eight values x (scale s > 0, inv about 1 / s): whole
// numbers nearest to x / s, ties to even, plus 8.  The quotient is x * inv,
// corrected by its exact remainder: quotients of two 16-bit values are either
// exactly between two whole numbers, which the correction restores, or further
// from there than any error here.  They lie within 7.02 unless the scale has
// lost bits (CLAMP).  The whole number comes out of the last bits of a sum with
// kRound, and the eight are put together modulo 2^32, constants and all.
template <bool CLAMP>
__device__ __forceinline__ uint32_t word_from(const float (&x)[8], float s, float inv)
{
    uint32_t word = 0u - (kRoundBits - 8u) * 0x11111111u;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const float t = x[r] * inv;
        float q = fmaf(fmaf(-t, s, x[r]), inv, t);
        if (CLAMP) q = fminf(fmaxf(q, -8.0f), 7.0f);
        word += __float_as_uint(q + kRound) << (4 * ((r >> 1) + 4 * (r & 1)));
    }
    return word;
}

// grid: x = 64 columns, y = 128 rows, z = experts.  Groups of 1 << shift.
template <bool BF16, bool ANY>
__global__ void __launch_bounds__(kThreads, 7) pack4_kernel(int64_t K, int64_t N, int shift, int64_t tiles,
                                                            const uint16_t *W, uint32_t *Q, uint16_t *S)
{
    __shared__ uint32_t tops[4][32];
    const int64_t n4 = (N + 3) / 4 * 4, words = (K + 7) / 8;
    const int64_t groups = (K + (1 << shift) - 1) >> shift, e = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = lane >> 3;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 64 + 8 * (lane & 7);
    const int cols = n >= N ? 0 : (N - n < 8 ? static_cast<int>(N - n) : 8);
    const int together = 1 << (shift - 5);  // warps that share a group
    for (int64_t tile = blockIdx.y; tile < tiles; tile += gridDim.y) {
        const int64_t k0 = tile * 128 + 32 * warp + 8 * block;
        const int rows = k0 >= K ? 0 : (K - k0 < 8 ? static_cast<int>(K - k0) : 8);
        uint4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = load8<ANY>(W + (e * K + k0 + r) * N + n, r < rows ? cols : 0);
        // Largest magnitude of each column, by its bits: they are in the order
        // of the values, those that are not finite above all others.
        uint32_t top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            top[c] = word_of(v[0], c) & 0x7fff7fffu;
#pragma unroll
            for (int r = 1; r < 8; ++r) top[c] = max_u16x2(top[c], word_of(v[r], c) & 0x7fff7fffu);
#pragma unroll
            for (int d = 8; d < 32; d *= 2) top[c] = max_u16x2(top[c], __shfl_xor_sync(0xffffffffu, top[c], d));
        }
        if (together > 1) {
            if (block == 0)
#pragma unroll
                for (int c = 0; c < 4; ++c) tops[warp][4 * (lane & 7) + c] = top[c];
            __syncthreads();
            const int first = warp & -together;
            for (int w = first; w < first + together; ++w)
#pragma unroll
                for (int c = 0; c < 4; ++c) top[c] = max_u16x2(top[c], tops[w][4 * (lane & 7) + c]);
            __syncthreads();
        }
        constexpr uint32_t kInfinite = BF16 ? 0x7f80u : 0x7c00u, kNan = 0x7fffu, kNormal = BF16 ? 0x0080u : 0x0400u;
        uint32_t bits[8], word[8];
        bool lost = false;  // scales that are subnormal numbers
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint32_t most = c < cols ? (c & 1 ? top[c >> 1] >> 16 : top[c >> 1] & 0xffffu) : 0u;
            // (Past the last column: scale 0, values 0.)
            bits[c] = most >= kInfinite ? kNan : to_bits<BF16>(seventh(to_float<BF16>(most)));
            lost |= bits[c] != 0 && bits[c] < kNormal;
        }
        lost = __any_sync(0xffffffffu, lost);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float s = to_float<BF16>(bits[c]);
            float x[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const uint32_t two = word_of(v[r], c >> 1);
                x[r] = BF16 ? __uint_as_float(c & 1 ? two & 0xffff0000u : two << 16) : to_float<BF16>(c & 1 ? two >> 16 : two & 0xffffu);
            }
            word[c] = word_from<false>(x, s, about_inverse(s));
        }
        if (lost) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                uint32_t b = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) b = i == c ? bits[i] : b;
                // (the reciprocal of a scale below 2^-126 has no fp32 value)
                float s = to_float<BF16>(b), x[8];
                const float lift = s < 1e-30f ? 0x1p100f : 1.0f;
                s *= lift;
#pragma unroll
                for (int r = 0; r < 8; ++r) x[r] = to_float<BF16>((word_of(v[r], c >> 1) >> (16 * (c & 1))) & 0xffffu) * lift;
                const uint32_t w = word_from<true>(x, s, about_inverse(s));
#pragma unroll
                for (int i = 0; i < 8; ++i) word[i] = i == c ? w : word[i];
            }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (bits[c] == 0 || bits[c] == kNan) word[c] = 0x88888888u;
        if (rows > 0) {
            uint32_t *q = Q + (e * words + k0 / 8) * n4 + n;
            if (n < n4) *reinterpret_cast<uint4 *>(q) = make_uint4(word[0], word[1], word[2], word[3]);
            if (n + 4 < n4) *reinterpret_cast<uint4 *>(q + 4) = make_uint4(word[4], word[5], word[6], word[7]);
            if ((k0 & ((1 << shift) - 1)) == 0) {
                uint16_t *s = S + (e * groups + (k0 >> shift)) * n4 + n;
                if (n < n4) *reinterpret_cast<uint2 *>(s) = make_uint2(bits[0] | bits[1] << 16, bits[2] | bits[3] << 16);
                if (n + 4 < n4) *reinterpret_cast<uint2 *>(s + 4) = make_uint2(bits[4] | bits[5] << 16, bits[6] | bits[7] << 16);
            }
        }
    }
}

// The pair of rows 2i, 2i + 1 of a word, as values q - 8, exact (as in few_kernel.cuh).
template <bool BF16>
__device__ __forceinline__ uint32_t pair_of(uint32_t word, int i)
{
    uint32_t m;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(m) : "r"(word >> (4 * i)), "r"(0x000f000fu), "r"(BF16 ? 0x43004300u : 0x64006400u));
    if constexpr (BF16) {
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&m), __float2bfloat162_rn(136.0f));
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&m), __float2half2_rn(1032.0f));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// The product of 4 bits and a 16-bit scale, rounded once.
template <bool BF16>
__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b)
{
    if constexpr (BF16) {
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// A row of the warp's 256 columns off 16-byte boundaries: lane's 8 elements o,
// `left` of the row's columns from its first lane's on.  Each lane stores the
// whole piece that begins among its elements (the next lane has the rest), and
// single elements what lies before the first piece and after the last.
__device__ __forceinline__ void store_any(uint16_t *row, const uint32_t (&o)[4], int lane, int64_t left)
{
    const int total = left < 256 ? static_cast<int>(left) : 256;
    const int skip = static_cast<int>(((16u - (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u)) & 15u) / 2);  // 0 .. 7
    uint4 hi;
    hi.x = __shfl_down_sync(0xffffffffu, o[0], 1);
    hi.y = __shfl_down_sync(0xffffffffu, o[1], 1);
    hi.z = __shfl_down_sync(0xffffffffu, o[2], 1);
    hi.w = __shfl_down_sync(0xffffffffu, o[3], 1);
    uint32_t v[4];
    realign16_steps(make_uint4(o[0], o[1], o[2], o[3]), hi, 2 * skip, v);
    const int at = 8 * lane + skip;
    if (at + 8 <= total) *reinterpret_cast<uint4 *>(row + at) = make_uint4(v[0], v[1], v[2], v[3]);
    // Elements before the first piece, of lane 0, by lanes 0 .. 6; those behind
    // the last piece, of the last lanes with any, by lanes 8 .. 15.
    const int end = total < skip ? total : skip + (total - skip) / 8 * 8;  // where the pieces end
    const int i = lane < 8 ? lane : end + lane - 8;
    const bool on = lane < 8 ? lane < skip && lane < total : lane < 16 && end >= skip && i < total;
    const int from = on ? i / 8 : 0;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __shfl_sync(0xffffffffu, o[j], from);
    const uint32_t x = word_of(make_uint4(w[0], w[1], w[2], w[3]), (i & 7) >> 1);
    if (on) row[i] = static_cast<uint16_t>(x >> (16 * (i & 1)));
}

// grid: x = 256 columns; y = rows of words; z = experts.  A warp takes a row of words.
template <bool BF16, bool ANY>
__global__ void __launch_bounds__(kThreads) unpack4_kernel(int64_t K, int64_t N, int shift, int64_t words,
                                                           const uint32_t *Q, const uint16_t *S, uint16_t *W)
{
    const int64_t n4 = (N + 3) / 4 * 4, groups = (K + (1 << shift) - 1) >> shift, e = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * 256, n = first + 8 * lane;
    for (int64_t b = blockIdx.y * static_cast<int64_t>(kThreads / 32) + warp; b < words;
         b += static_cast<int64_t>(gridDim.y) * (kThreads / 32)) {
        const uint32_t *q = Q + (e * words + b) * n4 + n;
        const uint16_t *s = S + (e * groups + (8 * b >> shift)) * n4 + n;
        const uint4 qa = ld_global_v4_if(q, n < n4), qb = ld_global_v4_if(q + 4, n + 4 < n4);
        uint2 sa = make_uint2(0, 0), sb = sa;
        if (n < n4) sa = *reinterpret_cast<const uint2 *>(s);
        if (n + 4 < n4) sb = *reinterpret_cast<const uint2 *>(s + 4);
        const uint32_t word[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
        const uint32_t scale[4] = {sa.x, sa.y, sb.x, sb.y};
        const int rows = K - 8 * b < 8 ? static_cast<int>(K - 8 * b) : 8;
        uint16_t *w = W + (e * K + 8 * b) * N + n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t even[4], odd[4];  // rows 2i and 2i + 1, two columns a word
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t a = pair_of<BF16>(word[2 * c], i), b2 = pair_of<BF16>(word[2 * c + 1], i);
                even[c] = times<BF16>(__byte_perm(a, b2, 0x5410), scale[c]);
                odd[c] = times<BF16>(__byte_perm(a, b2, 0x7632), scale[c]);
            }
            if constexpr (ANY) {
                uint16_t *row = W + (e * K + 8 * b + 2 * i) * N + first;
                if (2 * i < rows) store_any(row, even, lane, N - first);
                if (2 * i + 1 < rows) store_any(row + N, odd, lane, N - first);
            } else if (n < N) {
                if (2 * i < rows) *reinterpret_cast<uint4 *>(w + 2 * i * N) = make_uint4(even[0], even[1], even[2], even[3]);
                if (2 * i + 1 < rows) *reinterpret_cast<uint4 *>(w + (2 * i + 1) * N) = make_uint4(odd[0], odd[1], odd[2], odd[3]);
            }
        }
    }
}

bool off16(const void *p, int64_t N) { return reinterpret_cast<uintptr_t>(p) % 16 != 0 || N % 8 != 0; }

dim3 grid_of(int64_t x, int64_t y, int64_t z)
{
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y < 65535 ? y : 65535), static_cast<unsigned>(z));
}

int shift_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

}  // namespace

cudaError_t launch_pack4(bool bf16, int64_t experts, int64_t K, int64_t N, int group, const uint16_t *W, uint32_t *Q,
                         uint16_t *S, cudaStream_t s)
{
    const int64_t tiles = (K + 127) / 128;
    const dim3 grid = grid_of((N + 63) / 64, tiles, experts);
    const auto kernel = off16(W, N) ? (bf16 ? pack4_kernel<true, true> : pack4_kernel<false, true>)
                                    : (bf16 ? pack4_kernel<true, false> : pack4_kernel<false, false>);
    kernel<<<grid, kThreads, 0, s>>>(K, N, shift_of(group), tiles, W, Q, S);
    return cudaGetLastError();
}

cudaError_t launch_unpack4(bool bf16, int64_t experts, int64_t K, int64_t N, int group, const uint32_t *Q,
                           const uint16_t *S, uint16_t *W, cudaStream_t s)
{
    const int64_t words = (K + 7) / 8;
    const bool any = off16(W, N);
    const dim3 grid = grid_of((N + 255) / 256, (words + kThreads / 32 - 1) / (kThreads / 32), experts);
    const auto kernel = any ? (bf16 ? unpack4_kernel<true, true> : unpack4_kernel<false, true>)
                                    : (bf16 ? unpack4_kernel<true, false> : unpack4_kernel<false, false>);
    kernel<<<grid, kThreads, 0, s>>>(K, N, shift_of(group), words, Q, S, W);
    return cudaGetLastError();
}

}  // namespace gp
