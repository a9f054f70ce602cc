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

constexpr int kThreads = 128;
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

// min(|a|, b) with a's sign (b positive).
__device__ __forceinline__ float clamp_abs(float a, float b)
{
    float r;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The bits of 1.5 * 2^23 + q: adding rounds x / step to a whole number, to
// nearest even, and leaves q's byte lowest.
__device__ __forceinline__ uint32_t whole_bits(float x, float inv)
{
    return __float_as_uint(clamp_abs(x * inv, 127.f) + 12582912.f);
}

// Eight values (two to a word) of one group to their bytes.
template <bool BF16>
__device__ __forceinline__ uint2 quantise8(const uint32_t (&w)[4], uint32_t byte)
{
    const float inv = per_step(byte & 255u);
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        b[2 * i] = whole_bits(value_of<BF16>(w[i] & 0xffffu), inv);
        b[2 * i + 1] = whole_bits(BF16 ? __uint_as_float(w[i] & 0xffff0000u) : value_of<BF16>(w[i] >> 16), inv);
    }
    uint2 q;
    q.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    q.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    if (byte == kNanStep) q = make_uint2(0, 0);
    return q;
}

// The largest magnitude of 8 values, as bits (an infinity or NaN is above all others).
__device__ __forceinline__ uint32_t top8(const uint32_t (&w)[4])
{
    const uint32_t a = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(w[0] & a, w[1] & a), __vmaxu2(w[2] & a, w[3] & a));
    return max(m & 0xffffu, m >> 16);
}

// The largest over the 4 lanes of a group.
__device__ __forceinline__ uint32_t top_of_group(uint32_t top)
{
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    return max(top, __shfl_xor_sync(0xffffffffu, top, 2));
}

// Dense rows of whole groups on 16-byte boundaries: one run of 8-value
// pieces, four lanes to a group, FLIGHT pieces per thread in flight.
constexpr int kFlight = 4;

template <bool BF16>
__global__ void __launch_bounds__(kThreads) keep8_dense_kernel(const uint16_t *X, int64_t n, int8_t *Q, uint8_t *S)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kFlight) + threadIdx.x;
    uint4 x[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
        x[k] = make_uint4(0, 0, 0, 0);
        if (i0 + k * kThreads < n) x[k] = ldg_nc_v4(X + 8 * (i0 + k * kThreads));
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
        const int64_t i = i0 + k * kThreads;
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        const uint32_t byte = step_byte<BF16>(top_of_group(top8(w)));
        const uint2 q = quantise8<BF16>(w, byte);
        if (i < n) {
            *reinterpret_cast<uint2 *>(Q + 8 * i) = q;
            if ((i & 3) == 0) S[i >> 2] = static_cast<uint8_t>(byte);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 restore_piece(uint2 q, float s0, float s1, int first)
{
    // The piece's elements before `first` have step s0, the others s1.
    uint32_t o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint32_t w = u < 2 ? q.x : q.y;
        const int lo = static_cast<int8_t>(w >> (16 * (u & 1))), hi = static_cast<int8_t>(w >> (16 * (u & 1) + 8));
        o[u] = bits_of<BF16>(static_cast<float>(lo) * (2 * u < first ? s0 : s1)) |
               (bits_of<BF16>(static_cast<float>(hi) * (2 * u + 1 < first ? s0 : s1)) << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) restore8_dense_kernel(const int8_t *Q, const uint8_t *S, int64_t n, uint16_t *X)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kFlight) + threadIdx.x;
    uint2 q[kFlight];
    uint32_t s[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
        const int64_t i = i0 + k * kThreads;
        q[k] = make_uint2(0, 0);
        s[k] = 0;
        if (i < n) {
            q[k] = *reinterpret_cast<const uint2 *>(Q + 8 * i);
            s[k] = S[i >> 2];
        }
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
        const int64_t i = i0 + k * kThreads;
        const float step = step_of(s[k]);
        if (i < n) *reinterpret_cast<uint4 *>(X + 8 * i) = restore_piece<BF16>(q[k], step, step, 8);
    }
}

// ---- any width, pitch and alignment: a warp takes 256 values of a row

// Eight bytes at p; only aligned words that hold a byte of [begin, end) are read.
__device__ __forceinline__ uint2 load_bytes(const char *p, const char *begin, const char *end)
{
    const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 7u);
    const char *a = p - shift;
    uint2 lo = make_uint2(0, 0), hi = lo;
    if (a < end && a + 8 > begin) lo = *reinterpret_cast<const uint2 *>(a);
    if (shift && a + 8 < end && a + 16 > begin) hi = *reinterpret_cast<const uint2 *>(a + 8);
    const bool b4 = (shift & 4u) != 0;
    const uint32_t w0 = b4 ? lo.y : lo.x, w1 = b4 ? hi.x : lo.y, w2 = b4 ? hi.y : hi.x, sh = (shift & 3u) * 8u;
    return make_uint2(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh));
}

constexpr int kSpan = 256;        // values a warp takes at once

// Warps that share a row: a power of two, as many as it has spans for.  (A
// block for each of 32768 rows of 100 values takes 34 us, a warp 10.)
__host__ __device__ __forceinline__ int warps_of_row(int spans)
{
    int w = 1;
    while (w < kThreads / 32 && w < spans) w *= 2;
    return w;
}

// A warp's part of a row: a block takes one or several short rows, `parts`
// blocks share a row of more than `take` spans.
struct RowPart {
    int64_t row;
    int span;  // the warp's first span; it takes every `step`-th up to `end`
    int step;
    int end;
};

__device__ __forceinline__ RowPart row_part(int spans, uint32_t parts, int take)
{
    RowPart p;
    p.step = warps_of_row(spans);
    const uint32_t block = blockIdx.x / parts, warp = threadIdx.x / 32;
    const int first = static_cast<int>(blockIdx.x - block * parts) * take;
    const uint32_t shift = static_cast<uint32_t>(__ffs(p.step) - 1);
    p.row = static_cast<int64_t>(block) * ((kThreads / 32) >> shift) + (warp >> shift);
    p.span = first + static_cast<int>(warp & (static_cast<uint32_t>(p.step) - 1u));
    p.end = first + take < spans ? first + take : spans;
    return p;
}

// The bytes of a span meet in shared memory and leave as the destination's
// own 8-byte words (rows of bytes start anywhere).
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    keep8_kernel(const uint16_t *X, int64_t rows, int width, int64_t ldx, uint32_t parts, int take,
                 int8_t *Q, uint8_t *S)
{
    __shared__ __align__(16) uint8_t stage[kThreads / 32][kSpan + 16];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    uint8_t *mine = stage[threadIdx.x >> 5];
    const RowPart p = row_part((width + kSpan - 1) / kSpan, parts, take);
    if (p.row >= rows) return;
    const uint16_t *x = X + p.row * ldx;
    uint8_t *steps = S + p.row * ((width + 31) / 32);
    uint8_t *q = reinterpret_cast<uint8_t *>(Q) + p.row * width;
    // Bytes of a span before the destination's first 8-byte word: the same in every span of a row.
    const int head = static_cast<int>((8 - (reinterpret_cast<uintptr_t>(q) & 7u)) & 7u);
    for (int sp = p.span; sp < p.end; sp += p.step) {
        const int e0 = sp * kSpan, e = e0 + 8 * lane;
        uint32_t w[4] = {0, 0, 0, 0};
        if (e + 8 <= width) {
            cut_words8(load_words8(x + e, true), x + e, w);
        } else {
            for (int u = 0; u < 8 && e + u < width; ++u)
                w[u >> 1] |= static_cast<uint32_t>(x[e + u]) << (16 * (u & 1));
        }
        const uint32_t byte = step_byte<BF16>(top_of_group(top8(w)));
        *reinterpret_cast<uint2 *>(mine + 8 * lane) = quantise8<BF16>(w, byte);
        if ((lane & 3) == 0 && e < width) steps[e >> 5] = static_cast<uint8_t>(byte);
        __syncwarp();
        const int have = width - e0 < kSpan ? width - e0 : kSpan;
        const int at = head + 8 * lane;
        if (at + 8 <= have) {
            const uint2 lo = *reinterpret_cast<const uint2 *>(mine + 8 * lane);
            const uint2 hi = *reinterpret_cast<const uint2 *>(mine + 8 * lane + 8);
            const bool b4 = (head & 4) != 0;
            const uint32_t w0 = b4 ? lo.y : lo.x, w1 = b4 ? hi.x : lo.y, w2 = b4 ? hi.y : hi.x, sh = (head & 3) * 8;
            *reinterpret_cast<uint2 *>(q + e0 + at) =
                make_uint2(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh));
        } else {
            for (int u = at; u < have; ++u) q[e0 + u] = mine[u];
        }
        if (lane < head && lane < have) q[e0 + lane] = mine[lane];
        __syncwarp();
    }
}

// A thread restores the values of one of the destination's 16-byte words;
// they may lie in two groups.
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    restore8_kernel(const int8_t *Q, const uint8_t *S, int64_t rows, int width, uint32_t parts, int take,
                    uint16_t *X, int64_t ldx)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const RowPart p = row_part((width + 7 + kSpan - 1) / kSpan, parts, take);
    if (p.row >= rows) return;
    const char *begin = reinterpret_cast<const char *>(Q), *end = begin + rows * width, *q = begin + p.row * width;
    const uint8_t *s = S + p.row * ((width + 31) / 32);
    uint16_t *x = X + p.row * ldx;
    const int before = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) >> 1);
    for (int sp = p.span; sp < p.end; sp += p.step) {
        const int e = sp * kSpan + 8 * lane - before;
        if (e >= width || e + 8 <= 0) continue;
        const int g0 = e > 0 ? e >> 5 : 0, g1 = (e + 7 < width ? e + 7 : width - 1) >> 5;
        const uint2 b = load_bytes(q + e, begin, end);
        const float s0 = step_of(s[g0]), s1 = step_of(s[g1]);
        const uint4 v = restore_piece<BF16>(b, s0, s1, 32 * (g0 + 1) - e);
        if (e >= 0 && e + 8 <= width) {
            *reinterpret_cast<uint4 *>(x + e) = v;
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (e + u >= 0 && e + u < width) x[e + u] = static_cast<uint16_t>(w[u >> 1] >> (16 * (u & 1)));
        }
    }
}

// Rows to aligned rows, a warp per row.  With `offsets`, rows of an expert
// (per_expert rows each) that has no row to multiply are left out: raw bounds
// that do not rise from e to e + 1 give it none, however they are clamped.
__global__ void __launch_bounds__(kThreads)
    repitch_kernel(const uint16_t *src, int64_t rows, int64_t width, int64_t lds, uint16_t *dst, int64_t ldd,
                   const int32_t *offsets, int64_t per_expert)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
    if (r >= rows) return;
    if (offsets) {
        const int64_t e = r / per_expert;
        if (offsets[e + 1] <= offsets[e]) return;
    }
    const uint16_t *x = src + r * lds;
    uint16_t *o = dst + r * ldd;
    const int64_t whole = width / 8;
    constexpr int FLIGHT = 4;
    for (int64_t i = lane; i < whole; i += 32 * FLIGHT) {
        Words8 v[FLIGHT];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) v[u] = load_words8(x + 8 * (i + 32 * u), i + 32 * u < whole);
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            uint32_t w[4];
            cut_words8(v[u], x + 8 * (i + 32 * u), w);
            if (i + 32 * u < whole)
                *reinterpret_cast<uint4 *>(o + 8 * (i + 32 * u)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    if (8 * whole < ldd && lane < 8) o[8 * whole + lane] = 8 * whole + lane < width ? x[8 * whole + lane] : uint16_t(0);
}

template <class... P, class... A>
cudaError_t launch(void (*k)(P...), int64_t work, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(static_cast<unsigned>((work + kThreads - 1) / kThreads), 1, 1);
    c.blockDim = dim3(kThreads, 1, 1);
    c.stream = s;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = a;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k, static_cast<P>(args)...);
}

// Blocks for rows of `values` values (at most 2^30 and a few: places within a
// row are 32-bit).  A block takes up to 32 spans of a row; 8 of few rows, which
// leave SMs free.  Rows of 4001, kept: 64 rows 2.3 us with 8 spans, 3.3 with
// 32; 32768 rows 117 and 110.  (32768 rows of 4001 and 2001 with 256 threads:
// 121 and 72 us, 111 and 62 with 128.)
struct RowBlocks {
    int take;
    int64_t parts, all;
    RowBlocks(int64_t rows, int64_t values)
    {
        const int64_t spans = (values + kSpan - 1) / kSpan;
        const int of_block = kThreads / 32 / warps_of_row(static_cast<int>(spans));
        take = rows <= 1024 ? 8 : 32;
        parts = (spans + take - 1) / take;
        all = (rows + of_block - 1) / of_block * parts;
    }
};

// Rows that are one run of whole groups, on the accesses' boundaries, in at
// most 2^31 - 1 blocks.
bool dense(const void *X, int64_t ldx, const void *Q, int64_t rows, int64_t width)
{
    return width % 32 == 0 && ldx == width && reinterpret_cast<uintptr_t>(X) % 16 == 0 &&
           reinterpret_cast<uintptr_t>(Q) % 8 == 0 && rows * (width / 8) < (int64_t(1) << 39);
}

}  // namespace

cudaError_t launch_keep8(bool bf16, int64_t rows, int64_t width, const uint16_t *X, int64_t ldx, int8_t *Q,
                         uint8_t *S, cudaStream_t s)
{
    if (dense(X, ldx, Q, rows, width)) {
        const int64_t n = rows * (width / 8);
        return launch(bf16 ? keep8_dense_kernel<true> : keep8_dense_kernel<false>, (n + kFlight - 1) / kFlight, s, X, n,
                      Q, S);
    }
    const RowBlocks b(rows, width);
    return launch(bf16 ? keep8_kernel<true> : keep8_kernel<false>, b.all * kThreads, s, X, rows,
                  static_cast<int>(width), ldx, static_cast<uint32_t>(b.parts), b.take, Q, S);
}

cudaError_t launch_restore8(bool bf16, int64_t rows, int64_t width, const int8_t *Q, const uint8_t *S, uint16_t *X,
                            int64_t ldx, cudaStream_t s)
{
    if (dense(X, ldx, Q, rows, width)) {
        const int64_t n = rows * (width / 8);
        return launch(bf16 ? restore8_dense_kernel<true> : restore8_dense_kernel<false>, (n + kFlight - 1) / kFlight, s,
                      Q, S, n, X);
    }
    const RowBlocks b(rows, width + 7);
    return launch(bf16 ? restore8_kernel<true> : restore8_kernel<false>, b.all * kThreads, s, Q, S, rows,
                  static_cast<int>(width), static_cast<uint32_t>(b.parts), b.take, X, ldx);
}

cudaError_t launch_repitch(const uint16_t *src, int64_t rows, int64_t width, int64_t lds, uint16_t *dst, int64_t ldd,
                           const int32_t *offsets, int64_t per_expert, cudaStream_t s)
{
    return launch(repitch_kernel, rows * 32, s, src, rows, width, lds, dst, ldd, offsets, per_expert);
}

}  // namespace gp
