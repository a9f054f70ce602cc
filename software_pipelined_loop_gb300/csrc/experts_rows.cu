// experts_rows.cu -- tokens sorted by expert, their rows dealt out and the
// experts' rows summed back, with the gradient of that sum.
//
// A token t has top_k choices; choice j is slot s = t * top_k + j.  A stable
// counting sort by expert gives every slot a row.  Slots whose id is outside
// [0, experts) are dropped: they sort behind all others and are marked by the
// complement (rows[s] = ~r), so that every buffer of tokens * top_k rows has a
// place for them and nothing reads it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "experts.h"
#include "ptx.cuh"

namespace gp {
namespace {

// ------------------------------------------------------------------- sort

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kSortChunk = 2048;  // slots of a block, at least
constexpr int kSortBlocks = 256;      // blocks, at most

__device__ __forceinline__ int bin_of(int32_t id, int experts)
{
    return static_cast<uint32_t>(id) < static_cast<uint32_t>(experts) ? id : experts;
}

// Per block: how many of its slots each expert has (bin `experts`: dropped).
__global__ void __launch_bounds__(kSortThreads) route_count_kernel(const int32_t *ids, int64_t slots, int64_t chunk,
                                                                   int experts, int32_t *counts)
{
    extern __shared__ int32_t hist[];
    pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i <= experts; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    const int64_t beg = blockIdx.x * chunk, end = beg + chunk < slots ? beg + chunk : slots;
    for (int64_t s = beg + threadIdx.x; s < end; s += kSortThreads) atomicAdd(&hist[bin_of(ids[s], experts)], 1);
    __syncthreads();
    for (int i = threadIdx.x; i <= experts; i += kSortThreads)
        counts[static_cast<int64_t>(blockIdx.x) * (experts + 1) + i] = hist[i];
}

// The places: rows of the bins, then of the blocks within a bin, then of the
// warps within a block (each has consecutive slots), then of the lanes.
__global__ void __launch_bounds__(kSortThreads)
    route_place_kernel(const int32_t *ids, int64_t slots, int64_t chunk, int experts, const int32_t *counts,
                       int32_t *offsets, int32_t *slot_of_row, int32_t *rows)
{
    extern __shared__ int32_t sm[];
    const int bins = experts + 1;
    int32_t *total = sm, *before = sm + bins, *mine = sm + 2 * bins;  // mine: [warp][bin]
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) mine[i] = 0;
    __syncthreads();
    const int64_t per = (chunk + kSortWarps - 1) / kSortWarps;
    const int64_t block_end = (blockIdx.x + 1) * chunk < slots ? (blockIdx.x + 1) * chunk : slots;
    const int64_t beg = blockIdx.x * chunk + warp * per;
    const int64_t end = beg + per < block_end ? beg + per : block_end;
    for (int64_t s0 = beg; s0 < end; s0 += 32) {
        const bool has = s0 + lane < end;
        const int b = has ? bin_of(ids[s0 + lane], experts) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, b);
        if (has && (same & ((1u << lane) - 1u)) == 0) mine[warp * bins + b] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
        int32_t all = 0, prior = 0;
        if (counts) {
            for (unsigned k = 0; k < gridDim.x; ++k) {
                const int32_t c = counts[static_cast<int64_t>(k) * bins + b];
                all += c;
                if (k < blockIdx.x) prior += c;
            }
        } else {
            for (int w = 0; w < kSortWarps; ++w) all += mine[w * bins + b];
        }
        total[b] = all;
        before[b] = prior;
    }
    __syncthreads();
    if (warp == 0) {
        int32_t sum = 0;
        for (int b0 = 0; b0 < bins; b0 += 32) {
            const int b = b0 + lane;
            const int32_t n = b < bins ? total[b] : 0;
            int32_t x = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t u = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += u;
            }
            if (b < bins) total[b] = sum + x - n;  // rows of the bins before b
            sum += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
        if (blockIdx.x == 0) offsets[b] = total[b];
        int32_t at = total[b] + before[b];
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t n = mine[w * bins + b];
            mine[w * bins + b] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int64_t s0 = beg; s0 < end; s0 += 32) {
        const int64_t s = s0 + lane;
        const bool has = s < end;
        const int b = has ? bin_of(ids[s], experts) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, b);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int32_t r = 0;
        if (has) r = mine[warp * bins + b] + rank;
        __syncwarp();
        if (has && rank == 0) mine[warp * bins + b] = r + __popc(same);
        __syncwarp();
        if (has) {
            const bool kept = b < experts;
            rows[s] = kept ? r : ~r;
            slot_of_row[r] = kept ? static_cast<int32_t>(s) : ~static_cast<int32_t>(s);
        }
    }
}

int64_t sort_chunk(int64_t slots)
{
    int64_t c = (slots + kSortBlocks - 1) / kSortBlocks;
    if (c < kSortChunk) c = kSortChunk;
    return (c + kSortThreads - 1) / kSortThreads * kSortThreads;
}

int sort_blocks(int64_t slots) { return static_cast<int>((slots + sort_chunk(slots) - 1) / sort_chunk(slots)); }

// -------------------------------------------------------------- row pieces

template <bool BF16>
__device__ __forceinline__ float widen16(uint16_t v)
{
    if constexpr (BF16)
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else
        return __half2float(__ushort_as_half(v));
}

template <bool BF16>
__device__ __forceinline__ uint16_t narrow16(float v)
{
    if constexpr (BF16)
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        return __half_as_ushort(__float2half_rn(v));
}

// V 16-bit elements, moved as one access of 2 V bytes.
template <int V>
struct __align__(2 * V) Piece {
    uint16_t v[V];
};

// A block's threads work in groups of `lanes` threads, one token per group.
struct RowShape {
    int64_t tokens;
    int top_k;
    int64_t pieces;  // per row
    int lanes;
    int64_t rows;    // tokens * top_k: entries of the row table outside [0, rows) are passed over
};

// Rows of X to the rows of their choices: a token's row is read once and
// written top_k times (times the choice's weight, if there are weights).
template <bool BF16, int V>
__global__ void __launch_bounds__(256)
    dispatch_kernel(RowShape g, const uint16_t *X, int64_t ldx, const int32_t *rows, const float *weights,
                    uint16_t *Xs, int64_t ldxs)
{
    pdl_wait();
    pdl_launch_dependents();
    const int per_block = 256 / g.lanes, lane = threadIdx.x % g.lanes;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / g.lanes;
    if (t >= g.tokens) return;
    const int32_t *mine = rows + t * g.top_k;
    for (int64_t i = lane; i < g.pieces; i += g.lanes) {
        const Piece<V> x = reinterpret_cast<const Piece<V> *>(X + t * ldx)[i];
#pragma unroll 4
        for (int j = 0; j < g.top_k; ++j) {
            const int32_t r = mine[j];
            Piece<V> o = x;
            if (r < 0) {
#pragma unroll
                for (int u = 0; u < V; ++u) o.v[u] = 0;
            } else if (weights) {
                const float w = weights[t * g.top_k + j];
#pragma unroll
                for (int u = 0; u < V; ++u) o.v[u] = narrow16<BF16>(w * widen16<BF16>(x.v[u]));
            }
            const int64_t to = r < 0 ? ~r : r;
            if (to < g.rows) reinterpret_cast<Piece<V> *>(Xs + to * ldxs)[i] = o;
        }
    }
}

// y = sum over the token's kept choices of weight times the expert's row, in
// fp32 in the order of the choices, rounded once.
template <bool BF16, int V>
__global__ void __launch_bounds__(256)
    combine_kernel(RowShape g, const uint16_t *Ys, int64_t ldys, const int32_t *rows, const float *weights,
                   uint16_t *Y, int64_t ldy)
{
    pdl_wait();
    pdl_launch_dependents();
    const int per_block = 256 / g.lanes, lane = threadIdx.x % g.lanes;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / g.lanes;
    if (t >= g.tokens) return;
    const int32_t *mine = rows + t * g.top_k;
    for (int64_t i = lane; i < g.pieces; i += g.lanes) {
        float acc[V];
#pragma unroll
        for (int u = 0; u < V; ++u) acc[u] = 0.f;
        for (int j0 = 0; j0 < g.top_k; j0 += 8) {
            Piece<V> y[8];
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int32_t r = j0 + j < g.top_k ? mine[j0 + j] : -1;
                w[j] = 0.f;
                if (r >= 0 && r < g.rows) {
                    y[j] = reinterpret_cast<const Piece<V> *>(Ys + static_cast<int64_t>(r) * ldys)[i];
                    w[j] = weights ? weights[t * g.top_k + j0 + j] : 1.f;
                } else {
#pragma unroll
                    for (int u = 0; u < V; ++u) y[j].v[u] = 0;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int u = 0; u < V; ++u) acc[u] = fmaf(w[j], widen16<BF16>(y[j].v[u]), acc[u]);
        }
        Piece<V> o;
#pragma unroll
        for (int u = 0; u < V; ++u) o.v[u] = narrow16<BF16>(acc[u]);
        reinterpret_cast<Piece<V> *>(Y + t * ldy)[i] = o;
    }
}

constexpr int32_t kNoRow = INT32_MIN;

// One block per token: dYs[r] = weight * dY[t] and dweight = <Ys[r], dY[t]>
// for each of its choices, eight at a time; the dot products are summed in
// fp32, over the threads in a fixed order.
template <bool BF16, int V>
__global__ void __launch_bounds__(256)
    combine_grad_kernel(RowShape g, const uint16_t *dY, int64_t lddy, const uint16_t *Ys, int64_t ldys,
                        const int32_t *rows, const float *weights, uint16_t *dYs, int64_t lddys, float *dweights)
{
    // kNoRow's complement is 2^31 - 1, never a row.
    __shared__ float part[8][8];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int j0 = 0; j0 < g.top_k; j0 += 8) {
        int32_t r[8];
        float w[8], dot[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool has = j0 + j < g.top_k;
            r[j] = has ? rows[t * g.top_k + j0 + j] : 0;
            if (r[j] >= g.rows || ~r[j] >= g.rows) r[j] = kNoRow;
            w[j] = has && r[j] >= 0 ? (weights ? weights[t * g.top_k + j0 + j] : 1.f) : 0.f;
            dot[j] = 0.f;
        }
        for (int64_t i = threadIdx.x; i < g.pieces; i += blockDim.x) {
            const Piece<V> dy = reinterpret_cast<const Piece<V> *>(dY + t * lddy)[i];
            float d[V];
#pragma unroll
            for (int u = 0; u < V; ++u) d[u] = widen16<BF16>(dy.v[u]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j0 + j >= g.top_k) break;
                Piece<V> o;
                if (r[j] >= 0) {
                    const Piece<V> y = reinterpret_cast<const Piece<V> *>(Ys + static_cast<int64_t>(r[j]) * ldys)[i];
#pragma unroll
                    for (int u = 0; u < V; ++u) {
                        dot[j] = fmaf(d[u], widen16<BF16>(y.v[u]), dot[j]);
                        o.v[u] = narrow16<BF16>(w[j] * d[u]);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < V; ++u) o.v[u] = 0;
                }
                const int64_t to = r[j] < 0 ? ~r[j] : r[j];
                if (r[j] != kNoRow) reinterpret_cast<Piece<V> *>(dYs + to * lddys)[i] = o;
            }
        }
        if (dweights) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
                if (lane == 0) part[warp][j] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < 8 && j0 + static_cast<int>(threadIdx.x) < g.top_k) {
                float sum = 0.f;
                for (int k = 0; k < warps; ++k) sum += part[k][threadIdx.x];
                dweights[t * g.top_k + j0 + threadIdx.x] = sum;
            }
            __syncthreads();
        }
    }
}

// --------------------------------------------------------------- launching

// Elements per access that every row of a matrix allows.
int piece_of(const void *p, int64_t ld)
{
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(2 * ld);
    return bits % 16 == 0 ? 8 : (bits % 8 == 0 ? 4 : (bits % 4 == 0 ? 2 : 1));
}

int min_piece(int a, int b) { return a < b ? a : b; }

cudaLaunchConfig_t config(int64_t grid, int threads, int smem, cudaStream_t s, cudaLaunchAttribute *attr)
{
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    c.blockDim = dim3(threads, 1, 1);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = attr;
    c.numAttrs = 1;
    return c;
}

RowShape row_shape(int64_t tokens, int top_k, int64_t width, int v)
{
    RowShape g{tokens, top_k, width / v, 32, tokens * top_k};
    while (g.lanes < 256 && g.lanes < g.pieces) g.lanes *= 2;
    return g;
}

int64_t row_blocks(const RowShape &g) { return (g.tokens + 256 / g.lanes - 1) / (256 / g.lanes); }

// Calls f with the element type and piece width as template arguments.
template <class F>
cudaError_t with_piece(bool bf16, int v, F f)
{
#define GP_PIECE(V) (bf16 ? f.template operator()<true, V>() : f.template operator()<false, V>())
    return v == 8 ? GP_PIECE(8) : (v == 4 ? GP_PIECE(4) : (v == 2 ? GP_PIECE(2) : GP_PIECE(1)));
#undef GP_PIECE
}

int piece_width(int64_t width) { return width % 8 == 0 ? 8 : (width % 4 == 0 ? 4 : (width % 2 == 0 ? 2 : 1)); }

struct DispatchCall {
    int64_t tokens, width;
    int top_k;
    const uint16_t *X;
    int64_t ldx;
    const int32_t *rows;
    const float *weights;
    uint16_t *Xs;
    int64_t ldxs;
    cudaStream_t s;
    template <bool BF16, int V>
    cudaError_t operator()() const
    {
        const RowShape g = row_shape(tokens, top_k, width, V);
        cudaLaunchAttribute a[1];
        const cudaLaunchConfig_t c = config(row_blocks(g), 256, 0, s, a);
        return cudaLaunchKernelEx(&c, dispatch_kernel<BF16, V>, g, X, ldx, rows, weights, Xs, ldxs);
    }
};

struct CombineCall {
    int64_t tokens, width;
    int top_k;
    const uint16_t *Ys;
    int64_t ldys;
    const int32_t *rows;
    const float *weights;
    uint16_t *Y;
    int64_t ldy;
    cudaStream_t s;
    template <bool BF16, int V>
    cudaError_t operator()() const
    {
        const RowShape g = row_shape(tokens, top_k, width, V);
        cudaLaunchAttribute a[1];
        const cudaLaunchConfig_t c = config(row_blocks(g), 256, 0, s, a);
        return cudaLaunchKernelEx(&c, combine_kernel<BF16, V>, g, Ys, ldys, rows, weights, Y, ldy);
    }
};

struct CombineGradCall {
    int64_t tokens, width;
    int top_k;
    const uint16_t *dY;
    int64_t lddy;
    const uint16_t *Ys;
    int64_t ldys;
    const int32_t *rows;
    const float *weights;
    uint16_t *dYs;
    int64_t lddys;
    float *dweights;
    cudaStream_t s;
    template <bool BF16, int V>
    cudaError_t operator()() const
    {
        const RowShape g = row_shape(tokens, top_k, width, V);
        cudaLaunchAttribute a[1];
        const cudaLaunchConfig_t c = config(tokens, g.lanes, 0, s, a);
        return cudaLaunchKernelEx(&c, combine_grad_kernel<BF16, V>, g, dY, lddy, Ys, ldys, rows, weights, dYs, lddys,
                                  dweights);
    }
};

}  // namespace

int64_t route_scratch_bytes(int64_t slots, int experts)
{
    const int nb = sort_blocks(slots);
    return nb > 1 ? static_cast<int64_t>(nb) * (experts + 1) * 4 : 0;
}

int route_kernels(int64_t slots) { return sort_blocks(slots) > 1 ? 2 : 1; }

cudaError_t launch_route(int64_t slots, int experts, const int32_t *ids, int32_t *offsets, int32_t *slot_of_row,
                         int32_t *rows, int32_t *scratch, cudaStream_t s)
{
    const int64_t chunk = sort_chunk(slots);
    const int nb = sort_blocks(slots), bins = experts + 1;
    const int smem = (2 + kSortWarps) * bins * 4;
    constexpr int kMaxSmem = (2 + kSortWarps) * (kMaxExperts + 1) * 4;
    static std::atomic<int> done[128];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (!done[dev].load()) {
        e = cudaFuncSetAttribute(route_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        done[dev].store(1);
    }
    cudaLaunchAttribute a[1];
    if (nb > 1) {
        const cudaLaunchConfig_t c = config(nb, kSortThreads, bins * 4, s, a);
        if ((e = cudaLaunchKernelEx(&c, route_count_kernel, ids, slots, chunk, experts, scratch)) != cudaSuccess)
            return e;
    }
    const cudaLaunchConfig_t c = config(nb, kSortThreads, smem, s, a);
    return cudaLaunchKernelEx(&c, route_place_kernel, ids, slots, chunk, experts,
                              static_cast<const int32_t *>(nb > 1 ? scratch : nullptr), offsets, slot_of_row, rows);
}

cudaError_t launch_dispatch(bool bf16, int64_t tokens, int top_k, int64_t width, const uint16_t *X, int64_t ldx,
                            const int32_t *rows, const float *weights, uint16_t *Xs, int64_t ldxs, cudaStream_t s)
{
    const int v = min_piece(piece_width(width), min_piece(piece_of(X, ldx), piece_of(Xs, ldxs)));
    return with_piece(bf16, v, DispatchCall{tokens, width, top_k, X, ldx, rows, weights, Xs, ldxs, s});
}

cudaError_t launch_combine(bool bf16, int64_t tokens, int top_k, int64_t width, const uint16_t *Ys, int64_t ldys,
                           const int32_t *rows, const float *weights, uint16_t *Y, int64_t ldy, cudaStream_t s)
{
    const int v = min_piece(piece_width(width), min_piece(piece_of(Ys, ldys), piece_of(Y, ldy)));
    return with_piece(bf16, v, CombineCall{tokens, width, top_k, Ys, ldys, rows, weights, Y, ldy, s});
}

cudaError_t launch_combine_grad(bool bf16, int64_t tokens, int top_k, int64_t width, const uint16_t *dY, int64_t lddy,
                                const uint16_t *Ys, int64_t ldys, const int32_t *rows, const float *weights,
                                uint16_t *dYs, int64_t lddys, float *dweights, cudaStream_t s)
{
    const int v = min_piece(min_piece(piece_width(width), piece_of(dY, lddy)),
                            min_piece(piece_of(Ys, ldys), piece_of(dYs, lddys)));
    return with_piece(bf16, v, CombineGradCall{tokens, width, top_k, dY, lddy, Ys, ldys, rows, weights, dYs, lddys,
                                               dweights, s});
}

}  // namespace gp
