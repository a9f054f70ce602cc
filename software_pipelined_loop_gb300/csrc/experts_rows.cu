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
    for (int64_t s = beg + lane; s < end; s += 32) atomicAdd(&mine[warp * bins + bin_of(ids[s], experts)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
        int32_t all = 0, prior = 0;
        if (counts) {
#pragma unroll 16
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
    int32_t id = beg + lane < end ? ids[beg + lane] : 0;
    for (int64_t s0 = beg; s0 < end; s0 += 32) {
        const int64_t s = s0 + lane;
        const bool has = s < end;
        const int b = has ? bin_of(id, experts) : -1;
        if (s + 32 < end) id = ids[s + 32];
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
//
// A thread moves 8 elements, 16 bytes, at a time.  Where every row of every
// matrix starts on 16 bytes and holds whole pieces, a piece is one access
// (the kernels named *_wide).  Otherwise an output row is written in its own
// 16-byte words -- up to 7 single elements before the first and after the
// last -- and an input piece is cut from the two aligned words that hold it.

struct Piece {
    uint32_t w[4];
};

template <bool BF16>
__device__ __forceinline__ void widen8(const Piece &p, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            f[2 * i] = __uint_as_float(p.w[i] << 16);
            f[2 * i + 1] = __uint_as_float(p.w[i] & 0xffff0000u);
        } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&p.w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ Piece narrow8(const float (&f)[8])
{
    Piece p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            p.w[i] = *reinterpret_cast<const uint32_t *>(&v);
        } else {
            const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            p.w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
    }
    return p;
}

__device__ __forceinline__ Piece load_wide(const uint16_t *p)
{
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    return Piece{{v.x, v.y, v.z, v.w}};
}

__device__ __forceinline__ Piece cut(const Words8 &w, const uint16_t *p)
{
    Piece r;
    cut_words8(w, p, r.w);
    return r;
}

// p is on a 16-byte boundary.
__device__ __forceinline__ void store_wide(uint16_t *p, const Piece &v)
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

// An output row at any alignment: elements [0, head) and [head + 8 body, n)
// are written one by one, the others as `body` aligned pieces.
struct RowCut {
    int head, body, n;
    __device__ __forceinline__ RowCut(const uint16_t *row, int n_) : n(n_)
    {
        head = static_cast<int>(((16u - (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u)) & 15u) >> 1);
        if (head > n) head = n;
        body = (n - head) >> 3;
    }
    // Element of single number i (i < singles()).
    __device__ __forceinline__ int singles() const { return n - 8 * body; }
    __device__ __forceinline__ int single(int i) const { return i < head ? i : i + 8 * body; }
};

template <bool BF16>
__device__ __forceinline__ float widen1(uint16_t v)
{
    if constexpr (BF16)
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else
        return __half2float(__ushort_as_half(v));
}

template <bool BF16>
__device__ __forceinline__ uint16_t narrow1(float v)
{
    if constexpr (BF16)
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        return __half_as_ushort(__float2half_rn(v));
}

template <bool BF16>
__device__ __forceinline__ Piece scaled(const Piece &p, float w)
{
    float f[8];
    widen8<BF16>(p, f);
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] *= w;
    return narrow8<BF16>(f);
}

// A block's threads work in groups of `lanes` threads, one token per group.
struct RowShape {
    int64_t tokens;
    int top_k;
    int width;
    int lanes;
    int64_t rows;  // tokens * top_k: entries of the row table outside [0, rows) are passed over
};

// The kernels of a warp per choice: small blocks, so that an SM refills as
// soon as two rows are done (256 threads: 145 us where 64 take 129).
constexpr int kSlotThreads = 64;

// A warp writes 31 aligned 16-byte words of an output row at a time and reads
// the input row in the input's own: lane l loads the word that holds the
// first element of output word l, lane l + 1 has the rest.  Words off the row
// are not read.
constexpr int kWarpWords = 31;

__device__ __forceinline__ int misalign8(const uint16_t *x, int e)
{
    return static_cast<int>(((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x)) >> 1) + static_cast<uint32_t>(e)) & 7u);
}

__device__ __forceinline__ uint4 load_word(const uint16_t *x, int e, int width, bool on)
{
    const int at = e - misalign8(x, e);
    return ld_global_v4_if(x + at, on && at > -8 && at < width);
}

// Elements [e, e + 8) of x out of the warp's words (all lanes call it).
__device__ __forceinline__ Piece join_words(const uint4 &lo, const uint16_t *x, int e)
{
    uint4 hi;
    hi.x = __shfl_down_sync(0xffffffffu, lo.x, 1);
    hi.y = __shfl_down_sync(0xffffffffu, lo.y, 1);
    hi.z = __shfl_down_sync(0xffffffffu, lo.z, 1);
    hi.w = __shfl_down_sync(0xffffffffu, lo.w, 1);
    Piece r;
    realign16_steps(lo, hi, 2u * static_cast<uint32_t>(misalign8(x, e)), r.w);
    return r;
}

// Element of the first aligned word of an output row, at or before 0.
__device__ __forceinline__ int first_word(const uint16_t *row)
{
    return -static_cast<int>((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u) >> 1);
}

// Elements [e, e + 8) of the output row, those that it has.
__device__ __forceinline__ void store_word(uint16_t *row, int e, int width, const Piece &p)
{
    if (e >= 0 && e + 8 <= width) {
        store_wide(row + e, p);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (e + u >= 0 && e + u < width) row[e + u] = static_cast<uint16_t>(p.w[u >> 1] >> (16 * (u & 1)));
    }
}

// Rows of X to the rows of their choices (times the choice's weight, if
// there are weights): a token's row is read once from memory and written
// top_k times.  Bound by memory: 16384 tokens x 8 rows of 2048 bf16 take
// 90 us, 6.7 TB/s.
template <bool BF16>
__global__ void __launch_bounds__(256)
    dispatch_wide_kernel(RowShape g, const uint16_t *X, int64_t ldx, const int32_t *rows, const float *weights,
                         uint16_t *Xs, int64_t ldxs)
{
    pdl_wait();
    pdl_launch_dependents();
    const int per_block = 256 / g.lanes, lane = threadIdx.x % g.lanes;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / g.lanes;
    if (t >= g.tokens) return;
    const int32_t *mine = rows + t * g.top_k;
    for (int e = lane * 8; e < g.width; e += g.lanes * 8) {
        const Piece x = load_wide(X + t * ldx + e);
#pragma unroll 4
        for (int j = 0; j < g.top_k; ++j) {
            const int32_t r = mine[j];
            const int64_t to = r < 0 ? ~r : r;
            Piece p = x;
            if (r < 0)
                p = Piece{{0, 0, 0, 0}};
            else if (weights)
                p = scaled<BF16>(x, weights[t * g.top_k + j]);
            if (to < g.rows) store_wide(Xs + to * ldxs + e, p);
        }
    }
}

// The same at any alignment, a warp per choice: each word of the input row is
// loaded once (two loads for each output word took 129 us instead of 119,
// route included, for 16384 tokens x 8 rows of 2001 bf16).
template <bool BF16>
__global__ void __launch_bounds__(kSlotThreads)
    dispatch_kernel(RowShape g, const uint16_t *X, int64_t ldx, const int32_t *rows, const float *weights,
                    uint16_t *Xs, int64_t ldxs)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t s = static_cast<int64_t>(blockIdx.x) * (kSlotThreads / 32) + (threadIdx.x >> 5);
    if (s >= g.rows) return;
    const int32_t r = rows[s];
    const int64_t to = r < 0 ? ~r : r;
    if (to >= g.rows) return;
    const uint16_t *x = X + s / g.top_k * ldx;
    uint16_t *o = Xs + to * ldxs;
    const bool copied = r < 0 || !weights;
    const float w = copied ? 1.f : weights[s];
    constexpr int FLIGHT = 3;
    for (int e0 = first_word(o); e0 < g.width; e0 += 8 * kWarpWords * FLIGHT) {
        const int e = e0 + 8 * lane;
        uint4 v[FLIGHT];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) v[u] = load_word(x, e + 8 * kWarpWords * u, g.width, r >= 0);
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const Piece p = join_words(v[u], x, e + 8 * kWarpWords * u);
            if (lane < kWarpWords) store_word(o, e + 8 * kWarpWords * u, g.width, copied ? p : scaled<BF16>(p, w));
        }
    }
}

// y = sum over the token's kept choices of weight times the expert's row, in
// fp32 in the order of the choices, rounded once.  Eight rows are in flight
// per thread.
template <bool BF16>
__global__ void __launch_bounds__(256)
    combine_wide_kernel(RowShape g, const uint16_t *Ys, int64_t ldys, const int32_t *rows, const float *weights,
                        uint16_t *Y, int64_t ldy)
{
    pdl_wait();
    pdl_launch_dependents();
    const int per_block = static_cast<int>(blockDim.x) / g.lanes, lane = threadIdx.x % g.lanes;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / g.lanes;
    if (t >= g.tokens) return;
    const int32_t *mine = rows + t * g.top_k;
    constexpr int FLIGHT = 8;
    for (int e = lane * 8; e < g.width; e += g.lanes * 8) {
        float acc[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) acc[u] = 0.f;
        for (int j0 = 0; j0 < g.top_k; j0 += FLIGHT) {
            Piece p[FLIGHT];
            float w[FLIGHT];
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j) {
                const int32_t r = j0 + j < g.top_k ? mine[j0 + j] : -1;
                w[j] = 0.f;
                p[j] = Piece{{0, 0, 0, 0}};
                if (r >= 0 && r < g.rows) {
                    p[j] = load_wide(Ys + static_cast<int64_t>(r) * ldys + e);
                    w[j] = weights ? weights[t * g.top_k + j0 + j] : 1.f;
                }
            }
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j) {
                float f[8];
                widen8<BF16>(p[j], f);
#pragma unroll
                for (int u = 0; u < 8; ++u) acc[u] = fmaf(w[j], f[u], acc[u]);
            }
        }
        store_wide(Y + t * ldy + e, narrow8<BF16>(acc));
    }
}

// The same at any alignment.  The kept choices' rows and weights are
// listed once per token in shared memory.
template <bool BF16>
__global__ void __launch_bounds__(256)
    combine_kernel(RowShape g, const uint16_t *Ys, int64_t ldys, const int32_t *rows, const float *weights,
                   uint16_t *Y, int64_t ldy)
{
    __shared__ const uint16_t *row_of[8][kMaxTopK];
    __shared__ float weight_of[8][kMaxTopK];
    pdl_wait();
    pdl_launch_dependents();
    const int per_block = static_cast<int>(blockDim.x) / g.lanes, lane = threadIdx.x % g.lanes;
    const int slot = threadIdx.x / g.lanes;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + slot;
    if (t < g.tokens) {
        for (int j = lane; j < g.top_k; j += g.lanes) {
            const int32_t r = rows[t * g.top_k + j];
            const bool kept = r >= 0 && r < g.rows;
            row_of[slot][j] = kept ? Ys + static_cast<int64_t>(r) * ldys : nullptr;
            weight_of[slot][j] = kept && weights ? weights[t * g.top_k + j] : 1.f;
        }
    }
    __syncthreads();
    if (t >= g.tokens) return;
    uint16_t *y = Y + t * ldy;
    const RowCut own(y, g.width);
    constexpr int FLIGHT = 4;
    for (int i = lane; i < own.body; i += g.lanes) {
        const int e = own.head + 8 * i;
        float acc[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) acc[u] = 0.f;
        for (int j0 = 0; j0 < g.top_k; j0 += FLIGHT) {
            Words8 v[FLIGHT];
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j) {
                const uint16_t *row = j0 + j < g.top_k ? row_of[slot][j0 + j] : nullptr;
                v[j] = load_words8(row + e, row != nullptr);
            }
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j) {
                if (j0 + j >= g.top_k || !row_of[slot][j0 + j]) continue;
                const float w = weight_of[slot][j0 + j];
                float f[8];
                widen8<BF16>(cut(v[j], row_of[slot][j0 + j] + e), f);
#pragma unroll
                for (int u = 0; u < 8; ++u) acc[u] = fmaf(w, f[u], acc[u]);
            }
        }
        store_wide(y + e, narrow8<BF16>(acc));
    }
    if (lane < own.singles()) {
        const int e = own.single(lane);
        float acc = 0.f;
        for (int j = 0; j < g.top_k; ++j)
            if (row_of[slot][j]) acc = fmaf(weight_of[slot][j], widen1<BF16>(row_of[slot][j][e]), acc);
        y[e] = narrow1<BF16>(acc);
    }
}

constexpr int32_t kNoRow = INT32_MIN;  // its complement is 2^31 - 1, never a row

// One block per token: dYs[r] = weight * dY[t] and dweight = <Ys[r], dY[t]>
// for each of its choices, eight at a time, their loads in flight together;
// the dot products are summed in fp32, over the threads in a fixed order.
// Bound by memory: 8192 tokens x 8 rows of 4096 bf16 take 167 us, 6.8 TB/s,
// with three blocks an SM; 187 with two (112 registers), 181 with four (64).
template <bool BF16>
__global__ void __launch_bounds__(256, 3)
    combine_grad_wide_kernel(RowShape g, const uint16_t *dY, int64_t lddy, const uint16_t *Ys, int64_t ldys,
                             const int32_t *rows, const float *weights, uint16_t *dYs, int64_t lddys,
                             float *dweights)
{
    constexpr int FLIGHT = 8;
    __shared__ float part[8][FLIGHT];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int j0 = 0; j0 < g.top_k; j0 += FLIGHT) {
        int32_t r[FLIGHT];
        float w[FLIGHT], dot[FLIGHT];
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j) {
            const bool has = j0 + j < g.top_k;
            r[j] = has ? rows[t * g.top_k + j0 + j] : kNoRow;
            if (r[j] >= g.rows || ~r[j] >= g.rows) r[j] = kNoRow;
            w[j] = r[j] >= 0 ? (weights ? weights[t * g.top_k + j0 + j] : 1.f) : 0.f;
            dot[j] = 0.f;
        }
        for (int e = threadIdx.x * 8; e < g.width; e += blockDim.x * 8) {
            const Piece d = load_wide(dY + t * lddy + e);
            Piece y[FLIGHT];
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j) {
                y[j] = Piece{{0, 0, 0, 0}};
                if (r[j] >= 0) y[j] = load_wide(Ys + static_cast<int64_t>(r[j]) * ldys + e);
            }
            float fd[8];
            widen8<BF16>(d, fd);
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j) {
                if (r[j] == kNoRow) continue;
                if (r[j] >= 0) {  // (a dropped choice's sum stays zero: dY may hold an infinity or NaN)
                    float fy[8];
                    widen8<BF16>(y[j], fy);
#pragma unroll
                    for (int u = 0; u < 8; ++u) dot[j] = fmaf(fd[u], fy[u], dot[j]);
                }
                const int64_t to = r[j] < 0 ? ~r[j] : r[j];
                store_wide(dYs + to * lddys + e, r[j] < 0 ? Piece{{0, 0, 0, 0}} : scaled<BF16>(d, w[j]));
            }
        }
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
            if (lane == 0) part[warp][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < FLIGHT && j0 + static_cast<int>(threadIdx.x) < g.top_k) {
            float sum = 0.f;
            for (int k = 0; k < warps; ++k) sum += part[k][threadIdx.x];
            dweights[t * g.top_k + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

// The same at any alignment, a warp per choice (8192 x 8 rows of 3001: 157 us
// with forty warps an SM in blocks of 64 threads, 174 with 32; each word
// loaded once and passed between lanes, as in dispatch_kernel, 179).
template <bool BF16>
__global__ void __launch_bounds__(kSlotThreads, 20)
    combine_grad_kernel(RowShape g, const uint16_t *dY, int64_t lddy, const uint16_t *Ys, int64_t ldys,
                        const int32_t *rows, const float *weights, uint16_t *dYs, int64_t lddys, float *dweights)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t s = static_cast<int64_t>(blockIdx.x) * (kSlotThreads / 32) + (threadIdx.x >> 5);
    if (s >= g.rows) return;
    const int32_t r = rows[s];
    const int64_t to = r < 0 ? ~r : r;
    if (r < 0 || to >= g.rows) {
        if (lane == 0) dweights[s] = 0.f;
        if (to >= g.rows) return;
    }
    uint16_t *o = dYs + to * lddys;
    const RowCut row(o, g.width);
    if (r < 0) {
        for (int i = lane; i < row.body; i += 32) store_wide(o + row.head + 8 * i, Piece{{0, 0, 0, 0}});
        if (lane < row.singles()) o[row.single(lane)] = 0;
        return;
    }
    const uint16_t *d = dY + s / g.top_k * lddy, *y = Ys + to * ldys;
    const float w = weights ? weights[s] : 1.f;
    float dot = 0.f;
    constexpr int FLIGHT = 2;
    for (int i = lane; i < row.body; i += 32 * FLIGHT) {
        Words8 vd[FLIGHT], vy[FLIGHT];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int e = row.head + 8 * (i + 32 * u);
            const bool on = i + 32 * u < row.body;
            vy[u] = load_words8(y + e, on);
            vd[u] = load_words8(d + e, on);
        }
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int e = row.head + 8 * (i + 32 * u);
            float fd[8], fy[8];
            widen8<BF16>(cut(vd[u], d + e), fd);
            widen8<BF16>(cut(vy[u], y + e), fy);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                dot = fmaf(fd[k], fy[k], dot);
                fd[k] *= w;
            }
            if (i + 32 * u < row.body) store_wide(o + e, narrow8<BF16>(fd));
        }
    }
    if (lane < row.singles()) {
        const int e = row.single(lane);
        const float fd = widen1<BF16>(d[e]);
        dot = fmaf(fd, widen1<BF16>(y[e]), dot);
        o[e] = narrow1<BF16>(fd * w);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, k);
    if (lane == 0) dweights[s] = dot;
}

// --------------------------------------------------------------- launching

bool wide_rows(const void *p, int64_t ld) { return ((reinterpret_cast<uintptr_t>(p) | 2 * ld) & 15) == 0; }

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

RowShape row_shape(int64_t tokens, int top_k, int64_t width)
{
    // A group covers the row in one pass if 256 threads can; a longer row is
    // covered in as few thread passes as 256 or 128 threads leave idle least.
    RowShape g{tokens, top_k, static_cast<int>(width), 32, tokens * top_k};
    const int64_t pieces = (width + 7) / 8;
    while (g.lanes < 256 && g.lanes < pieces) g.lanes *= 2;
    if (pieces > 256 && (pieces + 127) / 128 * 128 < (pieces + 255) / 256 * 256) g.lanes = 128;
    return g;
}

int64_t row_blocks(const RowShape &g, int threads = 256)
{
    return (g.tokens + threads / g.lanes - 1) / (threads / g.lanes);
}

int64_t slot_blocks(const RowShape &g) { return (g.rows + kSlotThreads / 32 - 1) / (kSlotThreads / 32); }

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
    const bool wide = width % 8 == 0 && wide_rows(X, ldx) && wide_rows(Xs, ldxs);
    const RowShape g = row_shape(tokens, top_k, width);
    const auto k = wide ? (bf16 ? dispatch_wide_kernel<true> : dispatch_wide_kernel<false>)
                        : (bf16 ? dispatch_kernel<true> : dispatch_kernel<false>);
    cudaLaunchAttribute a[1];
    const cudaLaunchConfig_t c = wide ? config(row_blocks(g), 256, 0, s, a) : config(slot_blocks(g), kSlotThreads, 0, s, a);
    return cudaLaunchKernelEx(&c, k, g, X, ldx, rows, weights, Xs, ldxs);
}

constexpr int64_t kManyTokens = 1024;

cudaError_t launch_combine(bool bf16, int64_t tokens, int top_k, int64_t width, const uint16_t *Ys, int64_t ldys,
                           const int32_t *rows, const float *weights, uint16_t *Y, int64_t ldy, cudaStream_t s)
{
    const bool wide = width % 8 == 0 && wide_rows(Ys, ldys) && wide_rows(Y, ldy);
    RowShape g = row_shape(tokens, top_k, width);
    // Of more tokens than are resident at once, narrower groups in blocks of
    // 128 threads keep the SMs full to the end; of few, the widest groups are
    // done first.  Four rows of 2048 (3001) a token, us (other numbers of rows
    // were not swept):
    //   tokens          256          512        1024        2048         4093
    //   256 threads  2.4 (4.1)  3.5 (4.8)   5.1 (7.0)   9.3 (15.0)  21.3 (26.8)
    //   128 threads  2.9 (5.3)  3.5 (5.8)   5.2 (7.4)   8.8 (14.1)  19.0 (25.1)
    const bool many = tokens > kManyTokens;
    const int threads = many ? 128 : 256, most = many ? (wide ? 128 : 64) : 256;
    if (g.lanes > most) g.lanes = most;
    const auto k = wide ? (bf16 ? combine_wide_kernel<true> : combine_wide_kernel<false>)
                        : (bf16 ? combine_kernel<true> : combine_kernel<false>);
    cudaLaunchAttribute a[1];
    const cudaLaunchConfig_t c = config(row_blocks(g, threads), threads, 0, s, a);
    return cudaLaunchKernelEx(&c, k, g, Ys, ldys, rows, weights, Y, ldy);
}

cudaError_t launch_combine_grad(bool bf16, int64_t tokens, int top_k, int64_t width, const uint16_t *dY, int64_t lddy,
                                const uint16_t *Ys, int64_t ldys, const int32_t *rows, const float *weights,
                                uint16_t *dYs, int64_t lddys, float *dweights, cudaStream_t s)
{
    const bool wide = width % 8 == 0 && wide_rows(dY, lddy) && wide_rows(Ys, ldys) && wide_rows(dYs, lddys);
    const RowShape g = row_shape(tokens, top_k, width);
    const auto k = wide ? (bf16 ? combine_grad_wide_kernel<true> : combine_grad_wide_kernel<false>)
                        : (bf16 ? combine_grad_kernel<true> : combine_grad_kernel<false>);
    cudaLaunchAttribute a[1];
    const cudaLaunchConfig_t c = wide ? config(tokens, g.lanes, 0, s, a) : config(slot_blocks(g), kSlotThreads, 0, s, a);
    return cudaLaunchKernelEx(&c, k, g, dY, lddy, Ys, ldys, rows, weights, dYs, lddys, dweights);
}

}  // namespace gp
