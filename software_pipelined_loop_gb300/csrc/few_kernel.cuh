// few_kernel.cuh -- products of a few rows with large matrices: one matrix in
// 4 bits, or the matrices of the experts that a few tokens chose.
//
// out[r][n] = sum over k of X[r][k] * W[k][n], for at most 64 rows.  Every
// weight is read once and used for few rows, so the kernel is bound by the
// rate at which weights come from memory (in 4 bits, by what it takes to make
// 16-bit values of them); everything else is arranged around that:
//   - a warp takes 64 columns and walks over k in steps of 32 (4 bits: 64).  It
//     copies the weights, scales and rows of X of the next steps into a ring of
//     its own in shared memory, asynchronously, so that no block-wide barrier
//     stands between loads and products.  (Straight into registers the same
//     loads allowed half of the bytes in flight: 4 tokens x 8 of 64 experts of
//     4096 x 1536 took 154 us, 139 with the ring.)  Its loads run ahead into
//     its next unit of work;
//   - the products run on warp-level matrix instructions (m16n8k16) with the
//     weights as the 16-row operand and 8 rows of X as the 8-column operand.
//     The places of n and k in that operand are free as long as X has the same
//     order: with g = lane / 4 and t = lane % 4 a lane takes rows k = 8t .. 8t
//     + 7 of 32 and
//       16 bits: columns 8g .. 8g + 7 (one 16-byte load a row),
//       4 bits:  columns 4g .. 4g + 3 and 32 + 4g .. (a word of 8 rows each);
//     in 16 bits two rows' words are woven into (k, k + 1) pairs by byte
//     permutes, in 4 bits a word's pairs lie as the instruction wants them;
//   - X's operand is the 8 values k = 8t .. 8t + 7 of row g: one 16-byte load;
//   - 4-bit values become 1024 + q (fp16) or 128 + q (bf16) by a mask and an or,
//     exact, then the constant and the 8 are taken off, exact; the sum over a
//     group's products of a step is multiplied by the columns' scales in fp32,
//     so nothing is rounded before the end; hidden rows, operands of the next
//     product, are two rows there: their rounding and what that leaves;
//   - the 8 warps of a block and the blocks of a cluster share the products;
//     their sums meet in shared memory, in a fixed order.
//
// Measured (GB300, back to back, SM clock about 1.95 GHz): weights in 16 bits
// 6.0 to 6.6 TB/s where there are some 0.3 ms of them or more.  In 4 bits, one row
// x 16384 x 19456, whose 304 units fill all places, 4.8 (bf16) and 5.3 (fp16) TB/s;
// x 16384 x 16384, 256 units, 4.1 in the same time: 165 and 150 instructions of a
// warp for 32 x 64 weights, of which the logic operations that take words apart (7
// or 5 for 8 weights, at half rate) keep their pipe 62% busy.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "few.h"
#include "ptx.cuh"

namespace gp {

// ------------------------------------------------------------ small pieces

// d (+)= a * b.  FIXED: products stay in the order they are written in, where
// the compiler's own order would keep too many operands in registers.
template <bool BF16, bool FIXED>
__device__ __forceinline__ void few_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    if constexpr (BF16 && FIXED)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else if constexpr (FIXED)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same without an addend.
template <bool BF16, bool FIXED>
__device__ __forceinline__ void few_mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    if constexpr (BF16 && FIXED)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else if constexpr (FIXED)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

template <bool BF16>
__device__ __forceinline__ float few_float(uint32_t bits)
{
    if constexpr (BF16)
        return __uint_as_float(bits << 16);
    else
        return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

template <bool BF16>
__device__ __forceinline__ uint16_t few_round(float v)
{
    if constexpr (BF16)
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        return __half_as_ushort(__float2half_rn(v));
}

// What the rounding of a hidden value leaves is kept times this: of fp16 values it
// would mostly be below the normal numbers (it is 2^-12 of the value at most,
// and 16 at most), where bits are lost.
template <bool BF16>
constexpr float kFewLift = BF16 ? 1.0f : 2048.0f;

// Values i and i + 4 of a word of eight 4-bit values: the pair of rows 2i, 2i
// + 1.  (v & mask) | one is a single operation when both are in registers.  The
// fp16 mantissa holds the upper of two neighbouring values in its place, 16
// times as large, so that one shift serves two pairs; that of bf16 is too short.
template <bool BF16>
__device__ __forceinline__ uint32_t few_pair(uint32_t word, int i)
{
    uint32_t m;
    if constexpr (BF16) {
        asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(m) : "r"(word >> (4 * i)), "r"(0x000f000fu), "r"(0x43004300u));
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&m), __float2bfloat162_rn(136.0f));  // 128 + q
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const uint32_t w = word >> (8 * (i >> 1));
        __half2 v;
        if (i & 1) {
            asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(m) : "r"(w), "r"(0x00f000f0u), "r"(0x64006400u));
            v = __hfma2(*reinterpret_cast<const __half2 *>(&m), __float2half2_rn(0.0625f), __float2half2_rn(-72.0f));  // 1024 + 16 q
        } else {
            asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(m) : "r"(w), "r"(0x000f000fu), "r"(0x64006400u));
            v = __hsub2(*reinterpret_cast<const __half2 *>(&m), __float2half2_rn(1032.0f));  // 1024 + q
        }
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// Asynchronous copies into this CTA's shared memory: `bytes` of 16 or 8 from
// global memory, zeros behind them (0: nothing is read).
__device__ __forceinline__ void few_copy16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void few_copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void few_copy8(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void few_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Waits until at most N of this thread's groups are incomplete.
template <int N>
__device__ __forceinline__ void few_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The first `count` of eight 16-bit elements, zeros behind.
__device__ __forceinline__ uint4 few_first(uint4 v, int count)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (count <= 2 * i) w[i] = 0;
        else if (count == 2 * i + 1) w[i] &= 0xffffu;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void few_st_cluster(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The two halves of a cluster barrier.  The first arrival says nothing but that
// the block is there; a later one, that what the block has read may be written
// over by the others after their wait.
__device__ __forceinline__ void few_cluster_arrive_first()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

__device__ __forceinline__ void few_cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void few_cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------- table of items
//
// An item is an expert and up to CHUNK of the tokens that chose it, in order.
// A token that chose one expert twice is one row with the sum of both weights.
// Up to 32 choices are sorted by every warp on its own, in registers, into a
// table of its own: one load of the ids and no barrier stand before the first
// load of a weight.

struct FewTables {
    uint32_t *expert;  // items: expert
    uint32_t *span;    // items: first row | rows << 16
    uint32_t *row;     // rows: token | slot << 8
    float *weight;     // rows
};

__host__ __device__ constexpr int few_own_table_words() { return 4 * 32; }

// At most 32 choices; one table a warp.
template <int CHUNK>
__device__ __forceinline__ int few_build_warp(const FewParams &p, FewTables &t, uint32_t *smem)
{
    const int lane = threadIdx.x & 31, k = p.top_k, R = p.tokens * k;
    t.expert = smem + (threadIdx.x >> 5) * few_own_table_words();
    t.span = t.expert + 32;
    t.row = t.span + 32;
    t.weight = reinterpret_cast<float *>(t.row + 32);
    uint32_t e = 0xffffffffu;
    float w = 0.0f;
    if (lane < R) {
        e = static_cast<uint32_t>(p.ids[lane]);
        if (p.weights) w = p.weights[lane];
    }
    const bool valid = lane < R && e < static_cast<uint32_t>(p.experts);
    const int token = lane / k;
    const uint32_t below = (1u << lane) - 1u, same = __match_any_sync(0xffffffffu, valid ? e : 0xffffffffu);
    const int from = token * k;
    const uint32_t mine = same & ((k >= 32 ? 0xffffffffu : (1u << k) - 1u) << (from & 31));  // this token's, same expert
    const bool again = valid && (mine & below) != 0;
    const uint32_t rows = __ballot_sync(0xffffffffu, valid && !again);
    if (__any_sync(0xffffffffu, again)) {
        float sum = w;
        for (int j = 1; j < k; ++j) {
            const float v = __shfl_down_sync(0xffffffffu, w, j);
            if (lane + j < 32 && (mine >> (lane + j) & 1u)) sum += v;
        }
        w = sum;
    }
    const uint32_t peers = same & rows;
    const bool row = valid && !again, leader = row && (peers & below) == 0;
    const int count = __popc(peers);
    // Rows and items of this expert and the ones before it.
    const uint32_t both = leader ? count | (count + CHUNK - 1) / CHUNK << 16 : 0;
    uint32_t sum = both;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
    }
    const int items = static_cast<int>(__shfl_sync(0xffffffffu, sum, 31) >> 16);
    const uint32_t before = __shfl_sync(0xffffffffu, sum - both, row ? __ffs(peers) - 1 : 0);
    const int first = static_cast<int>(before & 0xffffu);
    if (row) {
        const int at = first + __popc(peers & below);
        t.row[at] = static_cast<uint32_t>(token) | static_cast<uint32_t>(lane) << 8;
        t.weight[at] = w;
    }
    if (leader) {
        int i = static_cast<int>(before >> 16);
        for (int c = 0; c < count; c += CHUNK, ++i) {
            t.expert[i] = e;
            t.span[i] = static_cast<uint32_t>(first + c) | static_cast<uint32_t>(min(count - c, CHUNK)) << 16;
        }
    }
    __syncwarp();
    return items;
}

// Any number of choices; one table a block.
template <int CHUNK>
__device__ __forceinline__ int few_build_block(const FewParams &p, FewTables &t, uint32_t *smem)
{
    const int tid = threadIdx.x, k = p.top_k, R = p.tokens * k;
    t.expert = smem;
    t.span = t.expert + p.max_items;
    t.row = t.span + p.max_items;
    t.weight = reinterpret_cast<float *>(t.row + R);
    uint32_t *mask = reinterpret_cast<uint32_t *>(t.weight + R);  // 2 x experts: tokens that chose the expert
    uint32_t *start = mask + 2 * p.experts;                        // experts: first row
    uint32_t *items_out = start + p.experts;
    const auto rows_of = [&](int e) { return __popc(mask[2 * e]) + __popc(mask[2 * e + 1]); };
    for (int i = tid; i < 2 * p.experts; i += blockDim.x) mask[i] = 0;
    __syncthreads();
    for (int s = tid; s < R; s += blockDim.x) {
        const uint32_t e = static_cast<uint32_t>(p.ids[s]);
        const int token = s / k;
        if (e < static_cast<uint32_t>(p.experts)) atomicOr(&mask[2 * e + (token >> 5)], 1u << (token & 31));
    }
    __syncthreads();
    if (tid < 32) {
        const int per = (p.experts + 31) / 32;
        const int lo = min(tid * per, p.experts), hi = min(lo + per, p.experts);
        uint32_t rows = 0, items = 0;
        for (int e = lo; e < hi; ++e) {
            const int n = rows_of(e);
            rows += n;
            items += (n + CHUNK - 1) / CHUNK;
        }
        uint32_t both = rows | items << 16;  // at most 4096 and (1024 experts, 4096 rows in 16s) 1216
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, both, d);
            if (tid >= d) both += v;
        }
        uint32_t row = (both & 0xffffu) - rows, item = (both >> 16) - items;
        for (int e = lo; e < hi; ++e) {
            const int n = rows_of(e);
            start[e] = row;
            for (int c = 0; c < n; c += CHUNK) {
                t.expert[item] = e;
                t.span[item++] = (row + c) | static_cast<uint32_t>(min(n - c, CHUNK)) << 16;
            }
            row += n;
        }
        if (tid == 31) *items_out = item;
    }
    __syncthreads();
    for (int s = tid; s < R; s += blockDim.x) {
        const int32_t e = p.ids[s];
        if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(p.experts)) continue;
        const int token = s / k;
        bool again = false;
        for (int i = token * k; i < s; ++i) again |= p.ids[i] == e;
        if (again) continue;
        float w = 0.0f;
        if (p.weights) {
            w = p.weights[s];
            for (int i = s + 1; i < (token + 1) * k; ++i)
                if (p.ids[i] == e) w += p.weights[i];
        }
        const uint32_t below = (1u << (token & 31)) - 1u;
        const int at = token < 32 ? __popc(mask[2 * e] & below) : __popc(mask[2 * e]) + __popc(mask[2 * e + 1] & below);
        t.row[start[e] + at] = static_cast<uint32_t>(token) | static_cast<uint32_t>(s) << 8;
        t.weight[start[e] + at] = w;
    }
    __syncthreads();
    return static_cast<int>(*items_out);
}

// ------------------------------------------------------------------ kernel

// A unit of work: 64 columns of an item (kFewFlat: an item).  A warp takes the
// steps [lo, hi) of the units `first`, `first` + `stride`, ...; its loads run
// ahead of its products into the next unit.
struct FewShare {
    int first, stride, units;  // units: the number of all
    int lo, hi;
};

// Where a warp's loads are, with this lane's places.
template <int MB>
struct FewWalk {
    int unit, step, blocks;
    int whole;                  // steps of the unit whose loads of weights are all inside the matrix
    const char *w;              // this lane's piece of the step's first row (4 bits: of its word row)
    const uint16_t *s;          // this lane's scales of the group
    const uint16_t *x[MB];      // this lane's 8 values of each row
    uint32_t x_bytes[MB];       // 16, or 0 for a place without a row
};

template <bool BF16, bool FOUR, bool ANY, int MB, int MODE>
struct FewKernel {
    static constexpr int DEPTH = few_depth<FOUR, MB>();
    static constexpr bool FIXED = MB > 1;
    static constexpr bool UP = MODE == kFewUp, FLAT = MODE == kFewFlat;
    static constexpr int PARTS = UP ? 1 : 2, CHUNK = few_chunk(MB, UP);  // rows of the products for a row of an item
    static constexpr bool ANY_W = ANY && !FOUR, ANY_X = ANY && UP;
    using Stage = FewStage<FOUR, ANY_W, ANY_X, MB>;

    const FewParams &p;
    const FewTables &t;
    const void *W;
    const uint16_t *S;
    int64_t n_first;   // the warp's columns in the first block of columns (kFewFlat: in this one)
    int64_t n4;
    FewShare share;
    int lane, g, l4;   // lane / 4, lane % 4
    uint32_t put, get; // this lane's first place of W in a stage: to copy to, to read

    __device__ __forceinline__ FewKernel(const FewParams &p_, const FewTables &t_, int matrix, int64_t n_first_,
                                         const FewShare &share_)
        : p(p_), t(t_), W(matrix ? p_.W[1] : p_.W[0]), S(matrix ? p_.S[1] : p_.S[0]), n_first(n_first_), share(share_)
    {
        lane = threadIdx.x & 31;
        g = lane >> 2;
        l4 = lane & 3;
        n4 = (p.N + 3) / 4 * 4;
        if constexpr (FOUR) {
            put = 256 * (lane >> 4) + 16 * ((lane & 15) ^ (2 * (lane >> 4)));
            get = 256 * l4 + 16 * (g ^ (2 * l4));
        } else {
            put = 128 * (lane >> 3) + 16 * ((lane & 7) ^ (lane >> 3));
            get = 1024 * l4 + 16 * (g ^ (2 * l4));
        }
    }

    // (K, and columns, are below 2^31 - 1023)
    __device__ __forceinline__ int K32() const { return static_cast<int>(p.K); }

    __device__ __forceinline__ int item_of(int unit) const { return FLAT ? unit : unit / p.columns; }

    // The warp's first column in a unit.
    __device__ __forceinline__ int64_t column_of(int unit) const
    {
        return FLAT ? n_first : n_first + static_cast<int64_t>(unit % p.columns) * (p.wide * kFewCols);
    }

    __device__ __forceinline__ int rows_of(int item) const
    {
        return p.ids ? static_cast<int>(t.span[item] >> 16) : min(p.tokens - item * CHUNK, CHUNK);
    }

    // A hidden row is two of the products' rows, its rounded values and their rest.
    __device__ __forceinline__ static int blocks_of(int rows) { return (PARTS * rows + 7) / 8; }

    // Element 0 of row i of an item's products, or of its first row where it has no such row.
    __device__ __forceinline__ const uint16_t *row_of(int item, int rows, int i) const
    {
        const uint16_t *X = !UP && (i & 1) ? p.X2 : p.X;
        if (!UP) i >>= 1;
        const int first = p.ids ? static_cast<int>(t.span[item] & 0xffffu) : item * CHUNK;
        int64_t r = first + (i < rows ? i : 0);
        if (p.ids) r = UP ? t.row[r] & 0xffu : t.row[r] >> 8;
        return X + r * p.ldx;
    }

    __device__ __forceinline__ void place(FewWalk<MB> &k) const
    {
        const int item = item_of(k.unit);
        const int64_t e = p.ids ? static_cast<int64_t>(t.expert[item]) : 0, n0 = column_of(k.unit);
        if constexpr (FOUR) {
            k.w = reinterpret_cast<const char *>(static_cast<const uint32_t *>(W) + (e * p.words + 8 * static_cast<int64_t>(k.step) + (lane >> 4)) * n4 + n0 + 4 * (lane & 15));
            k.s = S + (e * p.groups + ((2 * k.step + (lane >> 4)) >> p.group_shift)) * n4 + n0 + 4 * (lane & 15);
        } else {
            // (off 16-byte boundaries: the row, not the lane's piece of it)
            k.w = reinterpret_cast<const char *>(static_cast<const uint16_t *>(W) + (e * p.K + 32 * static_cast<int64_t>(k.step) + (lane >> 3)) * p.N + n0 + (ANY_W ? 0 : 8 * (lane & 7)));
        }
        k.whole = !ANY_W && n0 + kFewCols <= (FOUR ? n4 : p.N) ? static_cast<int>(p.K / Stage::STEP) : 0;
        const int rows = rows_of(item);
        k.blocks = blocks_of(rows);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            k.x_bytes[m] = 8 * m + g < PARTS * rows ? 16u : 0u;
            k.x[m] = row_of(item, rows, 8 * m + g) + Stage::STEP * static_cast<int64_t>(k.step) + (ANY_X ? 0 : 8 * l4);
        }
    }

    // On to the pointers of the step after this one, of the same unit.
    __device__ __forceinline__ void next_step(FewWalk<MB> &k) const
    {
        ++k.step;
        if constexpr (FOUR) {
            k.w += 32 * n4;  // 8 rows of words
            if (p.group_steps == 1) k.s += 2 * n4;
            else if (p.group_steps == 2 || (k.step & 1) == 0) k.s += n4;
        } else {
            k.w += 64 * p.N;
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) k.x[m] += Stage::STEP;
    }

    __device__ __forceinline__ void advance(FewWalk<MB> &k) const
    {
        if (k.step + 1 < share.hi) {
            next_step(k);
            return;
        }
        k.step = share.lo;
        k.unit += share.stride;
        if (k.unit < share.units) place(k);
    }

    // Neighbouring lanes copy neighbouring pieces (lanes that share a 32-byte
    // sector but lie apart cost two requests to the L2 cache).  Pieces of a row
    // are exchanged so that eight lanes that read together, two columns of rows
    // 8t + r (4 bits: t), t = 0 .. 3, use all banks: piece c of row i is at
    // c ^ (i % 8) ^ 2(i / 8), 4 bits: c ^ 2i.
    __device__ __forceinline__ void load_w(uint32_t st, const FewWalk<MB> &k) const
    {
        if constexpr (FOUR) {
            const uint32_t to = st + put, scales = st + Stage::SCALES + 8 * lane;
            if (k.step < k.whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i) few_copy16((to ^ (64u * (i & 1))) + 512 * i, k.w + 8 * i * n4);
                few_copy8(scales, k.s, 8);
            } else {
                const bool inside = column_of(k.unit) + 4 * (lane & 15) < n4;
                const int left = K32() - 64 * k.step;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    few_copy16((to ^ (64u * (i & 1))) + 512 * i, k.w + 8 * i * n4,
                               inside && 8 * (2 * i + (lane >> 4)) < left ? 16u : 0u);
                few_copy8(scales, k.s, inside && 32 * (lane >> 4) < left ? 8u : 0u);
            }
        } else if constexpr (!ANY_W) {
            const uint32_t to = st + put;
            if (k.step < k.whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i) few_copy16((to ^ (64u * (i & 1)) ^ (32u * (i >> 1))) + 512 * i, k.w + 8 * i * p.N);
            } else {
                const bool inside = column_of(k.unit) + 8 * (lane & 7) < p.N;
                const int left = K32() - (32 * k.step + (lane >> 3));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    few_copy16((to ^ (64u * (i & 1)) ^ (32u * (i >> 1))) + 512 * i, k.w + 8 * i * p.N,
                               inside && 4 * i < left ? 16u : 0u);
            }
        } else {
            // A row's 128 bytes lie in up to nine aligned pieces: eight by
            // neighbouring lanes, then the ninth of row `lane`.
            const int left = K32() - 32 * k.step, n_left = static_cast<int>(p.N) - static_cast<int>(column_of(k.unit));
            const int bytes = n_left < kFewCols ? (n_left > 0 ? 2 * n_left : -16) : 2 * kFewCols;
            if (left > 32 && n_left >= kFewCols) {
                // Whole rows, and others behind them: all nine pieces may be read.
                const uint32_t n32 = static_cast<uint32_t>(p.N), to = st + Stage::W_PITCH * (lane >> 3) + 16 * (lane & 7);
                const uint64_t row = reinterpret_cast<uint64_t>(k.w), piece = row + 16 * (lane & 7);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    few_copy16(to + Stage::W_GROUP * (i >> 1) + 4 * Stage::W_PITCH * (i & 1),
                               reinterpret_cast<const void *>((piece + static_cast<uint64_t>(n32) * (8u * i)) & ~uint64_t(15)));
                const uint64_t last = row + static_cast<uint64_t>(n32) * (2u * (lane - (lane >> 3)));
                few_copy16(st + Stage::W_GROUP * (lane >> 3) + Stage::W_PITCH * (lane & 7) + 128,
                           reinterpret_cast<const void *>((last & ~uint64_t(15)) + 128));
                return;
            }
#pragma unroll
            for (int i = 0; i < 9; ++i) {
                const int row = i < 8 ? 4 * i + (lane >> 3) : lane, piece = i < 8 ? lane & 7 : 8;
                const char *at = k.w + 2 * (row - (lane >> 3)) * p.N;
                const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15u);
                few_copy16(st + Stage::W_GROUP * (row >> 3) + Stage::W_PITCH * (row & 7) + 16 * piece, at - off + 16 * piece,
                           row < left && 16 * piece < off + bytes ? 16u : 0u);
            }
        }
    }

    // Rows of 128 bytes exchange their halves in odd rows, so that eight lanes
    // that read together, four pieces of two rows, use all banks.
    __device__ __forceinline__ void load_x(uint32_t st, const FewWalk<MB> &k) const
    {
        constexpr int HALVES = Stage::STEP / 32;
        const int left = K32() - Stage::STEP * k.step;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (MB > 1 && m >= k.blocks) break;
            const uint32_t to = st + Stage::X + Stage::X_BLOCK * m + Stage::X_PITCH * g;
            if constexpr (ANY_X) {
                const int bytes = left < Stage::STEP ? 2 * left : 2 * Stage::STEP;
                const char *at = reinterpret_cast<const char *>(k.x[m]);
                const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15u);
#pragma unroll
                for (int i = 0; i <= HALVES; ++i) {
                    const int piece = 4 * i + l4;
                    if (i < HALVES || l4 == 0)
                        few_copy16(to + 16 * piece, at - off + 16 * piece, 16 * piece < off + bytes ? k.x_bytes[m] : 0u);
                }
            } else {
                // Aligned rows hold whole pieces (hidden rows end in zeros).
                const uint32_t at = to + 16 * l4;
#pragma unroll
                for (int i = 0; i < HALVES; ++i) {
                    const uint32_t half = HALVES > 1 ? 64u * (i ^ (g & 1)) : 0u;
                    few_copy16(at + half, k.x[m] + 32 * i, k.step < k.whole || 32 * i + 8 * l4 < left ? k.x_bytes[m] : 0u);
                }
            }
        }
    }

    // Eight values of this lane's row of block m, from 32 * half + 8 * l4 on.
    __device__ __forceinline__ uint4 rows_x(uint32_t st, int m, int half, int off, int step) const
    {
        const uint32_t at = st + Stage::X + Stage::X_BLOCK * m + Stage::X_PITCH * g + 16 * l4;
        if constexpr (ANY_X) {
            uint32_t o[4];
            realign16_steps(ld_shared_v4(at + 64 * half), ld_shared_v4(at + 64 * half + 16), off, o);
            const uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
            if (step + 1 < static_cast<int>(p.steps)) return v;
            const int left = K32() - (Stage::STEP * step + 32 * half + 8 * l4);
            return few_first(v, left < 0 ? 0 : (left < 8 ? left : 8));
        } else {
            return ld_shared_v4(at + (Stage::STEP > 32 ? 64u * (half ^ (g & 1)) : 0u));
        }
    }

    // The loads of a step that is whole, and on to the next one of the unit.
    __device__ __forceinline__ void load_whole(uint32_t st, FewWalk<MB> &k, int64_t row) const
    {
        const uint32_t to = st + put;
        if constexpr (FOUR) {
            const char *w = k.w;
#pragma unroll
            for (int i = 0; i < 4; ++i, w += row) few_copy16((to ^ (64u * (i & 1))) + 512 * i, w);
            k.w = w;
            few_copy8(st + Stage::SCALES + 8 * lane, k.s, 8);
            ++k.step;
            if (p.group_steps == 1) k.s += 2 * n4;
            else if (p.group_steps == 2 || (k.step & 1) == 0) k.s += n4;
        } else {
            const char *w = k.w;
#pragma unroll
            for (int i = 0; i < 8; ++i, w += row) few_copy16((to ^ (64u * (i & 1)) ^ (32u * (i >> 1))) + 512 * i, w);
            k.w = w;
            ++k.step;
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (m < k.blocks) {
                const uint32_t at = st + Stage::X + Stage::X_BLOCK * m + Stage::X_PITCH * g + 16 * l4;
                if constexpr (FOUR) {
                    few_copy16(at ^ (64u * (g & 1)), k.x[m], k.x_bytes[m]);
                    few_copy16(at ^ (64u * (g & 1) ^ 64u), k.x[m] + 32, k.x_bytes[m]);
                } else {
                    few_copy16(at, k.x[m], k.x_bytes[m]);
                }
            }
            k.x[m] += Stage::STEP;
        }
    }

    // The eight weights of this lane's row r, whose row begins `off` bytes into its pieces.
    __device__ __forceinline__ uint4 weights_any(uint32_t st, int r, int off) const
    {
        const uint32_t at = st + Stage::W_GROUP * l4 + Stage::W_PITCH * r + 16 * g;
        uint32_t o[4];
        realign16_steps(ld_shared_v4(at), ld_shared_v4(at + 16), off, o);
        return make_uint4(o[0], o[1], o[2], o[3]);
    }

    // 4 bits: `SAME` halves of 32 products share their scales; their sums are
    // multiplied together.
    template <int SAME, int NB>
    __device__ __forceinline__ void multiply4(float (&acc)[4][MB][4], uint32_t st, int step,
                                              const int (&x_off)[MB]) const
    {
#pragma unroll
        for (int q = 0; q < 2; q += SAME) {
            uint4 x[SAME][NB];
#pragma unroll
            for (int i = 0; i < SAME; ++i)
#pragma unroll
                for (int m = 0; m < NB; ++m) x[i][m] = rows_x(st, m, q + i, x_off[m], step);
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                const uint2 scales = ld_shared_v2(st + Stage::SCALES + 128 * q + 64 * l + 8 * g);
                uint32_t w[SAME][4];
#pragma unroll
                for (int i = 0; i < SAME; ++i) {
                    const uint4 v = ld_shared_v4(st + get + 1024 * (q + i) + 128 * l);
                    w[i][0] = v.x;
                    w[i][1] = v.y;
                    w[i][2] = v.z;
                    w[i][3] = v.w;
                }
                // The sums of different columns and rows in turn, so that none
                // waits for its own last product: of both pairs of columns for 8
                // rows, of one for more (both take more registers than there are).
                constexpr int PAIRS = MB < 4 && NB == 1 ? 2 : 1;
#pragma unroll
                for (int h0 = 0; h0 < 2; h0 += PAIRS) {
                    float d[PAIRS][NB][4];
#pragma unroll
                    for (int i = 0; i < SAME; ++i)
#pragma unroll
                        for (int c = 0; c < 4; c += 2)
#pragma unroll
                            for (int h = 0; h < PAIRS; ++h) {
                                const uint32_t v0 = w[i][2 * (h0 + h)], v1 = w[i][2 * (h0 + h) + 1];
                                const uint32_t a0 = few_pair<BF16>(v0, c), a1 = few_pair<BF16>(v1, c);
                                const uint32_t a2 = few_pair<BF16>(v0, c + 1), a3 = few_pair<BF16>(v1, c + 1);
#pragma unroll
                                for (int m = 0; m < NB; ++m) {
                                    const uint32_t b0 = c ? x[i][m].z : x[i][m].x, b1 = c ? x[i][m].w : x[i][m].y;
                                    if (i == 0 && c == 0) few_mma_first<BF16, FIXED>(d[h][m], a0, a1, a2, a3, b0, b1);
                                    else few_mma<BF16, FIXED>(d[h][m], a0, a1, a2, a3, b0, b1);
                                }
                            }
#pragma unroll
                    for (int h = 0; h < PAIRS; ++h) {
                        const uint32_t sc = h0 + h ? scales.y : scales.x;
                        const float s0 = few_float<BF16>(sc & 0xffffu), s1 = few_float<BF16>(sc >> 16);
#pragma unroll
                        for (int m = 0; m < NB; ++m) {
                            float(&a)[4] = acc[2 * l + h0 + h][m];
                            a[0] = fmaf(s0, d[h][m][0], a[0]);
                            a[1] = fmaf(s0, d[h][m][1], a[1]);
                            a[2] = fmaf(s1, d[h][m][2], a[2]);
                            a[3] = fmaf(s1, d[h][m][3], a[3]);
                        }
                    }
                }
            }
        }
    }

    // acc[j][m]: columns pair j of this lane, rows 8m + 2 * l4 and the next:
    // (column, row), (column, row + 1), (column + 1, row), (column + 1, row + 1).
    // w_off, x_off: places of the step's operands off 16-byte boundaries.
    template <int NB>
    __device__ __forceinline__ void multiply(float (&acc)[4][MB][4], uint32_t st, int step, int w_off,
                                             const int (&x_off)[MB]) const
    {
        if constexpr (FOUR) {
            // (32 rows: the registers do not hold both halves' operands)
            if (MB < 4 && p.group_steps > 1) multiply4<MB < 4 ? 2 : 1, NB>(acc, st, step, x_off);
            else multiply4<1, NB>(acc, st, step, x_off);
        } else {
            uint4 x[NB];
#pragma unroll
            for (int m = 0; m < NB; ++m) x[m] = rows_x(st, m, 0, x_off[m], step);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    uint4 v;
                    if constexpr (ANY_W)
                        v = weights_any(st, 4 * h + r, (w_off + 2 * static_cast<int>(p.N & 7) * (4 * h + r)) & 15);
                    else
                        v = ld_shared_v4(((st + get) ^ (16u * (4 * h + r))) + 128 * (4 * h + r));
                    w[r][0] = v.x;
                    w[r][1] = v.y;
                    w[r][2] = v.z;
                    w[r][3] = v.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a0 = __byte_perm(w[0][j], w[1][j], 0x5410), a1 = __byte_perm(w[0][j], w[1][j], 0x7632);
                    const uint32_t a2 = __byte_perm(w[2][j], w[3][j], 0x5410), a3 = __byte_perm(w[2][j], w[3][j], 0x7632);
#pragma unroll
                    for (int m = 0; m < NB; ++m)
                        few_mma<BF16, FIXED>(acc[j][m], a0, a1, a2, a3, h ? x[m].z : x[m].x, h ? x[m].w : x[m].y);
                }
            }
        }
    }

    // (blocks without rows give columns that nobody reads)
    __device__ __forceinline__ void multiply_rows(float (&acc)[4][MB][4], uint32_t st, int step, int blocks, int w_off,
                                                  const int (&x_off)[MB]) const
    {
        if (MB > 2 && blocks > 2) multiply<MB>(acc, st, step, w_off, x_off);
        else if (MB > 1 && blocks > 1) multiply<MB < 2 ? 1 : 2>(acc, st, step, w_off, x_off);
        else multiply<1>(acc, st, step, w_off, x_off);
    }

    // First column of pair j of this lane, from n0.
    __device__ __forceinline__ int column(int j) const
    {
        return FOUR ? 32 * (j >> 1) + 4 * g + 2 * (j & 1) : 8 * g + 2 * j;
    }

    // A hidden row's sum from those of its rounded values and of their rest.  An
    // infinite weight makes infinities of both, of either sign, and NaN of a
    // rest of zero: there the sum is that of the rounded values.
    __device__ __forceinline__ static float both(float rounded, float rest)
    {
        return fabsf(rest) < INFINITY ? fmaf(rest, 1.0f / kFewLift<BF16>, rounded) : rounded;
    }

    // Adds the sums of an item, weighted, to the warp's sums of the tokens.
    __device__ __forceinline__ void add(float *sums, const float (&acc)[4][MB][4], int item) const
    {
        const int rows = static_cast<int>(t.span[item] >> 16), first = static_cast<int>(t.span[item] & 0xffffu);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int r = 4 * m + l4;
            if (r >= rows) break;
            const float w = t.weight[first + r];
            float *to = sums + (t.row[first + r] & 0xffu) * kFewCols;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float(&a)[4] = acc[j][m];
                float2 *v = reinterpret_cast<float2 *>(to + column(j));
                float2 old = *v;
                old.x = fmaf(w, both(a[0], a[1]), old.x);
                old.y = fmaf(w, both(a[2], a[3]), old.y);
                *v = old;
            }
        }
    }

    __device__ __forceinline__ static void clear(float (&acc)[4][MB][4])
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][m][i] = 0.0f;
    }

    // Bytes from an aligned piece to the first row of W (those of rows 8t are
    // the same) and to this lane's rows of X.  A step is a whole number of
    // pieces of X's row, and rows of W of any pitch: they stay within a unit.
    __device__ __forceinline__ void offsets(int unit, int &w_off, int (&x_off)[MB]) const
    {
        const int item = item_of(unit);
        if constexpr (ANY_W) {
            const int64_t e = p.ids ? static_cast<int64_t>(t.expert[item]) : 0;
            w_off = static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const uint16_t *>(W) + e * p.K * p.N + column_of(unit)) & 15u);
        }
        if constexpr (ANY_X) {
            const int rows = rows_of(item);
#pragma unroll
            for (int m = 0; m < MB; ++m) x_off[m] = static_cast<int>(reinterpret_cast<uintptr_t>(row_of(item, rows, 8 * m + g)) & 15u);
        }
    }

    // All products of the warp, from step `step` of its first unit on, `count`
    // steps, through its ring.  After a unit's last step here `done(unit, acc)`
    // takes the sums.
    template <class Done>
    __device__ __forceinline__ void walk(uint32_t ring, int step, int64_t count, Done done) const
    {
        float acc[4][MB][4];
        FewWalk<MB> k;
        k.unit = share.first;
        k.step = step;
        if (count > 0) place(k);
        FewWalk<MB> kx = k;
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (d < count) {
                load_w(ring + d * Stage::BYTES, k);
                advance(k);
            }
        if constexpr (!UP) pdl_wait();  // hidden rows come from the launch before
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (d < count) {
                load_x(ring + d * Stage::BYTES, kx);
                if (d + 1 < DEPTH) advance(kx);
            }
            few_commit();
        }
        if (FLAT && count == 0) return;
        const int64_t row = FOUR ? 8 * n4 : 8 * p.N;  // bytes from a lane's piece to its next one
        uint32_t st = ring;
        int64_t left = count;  // steps to go
        for (int unit = share.first; unit < share.units; unit += share.stride) {
            clear(acc);
            const int blocks = blocks_of(rows_of(item_of(unit)));
            int w_off = 0, x_off[MB];
            offsets(unit, w_off, x_off);
            const int last = left < share.hi - step ? step + static_cast<int>(left) : share.hi;
            const auto work = [&](auto load) {
                few_wait<DEPTH - 1>();
                __syncwarp();  // a lane's operands are other lanes' copies
                multiply_rows(acc, st, step, blocks, w_off, x_off);
                __syncwarp();
                load();
                few_commit();
                st = st == ring + (DEPTH - 1) * Stage::BYTES ? ring : st + Stage::BYTES;
            };
            while (step < last) {
                // Runs of steps whose loads are whole and lead on to the same unit: nothing else to look at.
                int run = 0;
                if (!ANY && left > DEPTH) {
                    run = min(last - step, min(k.whole, share.hi - 1) - k.step);
                    if (left - DEPTH < run) run = static_cast<int>(left - DEPTH);
                }
                if (run > 0) {
                    for (int i = 0; i < run; ++i) work([&] { load_whole(st, k, row); });
                    step += run;
                    left -= run;
                    continue;
                }
                work([&] {
                    if (left > DEPTH) {
                        load_w(st, k);
                        load_x(st, k);
                        advance(k);
                    }
                });
                ++step;
                --left;
            }
            done(unit, acc);
            if (FLAT && left == 0) break;
            step = share.lo;
        }
    }
};

// A block (of a cluster of `split`) takes units in turn: `wide` times 64 columns
// of an item (kFewFlat: the items, of its own columns).  Its warps share the
// products of 64 columns, or (wide > 1) so many each of several 64s; the blocks
// of a cluster share those of the same columns.
template <bool BF16, bool FOUR, bool ANY, int MB, int MODE>
__global__ void __launch_bounds__(32 * kFewWarps, few_blocks<MB>()) few_kernel(const __grid_constant__ FewParams p)
{
    using K = FewKernel<BF16, FOUR, ANY, MB, MODE>;
    constexpr bool UP = K::UP, FLAT = K::FLAT;
    extern __shared__ __align__(128) unsigned char few_smem[];
    const int tid = threadIdx.x, warp = tid >> 5, split = p.split;
    // The launch that makes hidden rows waits for everything before it and
    // only then lets the next one start, which may read what was there before
    // both, weights and choices, right away.
    if constexpr (UP) pdl_wait();
    pdl_launch_dependents();
    const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int matrices = UP ? p.matrices : 1;
    const int warps = kFewWarps / p.wide, each = warps / matrices;  // of 64 columns, of a matrix of theirs
    const int slab_rows = FLAT ? p.tokens : 8, slab = slab_rows * kFewCols;  // a warp's sums
    const int sent = few_sent(min(p.tokens, slab_rows));                     // those of a matrix that count, at most
    float *from_cluster = reinterpret_cast<float *>(few_smem + p.table_bytes);  // sums of other blocks
    float *sums = from_cluster + (split > 1 ? matrices * sent : 0);
    const uint32_t ring = smem_u32(sums) + kFewWarps * slab * 4 + warp * (K::DEPTH * K::Stage::BYTES);
    FewTables t{};
    int items = p.max_items;
    if (p.ids) {
        uint32_t *tables = reinterpret_cast<uint32_t *>(few_smem);
        items = p.tokens * p.top_k <= 32 ? few_build_warp<K::CHUNK>(p, t, tables) : few_build_block<K::CHUNK>(p, t, tables);
    }

    // Where the sum of row r and column n of an item is stored, and how.
    const auto finish = [&](int item, int r, int64_t n, float a, float b) {
        if (n >= p.out_cols) return;
        if (UP && p.silu) a = a / (1.0f + expf(-a));
        if (matrices == 2) a *= b;
        int64_t to = r;
        if constexpr (!FLAT) {
            if (p.ids) {
                const uint32_t row = (t.span[item] & 0xffffu) + r;
                to = t.row[row] >> 8;
                if constexpr (!UP) a *= t.weight[row];
            } else {
                to = static_cast<int64_t>(item) * K::CHUNK + r;
            }
        }
        if constexpr (MODE == kFewParts)
            static_cast<float *>(p.out)[to * p.ldo + n] = a;
        else {
            const uint16_t rounded = n < p.N ? few_round<BF16>(a) : static_cast<uint16_t>(0);
            static_cast<uint16_t *>(p.out)[to * p.ldo + n] = rounded;
            if (UP && p.rest) {  // (nothing is left of what is not finite)
                const float left = n < p.N ? (a - few_float<BF16>(rounded)) * kFewLift<BF16> : 0.0f;
                p.rest[to * p.ldo + n] = fabsf(left) < INFINITY ? few_round<BF16>(left) : static_cast<uint16_t>(0);
            }
        }
    };
    // Adds the warps' sums of `rows` rows, the first of them row r0 of the item,
    // then the cluster's, in order: every block sends its sums to the block
    // that will store them.  (more: this is not the last time.)
    const auto join = [&](int item, int64_t n0, int r0, int rows, bool more) {
        const int total = rows * kFewCols, part = (total + split - 1) / split;
        __syncthreads();
        if (split > 1) few_cluster_wait();  // the others have read what they had here before
        for (int c = 0; c < p.wide; ++c)
            for (int i = tid; i < total; i += 32 * kFewWarps) {
                float a = 0.0f, b = 0.0f;
#pragma unroll
                for (int w = 0; w < kFewWarps; ++w) {
                    const float v = w < warps ? sums[(c * warps + w) * slab + i] : 0.0f;
                    if (w < each) a += v;
                    else b += v;
                }
                if (split == 1) {
                    finish(item, r0 + i / kFewCols, n0 + c * kFewCols + i % kFewCols, a, b);
                } else {
                    const uint32_t to = mapa_shared(smem_u32(from_cluster) + 4 * (rank * part + i % part), i / part);
                    few_st_cluster(to, a);
                    if (matrices == 2) few_st_cluster(to + 4 * sent, b);
                }
            }
        if (split > 1) {
            __syncwarp();
            cluster_sync();
            for (int i = tid; i < part && rank * part + i < total; i += 32 * kFewWarps) {
                float a = 0.0f, b = 0.0f;
                for (int r = 0; r < split; ++r) {
                    a += from_cluster[r * part + i];
                    if (matrices == 2) b += from_cluster[sent + r * part + i];
                }
                const int at = rank * part + i;
                finish(item, r0 + at / kFewCols, n0 + at % kFewCols, a, b);
            }
            __syncwarp();
            if (more) few_cluster_arrive();
        }
        __syncthreads();
    };

    const int cluster = static_cast<int>(blockIdx.x) / split, clusters = static_cast<int>(gridDim.x) / split;
    if (split > 1 && (FLAT || cluster < items * p.columns)) few_cluster_arrive_first();
    if constexpr (FLAT) {
        const int64_t n0 = static_cast<int64_t>(cluster) * kFewCols;
        float *own = sums + warp * slab;
        for (int i = tid & 31; i < slab; i += 32) own[i] = 0.0f;
        __syncwarp();
        const int64_t total = static_cast<int64_t>(items) * p.steps;
        const uint32_t part = rank * kFewWarps + warp, parts = split * kFewWarps;
        // (a 64-bit division is some 200 cycles)
        const bool small = total < int64_t(1) << 26;
        const uint32_t total32 = static_cast<uint32_t>(total);
        const int64_t lo = small ? total32 * part / parts : total * part / parts;
        const int64_t hi = small ? total32 * (part + 1) / parts : total * (part + 1) / parts;
        const uint32_t first = small ? static_cast<uint32_t>(lo) / p.steps : static_cast<uint32_t>(lo / p.steps);
        const uint32_t ahead = static_cast<uint32_t>(lo - static_cast<int64_t>(first) * p.steps);
        const K k(p, t, 0, n0, FewShare{static_cast<int>(first), 1, items, 0, static_cast<int>(p.steps)});
        k.walk(ring, static_cast<int>(ahead), hi - lo,
               [&](int item, const float(&acc)[4][MB][4]) { k.add(own, acc, item); });
        join(0, n0, 0, p.tokens, false);
    } else {
        const uint32_t part = rank * each + warp % each, parts = split * each;  // at most 64
        const int lo = static_cast<int>(p.steps * part / parts), hi = static_cast<int>(p.steps * (part + 1) / parts);
        const int units = items * p.columns;
        const K k(p, t, warp % warps / each, warp / warps * kFewCols, FewShare{cluster, clusters, units, lo, hi});
        const int mine = cluster < units ? (units - cluster + clusters - 1) / clusters : 0;
        float *own = sums + warp * slab;
        k.walk(ring, lo, static_cast<int64_t>(mine) * (hi - lo), [&](int unit, const float(&acc)[4][MB][4]) {
            const int item = unit / p.columns, rows = k.rows_of(item);
            const int64_t n0 = static_cast<int64_t>(unit % p.columns) * (p.wide * kFewCols);
            // 8 rows at a time: of a block of the products, or of two where a row is two of theirs.
#pragma unroll
            for (int m0 = 0; m0 < MB; m0 += K::PARTS) {
                const int r0 = 8 / K::PARTS * m0;
                if (MB > K::PARTS && r0 >= rows) break;
#pragma unroll
                for (int m = m0; m < m0 + K::PARTS && m < MB; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float(&a)[4] = acc[j][m];
                        if constexpr (UP) {
                            *reinterpret_cast<float2 *>(own + 2 * k.l4 * kFewCols + k.column(j)) = make_float2(a[0], a[2]);
                            *reinterpret_cast<float2 *>(own + (2 * k.l4 + 1) * kFewCols + k.column(j)) = make_float2(a[1], a[3]);
                        } else {
                            *reinterpret_cast<float2 *>(own + (4 * (m - m0) + k.l4) * kFewCols + k.column(j)) =
                                make_float2(k.both(a[0], a[1]), k.both(a[2], a[3]));
                        }
                    }
                join(item, n0, r0, min(rows - r0, 8), r0 + 8 < rows || unit + clusters < units);
            }
        });
    }
}

// ------------------------------------------------------------------ launch

template <bool BF16, bool FOUR, bool ANY, int MB, int MODE>
cudaError_t launch_few_kernel(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    using K = FewKernel<BF16, FOUR, ANY, MB, MODE>;
    constexpr int kMaxSmem = 227 * 1024;
    const int rows = K::FLAT ? p.tokens : 8, sent = p.tokens < rows ? p.tokens : rows;
    const int smem = p.table_bytes + 4 * ((p.split > 1 ? p.matrices * few_sent(sent) : 0) + kFewWarps * rows * kFewCols) +
                     kFewWarps * K::DEPTH * K::Stage::BYTES;
    if (smem > kMaxSmem) return cudaErrorInvalidConfiguration;
    static std::atomic<int> done[128];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (!done[dev].load()) {
        e = cudaFuncSetAttribute(few_kernel<BF16, FOUR, ANY, MB, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMaxSmem);
        if (e != cudaSuccess) return e;
        done[dev].store(1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.grid, 1, 1);
    cfg.blockDim = dim3(32 * kFewWarps, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
    if (p.split > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = p.split;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    e = cudaLaunchKernelEx(&cfg, few_kernel<BF16, FOUR, ANY, MB, MODE>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Clusters of `split` blocks that run at once on the current device, for the
// kernels of two blocks an SM (MB 1) or of one (MB 4); 0 on an error.
template <int MB>
int few_room_of(int split)
{
    const auto kernel = few_kernel<true, false, false, MB, kFewUp>;
    constexpr int smem = MB < 4 ? 100 * 1024 : 200 * 1024;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split * 64, 1, 1);
    cfg.blockDim = dim3(32 * kFewWarps, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

template <bool BF16, bool FOUR, bool ANY, int MB>
cudaError_t launch_few_mode(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    if (l.mode == kFewUp) return launch_few_kernel<BF16, FOUR, ANY, MB, kFewUp>(l, p, s);
    // Hidden rows are always aligned: with weights in 4 bits nothing else can be off.
    constexpr bool any = ANY && !FOUR;
    if constexpr (MB < 4)
        if (l.mode == kFewFlat) return launch_few_kernel<BF16, FOUR, any, MB, kFewFlat>(l, p, s);
    if constexpr (MB == 1 || (FOUR && MB == 4))
        return cudaErrorInvalidConfiguration;
    else
        return l.mode == kFewParts ? launch_few_kernel<BF16, FOUR, any, MB, kFewParts>(l, p, s) : cudaErrorInvalidConfiguration;
}

template <bool BF16, bool FOUR>
cudaError_t launch_few_type(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    if (l.row_blocks == 1) return l.any ? launch_few_mode<BF16, FOUR, true, 1>(l, p, s) : launch_few_mode<BF16, FOUR, false, 1>(l, p, s);
    if (l.row_blocks == 2) return l.any ? launch_few_mode<BF16, FOUR, true, 2>(l, p, s) : launch_few_mode<BF16, FOUR, false, 2>(l, p, s);
    if constexpr (FOUR)
        if (l.any) return launch_few_mode<BF16, FOUR, true, 4>(l, p, s);
    return l.any ? cudaErrorInvalidConfiguration : launch_few_mode<BF16, FOUR, false, 4>(l, p, s);
}

}  // namespace gp
