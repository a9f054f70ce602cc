// few_kernel.cuh -- products of a few rows with large matrices: one matrix in
// 4 bits, or the matrices of the experts that a few tokens chose.
//
// out[r][n] = sum over k of X[r][k] * W[k][n], for at most 64 rows.  Every
// weight is read once and used for few rows, so the kernel is bound by the
// rate at which weights come from memory; everything else is arranged around
// loads that never wait for one another:
//   - a warp takes 64 columns and walks over k in steps of 32.  Its lanes load
//     16-byte pieces of the matrix straight into registers, a few steps ahead
//     of the products, without shared memory or barriers in between;
//   - the products run on warp-level matrix instructions (m16n8k16) with the
//     weights as the 16-row operand and 8 rows of X as the 8-column operand.
//     The places of n and k in that operand are free as long as X has the same
//     order, so a lane's own loads are its operand: with g = lane / 4 and
//     t = lane % 4 it has rows k = 8t .. 8t + 7 of a step and
//       16 bits: columns 8g .. 8g + 7 (one 16-byte load a row),
//       4 bits:  columns 4g .. 4g + 3 and 32 + 4g .. (a word of 8 rows each);
//     in 16 bits two rows' words are woven into (k, k + 1) pairs by byte
//     permutes, in 4 bits a word's pairs lie as the instruction wants them;
//   - X's operand is the 8 values k = 8t .. 8t + 7 of row g: one 16-byte load;
//   - 4-bit values become v + 1024 (fp16) or v + 128 (bf16) by one mask and or,
//     exact, then the constant and the 8 are taken off, exact; a step's sum is
//     multiplied by the columns' scales in fp32, so nothing is rounded before
//     the end but hidden rows, which are operands of the next product;
//   - the 8 warps of a block and the blocks of a cluster share the products;
//     their sums meet in shared memory, in a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "few.h"
#include "ptx.cuh"

namespace gp {

// ------------------------------------------------------------ small pieces

template <bool BF16>
__device__ __forceinline__ void few_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Values i and i + 4 of a word of eight 4-bit values: the pair of rows 2i, 2i + 1.
template <bool BF16>
__device__ __forceinline__ uint32_t few_pair(uint32_t word, int i)
{
    const uint32_t q = (word >> (4 * i)) & 0x000f000fu;
    if constexpr (BF16) {
        const uint32_t m = q | 0x43004300u;  // 128 + q
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&m), __float2bfloat162_rn(136.0f));
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const uint32_t m = q | 0x64006400u;  // 1024 + q
        const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&m), __float2half2_rn(1032.0f));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

__device__ __forceinline__ uint4 few_ld_v4(const void *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ uint2 few_ld_v2(const void *p)
{
    uint2 v;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// 8 bytes at p if `on`, else zeros.
__device__ __forceinline__ uint2 few_ld_v2_if(const void *p, bool on)
{
    uint2 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %3, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "@p ld.global.v2.u32 {%0, %1}, [%2];\n\t}"
        : "=&r"(v.x), "=&r"(v.y)
        : "l"(p), "r"(on ? 1u : 0u)
        : "memory");
    return v;
}

// Eight 16-bit elements at p, the first `count` of them (others: whatever is
// there, or zeros); any 2-byte alignment.  Only words that hold one of the
// first `count` are read.
__device__ __forceinline__ uint4 few_load8_any(const uint16_t *p, int count)
{
    const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
    const char *a = reinterpret_cast<const char *>(p) - s;
    const uint4 lo = ld_global_v4_if(a, count > 0);
    const uint4 hi = ld_global_v4_if(a + 16, count > 0 && static_cast<int>(s) + 2 * (count < 8 ? count : 8) > 16);
    uint32_t o[4];
    realign16_steps(lo, hi, s, o);
    return make_uint4(o[0], o[1], o[2], o[3]);
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

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
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
    const uint32_t items = __ballot_sync(0xffffffffu, leader);
    const int count = __popc(peers);
    int first = leader ? count : 0;  // sum of the rows of earlier items
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, first, d);
        if (lane >= d) first += v;
    }
    first -= leader ? count : 0;
    first = __shfl_sync(0xffffffffu, first, row ? __ffs(peers) - 1 : 0);
    if (row) {
        const int at = first + __popc(peers & below);
        t.row[at] = static_cast<uint32_t>(token) | static_cast<uint32_t>(lane) << 8;
        t.weight[at] = w;
    }
    if (leader) {
        const int i = __popc(items & below);
        t.expert[i] = e;
        t.span[i] = static_cast<uint32_t>(first) | static_cast<uint32_t>(count) << 16;
    }
    __syncwarp();
    return __popc(items);
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
        uint32_t both = rows | items << 16;  // at most 4096 and 1148
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

template <bool FOUR, int MB>
struct FewStage {
    uint4 w[FOUR ? 2 : 8];
    uint2 s[FOUR ? 2 : 1];
    uint4 x[MB];
};

// Where a warp's loads are: an item, a step of it, and this lane's places.
template <int MB>
struct FewWalk {
    int item, step, blocks;
    int group;                  // 4 bits: steps left in the group
    const char *w;              // this lane's piece of the step's first row (4 bits: of its word row)
    const uint16_t *s;          // this lane's scales of the group
    const uint16_t *x[MB];      // this lane's 8 values of each row (a place without a row: of the item's first)
};

template <bool BF16, bool FOUR, bool ANY, int MB, bool DOWN>
struct FewKernel {
    static constexpr int CHUNK = 8 * MB;
    static constexpr int DEPTH = FOUR ? 4 : 2;  // steps whose loads are in flight

    const FewParams &p;
    const FewTables &t;
    const void *W;
    const uint16_t *S;
    int64_t n0, n4;
    int g, l4;         // lane / 4, lane % 4
    int steps;
    int whole;         // steps whose loads of the warp are all inside the matrix
    int cols;          // 16 bits: this lane's columns inside the matrix (0 .. 8)
    bool on4[2];       // 4 bits: whether each piece is

    __device__ __forceinline__ FewKernel(const FewParams &p_, const FewTables &t_, int matrix, int64_t n0_)
        : p(p_), t(t_), W(matrix ? p_.W[1] : p_.W[0]), S(matrix ? p_.S[1] : p_.S[0]), n0(n0_)
    {
        const int lane = threadIdx.x & 31;
        g = lane >> 2;
        l4 = lane & 3;
        n4 = (p.N + 3) / 4 * 4;
        steps = static_cast<int>(p.steps);
        const bool wide = n0 + kFewCols <= (FOUR ? n4 : p.N);
        whole = wide && !ANY ? static_cast<int>(p.K / kFewStep) : 0;
        if constexpr (FOUR) {
            on4[0] = n0 + 4 * g < n4;
            on4[1] = n0 + 32 + 4 * g < n4;
        } else {
            const int64_t left = p.N - (n0 + 8 * g);
            cols = left < 0 ? 0 : (left < 8 ? static_cast<int>(left) : 8);
        }
    }

    __device__ __forceinline__ int rows_of(int item) const
    {
        return p.ids ? static_cast<int>(t.span[item] >> 16) : min(p.tokens - item * CHUNK, CHUNK);
    }

    __device__ __forceinline__ void place(FewWalk<MB> &k) const
    {
        const int64_t e = p.ids ? t.expert[k.item] : 0;
        if constexpr (FOUR) {
            const int group_rows = 32 * p.group_steps, gr = k.step / p.group_steps;
            const int64_t words = (p.K + 7) / 8, groups = (p.K + group_rows - 1) / group_rows;
            k.w = reinterpret_cast<const char *>(static_cast<const uint32_t *>(W) + (e * words + 4 * static_cast<int64_t>(k.step) + l4) * n4 + n0 + 4 * g);
            k.s = S + (e * groups + gr) * n4 + n0 + 4 * g;
            k.group = (gr + 1) * p.group_steps - k.step;
        } else {
            k.w = reinterpret_cast<const char *>(static_cast<const uint16_t *>(W) + (e * p.K + 32 * static_cast<int64_t>(k.step) + 8 * l4) * p.N + n0 + 8 * g);
        }
        const int rows = rows_of(k.item), first = p.ids ? static_cast<int>(t.span[k.item] & 0xffffu) : k.item * CHUNK;
        k.blocks = (rows + 7) / 8;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            int64_t r = first + (8 * m + g < rows ? 8 * m + g : 0);
            if (p.ids) r = DOWN ? t.row[r] >> 8 : t.row[r] & 0xffu;
            k.x[m] = p.X + r * p.ldx + 32 * static_cast<int64_t>(k.step) + 8 * l4;
        }
    }

    __device__ __forceinline__ void advance(FewWalk<MB> &k, int items) const
    {
        if (++k.step == steps) {
            k.step = 0;
            if (++k.item < items) place(k);
            return;
        }
        if constexpr (FOUR) {
            k.w += 16 * n4;  // 4 rows of words
            if (--k.group == 0) {
                k.s += n4;
                k.group = p.group_steps;
            }
        } else {
            k.w += 64 * p.N;
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) k.x[m] += 32;
    }

    __device__ __forceinline__ void load_w(FewStage<FOUR, MB> &st, const FewWalk<MB> &k) const
    {
        if (k.step < whole) {
            if constexpr (FOUR) {
#pragma unroll
                for (int l = 0; l < 2; ++l) st.w[l] = few_ld_v4(k.w + 128 * l);
#pragma unroll
                for (int l = 0; l < 2; ++l) st.s[l] = few_ld_v2(k.s + 32 * l);
            } else {
#pragma unroll
                for (int r = 0; r < 8; ++r) st.w[r] = few_ld_v4(k.w + 2 * r * p.N);
            }
            return;
        }
        const int64_t left = p.K - (32 * static_cast<int64_t>(k.step) + 8 * l4);  // rows from this lane's first
        if constexpr (FOUR) {
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                st.w[l] = ld_global_v4_if(k.w + 128 * l, left > 0 && on4[l]);
                st.s[l] = few_ld_v2_if(k.s + 32 * l, on4[l]);
            }
        } else {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const char *at = k.w + 2 * r * p.N;
                if constexpr (ANY)
                    st.w[r] = few_load8_any(reinterpret_cast<const uint16_t *>(at), r < left ? cols : 0);
                else
                    st.w[r] = ld_global_v4_if(at, r < left && cols > 0);
            }
        }
    }

    __device__ __forceinline__ void load_x(FewStage<FOUR, MB> &st, const FewWalk<MB> &k) const
    {
        // Aligned rows hold whole pieces (hidden rows end in zeros).
        const int64_t left = p.K - (32 * static_cast<int64_t>(k.step) + 8 * l4);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (MB > 1 && m >= k.blocks) break;
            if constexpr (ANY && !DOWN) {
                const int count = left < 0 ? 0 : (left < 8 ? static_cast<int>(left) : 8);
                st.x[m] = few_first(few_load8_any(k.x[m], count), count);
            } else {
                st.x[m] = ld_global_v4_if(k.x[m], left > 0);
            }
        }
    }

    // acc[j][m]: columns pair j of this lane, rows 8m + 2 * l4 and the next:
    // (column, row), (column, row + 1), (column + 1, row), (column + 1, row + 1).
    __device__ __forceinline__ void multiply(float (&acc)[4][MB][4], const FewStage<FOUR, MB> &st, int blocks) const
    {
        if constexpr (FOUR) {
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                const uint32_t w[4] = {st.w[l].x, st.w[l].y, st.w[l].z, st.w[l].w};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t u[2][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        u[0][i] = few_pair<BF16>(w[2 * h], i);
                        u[1][i] = few_pair<BF16>(w[2 * h + 1], i);
                    }
                    const uint32_t sc = h ? st.s[l].y : st.s[l].x;
                    const float s0 = few_float<BF16>(sc & 0xffffu), s1 = few_float<BF16>(sc >> 16);
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
                        if (MB > 1 && m >= blocks) break;
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        few_mma<BF16>(d, u[0][0], u[1][0], u[0][1], u[1][1], st.x[m].x, st.x[m].y);
                        few_mma<BF16>(d, u[0][2], u[1][2], u[0][3], u[1][3], st.x[m].z, st.x[m].w);
                        float(&a)[4] = acc[2 * l + h][m];
                        a[0] = fmaf(s0, d[0], a[0]);
                        a[1] = fmaf(s0, d[1], a[1]);
                        a[2] = fmaf(s1, d[2], a[2]);
                        a[3] = fmaf(s1, d[3], a[3]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w[4][4] = {{st.w[4 * h].x, st.w[4 * h].y, st.w[4 * h].z, st.w[4 * h].w},
                                          {st.w[4 * h + 1].x, st.w[4 * h + 1].y, st.w[4 * h + 1].z, st.w[4 * h + 1].w},
                                          {st.w[4 * h + 2].x, st.w[4 * h + 2].y, st.w[4 * h + 2].z, st.w[4 * h + 2].w},
                                          {st.w[4 * h + 3].x, st.w[4 * h + 3].y, st.w[4 * h + 3].z, st.w[4 * h + 3].w}};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a0 = __byte_perm(w[0][j], w[1][j], 0x5410), a1 = __byte_perm(w[0][j], w[1][j], 0x7632);
                    const uint32_t a2 = __byte_perm(w[2][j], w[3][j], 0x5410), a3 = __byte_perm(w[2][j], w[3][j], 0x7632);
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
                        if (MB > 1 && m >= blocks) break;
                        few_mma<BF16>(acc[j][m], a0, a1, a2, a3, h ? st.x[m].z : st.x[m].x, h ? st.x[m].w : st.x[m].y);
                    }
                }
            }
        }
    }

    // First column of pair j of this lane, from n0.
    __device__ __forceinline__ int column(int j) const
    {
        return FOUR ? 32 * (j >> 1) + 4 * g + 2 * (j & 1) : 8 * g + 2 * j;
    }

    // Adds the sums of an item, weighted, to the warp's sums of the tokens.
    __device__ __forceinline__ void add(float *sums, const float (&acc)[4][MB][4], int item) const
    {
        const int rows = static_cast<int>(t.span[item] >> 16), first = static_cast<int>(t.span[item] & 0xffffu);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (MB > 1 && 8 * m >= rows) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * m + 2 * l4 + i;
                if (r >= rows) continue;
                const float w = t.weight[first + r];
                float *to = sums + (t.row[first + r] & 0xffu) * kFewCols;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 *v = reinterpret_cast<float2 *>(to + column(j));
                    float2 old = *v;
                    old.x = fmaf(w, acc[j][m][i], old.x);
                    old.y = fmaf(w, acc[j][m][2 + i], old.y);
                    *v = old;
                }
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

    // The warp's `count` steps from step `step` of item `item` on; down: sums
    // by token in `sums`, else the item's in acc.
    __device__ __forceinline__ void walk(float (&acc)[4][MB][4], float *sums, int item, int step, int items,
                                         int count) const
    {
        clear(acc);
        FewStage<FOUR, MB> st[DEPTH];
        FewWalk<MB> k;
        k.item = item;
        k.step = step;
        if (count > 0) place(k);
        FewWalk<MB> kx = k;
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (d >= count) break;
            load_w(st[d], k);
            advance(k, items);
        }
        if constexpr (DOWN) pdl_wait();  // hidden rows come from the launch before
        int blocks = kx.blocks;
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (d >= count) break;
            load_x(st[d], kx);
            if (DOWN || d + 1 < DEPTH) advance(kx, items);
        }
        for (int i = 0; i < count; i += DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (i + d >= count) break;
                multiply(acc, st[d], blocks);
                if (i + d + DEPTH < count) {
                    load_w(st[d], k);
                    load_x(st[d], k);
                    advance(k, items);
                }
                if constexpr (DOWN) {
                    if (++step == steps || i + d + 1 == count) {
                        add(sums, acc, item);
                        clear(acc);
                        if (step == steps && i + d + 1 < count) {
                            step = 0;
                            ++item;
                            blocks = (rows_of(item) + 7) / 8;
                        }
                    }
                }
            }
        }
    }
};

// grid: x = column blocks x cluster blocks, y = items (down: 1).
template <bool BF16, bool FOUR, bool ANY, int MB, bool DOWN>
__global__ void __launch_bounds__(32 * kFewWarps, MB == 1 ? 2 : 1)
    few_kernel(const __grid_constant__ FewParams p, int split)
{
    using K = FewKernel<BF16, FOUR, ANY, MB, DOWN>;
    extern __shared__ __align__(16) unsigned char few_smem[];
    const int tid = threadIdx.x, warp = tid >> 5;
    // The launch that makes hidden rows waits for everything before it and
    // only then lets the next one start, which may read what was there before
    // both, weights and choices, right away.
    if constexpr (!DOWN) pdl_wait();
    pdl_launch_dependents();
    const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x / split) * kFewCols;
    float *sums = reinterpret_cast<float *>(few_smem + p.table_bytes);
    FewTables t{};
    int items = static_cast<int>(gridDim.y);
    if (p.ids) {
        uint32_t *tables = reinterpret_cast<uint32_t *>(few_smem);
        items = p.tokens * p.top_k <= 32 ? few_build_warp(p, t, tables) : few_build_block<K::CHUNK>(p, t, tables);
    }
    float acc[4][MB][4];
    int count;  // rows of sums
    if constexpr (DOWN) {
        count = p.tokens;
        float *own = sums + warp * (p.tokens * kFewCols);
        for (int i = tid & 31; i < p.tokens * kFewCols; i += 32) own[i] = 0.0f;
        __syncwarp();
        const int64_t total = static_cast<int64_t>(items) * p.steps;
        const int part = rank * kFewWarps + warp, parts = split * kFewWarps;
        const int64_t lo = total * part / parts, hi = total * (part + 1) / parts;
        const K k(p, t, 0, n0);
        k.walk(acc, own, static_cast<int>(lo / p.steps), static_cast<int>(lo % p.steps), items,
               static_cast<int>(hi - lo));
    } else {
        const int item = blockIdx.y;
        if (item >= items) return;  // the whole cluster
        const int warps = kFewWarps / p.matrices, matrix = warp / warps;
        const int part = rank * warps + warp % warps, parts = split * warps;
        const int64_t lo = p.steps * part / parts, hi = p.steps * (part + 1) / parts;
        const K k(p, t, matrix, n0);
        count = k.rows_of(item);
        k.walk(acc, nullptr, item, static_cast<int>(lo), item + 1, static_cast<int>(hi - lo));
        float *own = sums + warp * (K::CHUNK * kFewCols);
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<float2 *>(own + (8 * m + 2 * k.l4 + i) * kFewCols + k.column(j)) =
                        make_float2(acc[j][m][i], acc[j][m][2 + i]);
    }
    __syncthreads();

    // The warps' sums, then the cluster's, in order.
    const int slab = (DOWN ? p.tokens : K::CHUNK) * kFewCols, total = count * kFewCols;
    const bool two = !DOWN && p.matrices == 2;
    const int warps = two ? kFewWarps / 2 : kFewWarps;
    const auto finish = [&](int i, float a, float b) {
        const int r = i / kFewCols;
        const int64_t n = n0 + i % kFewCols;
        if (n >= p.out_cols) return;
        if (!DOWN && p.silu) a = a / (1.0f + expf(-a));
        if (two) a *= b;
        int64_t to = r;
        if (!DOWN)
            to = p.ids ? t.row[(t.span[blockIdx.y] & 0xffffu) + r] >> 8 : static_cast<int64_t>(blockIdx.y) * K::CHUNK + r;
        p.out[to * p.ldo + n] = n < p.N ? few_round<BF16>(a) : static_cast<uint16_t>(0);
    };
    for (int i = tid; i < total; i += 32 * kFewWarps) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float v = sums[w * slab + i];
            if (w < warps) a += v;
            else b += v;
        }
        if (split == 1) {
            finish(i, a, b);
        } else {
            sums[i] = a;
            if (two) sums[slab + i] = b;
        }
    }
    if (split == 1) return;
    cluster_sync();
    const uint32_t base = smem_u32(sums);
    for (int i = rank * (32 * kFewWarps) + tid; i < total; i += split * (32 * kFewWarps)) {
        float a = 0.0f, b = 0.0f;
        for (int r = 0; r < split; ++r) {
            a += ld_cluster_f32(mapa_shared(base + 4 * i, r));
            if (two) b += ld_cluster_f32(mapa_shared(base + 4 * (slab + i), r));
        }
        finish(i, a, b);
    }
    cluster_sync();  // others may still read this block's sums
}

// ------------------------------------------------------------------ launch

template <bool BF16, bool FOUR, bool ANY, int MB, bool DOWN>
cudaError_t launch_few_kernel(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    constexpr int kMaxSmem = 227 * 1024;
    if (l.smem_bytes > kMaxSmem) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaSuccess;
    if (l.smem_bytes > 48 * 1024 &&
        (e = cudaFuncSetAttribute(few_kernel<BF16, FOUR, ANY, MB, DOWN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  kMaxSmem)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.grid_x, l.grid_y, 1);
    cfg.blockDim = dim3(32 * kFewWarps, 1, 1);
    cfg.dynamicSmemBytes = l.smem_bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
    if (l.split > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = l.split;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    e = cudaLaunchKernelEx(&cfg, few_kernel<BF16, FOUR, ANY, MB, DOWN>, p, l.split);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool BF16, bool FOUR, bool ANY, int MB>
cudaError_t launch_few_rows(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    // Hidden rows are always aligned: with weights in 4 bits nothing else can be off.
    if constexpr (FOUR && ANY)
        return l.down ? launch_few_kernel<BF16, FOUR, false, MB, true>(l, p, s)
                      : launch_few_kernel<BF16, FOUR, ANY, MB, false>(l, p, s);
    else
        return l.down ? launch_few_kernel<BF16, FOUR, ANY, MB, true>(l, p, s)
                      : launch_few_kernel<BF16, FOUR, ANY, MB, false>(l, p, s);
}

template <bool BF16, bool FOUR>
cudaError_t launch_few_type(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    if (l.row_blocks == 1)
        return l.any ? launch_few_rows<BF16, FOUR, true, 1>(l, p, s) : launch_few_rows<BF16, FOUR, false, 1>(l, p, s);
    return l.any ? launch_few_rows<BF16, FOUR, true, 4>(l, p, s) : launch_few_rows<BF16, FOUR, false, 4>(l, p, s);
}

}  // namespace gp
