// few.h -- launchers of the kernels for a few rows (few_kernel.cuh,
// rows4_wide.cu) and of the weights' way into 4 bits and back (pack4.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gemmpipe.h"

namespace gp {

constexpr int kFewRows = 64;       // rows or tokens of a call, at most
constexpr int kFewCols = 64;       // output columns of a block
constexpr int kFewWarps = 8;       // warps of a block

// What a launch computes:
enum FewMode : int {
    kFewUp = 0,    // rows of X times a matrix, or the tokens' rows times their experts' matrices: hidden rows
    kFewFlat = 1,  // hidden rows times the experts' second matrices, summed by token in the block (few tokens)
    kFewParts = 2, // the same, one fp32 row for each choice: few_combine adds them
};

// Rows of an item: what `blocks` 8-row blocks of the products hold.  Hidden rows
// are in two parts, their rounding to the type and what that leaves, so that
// nothing is lost between the products, and take two rows each.
__host__ __device__ constexpr int few_chunk(int blocks, bool up) { return (up ? 8 : 4) * blocks; }

// One launch.  An item is an expert and up to few_chunk of the tokens that chose
// it, or (`ids` null) so many of `tokens` rows of X.
struct FewParams {
    const uint16_t *X;      // kFewUp: rows by token; else by slot
    const uint16_t *X2;     // not kFewUp: what their rounding left
    int64_t ldx;
    const int32_t *ids;     // tokens x top_k
    const float *weights;   // tokens x top_k (not kFewUp)
    const void *W[2];       // matrices experts x K x N (16 bits), or words experts x ceil(K / 8) x N4 (4 bits)
    const uint16_t *S[2];   // scales experts x ceil(K / group) x N4 (4 bits)
    void *out;              // 16 bits; kFewParts: fp32
    uint16_t *rest;         // kFewUp: what the rounding of out leaves (may be null)
    int64_t ldo;
    int64_t K, N;
    int64_t out_cols;       // columns of out: those past N are set to zero
    int64_t words, groups;  // ceil(K / 8), ceil(K / group) (4 bits)
    uint32_t steps;         // ceil(K / step): below 2^26
    int tokens, top_k, experts;
    int group_steps;        // group / 32
    int group_shift;        // log2 of it
    int matrices;           // 2: silu(first product) * second product
    int silu;               // 1: silu of the (first) product
    int max_items;
    int columns;            // blocks of columns: ceil(out_cols / (64 * wide))
    int split;              // blocks of a cluster (1 to 8), sharing the products of 64 columns
    int wide;               // 64s of columns of a block: 1, 2 or 4 (with split 1)
    int table_bytes;        // shared memory of the table of items
};

// What a warp copies for one step of 32 products (4 bits: 64): the rows of 64
// weights (16 bits: eight 16-byte pieces a row; off 16-byte boundaries nine,
// rows 8t .. 8t + 7 shifted by 2t pieces so that the lanes of a load use
// different banks; 4 bits: 8 rows of words, and the scales of both halves),
// and the values of the rows of X (off boundaries: a piece more).
template <bool FOUR, bool ANY_W, bool ANY_X, int MB>
struct FewStage {
    static constexpr int STEP = FOUR ? 64 : 32;
    static constexpr int W_PITCH = 144, W_GROUP = 8 * W_PITCH + 32;
    static constexpr int SCALES = 2048;
    static constexpr int X = FOUR ? 2048 + 256 : (ANY_W ? 4 * W_GROUP : 4096);
    static constexpr int X_PITCH = 2 * STEP + (ANY_X ? 16 : 0);
    static constexpr int X_BLOCK = 8 * X_PITCH;
    static constexpr int BYTES = X + MB * X_BLOCK;
};

// Blocks of an SM: two, but one where an item's sums take half of the registers
// of two.
template <int MB>
constexpr int few_blocks()
{
    return MB < 4 ? 2 : 1;
}

// Stages of a warp's ring: what lets two blocks run on an SM beside their sums
// and tables.  (A stage more made short calls slower by up to 5%: the first
// products wait for more copies of others.)
template <bool FOUR, int MB>
constexpr int few_depth()
{
    return (FOUR && MB == 1) || MB == 4 ? 3 : 2;
}

// Floats of a block's room for the cluster's sums of `rows` rows of a matrix (a
// multiple of 128 bytes: the rings follow).
__host__ __device__ constexpr int few_sent(int rows) { return rows * kFewCols + 32; }

struct FewLaunch {
    bool bf16, four, any;
    int mode;
    int row_blocks;         // 8-row blocks of an item: 1, 2 or 4
    int grid;               // blocks
    gemmpipe_status_t status;
};

// four: weights in 4 bits; any: operands off 16-byte boundaries.
cudaError_t launch_few_f16(const FewLaunch &l, const FewParams &p, cudaStream_t s);
cudaError_t launch_few_bf16(const FewLaunch &l, const FewParams &p, cudaStream_t s);

// Clusters of `split` (1 to 8) blocks that run at once on the current device:
// [0] of kernels with two blocks an SM, [1] with one.  0 on an error.
int few_room(int one, int split);

// Y[t] = sum of the rows of `parts` (tokens x top_k rows of `width`) that stand
// for a choice: one inside [0, experts), the token's first of that expert.
cudaError_t launch_few_combine(bool bf16, int tokens, int top_k, int experts, int64_t width, const int32_t *ids,
                               const float *parts, uint16_t *Y, int64_t ldy, cudaStream_t s);

// ---- some rows times weights in 4 bits (rows4_wide.cu)

struct WideParams {
    const uint16_t *X;
    int64_t ldx;
    const uint32_t *Q;
    const uint16_t *S;
    uint16_t *Y;
    int64_t ldy, N, n4, K;
    int M, group;
    int stages;            // ceil(K / wide_stage_k)
    int split;             // CTAs of a cluster, sharing a tile's k
    int64_t stall_stage;   // test hook: the stage that CTA 0 leaves unfilled (-1: none)
    int *status;
    uint64_t timeout_ns;
};

constexpr int kWideCols = 128;  // columns of a tile

// Products of a row in a stage of the ring.
constexpr int wide_stage_k(int group) { return group == 32 ? 64 : 128; }

// words: boxes of 128 x (stage / 8), not swizzled; rows: X, boxes of 64 x 64 (more than 32
// rows) or 64 x 32.
cudaError_t launch_rows4_wide(bool bf16, const CUtensorMap &words, const CUtensorMap &rows, const WideParams &p,
                              int grid, cudaStream_t s);

// ---- weights into 4 bits and back (pack4.cu)

cudaError_t launch_pack4(bool bf16, int64_t experts, int64_t K, int64_t N, int group, const uint16_t *W, uint32_t *Q,
                         uint16_t *S, cudaStream_t s);
cudaError_t launch_unpack4(bool bf16, int64_t experts, int64_t K, int64_t N, int group, const uint32_t *Q,
                           const uint16_t *S, uint16_t *W, cudaStream_t s);

}  // namespace gp
