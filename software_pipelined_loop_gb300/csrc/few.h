// few.h -- launchers of the kernels for a few rows (few_kernel.cuh) and of the
// weights' way into 4 bits and back (pack4.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gp {

constexpr int kFewRows = 64;       // rows or tokens of a call, at most
constexpr int kFewCols = 64;       // output columns of a block
constexpr int kFewWarps = 8;       // warps of a block, at most
constexpr int kFewStep = 32;       // products of a row per step

// One launch.  Products of rows with one matrix (`ids` null: `tokens` rows of X
// give `tokens` rows of `out`) or with the matrices of the experts that have
// rows: upwards from the tokens' rows to one hidden row per choice, or (`down`)
// from those to the weighted sum of each token.
struct FewParams {
    const uint16_t *X;      // rows by token; down: by slot
    int64_t ldx;
    const int32_t *ids;     // tokens x top_k
    const float *weights;   // tokens x top_k (down)
    const void *W[2];       // matrices experts x K x N (16 bits), or words experts x ceil(K / 8) x N4 (4 bits)
    const uint16_t *S[2];   // scales experts x ceil(K / group) x N4 (4 bits)
    uint16_t *out;
    int64_t ldo;
    int64_t K, N;
    int64_t out_cols;       // columns of out: those past N are set to zero
    int64_t steps;          // ceil(K / 32)
    int tokens, top_k, experts;
    int group_steps;        // group / 32
    int matrices;           // 2: silu(first product) * second product
    int silu;               // 1: silu of the (first) product
    int max_items;          // entries of the table of (expert, up to 8 * blocks of its rows)
    int table_bytes;        // shared memory before the sums
    int depth;              // stages of a warp's ring, 1 to 8
};

// What a warp copies for one step of 32 products: 32 rows of 64 weights (16
// bits: eight 16-byte pieces a row; off 16-byte boundaries nine, rows 8t .. 8t
// + 7 shifted by 2t pieces so that the lanes of a load use different banks; 4
// bits: 4 rows of words, and scales), and 32 values of the rows of X (off
// boundaries: five pieces a row).
template <bool FOUR, bool ANY_W, bool ANY_X, int MB>
struct FewStage {
    static constexpr int W_PITCH = 144, W_GROUP = 8 * W_PITCH + 32;
    static constexpr int SCALES = 1024;
    static constexpr int X = FOUR ? 1024 + 128 : (ANY_W ? 4 * W_GROUP : 4096);
    static constexpr int X_BLOCK = ANY_X ? 640 : 512;
    static constexpr int BYTES = X + MB * X_BLOCK;
};

constexpr int few_stage_bytes(bool four, bool any_w, bool any_x, int blocks)
{
    return (four ? 1024 + 128 : (any_w ? FewStage<false, true, true, 1>::X : 4096)) + blocks * (any_x ? 640 : 512);
}

struct FewLaunch {
    bool bf16, four, any, down;
    int row_blocks;         // 8-row blocks of an item: 1 or 4
    int split;              // blocks of a cluster, sharing the products
    int warps;              // warps of a block
    int grid_x, grid_y;
    int smem_bytes;
};

// four: weights in 4 bits; any: operands off 16-byte boundaries.
cudaError_t launch_few_f16(const FewLaunch &l, const FewParams &p, cudaStream_t s);
cudaError_t launch_few_bf16(const FewLaunch &l, const FewParams &p, cudaStream_t s);

cudaError_t launch_pack4(bool bf16, int64_t experts, int64_t K, int64_t N, int group, const uint16_t *W, uint32_t *Q,
                         uint16_t *S, cudaStream_t s);
cudaError_t launch_unpack4(bool bf16, int64_t experts, int64_t K, int64_t N, int group, const uint32_t *Q,
                           const uint16_t *S, uint16_t *W, cudaStream_t s);

}  // namespace gp
