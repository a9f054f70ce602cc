// few.h -- launchers of the kernels for a few rows (few_kernel.cuh) and of the
// weights' way into 4 bits and back (pack4.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gp {

constexpr int kFewRows = 64;       // rows or tokens of a call, at most
constexpr int kFewCols = 64;       // output columns of a block
constexpr int kFewWarps = 8;       // warps of a block
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
};

struct FewLaunch {
    bool bf16, four, any, down;
    int row_blocks;         // 8-row blocks of an item: 1 or 4
    int split;              // blocks of a cluster, sharing the products
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
