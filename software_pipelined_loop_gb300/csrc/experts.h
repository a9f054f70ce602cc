// experts.h -- host-side launchers of the expert-layer kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "grouped_params.h"

namespace gp {

// ---- grouped products (grouped.cu)

struct GroupedVariant {
    int mode;      // GroupedMode
    int bn;        // output rows per tile
    int tile_f;    // features per tile
    int pair;      // 1: CTA pairs, 256 features per tile; 0: single CTAs, 128 or 64
    int cta_bn;    // columns of the row operand per CTA
    int bk;        // products per stage
    int b_part;    // rows of a short copy of the row operand
    int smem_bytes;
    cudaError_t (*launch)(const GroupedMaps &, const GroupedParams &, int grid, cudaStream_t);
    int (*max_units)();  // co-resident CTAs (or CTA pairs) on the current device
};

const GroupedVariant *grouped_variant(int mode, int bn, int tile_f);

// ---- routing and rows (experts_rows.cu)

// Bytes of device scratch launch_route needs (0: none), and its launches.
int64_t route_scratch_bytes(int64_t slots, int experts);
int route_kernels(int64_t slots);
cudaError_t launch_route(int64_t slots, int experts, const int32_t *ids, int32_t *offsets, int32_t *slot_of_row,
                         int32_t *rows, int32_t *scratch, cudaStream_t s);
cudaError_t launch_dispatch(bool bf16, int64_t tokens, int top_k, int64_t width, const uint16_t *X, int64_t ldx,
                            const int32_t *rows, const float *weights, uint16_t *Xs, int64_t ldxs, cudaStream_t s);
cudaError_t launch_combine(bool bf16, int64_t tokens, int top_k, int64_t width, const uint16_t *Ys, int64_t ldys,
                           const int32_t *rows, const float *weights, uint16_t *Y, int64_t ldy, cudaStream_t s);
cudaError_t launch_combine_grad(bool bf16, int64_t tokens, int top_k, int64_t width, const uint16_t *dY, int64_t lddy,
                                const uint16_t *Ys, int64_t ldys, const int32_t *rows, const float *weights,
                                uint16_t *dYs, int64_t lddys, float *dweights, cudaStream_t s);

// ---- 8-bit copies (keep8.cu)

// rows * ceil((width + 7) / 8192) must fit the grid (2^31 - 1 blocks).
cudaError_t launch_keep8(bool bf16, int64_t rows, int64_t width, const uint16_t *X, int64_t ldx, int8_t *Q,
                         uint8_t *S, cudaStream_t s);
cudaError_t launch_restore8(bool bf16, int64_t rows, int64_t width, const int8_t *Q, const uint8_t *S, uint16_t *X,
                            int64_t ldx, cudaStream_t s);
// Copy of a pitched 16-bit matrix to pitch ldd >= width (columns past width:
// zeros); with `offsets`, only rows of experts (per_expert each) that have
// rows of their own to multiply.
cudaError_t launch_repitch(const uint16_t *src, int64_t rows, int64_t width, int64_t lds, uint16_t *dst, int64_t ldd,
                           const int32_t *offsets, int64_t per_expert, cudaStream_t s);

}  // namespace gp
