// grouped_params.h -- kernel arguments of the grouped products, shared by
// host and device code.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace gp {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kMaxSorted = 256;  // experts up to which the weight gradient sorts its work
constexpr int kMaxPartSlots = 512;

enum GroupedMode { kRows = 0, kRowsT = 1, kWeights = 2 };

// Tensor maps of one launch.  Rows: A the weights, B the row operand, BPart
// the same in boxes of fewer rows.  Weight gradient: A and B the two row operands,
// and each in boxes of 4 rows and of 1 row of 64 elements (from ALast, BLast).
enum GroupedMap { kMapA = 0, kMapB = 1, kMapBPart = 2, kMapALast = 2, kMapBLast = 4, kMaps = 6 };
struct GroupedMaps {
    CUtensorMap m[kMaps];
};

// The product of every expert e over its rows [offsets[e], offsets[e + 1]).
// The kernel computes it transposed, D[f][c]: f runs over `features`, the
// contiguous dimension of the output, c over rows of the output.
struct GroupedParams {
    const int32_t *offsets;  // experts + 1 row bounds, in device memory
    int experts;
    int64_t rows;            // rows of the row operands; the bounds are clamped to [0, rows]
    int64_t features;        // length of an output row
    int64_t out_rows;        // weight gradient: output rows per expert; else unused
    int64_t depth;           // products summed per value (weight gradient: the expert's rows instead)
    void *out;
    int64_t ldo;             // output row pitch in elements
    float *parts;            // weight gradient: sums of parts of an expert's rows, a slot per tile
    unsigned long long *part_counts;  // ... finished parts, one count per slot and epilogue warp of both CTAs
    uint32_t *launch;        // ... this launch's number, and how many warps have read it
    int32_t split_rows;      // ... an expert of more than 1.5 times as many is summed in parts (0: none is)
    int sorted;              // ... the longest sums go first (up to kMaxSorted experts)
    int bf16;
    int vec_store;           // output base and pitch allow 16-byte stores
    int a_groups, b_groups;  // 1: the operand's tensor map is in 64-column groups (one copy per k-block)
    uint64_t timeout_ns;
    int64_t stall_kb;        // test hook: CTA 0 leaves this k-block unfilled (-1: none)
    int *status;
};

}  // namespace gp
