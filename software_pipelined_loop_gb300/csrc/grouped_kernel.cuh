// grouped_kernel.cuh -- the pipelined tiled product with one weight matrix
// per group of rows ("expert"), for sm_103a.
//
//   rows times matrix      Y[r]  = X[r] . W[e]            (kRows)
//   gradient to the rows   dX[r] = dY[r] . W[e]^T         (kRowsT)
//   gradient to a matrix   dW[e] = sum over r of X[r]^T . dY[r]   (kWeights)
//
// for r in [offsets[e], offsets[e + 1]), the bounds read on the device.
//
// Every product is computed transposed: the 128 (or, over a CTA pair, 256)
// lanes of tensor memory are consecutive elements of the output's rows, and
// the accumulator's columns are output rows.  The ragged dimension -- an
// expert's rows -- is then the MMA's N, which may be any multiple of 16: a
// tile of 32 rows costs a quarter of a 128-row one, so a few rows per expert
// (token generation) stream the weights at the memory's rate.  A tile's last
// rows may belong to the next expert; they only make columns that are not
// stored.
//
// The ring, barriers and bounded waits are those of gemm_kernel.cuh.  Warps: a
// producer for each operand, filling stages of 64 products (128 in the tiles
// of 32 and 64 rows) by TMA, one that issues the MMAs, two epilogue
// warpgroups on double-buffered accumulators, and for the weight gradient one
// more producer, below.
//
// Weight gradient: the summed dimension is the expert's rows, and the 16 rows
// of an MMA step must all be its own (the next expert's, or unused ones, may
// be NaN).  The ring holds the expert's whole 16-row steps; its last 1 to 15
// rows go to a 16-row buffer of their own, in pieces of 4 rows and 1 row, the
// rows past the last one from outside the tensor, which reads as zeros.  A
// warp of its own loads that buffer as soon as the previous tile has left it,
// a whole tile ahead: these rows in the ring, whether cleared there by a warp
// or loaded in pieces, held the MMAs up for 0.9 us a tile (8192 tokens x 4 on
// 32 experts, 4096 x 1536: 309 us against 275).
#pragma once

#include "gemm_kernel.cuh"
#include "grouped_params.h"

#include <cuda_bf16.h>

namespace gp {

template <int MODE_, int BN_, bool PAIR_, int BK_ = 64, int BM_ = 128>
struct GroupedCfg {
    static constexpr int MODE = MODE_;
    static constexpr int BN = BN_;        // output rows per tile
    static constexpr bool PAIR = PAIR_;   // cluster of two CTAs, 256 features per tile
    static constexpr int CLUSTER = PAIR ? 2 : 1;
    static constexpr int BM = BM_;        // features per CTA: 128, or 64 (then in lanes 0-15 of each TMEM quarter)
    static constexpr int QF = BM / 4;     // features of an epilogue warp's TMEM quarter
    static constexpr int TILE_F = BM * CLUSTER;
    static constexpr int BK = BK_;        // products per stage
    static constexpr int SUBS = BK / 64;  // 64-product sub-tiles of an operand with products contiguous
    static constexpr bool A_MN = MODE != kRowsT;    // W[k][n] and dY[r][n]: features contiguous
    static constexpr bool B_MN = MODE == kWeights;  // X[r][k] of the weight gradient
    static constexpr int N_UNIT = 16 * CLUSTER;     // the MMA's columns are a multiple of this
    static constexpr int CTA_BN = BN / CLUSTER;     // columns of B each CTA holds
    static constexpr int A_BYTES = BM * BK * 2;
    static constexpr int B_BYTES = CTA_BN * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int ATOM_BYTES = BK * 128;     // 64 features (columns) x BK products
    static constexpr int A_SUB_BYTES = BM * 128, B_SUB_BYTES = CTA_BN * 128;
    static constexpr int RING_BYTES = 196608;
    static constexpr int STAGES = RING_BYTES / STAGE_BYTES < 16 ? RING_BYTES / STAGE_BYTES : 16;
    static constexpr int TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int EPI_WARP0 = 4, EPI_WARPS = 8;
    static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
    static constexpr int EPI_COLS = BN / 2;         // columns per epilogue warp
    static constexpr int EPI_BLOCK = EPI_COLS < 32 ? EPI_COLS : 32;

    static constexpr int B_PART_ROWS = BN <= 32 ? 16 : 32;  // rows of one short copy of the row operand
    static constexpr int B_PART_BYTES = B_PART_ROWS * 128;

    static constexpr int LAST_ROWS = 16;            // weight gradient: rows of an expert's last MMA step
    static constexpr int LAST_ATOM_BYTES = LAST_ROWS * 128;
    static constexpr int LAST_BYTES = MODE == kWeights ? STAGE_BYTES / BK * LAST_ROWS : 0;
    static constexpr int LAST_OFF = STAGES * STAGE_BYTES;

    static constexpr int STAGING_OFF = LAST_OFF + LAST_BYTES;
    static constexpr int STAGING_BYTES = EPI_WARPS * EPI_BLOCK * QF * 2;
    static constexpr int TABLE_OFF = STAGING_OFF + STAGING_BYTES;
    static constexpr int TABLE_BYTES = 2 * 4 * (kMaxExperts + 2) + (MODE == kWeights ? kMaxSorted : 0);
    static constexpr int CTL_OFF = TABLE_OFF + TABLE_BYTES;
    static constexpr int CTL_BYTES = 8 * (2 * STAGES + 7) + 16;
    static constexpr int SMEM_BYTES = 1024 + CTL_OFF + CTL_BYTES;

    static_assert(BN % 32 == 0 && BN >= 32 && BN <= 256, "MMA columns");
    static_assert(BM == 128 || (BM == 64 && MODE == kRows && !PAIR && BN == 32), "64 features: few rows, forward");
    static_assert(!PAIR || BN == 256, "pairs take 256 x 256 tiles");
    static_assert(B_BYTES % 1024 == 0 && TABLE_BYTES % 8 == 0, "alignment");
    static_assert(!B_MN || (CTA_BN % 64 == 0 && BK == 64), "64-column atoms, 64 rows a stage");
    static_assert(SMEM_BYTES <= 232448, "over the per-CTA shared-memory limit");
};

template <int STAGES>
struct GroupedCtl {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t last_full;   // weight gradient: the buffer of an expert's last rows
    uint64_t last_empty;
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

// Row bounds and tile numbers of the experts, made by every CTA at its
// start: start[e] (e <= E) and first[i], the tiles before the i-th expert in
// the order of work (their own order; weight gradient: order[i]).
struct GroupTable {
    int32_t *start;
    int32_t *first;
    uint8_t *order;  // null: their own order
    int E;
};

// Weight gradient: an expert's rows are summed in one part, or, where the
// matrices have too few tiles for the machine (split_rows > 0) and the expert
// has more than 1.5 split_rows rows, in parts of at most split_rows rows each
// (a multiple of 64, but for the last one's).
__device__ __forceinline__ int32_t rows_of_part(int32_t rows, int32_t split_rows)
{
    if (split_rows == 0 || rows - split_rows <= split_rows / 2) return rows;
    const int32_t parts = (rows - 1) / split_rows + 1;
    return ((rows - 1) / parts + 64) / 64 * 64;
}

__device__ __forceinline__ int32_t parts_of(int32_t rows, int32_t split_rows)
{
    const int32_t part = rows_of_part(rows, split_rows);
    return part == rows ? 1 : (rows - 1) / part + 1;
}

// Slot of an expert's first part of the first tile, in units of one matrix's
// tiles.  An expert of x = rows / split_rows > 1 has at most ceil(x) <=
// floor(2 x) parts, so experts do not meet.
__device__ __forceinline__ int32_t first_slot(int32_t start, int32_t split_rows)
{
    return static_cast<int32_t>(2 * static_cast<int64_t>(start) / split_rows);
}

// Expert of the i-th place in the order of work.
template <int MODE>
__device__ __forceinline__ int expert_at(const GroupTable &t, int i)
{
    return MODE == kWeights && t.order ? t.order[i] : i;
}

// All threads of the CTA.  The bounds are clamped to [0, rows] and made
// non-decreasing, so that nothing they hold can send an access outside.
template <class Cfg>
__device__ void make_table(const GroupedParams &p, GroupTable t)
{
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i <= t.E; i += Cfg::THREADS) {
        const int64_t v = p.offsets[i];
        t.start[i] = static_cast<int32_t>(v < 0 ? 0 : (v > p.rows ? p.rows : v));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int32_t top = 0;
        for (int b = 0; b <= t.E; b += 32) {
            const int i = b + lane;
            int32_t v = i <= t.E ? t.start[i] : 0;
            if (v < top) v = top;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t u = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d && u > v) v = u;
            }
            if (i <= t.E) t.start[i] = v;
            top = __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
    if (Cfg::MODE == kWeights && t.order) {
        // Longest sums first (first[] holds their lengths meanwhile).
        for (int i = threadIdx.x; i < t.E; i += Cfg::THREADS)
            t.first[i] = rows_of_part(t.start[i + 1] - t.start[i], p.split_rows);
        __syncthreads();
        for (int i = threadIdx.x; i < t.E; i += Cfg::THREADS) {
            const int32_t mine = t.first[i];
            int place = 0;
#pragma unroll 8
            for (int k = 0; k < t.E; ++k) {
                const int32_t other = t.first[k];
                place += other > mine || (other == mine && k < i);
            }
            t.order[place] = static_cast<uint8_t>(i);
        }
        __syncthreads();
    }
    if (threadIdx.x < 32) {
        const int32_t f_tiles = static_cast<int32_t>((p.features + Cfg::TILE_F - 1) / Cfg::TILE_F);
        const int32_t w_tiles = static_cast<int32_t>((p.out_rows + Cfg::BN - 1) / Cfg::BN);
        int32_t sum = 0;
        for (int b = 0; b < t.E; b += 32) {
            int32_t n = 0;
            if (b + lane < t.E) {
                const int e = expert_at<Cfg::MODE>(t, b + lane);
                const int32_t rows = t.start[e + 1] - t.start[e];
                n = f_tiles * (Cfg::MODE == kWeights ? w_tiles * parts_of(rows, p.split_rows)
                                                     : (rows + Cfg::BN - 1) / Cfg::BN);
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t u = __shfl_up_sync(0xffffffffu, n, d);
                if (lane >= d) n += u;
            }
            if (b + lane < t.E) t.first[b + lane + 1] = sum + n;
            sum += __shfl_sync(0xffffffffu, n, 31);
        }
        if (lane == 0) t.first[0] = 0;
    }
    __syncthreads();
}

struct GroupedTile {
    int e;           // expert
    int32_t row0;    // its first row (weight gradient: of the part)
    int32_t count;   // its rows (of the part)
    int32_t f0;      // first feature of the tile
    int32_t c0;      // first output row of the tile, within the expert
    int32_t cols;    // the MMA's columns: the tile's output rows, rounded up
    int32_t kbs;     // k-blocks in the ring
    int32_t last;    // products in the last of them (1 .. 64)
    int32_t extra;   // weight gradient: rows past the last whole 16 (0 .. 15)
    int32_t parts;   // weight gradient: parts of the expert's rows (1: the sums go to the output)
    int32_t slot;    // ... where this part's sums go
    int32_t slot0;   // ... and the first part's; `tiles` apart
    int32_t tiles;
};

// Tiles of a unit (CTA or pair).  Rows: round-robin, experts in order,
// features fastest, so that tiles in flight share rows and a few experts'
// weights.  Weight gradient: the tiles differ as the experts' rows do, so they
// are dealt out longest first, in turns of alternating direction.
template <class Cfg>
struct GroupedIter {
    GroupTable t;
    int32_t pos, unit, units, turn;
    int at;  // place of the latest tile's expert in the order of work
    int32_t f_tiles;

    __device__ __forceinline__ GroupedIter(const GroupedParams &p, GroupTable tab)
        : t(tab), pos(blockIdx.x / Cfg::CLUSTER), unit(pos), units(gridDim.x / Cfg::CLUSTER), turn(0), at(0),
          f_tiles(static_cast<int32_t>((p.features + Cfg::TILE_F - 1) / Cfg::TILE_F))
    {
    }

    __device__ __forceinline__ bool next(const GroupedParams &p, GroupedTile &w)
    {
        if (pos >= t.first[t.E]) return false;
        if (pos >= t.first[at + 1]) {
            // The expert of this tile: the last place with first[i] <= pos.
            // (A step at a time costs 1 us of a 64-expert call of one token.)
            int below = at + 1, above = t.E;
            while (above - below > 1) {
                const int mid = (below + above) >> 1;
                if (t.first[mid] <= pos)
                    below = mid;
                else
                    above = mid;
            }
            at = below;
        }
        int32_t in = pos - t.first[at];
        if constexpr (Cfg::MODE == kWeights) {
            ++turn;
            pos = turn * units + ((turn & 1) ? units - 1 - unit : unit);
        } else {
            pos += units;
        }
        w.e = expert_at<Cfg::MODE>(t, at);
        w.row0 = t.start[w.e];
        w.count = t.start[w.e + 1] - w.row0;
        w.parts = 1;
        if constexpr (Cfg::MODE == kWeights) {
            const int32_t rows = rows_of_part(w.count, p.split_rows);
            if (rows < w.count) {
                w.parts = (w.count - 1) / rows + 1;
                w.tiles = f_tiles * static_cast<int32_t>((p.out_rows + Cfg::BN - 1) / Cfg::BN);
                const int32_t part = in / w.tiles;
                in -= part * w.tiles;
                w.slot0 = first_slot(w.row0, p.split_rows) * w.tiles + in;
                w.slot = w.slot0 + part * w.tiles;
                w.row0 += part * rows;
                w.count = w.count - part * rows < rows ? w.count - part * rows : rows;
            }
        }
        const int32_t c = in / f_tiles;
        w.f0 = (in - c * f_tiles) * Cfg::TILE_F;
        if constexpr (Cfg::MODE == kWeights) {
            w.c0 = c * Cfg::BN;
            w.cols = Cfg::BN;
        } else {
            // Whole tiles, and a last one of as many columns as it needs.
            w.c0 = c * Cfg::BN;
            const int32_t left = w.count - w.c0;
            w.cols = left < Cfg::BN ? (left + Cfg::N_UNIT - 1) / Cfg::N_UNIT * Cfg::N_UNIT : Cfg::BN;
        }
        w.extra = Cfg::MODE == kWeights ? w.count & (Cfg::LAST_ROWS - 1) : 0;
        const int64_t depth = Cfg::MODE == kWeights ? w.count - w.extra : p.depth;
        w.kbs = static_cast<int32_t>((depth + Cfg::BK - 1) / Cfg::BK);
        w.last = static_cast<int32_t>(depth - static_cast<int64_t>(w.kbs - 1) * Cfg::BK);
        return true;
    }
};

// --------------------------------------------------------------- producer

template <class Cfg>
struct TileLoader {
    uint32_t bar;  // shared::cluster address for pairs

    __device__ __forceinline__ void load4(uint32_t dst, const CUtensorMap *m, int32_t x, int32_t y, int32_t z,
                                          int32_t v) const
    {
        if constexpr (Cfg::PAIR)
            tma_load_4d_pair(dst, m, bar, x, y, z, v);
        else
            tma_load_4d(dst, m, bar, x, y, z, v);
    }
    __device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap *m, int32_t x, int32_t y, int32_t z) const
    {
        if constexpr (Cfg::PAIR)
            tma_load_3d_pair(dst, m, bar, x, y, z);
        else
            tma_load_3d(dst, m, bar, x, y, z);
    }
    __device__ __forceinline__ void load2(uint32_t dst, const CUtensorMap *m, int32_t x, int32_t y) const
    {
        if constexpr (Cfg::PAIR)
            tma_load_2d_pair(dst, m, bar, x, y);
        else
            tma_load_2d(dst, m, bar, x, y);
    }

    // `rows` (1 .. 15) rows of 64 elements from (x, y) and zeros up to 16
    // rows: maps of 4- and 1-row boxes, `outside` the first row past the
    // tensor.  (The swizzle goes by the address, so pieces of any number of
    // rows land where one box would put them.)
    __device__ __forceinline__ void load_last_rows(uint32_t dst, const CUtensorMap *m4, const CUtensorMap *m1,
                                                   int32_t x, int32_t y, int32_t rows, int32_t outside) const
    {
        for (int32_t r = 0; r < Cfg::LAST_ROWS; r += 4) {
            if (r + 4 <= rows || r >= rows) {
                load2(dst + r * 128, m4, x, r < rows ? y + r : outside);
            } else {
                for (int32_t i = r; i < r + 4; ++i) load2(dst + i * 128, m1, x, i < rows ? y + i : outside);
            }
        }
    }
};

// Two warps run this loop, one for each operand, the whole warp with one
// elected lane issuing.  A stage costs a warp a few hundred cycles of issue
// whatever it holds (a passed wait 120, a barrier armed and two copies 260 --
// one warp for both operands kept a 64-feature tile and a 128-feature one to
// the same 470 cycles per 64 products), so the operands have a warp each and
// the next stage's barrier is looked at while this one's copies are issued.
template <class Cfg, bool A_SIDE>
__device__ void grouped_producer(const GroupedParams &p, const GroupedMaps &maps, uint32_t sbase,
                                 GroupedCtl<Cfg::STAGES> *ctl, GroupTable tab, const Waiter &w, uint32_t rank)
{
    const CUtensorMap *map = &maps.m[A_SIDE ? kMapA : kMapB];
    int stage = 0;
    uint32_t phase = 0;
    uint32_t armed = 0, armed_par = 0;
    int64_t kb_count = 0;
    bool ok = true, ready = false;
    const uint32_t full0 = smem_u32(&ctl->full[0]), empty0 = smem_u32(&ctl->empty[0]);
    const uint32_t full0_leader = Cfg::PAIR ? mapa_shared(full0, 0) : full0;
    GroupedIter<Cfg> it(p, tab);
    GroupedTile t;
    while (ok && it.next(p, t)) {
        const int32_t f0 = t.f0 + static_cast<int32_t>(rank) * Cfg::BM;
        const int32_t c0 = t.c0 + static_cast<int32_t>(rank) * (t.cols / Cfg::CLUSTER);
        // Copies of the row operand: one of all CTA_BN rows, or as many short
        // ones as hold the tile's columns when that is fewer rows.
        const int32_t parts = (t.cols / Cfg::CLUSTER + Cfg::B_PART_ROWS - 1) / Cfg::B_PART_ROWS;
        const bool whole = Cfg::MODE == kWeights || parts * Cfg::B_PART_ROWS >= Cfg::CTA_BN;
        const uint32_t bytes = Cfg::A_BYTES + (whole ? Cfg::B_BYTES : Cfg::SUBS * parts * Cfg::B_PART_BYTES);
        for (int32_t kb = 0; kb < t.kbs; ++kb, ++kb_count) {
            if (!ready && !__all_sync(0xffffffffu, w.wait(empty0 + 8u * stage, phase ^ 1u))) {
                ok = false;
                break;
            }
            const uint32_t so = 8u * static_cast<uint32_t>(stage);
            const uint32_t sa = sbase + stage * Cfg::STAGE_BYTES, sb = sa + Cfg::A_BYTES;
            const uint32_t bit = 1u << stage, this_phase = phase;
            if (++stage == Cfg::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            const bool free = mbar_test_wait(empty0 + 8u * stage, phase ^ 1u);
            if (blockIdx.x == 0 && kb_count == p.stall_kb) {
                ready = false;
                continue;
            }
            const int32_t k0 = kb * Cfg::BK;
            const TileLoader<Cfg> ld{full0_leader + so};
            if (elect_one_sync()) {
                if constexpr (A_SIDE) {
                    if (rank == 0) mbar_arrive_expect_tx(full0 + so, Cfg::CLUSTER * bytes);
                    if constexpr (Cfg::MODE == kRows) {
                        // W[e]: BK products x BM features, atoms of 64 features.
                        if (p.a_groups) {
                            ld.load4(sa, map, 0, k0, f0 / 64, t.e);
                        } else {
#pragma unroll
                            for (int j = 0; j < Cfg::BM / 64; ++j)
                                ld.load3(sa + j * Cfg::ATOM_BYTES, map, f0 + 64 * j, k0, t.e);
                        }
                    } else if constexpr (Cfg::MODE == kRowsT) {
#pragma unroll
                        for (int u = 0; u < Cfg::SUBS; ++u)
                            ld.load3(sa + u * Cfg::A_SUB_BYTES, map, k0 + 64 * u, f0, t.e);
                    } else if (p.a_groups) {
                        ld.load3(sa, map, 0, t.row0 + k0, f0 / 64);
                    } else {
                        ld.load2(sa, map, f0, t.row0 + k0);
                        ld.load2(sa + Cfg::ATOM_BYTES, map, f0 + 64, t.row0 + k0);
                    }
                } else if constexpr (Cfg::MODE == kWeights) {
                    if (p.b_groups) {
                        ld.load3(sb, map, 0, t.row0 + k0, c0 / 64);
                    } else {
#pragma unroll
                        for (int j = 0; j < Cfg::CTA_BN / 64; ++j)
                            ld.load2(sb + j * Cfg::ATOM_BYTES, map, c0 + 64 * j, t.row0 + k0);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < Cfg::SUBS; ++u) {
                        if (whole) {
                            ld.load2(sb + u * Cfg::B_SUB_BYTES, map, k0 + 64 * u, t.row0 + c0);
                        } else {
                            for (int32_t j = 0; j < parts; ++j)
                                ld.load2(sb + u * Cfg::B_SUB_BYTES + j * Cfg::B_PART_BYTES, &maps.m[kMapBPart],
                                         k0 + 64 * u, t.row0 + c0 + j * Cfg::B_PART_ROWS);
                        }
                    }
                }
            }
            ready = __all_sync(0xffffffffu, free);
            armed |= bit;
            armed_par = this_phase ? (armed_par | bit) : (armed_par & ~bit);
        }
    }
    if (ok && Cfg::PAIR && A_SIDE) {
        // The last MMA commits arrive on both CTAs' empty barriers: none may
        // be in flight when a CTA leaves.
        for (int s = 0; s < Cfg::STAGES && ok; ++s) {
            const uint32_t ph = s < stage ? phase ^ 1u : phase;
            ok = __all_sync(0xffffffffu, w.wait(empty0 + 8u * s, ph ^ 1u));
        }
    }
    if (!ok && armed) {
        // Let the copies that were started land before the CTA leaves: the
        // leader's first warp sees them on its barriers, the others give
        // them a bounded time.
        if (A_SIDE && rank == 0) {
            for (int s = 0; s < Cfg::STAGES; ++s)
                if (armed & (1u << s)) w.wait_drain(full0 + 8u * s, (armed_par >> s) & 1u, kDrainNs);
        } else {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 2000000ull) {
            }
        }
    }
}

// Weight gradient: one warp loads every tile's last rows (fewer than 16) into
// their buffer, a lane per 64-element atom: two of A, then B's.
template <class Cfg>
__device__ void last_rows_producer(const GroupedParams &p, const GroupedMaps &maps, uint32_t sbase,
                                   GroupedCtl<Cfg::STAGES> *ctl, GroupTable tab, const Waiter &w, uint32_t rank,
                                   int lane)
{
    constexpr int ATOMS = Cfg::LAST_BYTES / Cfg::LAST_ATOM_BYTES;
    const uint32_t full = smem_u32(&ctl->last_full);
    const TileLoader<Cfg> ld{Cfg::PAIR ? mapa_shared(full, 0) : full};
    uint32_t phase = 0;
    int64_t kb_count = 0;
    bool used = false, ok = true;
    GroupedIter<Cfg> it(p, tab);
    GroupedTile t;
    while (it.next(p, t)) {
        // (Test hook: a tile without ring k-blocks stalls here.)
        const bool stalled = blockIdx.x == 0 && t.kbs == 0 && kb_count == p.stall_kb;
        kb_count += t.kbs;
        if (t.extra == 0) continue;
        ok = __all_sync(0xffffffffu, w.wait(smem_u32(&ctl->last_empty), phase ^ 1u));
        if (!ok) break;
        if (stalled) {
            phase ^= 1u;
            continue;
        }
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(full, Cfg::CLUSTER * Cfg::LAST_BYTES);
        __syncwarp();
        if (lane < ATOMS) {
            const bool a = lane < 2;
            const int32_t x = a ? t.f0 + static_cast<int32_t>(rank) * Cfg::BM + 64 * lane
                                : t.c0 + static_cast<int32_t>(rank) * Cfg::CTA_BN + 64 * (lane - 2);
            const CUtensorMap *m = &maps.m[a ? kMapALast : kMapBLast];
            ld.load_last_rows(sbase + Cfg::LAST_OFF + lane * Cfg::LAST_ATOM_BYTES, m, m + 1, x,
                              t.row0 + t.count - t.extra, t.extra, static_cast<int32_t>(p.rows));
        }
        __syncwarp();
        used = true;
        phase ^= 1u;
    }
    if (used) {
        // The commit that frees the buffer has arrived, or (giving up) the
        // copies get a bounded time to land.
        if (ok) ok = __all_sync(0xffffffffu, w.wait(smem_u32(&ctl->last_empty), phase ^ 1u));
        if (!ok) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 2000000ull) {
            }
        }
    }
}

// -------------------------------------------------------------------- MMA

// A shared-memory descriptor `units` of 16 bytes on (the address field never
// carries out of the low word).
__device__ __forceinline__ uint64_t desc_plus(uint64_t desc, uint32_t units)
{
    return (desc & 0xffffffff00000000ull) | (static_cast<uint32_t>(desc) + units);
}

template <class Cfg>
__device__ void grouped_mma(const GroupedParams &p, uint32_t sbase, uint32_t tmem_base,
                            GroupedCtl<Cfg::STAGES> *ctl, GroupTable tab, const Waiter &w)
{
    const uint32_t idesc0 = umma_idesc_16bit_f32(Cfg::TILE_F, 0, p.bf16 != 0, Cfg::A_MN, Cfg::B_MN);
    const uint64_t dA0 = Cfg::A_MN ? umma_desc_sw128(sbase, Cfg::ATOM_BYTES, 1024) : umma_desc_sw128(sbase, 16, 1024);
    const uint64_t dB0 = Cfg::B_MN ? umma_desc_sw128(sbase + Cfg::A_BYTES, Cfg::ATOM_BYTES, 1024)
                                   : umma_desc_sw128(sbase + Cfg::A_BYTES, 16, 1024);
    auto mma = [](uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t add) {
        if constexpr (Cfg::PAIR)
            umma_f16_pair(d, da, db, idesc, add);
        else
            umma_f16(d, da, db, idesc, add);
    };
    auto commit = [](uint64_t *bar) {
        if constexpr (Cfg::PAIR)
            umma_commit_pair(smem_u32(bar), 3);
        else
            umma_commit(smem_u32(bar));
    };
    int stage = 0;
    uint32_t phase = 0, last_phase = 0;
    uint32_t acc = 0, acc_phase = 0;
    bool issued = false, ok = true, ready = false;
    const uint32_t full0 = smem_u32(&ctl->full[0]);
    GroupedIter<Cfg> it(p, tab);
    GroupedTile t;
    while (ok && it.next(p, t)) {
        if (t.kbs == 0 && t.extra == 0) continue;  // the empty sum: the epilogue writes zeros
        if (!__all_sync(0xffffffffu, w.wait(smem_u32(&ctl->tempty[acc]), acc_phase ^ 1u))) {
            ok = false;
            break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem_base + acc * Cfg::BN;
        const uint32_t idesc = idesc0 | (static_cast<uint32_t>(t.cols >> 3) << 17);
        for (int32_t kb = 0; kb < t.kbs; ++kb) {
            if (!ready && !__all_sync(0xffffffffu, w.wait(full0 + 8u * stage, phase))) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const int at = stage;
            if (++stage == Cfg::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            // The next stage's barrier, looked at while this one's MMAs are issued.
            const bool there = mbar_test_wait(full0 + 8u * stage, phase);
            const uint32_t so = static_cast<uint32_t>(at * Cfg::STAGE_BYTES) >> 4;
            const int steps = kb == t.kbs - 1 ? (t.last + 15) / 16 : Cfg::BK / 16;
            if (elect_one_sync()) {
#pragma unroll
                for (int kk = 0; kk < Cfg::BK / 16; ++kk) {
                    // 16 products on: rows of an atom, or 32 bytes within a 64-product sub-tile.
                    const uint32_t ak = (Cfg::A_MN ? kk * 2048 : (kk / 4) * Cfg::A_SUB_BYTES + (kk % 4) * 32) >> 4;
                    const uint32_t bk = (Cfg::B_MN ? kk * 2048 : (kk / 4) * Cfg::B_SUB_BYTES + (kk % 4) * 32) >> 4;
                    if (kk < steps)
                        mma(d, desc_plus(dA0, so + ak), desc_plus(dB0, so + bk), idesc, kb > 0 || kk > 0 ? 1u : 0u);
                }
                commit(&ctl->empty[at]);
            }
            ready = __all_sync(0xffffffffu, there);
            issued = true;
        }
        if constexpr (Cfg::MODE == kWeights) {
            if (ok && t.extra > 0) {
                ok = __all_sync(0xffffffffu, w.wait(smem_u32(&ctl->last_full), last_phase));
                if (ok) {
                    last_phase ^= 1u;
                    tc_fence_after_sync();
                    const uint32_t at = sbase + Cfg::LAST_OFF;
                    if (elect_one_sync()) {
                        mma(d, umma_desc_sw128(at, Cfg::LAST_ATOM_BYTES, 1024),
                            umma_desc_sw128(at + 2 * Cfg::LAST_ATOM_BYTES, Cfg::LAST_ATOM_BYTES, 1024), idesc,
                            t.kbs > 0 ? 1u : 0u);
                        commit(&ctl->last_empty);
                    }
                    __syncwarp();
                    issued = true;
                }
            }
        }
        if (!ok) break;
        if (elect_one_sync()) commit(&ctl->tfull[acc]);
        __syncwarp();
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
    }
    if (ok && Cfg::PAIR) {
        // The accumulators' last releases, the peer's among them, have landed.
        ok = __all_sync(0xffffffffu, w.wait(smem_u32(&ctl->tempty[acc]), acc_phase ^ 1u));
        ok = ok && __all_sync(0xffffffffu,
                              w.wait(smem_u32(&ctl->tempty[acc ^ 1u]), acc == 0 ? acc_phase ^ 1u : acc_phase));
    }
    if (!ok && issued) {
        if (elect_one_sync()) {
            if constexpr (Cfg::PAIR)
                umma_commit_pair(smem_u32(&ctl->drain), 1);
            else
                umma_commit(smem_u32(&ctl->drain));
        }
        __syncwarp();
        w.wait_drain(smem_u32(&ctl->drain), 0, kDrainNs);
    }
}

// --------------------------------------------------------------- epilogue

// Two fp32 sums rounded to 16 bits, `lo` in the low half.  (Volatile, so that
// it stays behind the wait for the tensor memory load it takes its inputs from.)
__device__ __forceinline__ uint32_t round_pair(uint32_t lo, uint32_t hi, bool bf16)
{
    uint32_t r;
    if (bf16)
        asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
    else
        asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
    return r;
}

// Stores a block of n (up to EPI_BLOCK) output rows x QF features whose fp32
// sums a warp holds as tensor memory gives them (lanes 0-15 of its quarter in
// lo, 16-31 in hi): rounded once to the output's type and turned through the
// warp's staging tile (16-byte chunks, XOR-swizzled by row: free of bank
// conflicts both ways), so that a store instruction writes 64 contiguous
// bytes of 8 rows.  `o` is the block's first element, `left` the features
// from there to the end of a row.
template <class Cfg>
__device__ __forceinline__ void store_block(const GroupedParams &p, uint32_t stg, int lane,
                                            const uint32_t (&lo)[Cfg::EPI_BLOCK / 2],
                                            const uint32_t (&hi)[Cfg::EPI_BLOCK / 2], uint16_t *o, int n, int64_t left)
{
    constexpr int NB = Cfg::EPI_BLOCK, QF = Cfg::QF;
    constexpr int ROW = QF * 2, CHUNKS = QF / 8;  // bytes and 16-byte chunks of a staged row
    const bool bf16 = p.bf16 != 0;
    // Address of chunk k of staged row c.
    auto staged = [stg](int c, int k) {
        return stg + c * ROW + ((k ^ (CHUNKS == 4 ? (c >> 1) & 3 : (c >> 2) & 1)) << 4);
    };
    if constexpr (QF == 32) {
        // Per 8 columns: lane / 8 = 8 features, lane % 8 = column.
#pragma unroll
        for (int i = 0; i < NB / 8; ++i)
            stmatrix_x4_trans(staged(8 * i + (lane & 7), lane >> 3), round_pair(lo[4 * i], lo[4 * i + 1], bf16),
                              round_pair(lo[4 * i + 2], lo[4 * i + 3], bf16),
                              round_pair(hi[4 * i], hi[4 * i + 1], bf16),
                              round_pair(hi[4 * i + 2], hi[4 * i + 3], bf16));
    } else {
        // Sixteen columns: the first 8 columns' two pieces of 8 features, then the others'.
        static_assert(QF == 32 || NB == 16, "one store");
        stmatrix_x4_trans(staged((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1), round_pair(lo[0], lo[1], bf16),
                          round_pair(lo[2], lo[3], bf16), round_pair(lo[4], lo[5], bf16),
                          round_pair(lo[6], lo[7], bf16));
    }
    __syncwarp();
    if (p.vec_store && QF <= left) {
        // 16-byte pieces, CHUNKS lanes to a row.
        constexpr int ROWS = 32 / CHUNKS;
        o += (lane / CHUNKS) * p.ldo + (lane % CHUNKS) * 8;
#pragma unroll
        for (int i = 0; i < NB; i += ROWS)
            if (i + lane / CHUNKS < n)
                *reinterpret_cast<uint4 *>(o + i * p.ldo) = ld_shared_v4(staged(i + lane / CHUNKS, lane % CHUNKS));
    } else if (lane < QF && lane < left) {
        // A feature per lane, row by row.  (Two rows at a time in the row's
        // own 4-byte words: 179 us where this takes 112.)
#pragma unroll 8
        for (int c = 0; c < n; ++c) o[c * p.ldo + lane] = ld_shared_u16(staged(c, lane >> 3) + (lane & 7) * 2);
    }
    __syncwarp();
}

// Where a warp's block j of a slot's sums begins: 32 lanes of one register
// after another, in the order of lo and hi.
template <class Cfg>
__device__ __forceinline__ float *part_of(const GroupedParams &p, int32_t slot, uint32_t rank, int e, int block)
{
    constexpr int BLOCKS = Cfg::EPI_COLS / Cfg::EPI_BLOCK;
    const int64_t at = ((static_cast<int64_t>(slot) * Cfg::CLUSTER + rank) * Cfg::EPI_WARPS + e) * BLOCKS + block;
    return p.parts + at * (Cfg::EPI_BLOCK * 32);
}

// Counts a finished part; true for the last of `parts`, which leaves the
// counter at zero for the next launch.  A count is of one launch only (its
// number is beside it), so that a launch that gave up leaves nothing behind.
// The number is in device memory and not an argument: a recorded launch has
// the same arguments each time.
__device__ __forceinline__ bool last_part(unsigned long long *count, uint32_t launch, int parts)
{
    unsigned long long seen = *reinterpret_cast<volatile unsigned long long *>(count), want;
    for (;;) {  // at most as often as there are other parts
        const uint32_t n = (seen >> 32) == launch ? static_cast<uint32_t>(seen) + 1 : 1u;
        const bool last = n == static_cast<uint32_t>(parts);
        want = last ? 0ull : (static_cast<unsigned long long>(launch) << 32) | n;
        const unsigned long long was = atomicCAS(count, seen, want);
        if (was == seen) return last;
        seen = was;
    }
}

// The launch's number; each of its `readers` asks once, and the last one moves
// the number on for the next launch.  (Read by every epilogue warp at its
// start, while the ring fills.  Moved on at the CTAs' ends instead, behind
// their stores, it took 1 to 2 us of a call.)
__device__ __forceinline__ uint32_t launch_number(uint32_t *launch, uint32_t readers)
{
    const uint32_t n = __ldcg(launch);
    __threadfence();
    if (atomicAdd(launch + 1, 1u) == readers - 1) {
        launch[1] = 0;
        launch[0] = n + 1;
    }
    return n;
}

// Accumulator lane l of warp quarter q is feature f0 + 32 q + l, column c the
// output row c0 + c.  (One staging tile per warpgroup, 256 contiguous bytes of
// 2 rows, and bulk tensor copies out of the staging tiles measured the same.)
// An accumulator is handed back with relaxed arrivals: a release at cluster
// scope waits for the warp's stores of the tile before, and held the MMAs up
// for it.  Weight gradient of 8192 rows on 32 experts, 2048 x 1024: 43 us, 60
// with releases, 31 with nothing stored; of 32768 rows on 32 experts,
// 4096 x 1536: 250, 261 and 233 us.
template <class Cfg>
__device__ void grouped_epilogue(const GroupedParams &p, uint32_t sbase, uint32_t tmem_base,
                                 GroupedCtl<Cfg::STAGES> *ctl, GroupTable tab, const Waiter &w, int warp, int lane,
                                 uint32_t rank)
{
    const int e = warp - Cfg::EPI_WARP0;
    const int q = warp & 3, h = e >> 2;
    constexpr int NB = Cfg::EPI_BLOCK, QF = Cfg::QF;
    const uint32_t stg = sbase + Cfg::STAGING_OFF + e * (NB * QF * 2);
    uint32_t acc = 0, acc_phase = 0;
    const uint32_t tempty0 = Cfg::PAIR ? mapa_shared(smem_u32(&ctl->tempty[0]), 0) : smem_u32(&ctl->tempty[0]);
    uint16_t *out = static_cast<uint16_t *>(p.out);
    uint32_t launch = 0;  // (of lane 0)
    if (Cfg::MODE == kWeights && p.split_rows > 0 && lane == 0)
        launch = launch_number(p.launch, gridDim.x * Cfg::EPI_WARPS);
    __syncwarp();
    GroupedIter<Cfg> it(p, tab);
    GroupedTile t;
    while (it.next(p, t)) {
        const int64_t f0 = static_cast<int64_t>(t.f0) + rank * Cfg::BM + q * QF;  // the warp's first feature
        const int64_t all = Cfg::MODE == kWeights ? p.out_rows : t.count;          // output rows of the expert
        const int64_t base = Cfg::MODE == kWeights ? p.out_rows * t.e : t.row0;
        // The tile's rows are its columns up to the expert's last row; this
        // warp takes the first or the second half of them.
        const int32_t half = ((t.cols / 2) + NB - 1) / NB * NB;
        const int64_t end = all - t.c0 < t.cols ? all - t.c0 : t.cols;
        const int32_t from = h ? half : 0;
        const int64_t to = h ? end : (end < half ? end : half);
        const bool empty = t.kbs == 0 && t.extra == 0;
        if (!empty) {
            if (!__all_sync(0xffffffffu, w.wait(smem_u32(&ctl->tfull[acc]), acc_phase))) return;
            tc_fence_after_sync();
        }
        const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * Cfg::BN;
        auto release = [&] {  // this warp has read its part of the accumulator
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (Cfg::PAIR)
                    mbar_arrive_cluster_relaxed(tempty0 + 8 * acc);
                else
                    mbar_arrive(tempty0 + 8 * acc);
            }
        };
        if (!empty && to <= from) release();
#pragma unroll 1
        for (int32_t j = from; j < to; j += NB) {
            uint32_t lo[NB / 2], hi[NB / 2];  // lanes 0-15 and 16-31 of the quarter
            if (empty) {
#pragma unroll
                for (int i = 0; i < NB / 2; ++i) lo[i] = hi[i] = 0;
            } else {
                if constexpr (NB == 32) {
                    tmem_ld_16x256b_x4(tbase + j, lo);
                    tmem_ld_16x256b_x4(tbase + j + (16u << 16), hi);
                } else {
                    tmem_ld_16x256b_x2(tbase + j, lo);
                    if constexpr (QF == 32) tmem_ld_16x256b_x2(tbase + j + (16u << 16), hi);
                }
                tmem_wait_ld();
                if (j + NB >= to) release();
            }
            if (Cfg::MODE == kWeights && t.parts > 1) {
                // A part of a sum: as it is, 128 contiguous bytes a register.
                float *o = part_of<Cfg>(p, t.slot, rank, e, (j - from) / NB) + lane;
#pragma unroll
                for (int i = 0; i < NB / 2; ++i) {
                    o[32 * i] = __uint_as_float(lo[i]);
                    o[32 * (NB / 2 + i)] = __uint_as_float(hi[i]);
                }
                continue;
            }
            const int n = to - j < NB ? static_cast<int>(to - j) : NB;
            store_block<Cfg>(p, stg, lane, lo, hi, out + (base + t.c0 + j) * p.ldo + f0, n, p.features - f0);
        }
        if constexpr (Cfg::MODE == kWeights) {
            if (t.parts > 1 && from < to) {
                // Whichever part of these sums comes last adds them all, in
                // the parts' order, and stores them: no warp waits for another.
                __threadfence();
                __syncwarp();
                bool last = false;
                if (lane == 0)
                    last = last_part(&p.part_counts[(t.slot0 * Cfg::CLUSTER + rank) * Cfg::EPI_WARPS + e], launch,
                                     t.parts);
                if (__any_sync(0xffffffffu, last)) {
                    __threadfence();
#pragma unroll 1
                    for (int32_t j = from; j < to; j += NB) {
                        float sum[NB];
#pragma unroll
                        for (int i = 0; i < NB; ++i) sum[i] = 0.f;
#pragma unroll 1
                        for (int k = 0; k < t.parts; ++k) {
                            const float *v =
                                part_of<Cfg>(p, t.slot0 + k * t.tiles, rank, e, (j - from) / NB) + lane;
#pragma unroll
                            for (int i = 0; i < NB; ++i) sum[i] += __ldcg(v + 32 * i);
                        }
                        uint32_t lo[NB / 2], hi[NB / 2];
#pragma unroll
                        for (int i = 0; i < NB / 2; ++i) {
                            lo[i] = __float_as_uint(sum[i]);
                            hi[i] = __float_as_uint(sum[NB / 2 + i]);
                        }
                        const int n = to - j < NB ? static_cast<int>(to - j) : NB;
                        store_block<Cfg>(p, stg, lane, lo, hi, out + (base + t.c0 + j) * p.ldo + f0, n,
                                         p.features - f0);
                    }
                }
            }
        }
        if (!empty) {
            acc ^= 1u;
            if (acc == 0) acc_phase ^= 1u;
        }
    }
    if constexpr (Cfg::MODE != kWeights) {
        // Rows of no expert are written as zeros.
        const int64_t head = tab.start[0], tail = tab.start[tab.E];
        const int64_t none = head + p.rows - tail;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * Cfg::EPI_WARPS + e; i < none;
             i += static_cast<int64_t>(gridDim.x) * Cfg::EPI_WARPS) {
            uint16_t *o = out + (i < head ? i : tail + (i - head)) * p.ldo;
            for (int64_t x = lane; x < p.features; x += 32) o[x] = 0;
        }
    }
}

// ----------------------------------------------------------------- kernel

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    grouped_kernel(const __grid_constant__ GroupedMaps maps, const GroupedParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    auto *ctl = reinterpret_cast<GroupedCtl<Cfg::STAGES> *>(smem + Cfg::CTL_OFF);
    GroupTable tab;
    tab.start = reinterpret_cast<int32_t *>(smem + Cfg::TABLE_OFF);
    tab.first = tab.start + kMaxExperts + 2;
    tab.order = Cfg::MODE == kWeights && p.sorted ? reinterpret_cast<uint8_t *>(tab.first + kMaxExperts + 2) : nullptr;
    tab.E = p.experts;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::STAGES; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        mbar_init(smem_u32(&ctl->last_full), 1);
        mbar_init(smem_u32(&ctl->last_empty), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctl->tfull[b]), 1);
            mbar_init(smem_u32(&ctl->tempty[b]), Cfg::CLUSTER * Cfg::EPI_WARPS);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.m[kMapA]);
        tma_prefetch_desc(&maps.m[kMapB]);
    }
    if (warp == 1) {
        if constexpr (Cfg::PAIR) {
            tmem_alloc_pair(smem_u32(&ctl->tmem_base), Cfg::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(&ctl->tmem_base), Cfg::TMEM_COLS);
            tmem_relinquish();
        }
    }
    pdl_wait();
    pdl_launch_dependents();
    make_table<Cfg>(p, tab);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (Cfg::PAIR) cluster_sync();  // the leader's barriers exist before the peer signals them
    tc_fence_after_sync();
    const uint32_t tmem_base = ctl->tmem_base;
    const Waiter w{&ctl->abort, p.status, p.timeout_ns};
    const uint32_t rank = Cfg::PAIR ? cluster_ctarank() : 0u;
    if (warp == 0) {
        grouped_producer<Cfg, true>(p, maps, sbase, ctl, tab, w, rank);
    } else if (warp == 3) {
        grouped_producer<Cfg, false>(p, maps, sbase, ctl, tab, w, rank);
    } else if (warp == 1) {
        if (rank == 0) grouped_mma<Cfg>(p, sbase, tmem_base, ctl, tab, w);
    } else if (warp == 2) {
        if constexpr (Cfg::MODE == kWeights) last_rows_producer<Cfg>(p, maps, sbase, ctl, tab, w, rank, lane);
    } else if (warp >= Cfg::EPI_WARP0) {
        grouped_epilogue<Cfg>(p, sbase, tmem_base, ctl, tab, w, warp, lane, rank);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (Cfg::PAIR) cluster_sync();  // no peer still signals or reads this CTA
    if (warp == 1) {
        tc_fence_after_sync();
        if constexpr (Cfg::PAIR)
            tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
        else
            tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace gp
