// rows4_wide.cu -- some rows times weights in 4 bits (more than 8, in groups of
// 32 more than 16), on the tensor cores' tensor memory.
//
// Y[m][n] = sum over k of X[m][k] * (q[k][n] - 8) * s[k / group][n].  With some
// tens of rows the warp-level matrix instructions of few_kernel.cuh are the
// bound (1024 products a cycle and SM; 64 rows x 16384 x 4096 in groups of 32:
// 38 us there; 64 rows x 4096 x 16384 in groups of 128: 54).  Here a CTA takes
// 128 columns and a range of k:
//   - producer warps fill a ring of stages with TMA copies of the words (rows
//     of 128) and of X's rows (128-byte swizzle);
//   - warpgroups take stages in turn: a thread has one column, turns its words
//     into 16-bit values and stores them to tensor memory -- as operand A of
//     the MMA, whose 128 rows are the columns; so weights pass not back through
//     shared memory;
//   - two MMA warps issue tcgen05.mma (128 x rows x 16) with X from shared
//     memory, every other stage each.
// Scales, by size of group:
//   - 64 and 128: the values are q - 8, exact, and each group of k has an
//     accumulator; one or two more warpgroups read it, a column and 32 rows a
//     thread, and add it to sums in registers, times the scale;
//   - 32: an accumulator handed over costs some 300 cycles, and there would be
//     four for 128 k.  The values are w = (q - 8) * s, which has at most 4 bits
//     more than the type holds: it is split into its rounding and the rest,
//     exactly, and both are multiplied, into one accumulator for all groups.
//     Infinities, and scales so large that w is past the type's largest value,
//     do not survive that: sums that are not finite are made again (wide_again).
// fp32 throughout, one rounding at the end.  The CTAs of a cluster share a
// tile's k; their sums meet in shared memory, in a fixed order.  Every wait is
// bounded (Waiter).
//
// What bounds it: tensor memory.  Storing 16 KB of values costs about 100
// cycles and the MMAs' reading them 128, and a stage passes through four or five
// kinds of warps in 450 cycles at least, whatever its size.  Split values are
// twice the bytes: 64 rows x 4096 x 16384 take 17 us in groups of 128, 19 of 64,
// 21 of 32 (as the others do: 30; the others as this one does: 22).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "few.h"
#include "gemm_kernel.cuh"

namespace gp {
namespace {

template <int MP_, int GROUP_>
struct WideCfg {
    static constexpr int MP = MP_, GROUP = GROUP_;          // rows of X, rounded up: the MMA's columns
    static constexpr bool SPLIT = GROUP == 32;              // values times scales, in two parts
    static constexpr int STAGE_K = wide_stage_k(GROUP), SUBS = STAGE_K / 64;
    static constexpr int EACH = SPLIT ? 0 : STAGE_K / GROUP;  // accumulators of a stage
    static constexpr int X_BYTES = SUBS * MP * 128, WORD_PITCH = 4 * kWideCols, WORD_BYTES = STAGE_K / 8 * WORD_PITCH;
    static constexpr int STAGE_BYTES = X_BYTES + WORD_BYTES;
    static constexpr int STAGES = (MP == 64 ? 6 : 8) * 128 / STAGE_K;
    // Warps: two producers, two that issue MMAs, warpgroups of sums (without SPLIT), warpgroups that unpack.
    static constexpr int PRODUCERS = 2, MMA_WARP0 = 2, MMA_WARPS = 2, END_WARP0 = 4;
    static constexpr int SUMS = 32, END_WARPS = 4 * (MP / SUMS);  // rows that a thread has at the end; warps that have some
    static constexpr int UNPACK_WARP0 = SPLIT ? END_WARP0 : END_WARP0 + END_WARPS, UNPACK_GROUPS = SPLIT ? 4 : 2;
    static constexpr int THREADS = 32 * UNPACK_WARP0 + 128 * UNPACK_GROUPS;
    // Tensor memory: a stage's values (SPLIT: and their rests) of 128 columns, accumulators of MP columns.
    static constexpr int PART_COLS = STAGE_K / 2, A_COLS = SPLIT ? 2 * PART_COLS : PART_COLS;
    static constexpr int A_BUFS = SPLIT ? 6 : 4, D_COL0 = A_BUFS * A_COLS;
    static constexpr int D_ROOM = (512 - D_COL0) / MP, D_MOST = SPLIT ? MMA_WARPS : EACH * (STAGES - 2);
    static constexpr int D_BUFS = D_ROOM < D_MOST ? D_ROOM : D_MOST;
    static constexpr int CTL_OFF = STAGES * STAGE_BYTES;
    static constexpr int SMEM_BYTES = 1024 + CTL_OFF + 512;

    static_assert(SPLIT ? D_BUFS == MMA_WARPS : D_BUFS >= 3 && D_BUFS >= EACH, "tensor memory");
    static_assert(A_BUFS < STAGES && D_BUFS < (SPLIT ? 512 : EACH * STAGES), "a stage's barrier outlasts its readers");
    // A barrier's phases are told apart by one bit: who waits for a phase has to
    // know that the one before is over.  So the users of a place in a ring are
    // the same warps each time round, and the producer of a stage has been
    // that of the one whose buffer of values it takes.  (Accumulators go round
    // in the order of the sums, and a warp's last use of one tells enough of
    // the uses before if there are three.)
    static_assert(STAGES % PRODUCERS == 0 && STAGES % UNPACK_GROUPS == 0 && STAGES % MMA_WARPS == 0, "phases");
    static_assert(A_BUFS % MMA_WARPS == 0 && A_BUFS % PRODUCERS == 0, "phases");
    static_assert(STAGE_BYTES % 1024 == 0 && SMEM_BYTES <= 232448 && SMEM_BYTES > 116 * 1024, "one CTA an SM");
    static_assert(MP * kWideCols * 4 <= CTL_OFF, "sums of the cluster in the ring's place");
};

template <class Cfg>
struct WideCtl {
    uint64_t full[Cfg::STAGES];     // copies of a stage have landed
    uint64_t a_full[Cfg::A_BUFS];   // its values are in tensor memory
    // Its products are done: the stage may be filled again, the values' buffer
    // too, and accumulators that end here be read.
    uint64_t done[Cfg::STAGES];
    uint64_t d_empty[Cfg::D_BUFS];  // an accumulator has been read (without SPLIT)
    uint64_t all_done;              // all products are done (SPLIT)
    uint64_t drain[Cfg::MMA_WARPS];
    uint32_t tmem_base;
    int abort;
};

// A place in a ring of N, and the parity of its barrier's phase.
template <int N>
struct Ring {
    int at = 0;
    uint32_t parity = 0;

    __device__ __forceinline__ void skip(int n)  // n at most N
    {
        at += n;
        if (at >= N) {
            at -= N;
            parity ^= 1u;
        }
    }

    __device__ __forceinline__ Ring back(int n) const  // n below N
    {
        Ring r{at - n, parity};
        if (r.at < 0) {
            r.at += N;
            r.parity ^= 1u;
        }
        return r;
    }
};

// A whole warp's bounded wait, without branches by lane.
__device__ __forceinline__ bool wait_for(const Waiter &w, const uint64_t *bar, uint32_t parity)
{
    const uint32_t at = smem_u32(bar);
    for (int i = 0; i < 16; ++i)
        if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
    return __all_sync(0xffffffffu, w.wait(at, parity));
}

template <bool BF16>
__device__ __forceinline__ float scale_of(uint16_t bits)
{
    if constexpr (BF16)
        return __uint_as_float(static_cast<uint32_t>(bits) << 16);
    else
        return __half2float(__ushort_as_half(bits));
}

template <bool BF16>
__device__ __forceinline__ uint16_t round_of(float v)
{
    if constexpr (BF16)
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        return __half_as_ushort(__float2half_rn(v));
}

// Values i and i + 4 of a word as 16-bit numbers q - 8: rows 2i and 2i + 1.
template <bool BF16>
__device__ __forceinline__ uint32_t pair_of(uint32_t word, int i)
{
    uint32_t m;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(m) : "r"(word >> (4 * i)), "r"(0x000f000fu), "r"(BF16 ? 0x43004300u : 0x64006400u));
    if constexpr (BF16) {  // 128 + q
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&m), __float2bfloat162_rn(136.0f));
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {               // 1024 + q
        const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&m), __float2half2_rn(1032.0f));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// A pair times the scale in both halves of `scale`: rounded, and what that is
// too large by, exactly.
template <bool BF16>
__device__ __forceinline__ void split_of(uint32_t pair, uint32_t scale, uint32_t &rounded, uint32_t &over)
{
    const uint32_t minus = scale ^ 0x80008000u;
    const auto split = [&](auto zero) {
        using T = decltype(zero);
        const T q = *reinterpret_cast<const T *>(&pair), s = *reinterpret_cast<const T *>(&scale);
        const T h = __hmul2_rn(q, s), o = __hfma2(q, *reinterpret_cast<const T *>(&minus), h);
        rounded = *reinterpret_cast<const uint32_t *>(&h);
        over = *reinterpret_cast<const uint32_t *>(&o);
    };
    if constexpr (BF16) split(__nv_bfloat162());
    else split(__half2());
}

// 32 columns of this thread's lane of tensor memory.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc].
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// The CTA's stages [lo, hi).
struct WideRange {
    int lo, hi;
};

__device__ __forceinline__ WideRange wide_range(const WideParams &p, int rank)
{
    const uint32_t stages = p.stages;  // below 2^25; a 64-bit division is some 200 cycles
    return WideRange{static_cast<int>(stages * rank / p.split), static_cast<int>(stages * (rank + 1) / p.split)};
}

template <class Cfg>
__device__ void wide_producer(const WideParams &p, const CUtensorMap *words, const CUtensorMap *rows, uint32_t sbase,
                              WideCtl<Cfg> *ctl, const Waiter &w, const WideRange &r, int col0, int mine)
{
    Ring<Cfg::STAGES> slot;
    slot.skip(mine);
    for (int i = r.lo + mine; i < r.hi; i += Cfg::PRODUCERS, slot.skip(Cfg::PRODUCERS)) {
        if (!wait_for(w, &ctl->done[slot.at], slot.parity ^ 1u)) {
            // Copies in flight land before the CTA's shared memory goes.
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 2000000ull) {
            }
            return;
        }
        if (static_cast<int64_t>(i - r.lo) == p.stall_stage && blockIdx.x == 0) continue;  // (test hook)
        if (elect_one_sync()) {
            const uint32_t bar = smem_u32(&ctl->full[slot.at]), at = sbase + slot.at * Cfg::STAGE_BYTES;
            mbar_arrive_expect_tx(bar, Cfg::STAGE_BYTES);
            tma_load_2d(at + Cfg::X_BYTES, words, bar, col0, Cfg::STAGE_K / 8 * i);
#pragma unroll
            for (int t = 0; t < Cfg::SUBS; ++t)
                tma_load_2d(at + Cfg::MP * 128 * t, rows, bar, Cfg::STAGE_K * i + 64 * t, 0);
        }
        __syncwarp();
    }
}

// The warpgroup's stages of this thread's column.  False: a wait ran out.
template <class Cfg, bool BF16>
__device__ bool wide_unpack(const WideParams &p, uint32_t sbase, uint32_t tmem, WideCtl<Cfg> *ctl, const Waiter &w,
                            const WideRange &r, int64_t n, int warp, int lane)
{
    constexpr int TURNS = Cfg::UNPACK_GROUPS;
    const int q = warp & 3, mine = (warp - Cfg::UNPACK_WARP0) >> 2;  // quarter of the columns, which stages
    const uint32_t at0 = sbase + Cfg::X_BYTES + 4u * (32 * q + lane);
    // SPLIT: scales of a stage's first and last 32 rows, loaded a turn ahead, into
    // two pairs of registers by turns (a move would wait for the load).  Past K
    // the last one again: x is zero there.
    const uint16_t *const column = p.S + (n < p.n4 ? n : 0);
    const int last = static_cast<int>((p.K - 1) / 32);
    int group = 2 * (r.lo + mine);
    uint32_t scales[2][2] = {};
    const auto fetch = [&](uint32_t(&s)[2]) {
        if constexpr (Cfg::SPLIT) {
            s[0] = __ldg(column + min(group, last) * p.n4);
            s[1] = __ldg(column + min(group + 1, last) * p.n4);
            group += 2 * TURNS;
        }
    };
    fetch(scales[0]);
    Ring<Cfg::STAGES> slot;
    Ring<Cfg::A_BUFS> a;
    slot.skip(mine);
    a.skip(mine);
    const auto unpack = [&](int i, const uint32_t(&scale)[2]) {
        if (!wait_for(w, &ctl->full[slot.at], slot.parity)) return false;
        const uint32_t at = at0 + slot.at * Cfg::STAGE_BYTES;
        const uint32_t to = tmem + (static_cast<uint32_t>(32 * q) << 16) + Cfg::A_COLS * a.at;
        const uint32_t s0 = scale[0] * 0x10001u, s1 = scale[1] * 0x10001u;
#pragma unroll
        for (int t = 0; t < Cfg::SUBS; ++t) {
            uint32_t v[32], over[32];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                const uint32_t word = ld_shared_b32(at + Cfg::WORD_PITCH * (8 * t + b));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t pair = pair_of<BF16>(word, j);
                    if constexpr (Cfg::SPLIT) split_of<BF16>(pair, b < 4 ? s0 : s1, v[4 * b + j], over[4 * b + j]);
                    else v[4 * b + j] = pair;
                }
            }
            if (t == 0 && i >= Cfg::A_BUFS) {
                // (the products before in this buffer; their barrier is not filled again before this stage is done)
                const Ring<Cfg::STAGES> before = slot.back(Cfg::A_BUFS);
                if (!wait_for(w, &ctl->done[before.at], before.parity)) return false;
                tc_fence_after_sync();
            }
            tmem_st_32x32b_x32(to + 32 * t, v);
            if constexpr (Cfg::SPLIT) tmem_st_32x32b_x32(to + Cfg::PART_COLS + 32 * t, over);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->a_full[a.at]));
        slot.skip(TURNS);
        a.skip(TURNS);
        return true;
    };
    const int stages = r.hi - r.lo;
    for (int i = mine; i < stages; i += 2 * TURNS) {
        fetch(scales[1]);
        if (!unpack(i, scales[0])) return false;
        if (i + TURNS >= stages) break;
        fetch(scales[0]);
        if (!unpack(i + TURNS, scales[1])) return false;
    }
    return true;
}

// Issuing a stage's MMAs and finding the next barriers ready takes a warp longer
// than anything else takes (8 MMAs 500 to 600 cycles, the rest as much again), so
// two warps take stages in turn, and the next barriers are looked at while the
// MMAs go out.
template <class Cfg, bool BF16>
__device__ void wide_mma(const WideParams &p, uint32_t sbase, uint32_t tmem, WideCtl<Cfg> *ctl, const Waiter &w,
                         const WideRange &r, int mine)
{
    constexpr int STEPS = Cfg::STAGE_K / 16, BLOCK = Cfg::GROUP / 16;
    const uint32_t idesc = umma_idesc_16bit_f32(128, Cfg::MP, BF16, false, false);
    const uint64_t b0 = umma_desc_sw128(sbase, 16, 1024);
    Ring<Cfg::STAGES> slot;
    Ring<Cfg::A_BUFS> a;
    Ring<Cfg::D_BUFS> d;
    const auto skip = [&](int stages) {
        slot.skip(stages);
        a.skip(stages);
        for (int j = 0; j < stages * Cfg::EACH; ++j) d.skip(1);
    };
    skip(mine);
    const int64_t rows = p.K - Cfg::STAGE_K * static_cast<int64_t>(r.lo);
    bool ok = true, ready = false, free = false, issued = false;
    for (int i = mine; i < r.hi - r.lo && ok; i += Cfg::MMA_WARPS) {
        const int64_t left = rows - Cfg::STAGE_K * static_cast<int64_t>(i);
        const int steps = left >= Cfg::STAGE_K ? STEPS : static_cast<int>((left + 15) / 16);
        const uint32_t b_lo = static_cast<uint32_t>(b0) + ((slot.at * Cfg::STAGE_BYTES) >> 4);
        const uint32_t a_at = tmem + Cfg::A_COLS * a.at;
        uint64_t *const done = &ctl->done[slot.at];
        if (!ready) ok = wait_for(w, &ctl->a_full[a.at], a.parity) && wait_for(w, &ctl->full[slot.at], slot.parity);
#pragma unroll
        for (int j0 = 0; j0 < STEPS; j0 += BLOCK) {
            if (j0 >= steps || !ok) break;
            if (!free) ok = wait_for(w, &ctl->d_empty[d.at], d.parity ^ 1u);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t d_at = tmem + Cfg::D_COL0 + Cfg::MP * d.at;
            d.skip(1);
            bool a_in = true, x_in = true;
            if (j0 + BLOCK >= STEPS) {
                slot.skip(1);
                a.skip(1);
                skip(Cfg::MMA_WARPS - 1);
                a_in = mbar_test_wait(smem_u32(&ctl->a_full[a.at]), a.parity);
                x_in = mbar_test_wait(smem_u32(&ctl->full[slot.at]), slot.parity);
            }
            const bool is_free = mbar_test_wait(smem_u32(&ctl->d_empty[d.at]), d.parity ^ 1u);
            if (elect_one_sync()) {
#pragma unroll
                for (int j = j0; j < j0 + BLOCK; ++j)  // (16 products on: 8 columns of A, 32 bytes of B, tiles of 64)
                    if (j < steps)
                        umma_f16_ta(d_at, a_at + 8 * j,
                                    (b0 & 0xffffffff00000000ull) | (b_lo + (j >> 2) * (Cfg::MP * 128 >> 4) + 2 * (j & 3)),
                                    idesc, j > j0 ? 1u : 0u);
                if (j0 + BLOCK >= steps) umma_commit(smem_u32(done));
            }
            issued = true;
            free = __all_sync(0xffffffffu, is_free);
            if (j0 + BLOCK >= STEPS) ready = __all_sync(0xffffffffu, a_in && x_in);
        }
    }
    if (!ok && issued) {
        if (elect_one_sync()) umma_commit(smem_u32(&ctl->drain[mine]));
        __syncwarp();
        w.wait_drain(smem_u32(&ctl->drain[mine]), 0, kDrainNs);
    }
}

// SPLIT: values and rests of all groups into one accumulator of the warp's own
// (MMAs of different warps are not ordered).  X has landed where the words have,
// which the warps that unpacked them saw.
template <class Cfg, bool BF16>
__device__ void wide_mma_split(const WideParams &p, uint32_t sbase, uint32_t tmem, WideCtl<Cfg> *ctl, const Waiter &w,
                         const WideRange &r, int mine)
{
    constexpr int STEPS = Cfg::STAGE_K / 16;
    const uint32_t idesc = umma_idesc_16bit_f32(128, Cfg::MP, BF16, false, false), minus = idesc | 1u << 13;  // A negated
    const uint64_t b0 = umma_desc_sw128(sbase, 16, 1024);
    const uint32_t d_at = tmem + Cfg::D_COL0 + Cfg::MP * mine;
    Ring<Cfg::STAGES> slot;
    Ring<Cfg::A_BUFS> a;
    slot.skip(mine);
    a.skip(mine);
    const int stages = r.hi - r.lo;
    bool ok = true, issued = false;
    for (int i = mine; i < stages; i += Cfg::MMA_WARPS) {
        const int64_t left = p.K - Cfg::STAGE_K * static_cast<int64_t>(r.lo + i);
        const int steps = left >= Cfg::STAGE_K ? STEPS : static_cast<int>((left + 15) / 16);
        const uint32_t b_lo = static_cast<uint32_t>(b0) + ((slot.at * Cfg::STAGE_BYTES) >> 4);
        const uint32_t a_at = tmem + Cfg::A_COLS * a.at;
        if (!(ok = wait_for(w, &ctl->a_full[a.at], a.parity))) break;
        tc_fence_after_sync();
        if (elect_one_sync()) {
#pragma unroll
            for (int j = 0; j < STEPS; ++j)  // (16 products on: 8 columns of A, 32 bytes of B)
                if (j < steps) {
                    const uint64_t b = (b0 & 0xffffffff00000000ull) | (b_lo + 2 * j);
                    umma_f16_ta(d_at, a_at + 8 * j, b, idesc, issued || j > 0 ? 1u : 0u);
                    umma_f16_ta(d_at, a_at + Cfg::PART_COLS + 8 * j, b, minus, 1u);
                }
            umma_commit(smem_u32(&ctl->done[slot.at]));
            if (i + Cfg::MMA_WARPS >= stages) umma_commit(smem_u32(&ctl->all_done));
        }
        issued = true;
        slot.skip(Cfg::MMA_WARPS);
        a.skip(Cfg::MMA_WARPS);
    }
    if (!ok && issued) {
        if (elect_one_sync()) umma_commit(smem_u32(&ctl->drain[mine]));
        __syncwarp();
        w.wait_drain(smem_u32(&ctl->drain[mine]), 0, kDrainNs);
    }
}

// This thread's column's sums over the CTA's groups, of 32 of the rows.
template <class Cfg, bool BF16>
__device__ void wide_sums(const WideParams &p, uint32_t tmem, WideCtl<Cfg> *ctl, const Waiter &w, const WideRange &r, int64_t n,
                          int warp, int lane, float (&sum)[Cfg::SUMS])
{
#pragma unroll
    for (int m = 0; m < Cfg::SUMS; ++m) sum[m] = 0.0f;
    const int64_t k0 = Cfg::STAGE_K * static_cast<int64_t>(r.lo), k1 = Cfg::STAGE_K * static_cast<int64_t>(r.hi);
    const int64_t rows = (k1 < p.K ? k1 : p.K) - k0;
    const int groups = rows > 0 ? static_cast<int>((rows + Cfg::GROUP - 1) / Cfg::GROUP) : 0;
    constexpr int EACH = Cfg::EACH;
    Ring<Cfg::STAGES> slot;
    Ring<Cfg::D_BUFS> d;
    const int part = (warp - Cfg::END_WARP0) >> 2;
    const uint32_t at0 = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + Cfg::D_COL0 + Cfg::SUMS * part;
    // This column's scales, AHEAD stages ahead in registers: a load takes a
    // stage or two, and the loop is short.
    constexpr int AHEAD = 3;
    const uint16_t *scale = p.S + k0 / Cfg::GROUP * p.n4 + (n < p.n4 ? n : 0);
    uint16_t next[AHEAD][EACH];
    int loaded = 0;  // groups
    const auto fetch = [&](uint16_t(&s)[EACH]) {
#pragma unroll
        for (int u = 0; u < EACH; ++u, ++loaded, scale += p.n4) s[u] = loaded < groups ? __ldg(scale) : uint16_t(0);
    };
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) fetch(next[a]);
    bool ok = true;
    for (int g0 = 0; ok && g0 < groups;) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a, g0 += EACH, slot.skip(1)) {
            if (g0 >= groups) break;
            float s[EACH];
#pragma unroll
            for (int u = 0; u < EACH; ++u) s[u] = scale_of<BF16>(next[a][u]);
            fetch(next[a]);
            // (not filled again before STAGES more, and accumulators do not reach that far)
            ok = wait_for(w, &ctl->done[slot.at], slot.parity);
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int u = 0; u < EACH; ++u) {
                if (g0 + u >= groups) break;
                uint32_t v[Cfg::SUMS];
                tmem_ld_32x32b_x32(at0 + Cfg::MP * d.at, v);
                tmem_wait_ld();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->d_empty[d.at]));
                d.skip(1);
#pragma unroll
                for (int m = 0; m < Cfg::SUMS; ++m) sum[m] = fmaf(s[u], __uint_as_float(v[m]), sum[m]);
            }
        }
    }
}

// SPLIT: the sums of the CTA's k that are not finite, again, group by group as
// they are written down: 8 rows at a time, a thread a column of them, and the
// warpgroups that unpack take groups in turn.  All threads of the CTA come here,
// with its sums in `sums` (MP x 128).  64 rows x 2^18 x 128, every sum infinite:
// 8.4 ms, one row of them 1.2 (all finite 0.13; by one thread a sum of all the
// cluster's k: 104).
template <class Cfg, bool BF16>
__device__ __noinline__ void wide_again(const WideParams &p, WideRange r, int64_t n, int warp, float *sums)
{
    constexpr int ROWS = 8, TEAMS = Cfg::UNPACK_GROUPS, EACH = Cfg::STAGE_K / Cfg::GROUP;
    static_assert((Cfg::MP + TEAMS * ROWS) * kWideCols * 4 <= Cfg::CTL_OFF, "sums and parts in the ring's place");
    float *const parts = sums + Cfg::MP * kWideCols;  // TEAMS x ROWS x 128
    const int column = static_cast<int>(threadIdx.x) & 127, team = (warp - Cfg::UNPACK_WARP0) >> 2;
    const bool on = warp >= Cfg::UNPACK_WARP0 && n < p.N;
    const int64_t groups = (p.K + Cfg::GROUP - 1) / Cfg::GROUP, first = static_cast<int64_t>(r.lo) * EACH;
    const int64_t last = static_cast<int64_t>(r.hi) * EACH < groups ? static_cast<int64_t>(r.hi) * EACH : groups;
    for (int m0 = 0; m0 < p.M; m0 += ROWS) {
        bool bad = false;
        if (on)
            for (int i = 0; i < ROWS && m0 + i < p.M; ++i) bad |= !isfinite(sums[(m0 + i) * kWideCols + column]);
        if (!__syncthreads_or(bad)) continue;
        float sum[ROWS] = {};
        for (int64_t g = first + team; bad && g < last; g += TEAMS) {
            float part[ROWS] = {};
#pragma unroll
            for (int b = 0; b < Cfg::GROUP / 8; ++b) {
                const int64_t k = Cfg::GROUP * g + 8 * b;
                if (k >= p.K) break;
                const int count = p.K - k < 8 ? static_cast<int>(p.K - k) : 8;
                const uint32_t word = p.Q[(k >> 3) * p.n4 + n];
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    // (a whole piece of 16 bytes, of which the first is inside the row)
                    const uint4 v = *reinterpret_cast<const uint4 *>(p.X + (m0 + i < p.M ? m0 + i : m0) * p.ldx + k);
                    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int q = static_cast<int>(word >> (4 * ((j & 1 ? 4 : 0) + (j >> 1))) & 15u);
                        const uint16_t bits = static_cast<uint16_t>(x[j >> 1] >> (16 * (j & 1)));
                        if (j < count) part[i] = fmaf(scale_of<BF16>(bits), static_cast<float>(q - 8), part[i]);
                    }
                }
            }
            const float s = scale_of<BF16>(p.S[g * p.n4 + n]);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) sum[i] = fmaf(s, part[i], sum[i]);
        }
        if (on)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) parts[(team * ROWS + i) * kWideCols + column] = sum[i];
        __syncthreads();
        if (on)
            for (int i = team; i < ROWS && m0 + i < p.M; i += TEAMS) {
                float &to = sums[(m0 + i) * kWideCols + column];
                if (isfinite(to)) continue;
                float all = 0.0f;
                for (int t = 0; t < TEAMS; ++t) all += parts[(t * ROWS + i) * kWideCols + column];
                to = all;
            }
        __syncthreads();
    }
}

template <class Cfg, bool BF16>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    rows4_wide_kernel(const __grid_constant__ CUtensorMap words, const __grid_constant__ CUtensorMap rows,
                      const __grid_constant__ WideParams p)
{
    extern __shared__ __align__(1024) uint8_t wide_smem[];
    const uint32_t raw = smem_u32(wide_smem), pad = (1024u - (raw & 1023u)) & 1023u, sbase = raw + pad;
    auto *ctl = reinterpret_cast<WideCtl<Cfg> *>(wide_smem + pad + Cfg::CTL_OFF);
    static_assert(sizeof(WideCtl<Cfg>) <= 512, "control block");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const WideRange r = wide_range(p, rank);
    const int stages = r.hi - r.lo, accumulators = stages < Cfg::MMA_WARPS ? stages : Cfg::MMA_WARPS;
    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::STAGES; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->done[s]), 1);
        }
        for (int a = 0; a < Cfg::A_BUFS; ++a) mbar_init(smem_u32(&ctl->a_full[a]), 4);
        for (int d = 0; d < Cfg::D_BUFS; ++d) mbar_init(smem_u32(&ctl->d_empty[d]), Cfg::END_WARPS);
        mbar_init(smem_u32(&ctl->all_done), accumulators);
        for (int i = 0; i < Cfg::MMA_WARPS; ++i) mbar_init(smem_u32(&ctl->drain[i]), 1);
        ctl->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&words);
        tma_prefetch_desc(&rows);
    }
    if (warp == Cfg::MMA_WARP0) {
        tmem_alloc(smem_u32(&ctl->tmem_base), 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_launch_dependents();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    const Waiter w{&ctl->abort, p.status, p.timeout_ns};
    const int64_t col0 = static_cast<int64_t>(blockIdx.x / p.split) * kWideCols;
    // At the end a warpgroup has SUMS rows, a thread a column of them.
    const int column = static_cast<int>(threadIdx.x) & 127, row0 = Cfg::SUMS * ((warp - Cfg::END_WARP0) >> 2);
    const bool ends = warp >= Cfg::END_WARP0 && warp < Cfg::END_WARP0 + Cfg::END_WARPS;
    const int64_t n = col0 + column;
    const auto store = [&](int m, float v) { p.Y[m * p.ldy + n] = round_of<BF16>(v); };
    float *sums = reinterpret_cast<float *>(wide_smem + pad);  // in the ring's place, once every stage is done
    bool bad = false;  // a sum that is not finite
    if (warp < Cfg::PRODUCERS) {
        wide_producer<Cfg>(p, &words, &rows, sbase, ctl, w, r, static_cast<int>(col0), warp);
    } else if (warp < Cfg::END_WARP0) {
        if constexpr (Cfg::SPLIT) wide_mma_split<Cfg, BF16>(p, sbase, tmem, ctl, w, r, warp - Cfg::MMA_WARP0);
        else wide_mma<Cfg, BF16>(p, sbase, tmem, ctl, w, r, warp - Cfg::MMA_WARP0);
    } else {
        bool ok = true;
        if (warp >= Cfg::UNPACK_WARP0) ok = wide_unpack<Cfg, BF16>(p, sbase, tmem, ctl, w, r, n, warp, lane);
        if (ends) {
            float sum[Cfg::SUMS] = {};
            if constexpr (!Cfg::SPLIT) {
                wide_sums<Cfg, BF16>(p, tmem, ctl, w, r, n, warp, lane, sum);
            } else if (ok && wait_for(w, &ctl->all_done, 0)) {
                tc_fence_after_sync();
                const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + Cfg::D_COL0 + row0;
                for (int d = 0; d < accumulators; ++d) {
                    uint32_t v[Cfg::SUMS];
                    tmem_ld_32x32b_x32(at + Cfg::MP * d, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int m = 0; m < Cfg::SUMS; ++m) sum[m] += __uint_as_float(v[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < Cfg::SUMS; ++m) {
                if (row0 + m >= p.M) break;
                if (Cfg::SPLIT || p.split > 1) sums[(row0 + m) * kWideCols + column] = sum[m];
                else if (n < p.N) store(row0 + m, sum[m]);
                bad |= Cfg::SPLIT && n < p.N && !isfinite(sum[m]);
            }
        }
    }
    __syncwarp();
    if constexpr (Cfg::SPLIT) {
        // (a wait that ran out leaves anything)
        if (__syncthreads_or(bad) && ctl->abort == 0) wide_again<Cfg, BF16>(p, r, n, warp, sums);
        if (p.split == 1 && ends && n < p.N)
            for (int m = row0; m < row0 + Cfg::SUMS && m < p.M; ++m) store(m, sums[m * kWideCols + column]);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == Cfg::MMA_WARP0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
    if (p.split == 1) return;
    cluster_sync();
    if (ends && n < p.N)
        for (int m = row0 + rank; m < p.M && m < row0 + Cfg::SUMS; m += p.split) {
            float v = 0.0f;
            for (int c = 0; c < p.split; ++c) v += ld_cluster_f32(mapa_shared(sbase + 4 * (m * kWideCols + column), c));
            store(m, v);
        }
    cluster_sync();  // others may still read this CTA's sums
}

template <class Cfg, bool BF16>
cudaError_t launch(const CUtensorMap &words, const CUtensorMap &rows, const WideParams &p, int grid, cudaStream_t s)
{
    const auto kernel = rows4_wide_kernel<Cfg, BF16>;
    static std::atomic<int> done[128];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (!done[dev].load()) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        done[dev].store(1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, words, rows, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows4_wide(bool bf16, const CUtensorMap &words, const CUtensorMap &rows, const WideParams &p,
                              int grid, cudaStream_t s)
{
    const auto of_group = [&](auto group) {
        constexpr int GROUP = decltype(group)::value;
        if (p.M > 32)
            return bf16 ? launch<WideCfg<64, GROUP>, true>(words, rows, p, grid, s)
                        : launch<WideCfg<64, GROUP>, false>(words, rows, p, grid, s);
        return bf16 ? launch<WideCfg<32, GROUP>, true>(words, rows, p, grid, s)
                    : launch<WideCfg<32, GROUP>, false>(words, rows, p, grid, s);
    };
    if (p.group == 32) return of_group(std::integral_constant<int, 32>());
    if (p.group == 64) return of_group(std::integral_constant<int, 64>());
    return of_group(std::integral_constant<int, 128>());
}

}  // namespace gp
