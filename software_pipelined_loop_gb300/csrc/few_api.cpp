// few_api.cpp -- the entry points for a few tokens of include/gemmpipe.h:
// rows times weights in 4 bits, the whole expert layer, and the weights' way
// into 4 bits and back.  Argument checks and the choice of the launch.
#include "gemmpipe.h"

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <utility>

#include "api_internal.h"
#include "few.h"
#include "grouped_params.h"
#include "variants.h"

namespace {

using gp::ApiDevice;
using gp::FewLaunch;
using gp::FewParams;

constexpr int64_t kMaxDim = 2147483647 - 1023;  // sizes rounded up to a block stay in 32 bits
constexpr int64_t kMaxElems = int64_t(1) << 56;

bool misaligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }
bool bad_pointer(const void *p, int bytes) { return !p || misaligned(p, bytes); }
bool bad_dim(int64_t v) { return v < 0 || v > kMaxDim; }
bool bad_type(int type) { return type != GEMMPIPE_F16 && type != GEMMPIPE_BF16; }
bool bad_group(int64_t group) { return group != 32 && group != 64 && group != 128; }
bool bad_pitch(int64_t width, int64_t ld) { return ld < width || ld > 2147483647; }
bool bad_experts(int64_t E) { return E < 1 || E > gp::kMaxExperts; }
// Matrices E x K x N.
bool bad_matrices(int64_t E, int64_t K, int64_t N)
{
    return bad_dim(K) || bad_dim(N) || (K > 0 && N > 0 && (K + 127) > kMaxElems / (E * (N + 3)));
}

gemmpipe_status_t check_all(std::initializer_list<std::pair<const void *, int>> ps)
{
    for (const auto &p : ps) {
        if (!p.first) continue;  // optional
        const gemmpipe_status_t st = gp::api_check_pointer(p.first, p.second);
        if (st != GEMMPIPE_OK) return st;
    }
    return GEMMPIPE_OK;
}

cudaStream_t stream_of(gemmpipe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Nothing thrown leaves an entry point.
template <class F>
gemmpipe_status_t guarded(F f)
{
    try {
        return f();
    } catch (...) {
        return GEMMPIPE_ERR_INTERNAL;
    }
}

gemmpipe_status_t zero_rows(void *out, int64_t rows, int64_t width, int64_t ld, cudaStream_t s)
{
    const cudaError_t e = cudaMemset2DAsync(out, static_cast<size_t>(ld) * 2, 0, static_cast<size_t>(width) * 2,
                                            static_cast<size_t>(rows), s);
    if (e == cudaSuccess) return GEMMPIPE_OK;
    cudaGetLastError();
    return GEMMPIPE_ERR_LAUNCH;
}

int64_t align128(int64_t x) { return (x + 127) / 128 * 128; }

// The launch for `p` (sizes, matrices and ids set).  Items of the first product
// hold 8 rows of up to 8 tokens; above, 16 rows, or 32 where the experts have more
// on average.  Those of the second product, whose rows are two each, hold 4 rows
// of up to 4 tokens; above, 8, or, of weights in 16 bits, 16 where the experts have
// more on average (64 tokens x 8 of 16 experts of 4096 x 1536 181 us, 199 in 8s; of 64
// experts 415 and 408; in 4 bits 203 and 187, 237 and 224).
FewLaunch few_launch(FewParams *p, bool bf16, bool four, bool any, int mode)
{
    FewLaunch l{};
    l.bf16 = bf16;
    l.four = four;
    l.any = any;
    l.mode = mode;
    const int64_t slots = static_cast<int64_t>(p->tokens) * p->top_k;
    const int64_t used = !p->ids ? 1 : (slots < p->experts ? slots : p->experts);  // experts with rows, at most
    const bool up = mode == gp::kFewUp;
    const bool many = p->tokens > 16 && slots > 16 * used && !(any && !four);
    l.row_blocks = p->tokens <= (up ? 8 : 4) ? 1 : (many && (up || (mode == gp::kFewParts && !four)) ? 4 : 2);
    const int64_t chunk = gp::few_chunk(l.row_blocks, up);
    p->steps = static_cast<uint32_t>((p->K + (four ? 63 : 31)) / (four ? 64 : 32));
    p->group_shift = p->group_steps == 4 ? 2 : p->group_steps == 2 ? 1 : 0;
    p->words = (p->K + 7) / 8;
    p->groups = (p->K + 32 * p->group_steps - 1) / (32 * p->group_steps);
    int64_t items = (p->tokens + chunk - 1) / chunk;
    p->max_items = static_cast<int>(items);
    p->table_bytes = 0;
    if (p->ids) {
        // An item for each expert with rows, and one more for each further chunk
        // of them: taken by the blocks of the first ones.
        items = used;
        p->max_items = static_cast<int>(used + (p->tokens > chunk ? slots / chunk : 0));
        const int64_t words = 2 * static_cast<int64_t>(p->max_items) + 2 * slots + 3 * static_cast<int64_t>(p->experts) + 1;
        p->table_bytes = static_cast<int>(slots <= 32 ? 4 * gp::kFewWarps * 128 : align128(4 * words));
    }
    // Units of work: 64 columns of an item each (kFewFlat: of all items).  The
    // experts that have rows are not known here: as many as tokens that choose
    // any of them alike would reach.
    const bool all = mode == gp::kFewFlat;
    const int64_t columns = (p->out_cols + gp::kFewCols - 1) / gp::kFewCols;
    double reached = static_cast<double>(items);
    if (p->ids && p->top_k < p->experts)
        reached = p->experts * (1.0 - std::pow(1.0 - static_cast<double>(p->top_k) / p->experts, p->tokens));
    const double units = static_cast<double>(columns) * (all ? 1.0 : reached);
    const double steps = static_cast<double>(p->steps) * (all ? reached : p->matrices);
    // Blocks of a cluster share a unit's products.  Time in us: rounds of units
    // over the clusters that run at once, each the steps of a warp (measured
    // with all warps of an SM at work) and the end of a unit.
    const int one = l.row_blocks == 4;
    const double step_us = four ? 1.0 : 1.45;
    double best = 0.0;
    int64_t room = 0;
    p->split = 0;
    for (int split = 1; split <= 8; ++split) {
        const int64_t at_once = gp::few_room(one, split);
        if (at_once < 1 || (split > 1 && units > at_once)) continue;
        const double warp_steps = std::ceil(steps / (gp::kFewWarps * split));
        const double us = std::ceil(units / at_once) * (warp_steps * step_us + (split == 1 ? 1.0 : 1.7));
        if (p->split == 0 || us < best) {
            best = us;
            p->split = split;
            room = at_once;
        }
    }
    l.status = GEMMPIPE_ERR_LAUNCH;
    if (p->split == 0) return l;  // (the device did not say)
    // Short sums: a warp takes four steps at least where there are units
    // enough, by sharing its columns with fewer others.
    p->wide = 1;
    while (!all && p->split == 1 && p->wide < 4 && units >= 2.0 * room * p->wide &&
           4 * gp::kFewWarps > steps * p->wide)
        p->wide *= 2;
    p->columns = static_cast<int>((columns + p->wide - 1) / p->wide);
    // (units are counted in 32 bits)
    const bool counted = static_cast<int64_t>(p->columns) * p->max_items < int64_t(1) << 30;
    l.status = counted ? GEMMPIPE_OK : GEMMPIPE_ERR_INVALID_VALUE;
    const int64_t clusters = static_cast<int64_t>(p->columns) * (all ? 1 : items);
    l.grid = static_cast<int>((all || clusters <= 4 * room ? clusters : room) * p->split);
    return l;
}

cudaError_t launch(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    return l.bf16 ? gp::launch_few_bf16(l, p, s) : gp::launch_few_f16(l, p, s);
}

// Tensor map of rows x n4 words, boxes of a stage of 128 columns (one copy: the
// 128-byte swizzle would take four, and a copy costs its warp 100 cycles).
bool encode_words(CUtensorMap *m, const uint32_t *Q, int64_t rows, int64_t n4, int group)
{
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<void *> encode{nullptr};
    void *f = encode.load();
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess || !f) {
            cudaGetLastError();
            return false;
        }
        encode.store(f);
    }
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(n4), static_cast<cuuint64_t>(rows)};
    const cuuint64_t pitch[1] = {static_cast<cuuint64_t>(4 * n4)};
    const cuuint32_t box[2] = {gp::kWideCols, static_cast<cuuint32_t>(gp::wide_stage_k(group) / 8)}, each[2] = {1, 1};
    return reinterpret_cast<Encode>(f)(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint32_t *>(Q), dims, pitch, box,
                                       each, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Some aligned rows times 4 bits: tiles of 128 columns on tcgen05.  16 rows in
// groups of 128 (64): 4096 x 16384 13.8 (15.8) us there and 16.6 (16.6) as few
// rows, 16384 x 4096 15.4 (17.3) and 18.1 (18.1), 2048 x 2048 6.3 (6.7) and 7.2
// (7.2); 8 rows x 4096 x 16384 in groups of 128 13.5 and 12.6.  In groups of 32, 17
// rows there and 16 as few rows: 19.3 and 17.5, 21.1 and 18.9, 6.8 and 7.0; 32 rows
// x 4096 x 16384 19.5 and 31.
bool wide_rows4(int64_t M, int64_t N, int64_t K, int64_t group, const void *X, int64_t ldx)
{
    return M > (group == 32 ? 16 : 8) && N <= (int64_t(1) << 29) && K <= (int64_t(1) << 30) && !misaligned(X, 16) &&
           ldx % 8 == 0;
}

gemmpipe_status_t rows4_wide(bool bf16, int64_t M, int64_t N, int64_t K, int64_t group, const uint16_t *X, int64_t ldx,
                             const uint32_t *Q, const uint16_t *S, uint16_t *Y, int64_t ldy, cudaStream_t s)
{
    gp::WideParams p;
    std::memset(&p, 0, sizeof(p));
    p.X = X;
    p.ldx = ldx;
    p.Q = Q;
    p.S = S;
    p.Y = Y;
    p.ldy = ldy;
    p.N = N;
    p.n4 = (N + 3) / 4 * 4;
    p.K = K;
    p.M = static_cast<int>(M);
    p.group = static_cast<int>(group);
    const int stage_k = gp::wide_stage_k(p.group);
    p.stages = static_cast<int>((K + stage_k - 1) / stage_k);
    const int64_t tiles = (N + gp::kWideCols - 1) / gp::kWideCols;
    // As many CTAs a tile as run at once, of 256 products at least.
    p.split = 1;
    for (int split = 2; split <= 8; ++split)
        if (tiles <= gp::few_room(1, split) && 256 * (split - 1) < K) p.split = split;
    CUtensorMap words, rows;
    const uint64_t xd[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(M)};
    const uint64_t xs[1] = {static_cast<uint64_t>(2 * ldx)};
    const uint32_t xb[2] = {64, M > 32 ? 64u : 32u};
    if (!encode_words(&words, Q, (K + 7) / 8, p.n4, p.group) || !gp::api_encode_16bit(&rows, bf16, 2, X, xd, xs, xb))
        return GEMMPIPE_ERR_INTERNAL;
    p.timeout_ns = 2000000000ull + static_cast<uint64_t>(p.stages) * 10000ull;
    p.stall_stage = gp::api_take_stall(&p.timeout_ns);
    if (gp::status_word(&p.status) != cudaSuccess) {
        cudaGetLastError();
        return GEMMPIPE_ERR_LAUNCH;
    }
    return gp::api_launch(true, s, 1, [&] {
        return gp::launch_rows4_wide(bf16, words, rows, p, static_cast<int>(tiles * p.split), s);
    });
}

struct Matrices {  // W of an expert step: 16 bits, or words with scales
    const void *W[3];
    const uint16_t *S[3];
    int64_t group;  // 0: 16 bits
};

gemmpipe_status_t expert_step(int type, int64_t T, int64_t top_k, int64_t E, int64_t C, int64_t H, const uint16_t *X,
                              int64_t ldx, const int32_t *experts, const float *weights, const Matrices &m,
                              uint16_t *hidden, uint16_t *Y, int64_t ldy, gemmpipe_stream_t stream)
{
    const bool four = m.group != 0, gated = m.W[2] != nullptr;
    if (bad_type(type) || T < 0 || T > gp::kFewRows || top_k < 1 || top_k > gp::kMaxTopK || bad_experts(E) ||
        bad_matrices(E, C, H) || bad_matrices(E, H, C) || bad_pitch(C, ldx) || bad_pitch(C, ldy) ||
        (four && bad_group(m.group)))
        return GEMMPIPE_ERR_INVALID_VALUE;
    if (T == 0 || C == 0) return GEMMPIPE_OK;
    if (bad_pointer(Y, 2)) return GEMMPIPE_ERR_INVALID_VALUE;
    const int wa = four ? 16 : 2, sa = four ? 8 : 1;
    if (H > 0) {
        if (bad_pointer(X, 2) || bad_pointer(experts, 4) || bad_pointer(weights, 4) || bad_pointer(hidden, 16))
            return GEMMPIPE_ERR_INVALID_VALUE;
        for (int i = 0; i < (gated ? 3 : 2); ++i)
            if (bad_pointer(m.W[i], wa) || (four && bad_pointer(m.S[i], sa))) return GEMMPIPE_ERR_INVALID_VALUE;
    }
    if (four && !gated && m.S[2]) return GEMMPIPE_ERR_INVALID_VALUE;  // scales without their words
    ApiDevice d;
    gemmpipe_status_t st = gp::api_device(&d);
    if (st != GEMMPIPE_OK) return st;
    if ((st = check_all({{Y, 2}})) != GEMMPIPE_OK) return st;
    cudaStream_t s = stream_of(stream);
    if (H == 0) return zero_rows(Y, T, C, ldy, s);
    if ((st = check_all({{X, 2}, {experts, 4}, {weights, 4}, {hidden, 16}})) != GEMMPIPE_OK) return st;
    for (int i = 0; i < 3; ++i)
        if ((st = check_all({{m.W[i], wa}, {m.S[i], sa}})) != GEMMPIPE_OK) return st;

    const int64_t ldh = (H + 7) / 8 * 8;
    FewParams up;
    std::memset(&up, 0, sizeof(up));
    up.ids = experts;
    up.tokens = static_cast<int>(T);
    up.top_k = static_cast<int>(top_k);
    up.experts = static_cast<int>(E);
    up.group_steps = four ? static_cast<int>(m.group / 32) : 1;
    FewParams down = up;
    up.X = X;
    up.ldx = ldx;
    up.W[0] = m.W[0];
    up.S[0] = m.S[0];
    up.W[1] = m.W[2];
    up.S[1] = m.S[2];
    up.matrices = gated ? 2 : 1;
    up.silu = 1;
    up.K = C;
    up.N = H;
    up.out = hidden;
    up.ldo = up.out_cols = ldh;
    down.X = hidden;
    down.ldx = ldh;
    down.weights = weights;
    down.W[0] = m.W[1];
    down.S[0] = m.S[1];
    down.matrices = 1;
    down.K = H;
    down.N = down.out_cols = C;
    down.out = Y;
    down.ldo = ldy;
    const bool rows_off = misaligned(X, 16) || ldx % 8 || C % 8;
    const bool up_off = rows_off || (!four && (misaligned(m.W[0], 16) || misaligned(m.W[2], 16) || H % 8));
    const bool down_off = !four && (misaligned(m.W[1], 16) || C % 8);
    const bool bf16 = type == GEMMPIPE_BF16;
    // The second products of a few tokens are summed where they are made, as many
    // as leave room for two blocks on an SM; those of more go by way of the
    // workspace, a row for each choice.  12 tokens x 4 of 32 experts of 2048 x 1024
    // 59 us and 65 that way (4 bits: 36 and 42), x 8 of 64 of 4096 x 1536 218 and 221
    // (107 and 106); 16 tokens 77 and 68 (42 and 45), 251 and 244 (124 and 126).
    const bool flat = T <= (four ? 16 : 12);
    const FewLaunch lu = few_launch(&up, bf16, four, up_off, gp::kFewUp);
    const FewLaunch ld = few_launch(&down, bf16, four, down_off, flat ? gp::kFewFlat : gp::kFewParts);
    if (lu.status != GEMMPIPE_OK || ld.status != GEMMPIPE_OK) return lu.status != GEMMPIPE_OK ? lu.status : ld.status;
    // What the rounding of hidden rows leaves is in the workspace, and before the
    // sums the rows for each choice.
    const gp::ApiOrder order(d.dev, s);
    const int64_t rest_bytes = align128(2 * T * top_k * ldh);
    void *ws = nullptr;
    if ((st = gp::api_workspace(d.dev, s, rest_bytes + (flat ? 0 : 4 * T * top_k * C), &ws)) != GEMMPIPE_OK) return st;
    float *parts = reinterpret_cast<float *>(static_cast<char *>(ws) + rest_bytes);
    up.rest = static_cast<uint16_t *>(ws);
    down.X2 = up.rest;
    if (!flat) {
        down.out = parts;
        down.ldo = C;
    }
    return gp::api_launch(true, s, flat ? 2 : 3, [&] {
        cudaError_t e = launch(lu, up, s);
        if (e == cudaSuccess) e = launch(ld, down, s);
        if (e == cudaSuccess && !flat)
            e = gp::launch_few_combine(bf16, static_cast<int>(T), static_cast<int>(top_k), static_cast<int>(E), C,
                                       experts, parts, Y, ldy, s);
        return e;
    });
}

}  // namespace

extern "C" {

gemmpipe_status_t gemm_rows4(int type, int64_t M, int64_t N, int64_t K, int64_t group, const void *X, int64_t ldx,
                             const uint32_t *Q, const void *S, void *Y, int64_t ldy, gemmpipe_stream_t stream)
{
    return guarded([&] {
        if (bad_type(type) || M < 0 || M > gp::kFewRows || bad_matrices(1, K, N) || bad_group(group) ||
            bad_pitch(K, ldx) || bad_pitch(N, ldy))
            return GEMMPIPE_ERR_INVALID_VALUE;
        if (M == 0 || N == 0) return GEMMPIPE_OK;
        if (bad_pointer(Y, 2) || (K > 0 && (bad_pointer(X, 2) || bad_pointer(Q, 16) || bad_pointer(S, 8))))
            return GEMMPIPE_ERR_INVALID_VALUE;
        ApiDevice d;
        gemmpipe_status_t st = gp::api_device(&d);
        if (st != GEMMPIPE_OK) return st;
        if ((st = check_all({{Y, 2}})) != GEMMPIPE_OK) return st;
        cudaStream_t s = stream_of(stream);
        if (K == 0) return zero_rows(Y, M, N, ldy, s);
        if ((st = check_all({{X, 2}, {Q, 16}, {S, 8}})) != GEMMPIPE_OK) return st;
        const bool bf16 = type == GEMMPIPE_BF16;
        if (wide_rows4(M, N, K, group, X, ldx))
            return rows4_wide(bf16, M, N, K, group, static_cast<const uint16_t *>(X), ldx, Q,
                              static_cast<const uint16_t *>(S), static_cast<uint16_t *>(Y), ldy, s);
        FewParams p;
        std::memset(&p, 0, sizeof(p));
        p.X = static_cast<const uint16_t *>(X);
        p.ldx = ldx;
        p.W[0] = Q;
        p.S[0] = static_cast<const uint16_t *>(S);
        p.matrices = 1;
        p.out = static_cast<uint16_t *>(Y);
        p.ldo = ldy;
        p.K = K;
        p.N = p.out_cols = N;
        p.tokens = static_cast<int>(M);
        p.top_k = 1;
        p.experts = 1;
        p.group_steps = static_cast<int>(group / 32);
        const bool off = misaligned(X, 16) || ldx % 8 || K % 8;
        const FewLaunch l = few_launch(&p, bf16, true, off, gp::kFewUp);
        if (l.status != GEMMPIPE_OK) return l.status;
        return gp::api_launch(true, s, 1, [&] { return launch(l, p, s); });
    });
}

gemmpipe_status_t gemmpipe_expert_step(int type, int64_t T, int64_t top_k, int64_t E, int64_t C, int64_t H,
                                       const void *X, int64_t ldx, const int32_t *experts, const float *weights,
                                       const void *W1, const void *W2, const void *W3, void *hidden, void *Y,
                                       int64_t ldy, gemmpipe_stream_t stream)
{
    return guarded([&] {
        const Matrices m{{W1, W2, W3}, {nullptr, nullptr, nullptr}, 0};
        return expert_step(type, T, top_k, E, C, H, static_cast<const uint16_t *>(X), ldx, experts, weights, m,
                           static_cast<uint16_t *>(hidden), static_cast<uint16_t *>(Y), ldy, stream);
    });
}

gemmpipe_status_t gemmpipe_expert_step4(int type, int64_t T, int64_t top_k, int64_t E, int64_t C, int64_t H,
                                        int64_t group, const void *X, int64_t ldx, const int32_t *experts,
                                        const float *weights, const uint32_t *Q1, const void *S1, const uint32_t *Q2,
                                        const void *S2, const uint32_t *Q3, const void *S3, void *hidden, void *Y,
                                        int64_t ldy, gemmpipe_stream_t stream)
{
    return guarded([&] {
        if (bad_group(group)) return GEMMPIPE_ERR_INVALID_VALUE;
        const Matrices m{{Q1, Q2, Q3},
                         {static_cast<const uint16_t *>(S1), static_cast<const uint16_t *>(S2),
                          static_cast<const uint16_t *>(S3)},
                         group};
        return expert_step(type, T, top_k, E, C, H, static_cast<const uint16_t *>(X), ldx, experts, weights, m,
                           static_cast<uint16_t *>(hidden), static_cast<uint16_t *>(Y), ldy, stream);
    });
}

gemmpipe_status_t gemmpipe_pack4(int type, int64_t E, int64_t K, int64_t N, int64_t group, const void *W, uint32_t *Q,
                                 void *S, gemmpipe_stream_t stream)
{
    return guarded([&] {
        if (bad_type(type) || bad_experts(E) || bad_matrices(E, K, N) || bad_group(group))
            return GEMMPIPE_ERR_INVALID_VALUE;
        if (K == 0 || N == 0) return GEMMPIPE_OK;
        if (bad_pointer(W, 2) || bad_pointer(Q, 16) || bad_pointer(S, 8)) return GEMMPIPE_ERR_INVALID_VALUE;
        ApiDevice d;
        gemmpipe_status_t st = gp::api_device(&d);
        if (st != GEMMPIPE_OK) return st;
        if ((st = check_all({{W, 2}, {Q, 16}, {S, 8}})) != GEMMPIPE_OK) return st;
        cudaStream_t s = stream_of(stream);
        return gp::api_launch(false, s, 1, [&] {
            return gp::launch_pack4(type == GEMMPIPE_BF16, E, K, N, static_cast<int>(group),
                                    static_cast<const uint16_t *>(W), Q, static_cast<uint16_t *>(S), s);
        });
    });
}

gemmpipe_status_t gemmpipe_unpack4(int type, int64_t E, int64_t K, int64_t N, int64_t group, const uint32_t *Q,
                                   const void *S, void *W, gemmpipe_stream_t stream)
{
    return guarded([&] {
        if (bad_type(type) || bad_experts(E) || bad_matrices(E, K, N) || bad_group(group))
            return GEMMPIPE_ERR_INVALID_VALUE;
        if (K == 0 || N == 0) return GEMMPIPE_OK;
        if (bad_pointer(W, 2) || bad_pointer(Q, 16) || bad_pointer(S, 8)) return GEMMPIPE_ERR_INVALID_VALUE;
        ApiDevice d;
        gemmpipe_status_t st = gp::api_device(&d);
        if (st != GEMMPIPE_OK) return st;
        if ((st = check_all({{W, 2}, {Q, 16}, {S, 8}})) != GEMMPIPE_OK) return st;
        cudaStream_t s = stream_of(stream);
        return gp::api_launch(false, s, 1, [&] {
            return gp::launch_unpack4(type == GEMMPIPE_BF16, E, K, N, static_cast<int>(group), Q,
                                      static_cast<const uint16_t *>(S), static_cast<uint16_t *>(W), s);
        });
    });
}

}  // extern "C"
