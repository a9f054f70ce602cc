// experts_api.cpp -- the expert-layer entry points of include/gemmpipe.h:
// argument checks, choice of the kernel variant, tensor maps and workspaces.
#include "gemmpipe.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>
#include <initializer_list>
#include <utility>

#include "api_internal.h"
#include "experts.h"
#include "variants.h"

namespace {

using gp::ApiDevice;
using gp::GroupedParams;
using gp::GroupedVariant;

constexpr int64_t kMaxDim = 2147483647;
constexpr int64_t kMaxElems = int64_t(1) << 56;

bool misaligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

bool bad_dim(int64_t v) { return v < 0 || v > kMaxDim; }

// A matrix of `rows` rows of `width` elements, `ld` apart.
bool bad_matrix(int64_t rows, int64_t width, int64_t ld)
{
    return bad_dim(rows) || bad_dim(width) || ld < width || ld > kMaxDim || (ld > 0 && rows > kMaxElems / ld);
}

bool bad_type(int type) { return type != GEMMPIPE_F16 && type != GEMMPIPE_BF16; }

// Null or misaligned where something is to be read or written.
bool bad_pointer(const void *p, int bytes) { return !p || misaligned(p, bytes); }

constexpr int64_t kMaxWidth = int64_t(1) << 30;  // elements of a row of the rows' operators (32-bit places)

// Rows in 8 bits: a block takes 8192 values of a row of many.
bool bad_kept(int64_t rows, int64_t width, int64_t ld)
{
    return width > kMaxWidth || bad_matrix(rows, width, ld) || (rows > 0 && (width + 7) / 8192 + 1 > kMaxDim / rows);
}

// ----------------------------------------------------------- routing, rows

struct Tokens {
    int64_t T, k, R;
};

bool bad_tokens(int64_t T, int64_t top_k, Tokens *t)
{
    if (bad_dim(T) || top_k < 1 || top_k > gp::kMaxTopK || T > kMaxDim / top_k) return true;
    *t = Tokens{T, top_k, T * top_k};
    return false;
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

// --------------------------------------------------------- grouped products

struct Rows {         // a 16-bit row operand
    const uint16_t *p;
    int64_t width, ld;
};

bool tma_ok(const void *p, int64_t ld) { return !misaligned(p, 16) && ld % 8 == 0; }
int64_t round64(int64_t x) { return (x + 63) / 64 * 64; }
constexpr int64_t kLeastSplit = 2048;  // rows of a part, at least: a part costs about 4 us more than its products

int64_t round8(int64_t x) { return (x + 7) / 8 * 8; }
int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// An operand that TMA cannot describe, to be copied to `to` in the workspace
// with its pitch rounded up to 16 bytes.
struct Pad {
    const uint16_t *from;
    int64_t rows, width, ld;
    uint16_t *to;
    const int32_t *offsets;  // weights of few rows: only the experts that have any
    int64_t per_expert;
};

// Dense operands go two to a launch: 16372 rows and 24 x 4107 weight rows of
// 1001 columns in 73 us, 82 us one by one.
gemmpipe_status_t pad_operands(Pad *pads, int n, const ApiDevice &d, cudaStream_t s)
{
    gemmpipe_status_t st = GEMMPIPE_OK;
    int dense = 0;
    for (int i = 0; i < n && st == GEMMPIPE_OK; ++i) {
        const Pad p = pads[i];
        if (p.ld == p.width && !p.offsets) {
            pads[dense++] = p;
        } else {
            st = gp::api_launch(false, s, 1, [&] {
                return gp::launch_repitch(p.from, p.rows, p.width, p.ld, p.to, round8(p.width), p.offsets,
                                          p.per_expert, s);
            });
        }
    }
    if (dense == 0 || st != GEMMPIPE_OK) return st;
    const Pad a = pads[0], b = dense > 1 ? pads[1] : Pad{a.from, 0, 0, 0, a.to, nullptr, 1};
    return gp::api_launch(false, s, 1, [&] {
        return gp::launch_pad_f16(a.from, a.rows, a.width, a.to, round8(a.width), b.from, b.rows, b.width, b.to,
                                  dense > 1 ? round8(b.width) : 8, d.sms, s);
    });
}

// 64 elements x box_rows rows of a row operand.
bool encode_rows(CUtensorMap *m, bool bf16, const Rows &r, int64_t rows, uint32_t box_rows)
{
    const uint64_t dims[2] = {static_cast<uint64_t>(r.width), static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {static_cast<uint64_t>(r.ld) * 2};
    const uint32_t box[2] = {64, box_rows};
    return gp::api_encode_16bit(m, bf16, 2, r.p, dims, strides, box);
}

// The same as 64-element groups, `groups` of them in one copy (width a
// multiple of 64).
bool encode_row_groups(CUtensorMap *m, bool bf16, const Rows &r, int64_t rows, uint32_t groups)
{
    const uint64_t dims[3] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(r.width / 64)};
    const uint64_t strides[2] = {static_cast<uint64_t>(r.ld) * 2, 128};
    const uint32_t box[3] = {64, 64, groups};
    return gp::api_encode_16bit(m, bf16, 3, r.p, dims, strides, box);
}

// Weights experts x rows x width: boxes of 64 elements x box_rows rows of
// one expert, or (grouped) `groups` x 64 elements x box_rows rows in one copy.
bool encode_weights(CUtensorMap *m, bool bf16, const uint16_t *w, int64_t experts, int64_t rows, int64_t width,
                    int64_t ld, uint32_t box_rows)
{
    const uint64_t dims[3] = {static_cast<uint64_t>(width), static_cast<uint64_t>(rows),
                              static_cast<uint64_t>(experts)};
    const uint64_t strides[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(rows * ld) * 2};
    const uint32_t box[3] = {64, box_rows, 1};
    return gp::api_encode_16bit(m, bf16, 3, w, dims, strides, box);
}

bool encode_weight_groups(CUtensorMap *m, bool bf16, const uint16_t *w, int64_t experts, int64_t rows, int64_t width,
                          int64_t ld, uint32_t box_rows, uint32_t groups)
{
    const uint64_t dims[4] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(width / 64),
                              static_cast<uint64_t>(experts)};
    const uint64_t strides[3] = {static_cast<uint64_t>(ld) * 2, 128, static_cast<uint64_t>(rows * ld) * 2};
    const uint32_t box[4] = {64, box_rows, groups, 1};
    return gp::api_encode_16bit(m, bf16, 4, w, dims, strides, box);
}

// Rows per tile, by the mean number of rows of an expert: the bounds are on
// the device, so rows that no expert has and experts without rows count too,
// and rows that fall on a few of many experts get smaller tiles than would be
// best.  Measured on 64 experts of 4096 x 1536 alone, forward (gradient to the
// rows), us:
//   mean    32 rows        64             128            256
//     16    118.6 (122.1)  123.7 (121.5)  122.9 (125.8)  124.8 (128.1)
//     32    129.6 (133.8)  120.6 (124.7)  130.6 (127.3)  126.8 (129.9)
//     64    165.8 (174.7)  134.2 (138.9)  129.4 (134.6)  137.3 (133.6)
//     96    212.1 (223.0)  157.1 (161.6)  141.3 (143.8)  138.6 (137.0)
int rows_per_tile(int64_t R, int64_t E)
{
    const int64_t mean = (R + E - 1) / E;
    return mean <= 16 ? 32 : (mean <= 32 ? 64 : (mean <= 64 ? 128 : 256));
}

struct Product {
    int mode;
    int type;
    int64_t R, N, K, E;  // weights: K x N per expert
    Rows rows;           // X (K wide) or dY (N wide); weight gradient: X
    Rows grad;           // weight gradient: dY
    const uint16_t *W;
    const int32_t *offsets;
    uint16_t *out;
    int64_t ldo;
    // Weight gradient from 8-bit rows: restored into the workspace first.
    const int8_t *Q = nullptr;
    const uint8_t *S = nullptr;
};

gemmpipe_status_t zero_rows(uint16_t *out, int64_t rows, int64_t width, int64_t ld, cudaStream_t s)
{
    const cudaError_t e = cudaMemset2DAsync(out, static_cast<size_t>(ld) * 2, 0, static_cast<size_t>(width) * 2,
                                            static_cast<size_t>(rows), s);
    if (e == cudaSuccess) return GEMMPIPE_OK;
    cudaGetLastError();
    return GEMMPIPE_ERR_LAUNCH;
}

gemmpipe_status_t run_product(Product q, const ApiDevice &d, cudaStream_t s)
{
    const bool weights = q.mode == gp::kWeights, bf16 = q.type == GEMMPIPE_BF16;
    const int64_t features = q.mode == gp::kRowsT ? q.K : q.N;
    // An empty sum leaves zeros.
    if (weights && q.R == 0) return zero_rows(q.out, q.E * q.K, q.N, q.ldo, s);
    if (!weights && (q.mode == gp::kRows ? q.K : q.N) == 0) return zero_rows(q.out, q.R, features, q.ldo, s);

    const int bn = weights ? 256 : rows_per_tile(q.R, q.E);
    // Tiles of all experts, at most (the bounds are on the device).
    const int64_t row_tiles = weights ? q.E * ((q.K + bn - 1) / bn) : q.R / bn + (q.R < q.E ? q.R : q.E);
    // 64-feature tiles where there is an SM for each of them: the rate at
    // which a CTA streams weights is bound by its shared memory.  (Eight rows
    // on 64 experts: 2048 x 1024 8.3 us, 8.6 with 128 features; 8192 x 1024
    // 24.3 and 27.8; 2048 x 1536, 192 tiles of 64, 12.9 and 10.4.)
    const bool narrow = q.mode == gp::kRows && bn == 32 && row_tiles * ((features + 63) / 64) <= d.sms;
    const GroupedVariant *v = gp::grouped_variant(q.mode, bn, bn == 256 ? 256 : (narrow ? 64 : 128));
    if (!v) return GEMMPIPE_ERR_INTERNAL;
    if (v->smem_bytes > d.smem_optin) return GEMMPIPE_ERR_UNSUPPORTED_DEVICE;
    const int64_t f_tiles = (features + v->tile_f - 1) / v->tile_f;
    if (row_tiles > kMaxDim / 4 / f_tiles) return GEMMPIPE_ERR_INVALID_VALUE;

    // Operands that TMA cannot describe are copied to aligned rows.
    const bool pad_x = q.Q == nullptr && !tma_ok(q.rows.p, q.rows.ld);
    const bool pad_g = weights && !tma_ok(q.grad.p, q.grad.ld);
    const bool pad_w = !weights && !tma_ok(q.W, q.N);
    const int64_t wld = pad_w ? round8(q.N) : q.N;
    const int64_t need_x = pad_x || q.Q ? align256(2 * q.R * round8(q.rows.width)) : 0;
    const int64_t need_g = pad_g ? align256(2 * q.R * round8(q.grad.width)) : 0;
    const int64_t need_w = pad_w ? align256(2 * q.E * q.K * wld) : 0;
    // Weight gradient of fewer tiles per matrix than CTA pairs: an expert of
    // far more rows than the others would leave most pairs idle while a few
    // sum them, so sums longer than 1.5 times a pair's even share are split.
    const int64_t units = v->max_units();
    if (units < 1) return GEMMPIPE_ERR_LAUNCH;
    int64_t split_rows = 0, slots = 0;
    const int64_t matrix_tiles = weights ? f_tiles * ((q.K + bn - 1) / bn) : 0;
    if (weights && matrix_tiles < units) {
        split_rows = round64(q.R * matrix_tiles / units + 1);
        if (split_rows < kLeastSplit) split_rows = kLeastSplit;
        slots = (2 * q.R / split_rows + 1) * matrix_tiles;
        if (split_rows + split_rows / 2 >= q.R || slots > gp::kMaxPartSlots) split_rows = slots = 0;
    }
    const gp::ApiOrder order(d.dev, s);
    gemmpipe_status_t st = GEMMPIPE_OK;
    const uint16_t *W = q.W;
    void *ws = nullptr;
    if (need_x + need_g + need_w > 0) {
        if ((st = gp::api_workspace(d.dev, s, need_x + need_g + need_w, &ws)) != GEMMPIPE_OK) return st;
        uint16_t *to_x = static_cast<uint16_t *>(ws), *to_g = to_x + need_x / 2, *to_w = to_g + need_g / 2;
        Pad pads[2];  // of a rows product X or dY, and W; of a weight gradient X and dY
        int n = 0;
        if (pad_x) pads[n++] = Pad{q.rows.p, q.R, q.rows.width, q.rows.ld, to_x, nullptr, 1};
        if (pad_g) pads[n++] = Pad{q.grad.p, q.R, q.grad.width, q.grad.ld, to_g, nullptr, 1};
        // With few rows many experts may have none: their weights stay out
        // (4096 x 1001, 64 experts: one token x 8 61 us, 177 with all copied;
        // 64 tokens, where all experts have rows, 252 either way).
        if (pad_w) pads[n++] = Pad{q.W, q.E * q.K, q.N, q.N, to_w, bn == 32 ? q.offsets : nullptr, q.K};
        if ((st = pad_operands(pads, n, d, s)) != GEMMPIPE_OK) return st;
        if (q.Q) {
            st = gp::api_launch(false, s, 1, [&] {
                return gp::launch_restore8(bf16, q.R, q.K, q.Q, q.S, to_x, round8(q.K), s);
            });
            if (st != GEMMPIPE_OK) return st;
        }
        if (need_x) q.rows = Rows{to_x, q.rows.width, round8(q.rows.width)};
        if (pad_g) q.grad = Rows{to_g, q.grad.width, round8(q.grad.width)};
        if (pad_w) W = to_w;
    }

    GroupedParams p;
    std::memset(&p, 0, sizeof(p));
    gp::GroupedMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    CUtensorMap *m = maps.m;
    bool ok = true;
    if (weights) {
        p.a_groups = q.grad.width % 64 == 0;
        p.b_groups = q.rows.width % 64 == 0;
        ok = (p.a_groups ? encode_row_groups(&m[gp::kMapA], bf16, q.grad, q.R, 2)
                         : encode_rows(&m[gp::kMapA], bf16, q.grad, q.R, 64)) &&
             (p.b_groups ? encode_row_groups(&m[gp::kMapB], bf16, q.rows, q.R, v->cta_bn / 64)
                         : encode_rows(&m[gp::kMapB], bf16, q.rows, q.R, 64));
        const uint32_t last[2] = {4, 1};
        for (int i = 0; i < 2 && ok; ++i)
            ok = encode_rows(&m[gp::kMapALast + i], bf16, q.grad, q.R, last[i]) &&
                 encode_rows(&m[gp::kMapBLast + i], bf16, q.rows, q.R, last[i]);
        p.out_rows = q.K;
    } else {
        p.a_groups = q.mode == gp::kRows && q.N % 64 == 0;
        ok = (p.a_groups ? encode_weight_groups(&m[gp::kMapA], bf16, W, q.E, q.K, q.N, wld, v->bk, v->tile_f / (v->pair ? 128 : 64))
                         : encode_weights(&m[gp::kMapA], bf16, W, q.E, q.K, q.N, wld, q.mode == gp::kRows ? v->bk : 128)) &&
             encode_rows(&m[gp::kMapB], bf16, q.rows, q.R, v->cta_bn) &&
             encode_rows(&m[gp::kMapBPart], bf16, q.rows, q.R, v->b_part);
        p.depth = q.mode == gp::kRows ? q.K : q.N;
    }
    if (!ok) return GEMMPIPE_ERR_INTERNAL;
    p.offsets = q.offsets;
    p.experts = static_cast<int>(q.E);
    p.rows = q.R;
    p.features = features;
    p.out = q.out;
    p.ldo = q.ldo;
    p.bf16 = bf16 ? 1 : 0;
    p.vec_store = tma_ok(q.out, q.ldo) ? 1 : 0;
    p.timeout_ns = 2000000000ull + static_cast<uint64_t>((weights ? q.R : p.depth) / 64 + 1) * 10000ull;
    p.stall_kb = gp::api_take_stall(&p.timeout_ns);
    if (split_rows > 0) {
        // A count per slot and epilogue warp of both CTAs, the launch's
        // number, then 256 KiB a slot, on 4 KiB (on 256 bytes 2 experts of
        // 20000 rows, 512 x 512, take 49.4 us where this takes 47.7).
        constexpr int64_t kCounts = gp::kMaxPartSlots * 16 * 8, kHead = kCounts + 4096;
        void *parts = nullptr;
        if ((st = gp::api_parts_workspace(d.dev, s, kHead, slots * 256 * 256 * 4, &parts)) != GEMMPIPE_OK) return st;
        char *base = static_cast<char *>(parts);
        p.part_counts = reinterpret_cast<unsigned long long *>(base);
        p.launch = reinterpret_cast<uint32_t *>(base + kCounts);
        p.parts = reinterpret_cast<float *>(base + kHead);
        p.split_rows = static_cast<int32_t>(split_rows);
    }
    if (gp::status_word(&p.status) != cudaSuccess) {
        cudaGetLastError();
        return GEMMPIPE_ERR_LAUNCH;
    }
    // Tiles at most: whole sums, and the parts of split ones.
    const int64_t tiles = row_tiles * f_tiles + slots;
    p.sorted = weights && tiles > units && q.E > 1 && q.E <= gp::kMaxSorted ? 1 : 0;
    const int grid = static_cast<int>((v->pair ? 2 : 1) * (tiles < units ? tiles : units));
    return gp::api_launch(true, s, 1, [&] { return v->launch(maps, p, grid, s); });
}

// Sizes common to the grouped products.  The kernel counts rows and features
// in 32 bits, up to a tile past the last one.
bool bad_product(int type, int64_t R, int64_t N, int64_t K, int64_t E)
{
    constexpr int64_t kMost = kMaxDim - 1023;
    return bad_type(type) || bad_dim(R) || bad_dim(N) || bad_dim(K) || R > kMost || N > kMost || K > kMost || E < 1 || E > gp::kMaxExperts ||
           (N > 0 && K > kMaxElems / (E * (N + 8)));
}

cudaStream_t stream_of(gemmpipe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Nothing thrown (allocation of the library's own tables) leaves an entry point.
template <class F>
gemmpipe_status_t guarded(F f)
{
    try {
        return f();
    } catch (...) {
        return GEMMPIPE_ERR_INTERNAL;
    }
}

gemmpipe_status_t rows_product(int mode, int type, int64_t R, int64_t N, int64_t K, int64_t E, const uint16_t *in,
                               int64_t ldi, const int32_t *offsets, const uint16_t *W, uint16_t *out, int64_t ldo,
                               gemmpipe_stream_t stream)
{
    const int64_t wi = mode == gp::kRows ? K : N, wo = mode == gp::kRows ? N : K;
    if (bad_product(type, R, N, K, E) || bad_matrix(R, wi, ldi) || bad_matrix(R, wo, ldo))
        return GEMMPIPE_ERR_INVALID_VALUE;
    if (R == 0 || wo == 0) return GEMMPIPE_OK;
    if (bad_pointer(out, 2) || bad_pointer(offsets, 4) || (wi > 0 && (bad_pointer(in, 2) || bad_pointer(W, 2))))
        return GEMMPIPE_ERR_INVALID_VALUE;
    ApiDevice d;
    gemmpipe_status_t st = gp::api_device(&d);
    if (st != GEMMPIPE_OK) return st;
    if ((st = check_all({{out, 2}, {offsets, 4}})) != GEMMPIPE_OK) return st;
    if (wi > 0 && (st = check_all({{in, 2}, {W, 2}})) != GEMMPIPE_OK) return st;
    Product q{};
    q.mode = mode;
    q.type = type;
    q.R = R;
    q.N = N;
    q.K = K;
    q.E = E;
    q.rows = Rows{in, wi, ldi};
    q.W = W;
    q.offsets = offsets;
    q.out = out;
    q.ldo = ldo;
    return run_product(q, d, stream_of(stream));
}

gemmpipe_status_t weights_product(int type, int64_t R, int64_t N, int64_t K, int64_t E, const uint16_t *X,
                                  int64_t ldx, const int8_t *Q, const uint8_t *S, bool kept, const uint16_t *dY,
                                  int64_t lddy, const int32_t *offsets, uint16_t *dW, gemmpipe_stream_t stream)
{
    if (bad_product(type, R, N, K, E) || bad_matrix(R, K, ldx) || bad_matrix(R, N, lddy) ||
        (kept && bad_kept(R, K, K)))
        return GEMMPIPE_ERR_INVALID_VALUE;
    if (N == 0 || K == 0) return GEMMPIPE_OK;
    if (bad_pointer(dW, 2) || bad_pointer(offsets, 4)) return GEMMPIPE_ERR_INVALID_VALUE;
    if (R > 0 && (bad_pointer(dY, 2) || (kept ? !Q || !S : bad_pointer(X, 2)))) return GEMMPIPE_ERR_INVALID_VALUE;
    ApiDevice d;
    gemmpipe_status_t st = gp::api_device(&d);
    if (st != GEMMPIPE_OK) return st;
    if ((st = check_all({{dW, 2}, {offsets, 4}})) != GEMMPIPE_OK) return st;
    if (R > 0 && (st = kept ? check_all({{dY, 2}, {Q, 1}, {S, 1}}) : check_all({{dY, 2}, {X, 2}})) != GEMMPIPE_OK)
        return st;
    Product q{};
    q.mode = gp::kWeights;
    q.type = type;
    q.R = R;
    q.N = N;
    q.K = K;
    q.E = E;
    q.rows = Rows{X, K, ldx};
    q.grad = Rows{dY, N, lddy};
    q.offsets = offsets;
    q.out = dW;
    q.ldo = N;
    q.Q = kept ? Q : nullptr;
    q.S = S;
    return run_product(q, d, stream_of(stream));
}

}  // namespace

extern "C" {

gemmpipe_status_t gemmpipe_route(int64_t T, int64_t top_k, int64_t E, const int32_t *experts, int32_t *offsets,
                                 int32_t *slots, int32_t *rows, gemmpipe_stream_t stream)
{
    return guarded([&] {
        Tokens t;
        if (bad_tokens(T, top_k, &t) || E < 1 || E > gp::kMaxExperts || bad_pointer(offsets, 4))
            return GEMMPIPE_ERR_INVALID_VALUE;
        if (t.R > 0 && (bad_pointer(experts, 4) || bad_pointer(slots, 4) || bad_pointer(rows, 4)))
            return GEMMPIPE_ERR_INVALID_VALUE;
        ApiDevice d;
        gemmpipe_status_t st = gp::api_device(&d);
        if (st != GEMMPIPE_OK) return st;
        if ((st = check_all({{offsets, 4}})) != GEMMPIPE_OK) return st;
        cudaStream_t s = stream_of(stream);
        if (t.R == 0) return zero_rows(reinterpret_cast<uint16_t *>(offsets), 1, 2 * (E + 1), 2 * (E + 1), s);
        if ((st = check_all({{experts, 4}, {slots, 4}, {rows, 4}})) != GEMMPIPE_OK) return st;
        const gp::ApiOrder order(d.dev, s);
        void *ws = nullptr;
        const int64_t bytes = gp::route_scratch_bytes(t.R, static_cast<int>(E));
        if (bytes > 0 && (st = gp::api_workspace(d.dev, s, bytes, &ws)) != GEMMPIPE_OK) return st;
        return gp::api_launch(false, s, gp::route_kernels(t.R), [&] {
            return gp::launch_route(t.R, static_cast<int>(E), experts, offsets, slots, rows,
                                    static_cast<int32_t *>(ws), s);
        });
    });
}

gemmpipe_status_t gemmpipe_dispatch(int type, int64_t T, int64_t top_k, int64_t C, const void *X, int64_t ldx,
                                    const int32_t *rows, const float *weights, void *Xs, int64_t ldxs,
                                    gemmpipe_stream_t stream)
{
    return guarded([&] {
        Tokens t;
        if (bad_type(type) || bad_tokens(T, top_k, &t) || C > kMaxWidth || bad_matrix(T, C, ldx) ||
            bad_matrix(t.R, C, ldxs))
            return GEMMPIPE_ERR_INVALID_VALUE;
        if (T == 0 || C == 0) return GEMMPIPE_OK;
        if (bad_pointer(X, 2) || bad_pointer(Xs, 2) || bad_pointer(rows, 4) || misaligned(weights, 4))
            return GEMMPIPE_ERR_INVALID_VALUE;
        ApiDevice d;
        gemmpipe_status_t st = gp::api_device(&d);
        if (st != GEMMPIPE_OK) return st;
        if ((st = check_all({{X, 2}, {Xs, 2}, {rows, 4}, {weights, 4}})) != GEMMPIPE_OK) return st;
        cudaStream_t s = stream_of(stream);
        return gp::api_launch(false, s, 1, [&] {
            return gp::launch_dispatch(type == GEMMPIPE_BF16, T, static_cast<int>(top_k), C,
                                       static_cast<const uint16_t *>(X), ldx, rows, weights,
                                       static_cast<uint16_t *>(Xs), ldxs, s);
        });
    });
}

gemmpipe_status_t gemmpipe_combine(int type, int64_t T, int64_t top_k, int64_t C, const void *Ys, int64_t ldys,
                                   const int32_t *rows, const float *weights, void *Y, int64_t ldy,
                                   gemmpipe_stream_t stream)
{
    return guarded([&] {
        Tokens t;
        if (bad_type(type) || bad_tokens(T, top_k, &t) || C > kMaxWidth || bad_matrix(t.R, C, ldys) ||
            bad_matrix(T, C, ldy))
            return GEMMPIPE_ERR_INVALID_VALUE;
        if (T == 0 || C == 0) return GEMMPIPE_OK;
        if (bad_pointer(Ys, 2) || bad_pointer(Y, 2) || bad_pointer(rows, 4) || misaligned(weights, 4))
            return GEMMPIPE_ERR_INVALID_VALUE;
        ApiDevice d;
        gemmpipe_status_t st = gp::api_device(&d);
        if (st != GEMMPIPE_OK) return st;
        if ((st = check_all({{Ys, 2}, {Y, 2}, {rows, 4}, {weights, 4}})) != GEMMPIPE_OK) return st;
        cudaStream_t s = stream_of(stream);
        return gp::api_launch(false, s, 1, [&] {
            return gp::launch_combine(type == GEMMPIPE_BF16, T, static_cast<int>(top_k), C,
                                      static_cast<const uint16_t *>(Ys), ldys, rows, weights,
                                      static_cast<uint16_t *>(Y), ldy, s);
        });
    });
}

gemmpipe_status_t gemmpipe_combine_grad(int type, int64_t T, int64_t top_k, int64_t C, const void *dY, int64_t lddy,
                                        const void *Ys, int64_t ldys, const int32_t *rows, const float *weights,
                                        void *dYs, int64_t lddys, float *dweights, gemmpipe_stream_t stream)
{
    return guarded([&] {
        Tokens t;
        if (bad_type(type) || bad_tokens(T, top_k, &t) || C > kMaxWidth || bad_matrix(T, C, lddy) ||
            bad_matrix(t.R, C, ldys) || bad_matrix(t.R, C, lddys))
            return GEMMPIPE_ERR_INVALID_VALUE;
        if (T == 0) return GEMMPIPE_OK;
        if (bad_pointer(rows, 4) || misaligned(weights, 4) || bad_pointer(dweights, 4))
            return GEMMPIPE_ERR_INVALID_VALUE;
        if (C > 0 && (bad_pointer(dY, 2) || bad_pointer(Ys, 2) || bad_pointer(dYs, 2)))
            return GEMMPIPE_ERR_INVALID_VALUE;
        ApiDevice d;
        gemmpipe_status_t st = gp::api_device(&d);
        if (st != GEMMPIPE_OK) return st;
        if ((st = check_all({{rows, 4}, {weights, 4}, {dweights, 4}})) != GEMMPIPE_OK) return st;
        if (C > 0 && (st = check_all({{dY, 2}, {Ys, 2}, {dYs, 2}})) != GEMMPIPE_OK) return st;
        cudaStream_t s = stream_of(stream);
        return gp::api_launch(false, s, 1, [&] {
            return gp::launch_combine_grad(type == GEMMPIPE_BF16, T, static_cast<int>(top_k), C,
                                           static_cast<const uint16_t *>(dY), lddy, static_cast<const uint16_t *>(Ys),
                                           ldys, rows, weights, static_cast<uint16_t *>(dYs), lddys, dweights, s);
        });
    });
}

gemmpipe_status_t gemm_grouped(int type, int64_t R, int64_t N, int64_t K, int64_t E, const void *X, int64_t ldx,
                               const int32_t *offsets, const void *W, void *Y, int64_t ldy, gemmpipe_stream_t stream)
{
    return guarded([&] {
        return rows_product(gp::kRows, type, R, N, K, E, static_cast<const uint16_t *>(X), ldx, offsets,
                            static_cast<const uint16_t *>(W), static_cast<uint16_t *>(Y), ldy, stream);
    });
}

gemmpipe_status_t gemm_grouped_dx(int type, int64_t R, int64_t N, int64_t K, int64_t E, const void *dY, int64_t lddy,
                                  const int32_t *offsets, const void *W, void *dX, int64_t lddx,
                                  gemmpipe_stream_t stream)
{
    return guarded([&] {
        return rows_product(gp::kRowsT, type, R, N, K, E, static_cast<const uint16_t *>(dY), lddy, offsets,
                            static_cast<const uint16_t *>(W), static_cast<uint16_t *>(dX), lddx, stream);
    });
}

gemmpipe_status_t gemm_grouped_dw(int type, int64_t R, int64_t N, int64_t K, int64_t E, const void *X, int64_t ldx,
                                  const void *dY, int64_t lddy, const int32_t *offsets, void *dW,
                                  gemmpipe_stream_t stream)
{
    return guarded([&] {
        return weights_product(type, R, N, K, E, static_cast<const uint16_t *>(X), ldx, nullptr, nullptr, false,
                               static_cast<const uint16_t *>(dY), lddy, offsets, static_cast<uint16_t *>(dW), stream);
    });
}

gemmpipe_status_t gemm_grouped_dw8(int type, int64_t R, int64_t N, int64_t K, int64_t E, const int8_t *Q,
                                   const uint8_t *S, const void *dY, int64_t lddy, const int32_t *offsets, void *dW,
                                   gemmpipe_stream_t stream)
{
    return guarded([&] {
        return weights_product(type, R, N, K, E, nullptr, K, Q, S, true, static_cast<const uint16_t *>(dY), lddy,
                               offsets, static_cast<uint16_t *>(dW), stream);
    });
}

gemmpipe_status_t gemmpipe_keep8(int type, int64_t R, int64_t C, const void *X, int64_t ldx, int8_t *Q, uint8_t *S,
                                 gemmpipe_stream_t stream)
{
    return guarded([&] {
        if (bad_type(type) || bad_kept(R, C, ldx)) return GEMMPIPE_ERR_INVALID_VALUE;
        if (R == 0 || C == 0) return GEMMPIPE_OK;
        if (bad_pointer(X, 2) || !Q || !S) return GEMMPIPE_ERR_INVALID_VALUE;
        ApiDevice d;
        gemmpipe_status_t st = gp::api_device(&d);
        if (st != GEMMPIPE_OK) return st;
        if ((st = check_all({{X, 2}, {Q, 1}, {S, 1}})) != GEMMPIPE_OK) return st;
        cudaStream_t s = stream_of(stream);
        return gp::api_launch(false, s, 1, [&] {
            return gp::launch_keep8(type == GEMMPIPE_BF16, R, C, static_cast<const uint16_t *>(X), ldx, Q, S, s);
        });
    });
}

gemmpipe_status_t gemmpipe_restore8(int type, int64_t R, int64_t C, const int8_t *Q, const uint8_t *S, void *X,
                                    int64_t ldx, gemmpipe_stream_t stream)
{
    return guarded([&] {
        if (bad_type(type) || bad_kept(R, C, ldx)) return GEMMPIPE_ERR_INVALID_VALUE;
        if (R == 0 || C == 0) return GEMMPIPE_OK;
        if (bad_pointer(X, 2) || !Q || !S) return GEMMPIPE_ERR_INVALID_VALUE;
        ApiDevice d;
        gemmpipe_status_t st = gp::api_device(&d);
        if (st != GEMMPIPE_OK) return st;
        if ((st = check_all({{X, 2}, {Q, 1}, {S, 1}})) != GEMMPIPE_OK) return st;
        cudaStream_t s = stream_of(stream);
        return gp::api_launch(false, s, 1, [&] {
            return gp::launch_restore8(type == GEMMPIPE_BF16, R, C, Q, S, static_cast<uint16_t *>(X), ldx, s);
        });
    });
}

}  // extern "C"
