// Host-side argument checks for the C ABI in include/q8_linear.h.
//
// Pure C++ (no HIP): every check runs before anything is enqueued, and the same
// header builds with g++ for CPU-only tests.  Each function returns Q8_OK or the
// error code, and writes a description into `msg` (capacity `cap`).
#pragma once

#include <stdint.h>
#include <stdio.h>

#include "../../include/q8_linear.h"

namespace q8v {

constexpr int64_t kQK = 32;           // quants per Q8_0 block
constexpr int64_t kBlockBytes = 34;   // binary16 scale + 32 int8
constexpr int64_t kKAlign = 256;      // K multiple: 8 blocks = 272 bytes = 17 x 16 bytes
constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxExperts = 256;
constexpr int64_t kMoeMaxDim = 16384;  // one staged activation row fits in 64 KB of LDS

inline int64_t row_bytes(int64_t k) { return (k / kQK) * kBlockBytes; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline q8_status fail(char* msg, size_t cap, q8_status s, const char* fmt, long long a = 0, long long b = 0) {
    if (msg && cap) snprintf(msg, cap, fmt, a, b);
    return s;
}

// K (or H, F) of a Q8_0 operand.
inline q8_status check_k(const char* what, int64_t k, char* msg, size_t cap) {
    if (k <= 0 || k > kMaxDim || k % kKAlign != 0) {
        if (msg && cap) snprintf(msg, cap, "%s=%lld must be a positive multiple of 256 (at most 2^30)", what, (long long)k);
        return Q8_ERR_SHAPE;
    }
    return Q8_OK;
}

inline q8_status check_dim(const char* what, int64_t v, char* msg, size_t cap) {
    if (v < 0 || v > kMaxDim) {
        if (msg && cap) snprintf(msg, cap, "%s=%lld out of range [0, 2^30]", what, (long long)v);
        return Q8_ERR_SHAPE;
    }
    return Q8_OK;
}

// Shared by q8_linear (n_out = n) and the fused gate_up call (n_out = f, weight rows 2f).
inline q8_status check_linear(const void* w, int64_t n_out, int64_t k, const float* x, int64_t m, int64_t ldx,
                              const float* y, int64_t ldy, char* msg, size_t cap) {
    q8_status s;
    if ((s = check_dim("n", n_out, msg, cap)) != Q8_OK) return s;
    if ((s = check_dim("m", m, msg, cap)) != Q8_OK) return s;
    if ((s = check_k("k", k, msg, cap)) != Q8_OK) return s;
    if (ldx < k) return fail(msg, cap, Q8_ERR_SHAPE, "ldx=%lld < k=%lld", ldx, k);
    if (ldy < n_out) return fail(msg, cap, Q8_ERR_SHAPE, "ldy=%lld < n=%lld", ldy, n_out);
    if (ldx > kMaxDim || ldy > kMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "leading dimension above 2^30");
    if (m == 0 || n_out == 0) return Q8_OK;  // nothing to do; pointers may be anything
    if (!w || !x || !y) return fail(msg, cap, Q8_ERR_NULL, "null pointer (w, x or y)");
    if (!aligned(w, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "weight pointer not 16-byte aligned");
    if (!aligned(x, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "x pointer not 16-byte aligned");
    if (ldx % 4 != 0) return fail(msg, cap, Q8_ERR_ALIGN, "ldx=%lld not a multiple of 4", ldx);
    if (!aligned(y, 4)) return fail(msg, cap, Q8_ERR_ALIGN, "output pointer not 4-byte aligned");
    return Q8_OK;
}

// The integer q8 x q8 linears: codes xq [m][k] and scales xd [m][k/32], contiguous.
inline q8_status check_linear_q8act(const void* w, int64_t n_out, int64_t k, const void* xq, const void* xd,
                                    int64_t m, const float* y, int64_t ldy, char* msg, size_t cap) {
    q8_status s;
    if ((s = check_dim("n", n_out, msg, cap)) != Q8_OK) return s;
    if ((s = check_dim("m", m, msg, cap)) != Q8_OK) return s;
    if ((s = check_k("k", k, msg, cap)) != Q8_OK) return s;
    if (ldy < n_out) return fail(msg, cap, Q8_ERR_SHAPE, "ldy=%lld < n=%lld", ldy, n_out);
    if (ldy > kMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "leading dimension above 2^30");
    if (m * k > (int64_t(1) << 40)) return fail(msg, cap, Q8_ERR_SHAPE, "m*k=%lld above 2^40", m * k);
    if (m == 0 || n_out == 0) return Q8_OK;
    if (!w || !xq || !xd || !y) return fail(msg, cap, Q8_ERR_NULL, "null pointer (w, xq, xd or y)");
    if (!aligned(w, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "weight pointer not 16-byte aligned");
    if (!aligned(xq, 16) || !aligned(xd, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "xq or xd not 16-byte aligned");
    if (!aligned(y, 4)) return fail(msg, cap, Q8_ERR_ALIGN, "output pointer not 4-byte aligned");
    return Q8_OK;
}

inline q8_status check_quantize_act(const float* x, int64_t m, int64_t k, int64_t ldx, const void* xq,
                                    const void* xd, char* msg, size_t cap) {
    q8_status s;
    if ((s = check_dim("m", m, msg, cap)) != Q8_OK) return s;
    if ((s = check_k("k", k, msg, cap)) != Q8_OK) return s;
    if (ldx < k || ldx > kMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "ldx=%lld < k=%lld", ldx, k);
    if (m * k > (int64_t(1) << 40)) return fail(msg, cap, Q8_ERR_SHAPE, "m*k=%lld above 2^40", m * k);
    if (m == 0) return Q8_OK;
    if (!x || !xq || !xd) return fail(msg, cap, Q8_ERR_NULL, "null pointer (x, xq or xd)");
    if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(xd, 16))
        return fail(msg, cap, Q8_ERR_ALIGN, "x, xq or xd not 16-byte aligned");
    if (ldx % 4 != 0) return fail(msg, cap, Q8_ERR_ALIGN, "ldx=%lld not a multiple of 4", ldx);
    return Q8_OK;
}

inline q8_status check_route(const float* x, int64_t m, int64_t h, int64_t ldx, const float* w_router, int64_t n_exp,
                             int32_t k, const int32_t* idx, const float* wts, char* msg, size_t cap) {
    q8_status s;
    if ((s = check_dim("m", m, msg, cap)) != Q8_OK) return s;
    if ((s = check_k("h", h, msg, cap)) != Q8_OK) return s;
    if (n_exp < 1 || n_exp > kMaxExperts) return fail(msg, cap, Q8_ERR_SHAPE, "n_exp=%lld out of range [1, 256]", n_exp);
    if (k < 1 || k > n_exp) return fail(msg, cap, Q8_ERR_SHAPE, "k=%lld out of range [1, n_exp=%lld]", k, n_exp);
    if (ldx < h || ldx > kMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "ldx=%lld < h=%lld", ldx, h);
    if (m == 0) return Q8_OK;
    if (!x || !w_router || !idx || !wts) return fail(msg, cap, Q8_ERR_NULL, "null pointer (x, w_router, topk_idx or topk_w)");
    if (!aligned(x, 16) || !aligned(w_router, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "x or w_router not 16-byte aligned");
    if (ldx % 4 != 0) return fail(msg, cap, Q8_ERR_ALIGN, "ldx=%lld not a multiple of 4", ldx);
    if (!aligned(idx, 4) || !aligned(wts, 4)) return fail(msg, cap, Q8_ERR_ALIGN, "topk outputs not 4-byte aligned");
    return Q8_OK;
}

// Workspace of the two-pass router: the float32 logits [m][n_exp].
inline size_t route_workspace_bytes(int64_t m, int64_t n_exp) {
    const size_t b = sizeof(float) * size_t(m) * size_t(n_exp);
    return b ? (b + 255) / 256 * 256 : 256;
}

inline q8_status check_route_workspace(int64_t m, int64_t n_exp, const void* ws, size_t ws_bytes, char* msg,
                                       size_t cap) {
    if (!ws) return fail(msg, cap, Q8_ERR_WORKSPACE, "workspace is NULL");
    const size_t need = route_workspace_bytes(m, n_exp);
    if (ws_bytes < need) return fail(msg, cap, Q8_ERR_WORKSPACE, "workspace %lld bytes < required %lld", (long long)ws_bytes, (long long)need);
    if (!aligned(ws, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "workspace not 16-byte aligned");
    return Q8_OK;
}

// The grouped MoE call runs on the bf16 matrix cores (expert-grouped 128-row tiles) when
// the routed pairs average at least this many per expert, else on the float32 GEMV
// passes (decode).  Measured on the Qwen3-30B-A3B layer (128 experts): at 4 pairs per
// expert the GEMV passes are faster (about 300 us against 330), at 8 the tiles (333
// against 518 us: the GEMV passes stream an expert's weights once per 4 tokens).
constexpr int64_t kMoeMatrixCorePairsPerExpert = 8;
inline bool moe_uses_matrix_cores(int64_t n_pairs, int64_t n_exp) {
    return n_pairs >= kMoeMatrixCorePairsPerExpert * n_exp;
}

// Workspace of the grouped MoE call: a route plan plus the hidden activations.
struct MoeWorkspace {
    size_t offsets_off, sorted_off, inv_off, active_off, tiles_off, hidden_off, out_off, total;
};

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline MoeWorkspace moe_workspace_layout(int64_t m, int32_t k, int64_t n_exp, int64_t f, int64_t h) {
    MoeWorkspace w{};
    const size_t pairs = size_t(m) * size_t(k);
    size_t off = 0;
    w.offsets_off = off; off = round_up(off + sizeof(int32_t) * size_t(n_exp + 1), 256);
    w.sorted_off = off;  off = round_up(off + sizeof(int32_t) * pairs, 256);
    w.inv_off = off;     off = round_up(off + sizeof(int32_t) * pairs, 256);
    w.active_off = off;  off = round_up(off + sizeof(int32_t) * size_t(n_exp + 1), 256);
    w.tiles_off = off;   off = round_up(off + sizeof(int32_t) * size_t(n_exp + 1), 256);
    w.hidden_off = off;  off = round_up(off + sizeof(float) * pairs * 2 * size_t(f), 256);  // gate and up rows
    w.out_off = off;     off = round_up(off + sizeof(float) * pairs * size_t(h), 256);
    w.total = off;
    return w;
}

// Arguments of the grouped MoE call other than its workspace.
inline q8_status check_moe_args(const void* wgu, const void* wdn, int64_t n_exp, int64_t f, int64_t h, const float* x,
                                int64_t m, int64_t ldx, const int32_t* idx, const float* wts, int32_t k,
                                const float* y, int64_t ldy, char* msg, size_t cap) {
    q8_status s;
    if ((s = check_dim("m", m, msg, cap)) != Q8_OK) return s;
    if ((s = check_k("h", h, msg, cap)) != Q8_OK) return s;
    if ((s = check_k("f", f, msg, cap)) != Q8_OK) return s;
    if (h > kMoeMaxDim || f > kMoeMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "h=%lld and f=%lld must be at most 16384", h, f);
    if (n_exp < 1 || n_exp > kMaxExperts) return fail(msg, cap, Q8_ERR_SHAPE, "n_exp=%lld out of range [1, 256]", n_exp);
    if (k < 1 || k > n_exp) return fail(msg, cap, Q8_ERR_SHAPE, "k=%lld out of range [1, n_exp=%lld]", k, n_exp);
    if (ldx < h || ldx > kMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "ldx=%lld < h=%lld", ldx, h);
    if (ldy < h || ldy > kMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "ldy=%lld < h=%lld", ldy, h);
    if (m * int64_t(k) > (int64_t(1) << 24)) return fail(msg, cap, Q8_ERR_SHAPE, "m*k=%lld above 2^24", m * int64_t(k));
    if (m == 0) return Q8_OK;
    if (!wgu || !wdn || !x || !idx || !wts || !y) return fail(msg, cap, Q8_ERR_NULL, "null pointer among the tensor arguments");
    if (!aligned(wgu, 16) || !aligned(wdn, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "expert stacks not 16-byte aligned");
    if (!aligned(x, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "x not 16-byte aligned");
    if (ldx % 4 != 0) return fail(msg, cap, Q8_ERR_ALIGN, "ldx=%lld not a multiple of 4", ldx);
    if (!aligned(idx, 4) || !aligned(wts, 4) || !aligned(y, 4)) return fail(msg, cap, Q8_ERR_ALIGN, "topk or y not 4-byte aligned");
    return Q8_OK;
}

inline q8_status check_moe(const void* wgu, const void* wdn, int64_t n_exp, int64_t f, int64_t h, const float* x,
                           int64_t m, int64_t ldx, const int32_t* idx, const float* wts, int32_t k, const float* y,
                           int64_t ldy, const void* ws, size_t ws_bytes, char* msg, size_t cap) {
    q8_status s = check_moe_args(wgu, wdn, n_exp, f, h, x, m, ldx, idx, wts, k, y, ldy, msg, cap);
    if (s != Q8_OK || m == 0) return s;
    if (!ws) return fail(msg, cap, Q8_ERR_WORKSPACE, "workspace is NULL");
    const size_t need = moe_workspace_layout(m, k, n_exp, f, h).total;
    if (ws_bytes < need) return fail(msg, cap, Q8_ERR_WORKSPACE, "workspace %lld bytes < required %lld", (long long)ws_bytes, (long long)need);
    if (!aligned(ws, 256)) return fail(msg, cap, Q8_ERR_ALIGN, "workspace not 256-byte aligned");
    return Q8_OK;
}

// ------------------------------------------------------------- low-rank adapters

constexpr int32_t kLoraMaxAdapters = 256;  // bins of the row sort
constexpr int32_t kLoraMaxRank = 256;

// The adapter stack beside a matrix of n rows and width k, for m rows of x.
inline q8_status check_lora(const q8_lora* lo, int64_t n, int64_t m, char* msg, size_t cap) {
    if (!lo) return fail(msg, cap, Q8_ERR_NULL, "lora is NULL");
    if (lo->type < Q8_LORA_F32 || lo->type > Q8_LORA_BF16) return fail(msg, cap, Q8_ERR_SHAPE, "lora type=%lld is none of Q8_LORA_*", lo->type);
    if (lo->n_adapters < 0 || lo->n_adapters > kLoraMaxAdapters)
        return fail(msg, cap, Q8_ERR_SHAPE, "n_adapters=%lld out of range [0, 256]", lo->n_adapters);
    if (lo->rank < 8 || lo->rank > kLoraMaxRank || lo->rank % 8 != 0)
        return fail(msg, cap, Q8_ERR_SHAPE, "rank=%lld must be a multiple of 8 in [8, 256]", lo->rank);
    if (lo->n_sections < 1 || lo->n_sections > Q8_LORA_MAX_SECTIONS)
        return fail(msg, cap, Q8_ERR_SHAPE, "n_sections=%lld out of range [1, 4]", lo->n_sections);
    int64_t sum = 0;
    for (int s = 0; s < lo->n_sections; ++s) {
        if (lo->section_rows[s] < 0 || lo->section_rows[s] > n)
            return fail(msg, cap, Q8_ERR_SHAPE, "a section has %lld rows of %lld", lo->section_rows[s], n);
        sum += lo->section_rows[s];
    }
    if (sum != n) return fail(msg, cap, Q8_ERR_SHAPE, "the sections have %lld rows, the matrix %lld", sum, n);
    if (m == 0 || n == 0 || lo->n_adapters == 0) return Q8_OK;
    if (!lo->a || !lo->b || !lo->adapter) return fail(msg, cap, Q8_ERR_NULL, "null pointer (lora a, b or adapter)");
    if (!aligned(lo->a, 16) || !aligned(lo->b, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "lora a or b not 16-byte aligned");
    if (!aligned(lo->adapter, 4) || !aligned(lo->ranks, 4) || !aligned(lo->scale, 4))
        return fail(msg, cap, Q8_ERR_ALIGN, "lora adapter, ranks or scale not 4-byte aligned");
    return Q8_OK;
}

// What the workspace sizes depend on.
inline bool lora_sizes_valid(const q8_lora& lo) {
    return lo.rank >= 8 && lo.rank <= kLoraMaxRank && lo.rank % 8 == 0 && lo.n_sections >= 1 &&
           lo.n_sections <= Q8_LORA_MAX_SECTIONS;
}

// Rows up to which the packed adapter calls keep float32 accuracy; from here on their
// shared product is q8_linear's, on the bf16 matrix cores.
constexpr int64_t kPrefillRows = 256;

// The matrix-core form of the correction (many rows): rows sorted by adapter in tiles of 64,
// the inner products in parts of k (enough blocks for few tiles).
constexpr int64_t kLoraTiledRows = 48;
inline int64_t lora_max_tiles(int64_t m, int64_t n_adapters) { return m / 64 + (m < n_adapters + 1 ? m : n_adapters + 1); }
// It takes two launches more, the form for few rows reads its adapter for every row: the
// latter is left once those reads would be 160 MB.  Measured, in us, few rows | matrix
// cores, 1 and 32 adapters in use: 6144 x 4096, three sections of rank 16 (0.6 MB a row), 192
// rows 21.5 | 23.1 and 23.6 | 30.3, 384 rows 36.4 | 25.9 and 38.5 | 32.9; of rank 64 (2.4 MB a
// row), 64 rows 24.6 | 32.7 and 29.7 | 51.0, 128 rows 44.7 | 35.3 and 50.5 | 53.1; 1024 x 1024,
// rank 8 in float32, 512 rows 11.7 | 17.5, 2048 rows 34.4 | 24.6.  The last launch's grid has
// to fit 32 bits of threads.
constexpr int64_t kLoraTiledBytes = int64_t(160) << 20;
constexpr int64_t kLoraOuterColumns = 128;  // outputs of a block of the last launch
inline bool lora_uses_matrix_cores(const q8_lora& lo, int64_t m, int64_t n, int64_t k) {
    if (m < kLoraTiledRows) return false;
    const int64_t row = (int64_t(lo.n_sections) * k + n) * lo.rank * (lo.type == Q8_LORA_F32 ? 4 : 2);
    const int64_t blocks = n / kLoraOuterColumns + 2 * Q8_LORA_MAX_SECTIONS + 1;
    // m * row >= kLoraTiledBytes; the product itself can pass 63 bits
    return row >= (kLoraTiledBytes + m - 1) / m && lora_max_tiles(m, lo.n_adapters) * blocks * 256 < (int64_t(1) << 32);
}
inline int64_t lora_parts(int64_t m) {
    if (m < kLoraTiledRows) return 1;
    const int64_t tiles = (m + 31) / 32;
    return tiles >= 512 ? 1 : tiles > 64 ? (512 + tiles - 1) / tiles : 8;
}

// Workspace of the adapter calls: the inner products u [parts][m][n_sections * rank], the rows
// sorted by adapter and their tiles; the packed calls add what their shared product needs.
struct LoraWorkspace {
    size_t u_off, split_off, sorted_off, tiles_off, count_off, base_off, total;
};

inline LoraWorkspace lora_workspace_layout(int64_t m, int32_t n_sections, int32_t rank, size_t base_bytes) {
    LoraWorkspace w{};
    size_t off = 0;
    w.u_off = off;
    off = round_up(off + sizeof(float) * size_t(lora_parts(m)) * size_t(m) * size_t(n_sections) * size_t(rank), 256);
    const size_t tiles = m < kLoraTiledRows ? 0 : size_t(lora_max_tiles(m, kLoraMaxAdapters));
    // u split in three bf16 parts, by tiles of 64 rows
    w.split_off = off;  off = round_up(off + 6 * 64 * tiles * size_t(n_sections) * size_t(rank), 256);
    w.sorted_off = off; off = round_up(off + sizeof(int32_t) * size_t(m), 256);
    w.tiles_off = off;  off = round_up(off + 16 * tiles, 256);
    w.count_off = off;  off = round_up(off + sizeof(int32_t), 256);
    w.base_off = off;   off = round_up(off + base_bytes, 256);
    w.total = off;
    return w;
}

// The packed calls run on the digit tiles (digit_tiles.h) from two rows to the prefill rows,
// for widths up to 64 slices and fused matrices whose up rows lie within 32-bit byte offsets
// of their gate rows; one row on q8_linear's one-row kernel with the correction behind its
// sums; the rest on q8_linear's kernels and the correction in launches of its own.  Measured,
// in us, at 1 | 2 | 16 | 255 rows, rank 16: 6144 x 4096 on tiles 15.0 | 15.1 | 21 | 116, otherwise
// 11.3 | 15.6 | 27.5 | 346; fused 24576 x 4096 28.0 | 28.3 | 37 | 377 and 23.4 | 31.7 | 59.9 |
// 850; 4096 x 12288 24.3 | 24.2 | 33 | 262 and 16.6 | 26.3 | 48.5 | 633.
// Neither m within its range nor the adapters decide, so that a row has the same bits whatever
// rows share the call.  That costs where ranks are high and rows many, as every row reads its
// adapter anew.  Measured, in us, at 16, 64, 128 and 255 rows, 16 adapters in use, the call | the
// tiles without adapters and lora_add behind them: 6144 x 4096, three sections, rank 16 in bf16
// 22.1 | 28.0, 39.4 | 45.2, 64.0 | 71.3, 117 | 123; rank 64 in bf16 30.0 | 35.2, 58.5 | 61.2, 97.1 |
// 98.3, 180 | 147; rank 256 in float32 86 | 94, 221 | 187, 409 | 215, 782 | 279; 8192 x 12288, rank 64
// in bf16 64.6 | 63.7, 187 | 167, 362 | 276, 712 | 501.
constexpr int64_t kLoraTilesMaxK = 16384;
constexpr int64_t kLoraTilesMaxRange = 16 * 256;  // of k without a cut
constexpr int64_t kLoraMaxRanges = 6;             // at most two more than the fewest, 4
inline bool lora_uses_tiles(int64_t m, int64_t n, int64_t k) {
    return m > 1 && m < kPrefillRows && k <= kLoraTilesMaxK && n * row_bytes(k) < (int64_t(1) << 31);
}
inline bool lora_uses_one_row(int64_t m, int64_t k) { return m == 1 && k <= kLoraTilesMaxK; }
// Row groups of four, as many as any form has.
inline int64_t lora_row_groups(int64_t m) { return (m + 3) / 4; }

// Workspace behind the adapters', from its start: four words a row, the digits, and for a
// cut k the ranges' sums and their counts (a tile: 16 rows of the matrix).
struct LoraTilesWorkspace {
    size_t rows_off, dig_off, partial_off, arrived_off, total;
};
inline LoraTilesWorkspace lora_tiles_workspace_layout(int64_t m, int64_t n, int64_t k) {
    LoraTilesWorkspace w{};
    const bool cut = k > kLoraTilesMaxRange;
    const size_t tiles = size_t((n + 15) / 16 + 1);  // + 1: gate and up rows round up apart
    const size_t rows = size_t((m + 15) / 16 * 16);
    size_t off = 0;
    w.rows_off = off;    off = round_up(off + 16 * size_t(m), 256);
    w.dig_off = off;     off = round_up(off + 4 * size_t(m) * size_t(k), 256);
    w.partial_off = off; off = round_up(off + (cut ? sizeof(float) * size_t(kLoraMaxRanges) * tiles * 16 * rows : 0), 256);
    w.arrived_off = off; off = round_up(off + (cut ? sizeof(uint32_t) * size_t(lora_row_groups(m)) * tiles : 0), 256);
    w.total = off;
    return w;
}

// Workspace behind the adapters': that, or the fused call's shared product; the plain call,
// whose product goes straight into y, needs nothing there (lora_linear_bytes).
inline size_t lora_base_bytes(int64_t m, int64_t n, int64_t k) {
    if (lora_uses_one_row(m, k)) return 0;
    if (lora_uses_tiles(m, n, k)) return lora_tiles_workspace_layout(m, n, k).total;
    return sizeof(float) * size_t(m) * size_t(n);
}

// The whole workspace that a packed call needs.
inline size_t lora_linear_bytes(int64_t m, int64_t n, int64_t k, bool fused, int32_t n_sections, int32_t rank) {
    const size_t base = fused || lora_uses_tiles(m, n, k) ? lora_base_bytes(m, n, k) : 0;
    return lora_workspace_layout(m, n_sections, rank, base).total;
}

inline q8_status check_workspace(size_t need, const void* ws, size_t ws_bytes, char* msg, size_t cap) {
    if (!ws) return fail(msg, cap, Q8_ERR_WORKSPACE, "workspace is NULL");
    if (ws_bytes < need) return fail(msg, cap, Q8_ERR_WORKSPACE, "workspace %lld bytes < required %lld", (long long)ws_bytes, (long long)need);
    if (!aligned(ws, 256)) return fail(msg, cap, Q8_ERR_ALIGN, "workspace not 256-byte aligned");
    return Q8_OK;
}

// Sizes the row sort and the grids of the adapter calls take.
inline q8_status check_lora_rows(int64_t m, char* msg, size_t cap) {
    if (m > (int64_t(1) << 22)) return fail(msg, cap, Q8_ERR_SHAPE, "m=%lld above 2^22 rows", m);
    return Q8_OK;
}

// lora_add (n_out = n, n_in = n) and lora_gate_up_silu (n_out = f, n_in = 2f).
inline q8_status check_lora_add(const float* y, int64_t n_in, int64_t ldy, const float* x, int64_t m, int64_t k,
                                int64_t ldx, const q8_lora* lo, const float* out, int64_t n_out, int64_t ldo,
                                char* msg, size_t cap) {
    q8_status s;
    if ((s = check_dim("n", n_in, msg, cap)) != Q8_OK) return s;
    if ((s = check_dim("m", m, msg, cap)) != Q8_OK) return s;
    if ((s = check_k("k", k, msg, cap)) != Q8_OK) return s;
    if ((s = check_lora_rows(m, msg, cap)) != Q8_OK) return s;
    if (ldx < k || ldx > kMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "ldx=%lld < k=%lld, or above 2^30", ldx, k);
    if (ldy < n_in || ldy > 2 * kMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "leading dimension %lld of the product < %lld, or above 2^31", ldy, n_in);
    if (ldo < n_out || ldo > kMaxDim) return fail(msg, cap, Q8_ERR_SHAPE, "leading dimension %lld of the output < %lld, or above 2^30", ldo, n_out);
    if ((s = check_lora(lo, n_in, m, msg, cap)) != Q8_OK) return s;
    if (m == 0 || n_in == 0) return Q8_OK;
    if (!y || !x || !out) return fail(msg, cap, Q8_ERR_NULL, "null pointer (the product, x or the output)");
    if (!aligned(x, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "x pointer not 16-byte aligned");
    if (ldx % 4 != 0) return fail(msg, cap, Q8_ERR_ALIGN, "ldx=%lld not a multiple of 4", ldx);
    if (!aligned(y, 4) || !aligned(out, 4)) return fail(msg, cap, Q8_ERR_ALIGN, "the product or the output not 4-byte aligned");
    return Q8_OK;
}

// ----------------------------------------------------- the whole mixture-of-experts layer

// q8_moe_layer runs in two launches on the digit tiles (digit_tiles.h) below the matrix-core
// switch of the grouped call, up to kMoeLayerMaxTokens tokens (every block selects all tokens'
// experts and holds their lists), at most 64 experts a token (a lane each) and widths of at
// most 24 slices of 256 (three a wave); else the routing and the grouped mixture follow each
// other.  Measured, in us, two launches | the calls one after the other (routing in its two-pass
// form): 8 of 128 experts of 768 x 2048 at 1 token 31.2 | 42.4, 16 95.6 | 129, 64 156 | 271, 127 236 |
// 452; 2 of 64 at 128 tokens 102 | 163; 2 of 8 experts of 2048 x 2048 at 31 tokens 65.3 | 132.
constexpr int64_t kMoeLayerMaxTokens = 128;
constexpr int64_t kMoeLayerMaxWidth = 24 * 256;
inline bool moe_layer_uses_tiles(int64_t m, int32_t k, int64_t n_exp, int64_t f, int64_t h) {
    return m <= kMoeLayerMaxTokens && k <= 64 && h <= kMoeLayerMaxWidth && f <= kMoeLayerMaxWidth &&
           !moe_uses_matrix_cores(m * int64_t(k), n_exp);
}

// Flags and counters of the two-launch form: claims of the chunks of two lists, the jobs' and
// the down tiles' counts.  Jobs: an expert's tokens in eights, m * k < 8 * n_exp <= 2048 pairs.
constexpr int kLayerMaxChunks = 512;
constexpr int kLayerMaxJobs = 512;
constexpr size_t kLayerCounterBytes = 128 * size_t(16 + 2 * kLayerMaxChunks + kLayerMaxJobs);

// Workspace of q8_moe_layer: the logits, then what its form needs.
struct MoeLayerWorkspace {
    size_t logits_off, total;
    size_t idx_off, w_off, moe_off;                                          // routing, then mixture
    size_t dig_off, exps_off, hidden_off, max_off, out_off, count_off;       // two launches
};

inline MoeLayerWorkspace moe_layer_workspace_layout(int64_t m, int32_t k, int64_t n_exp, int64_t f, int64_t h) {
    MoeLayerWorkspace w{};
    const size_t pairs = size_t(m) * size_t(k);
    size_t off = 0;
    w.logits_off = off; off = round_up(off + route_workspace_bytes(m, n_exp), 256);
    if (moe_layer_uses_tiles(m, k, n_exp, f, h)) {
        w.count_off = off;  off = round_up(off + kLayerCounterBytes, 256);
        w.max_off = off;    off = round_up(off + sizeof(uint32_t) * pairs, 256);
        w.exps_off = off;   off = round_up(off + sizeof(int32_t) * size_t(m), 256);
        w.dig_off = off;    off = round_up(off + 4 * size_t(m) * size_t(h), 256);
        w.hidden_off = off; off = round_up(off + sizeof(float) * pairs * size_t(f), 256);
        w.out_off = off;    off = round_up(off + sizeof(float) * pairs * size_t(h), 256);
    } else {
        w.idx_off = off;    off = round_up(off + sizeof(int32_t) * pairs, 256);
        w.w_off = off;      off = round_up(off + sizeof(float) * pairs, 256);
        w.moe_off = off;    off += moe_workspace_layout(m, k, n_exp, f, h).total;
    }
    w.total = off;
    return w;
}

inline q8_status check_moe_layer(const float* wr, const void* wgu, const void* wdn, int64_t n_exp, int64_t f,
                                 int64_t h, const float* x, int64_t m, int64_t ldx, int32_t k, float top_p,
                                 const float* y, int64_t ldy, const void* ws, size_t ws_bytes, char* msg, size_t cap) {
    // the routing lives in the workspace: x stands for its pointers in the mixture's checks
    q8_status s = check_moe_args(wgu, wdn, n_exp, f, h, x, m, ldx, reinterpret_cast<const int32_t*>(x), x, k, y, ldy, msg, cap);
    if (s != Q8_OK) return s;
    if (!(top_p > 0.0f && top_p <= 1.0f)) return fail(msg, cap, Q8_ERR_SHAPE, "top_p must be in (0, 1]");
    if (m == 0) return Q8_OK;
    if (!wr) return fail(msg, cap, Q8_ERR_NULL, "w_router is NULL");
    if (!aligned(wr, 16)) return fail(msg, cap, Q8_ERR_ALIGN, "w_router not 16-byte aligned");
    return check_workspace(moe_layer_workspace_layout(m, k, n_exp, f, h).total, ws, ws_bytes, msg, cap);
}

}  // namespace q8v
