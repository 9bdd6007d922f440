// Host-only check of the adapter calls' and the whole MoE layer's argument validation and
// workspace layouts (q8_validate.h) under AddressSanitizer and UndefinedBehaviorSanitizer:
// accepted boundary values and each error path, with message buffers of exact size, of
// capacity 1, and absent; the layouts and the choice of forms at the smallest and largest
// accepted sizes.  Built with g++ (no HIP).
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "q8_validate.h"

using namespace q8v;

static int failures = 0;
#define EXPECT(expr, want)                                                                           \
    do {                                                                                             \
        const long long got_ = (long long)(expr), want_ = (long long)(want);                         \
        if (got_ != want_) {                                                                         \
            fprintf(stderr, "%s:%d: %s -> %lld, expected %lld\n", __FILE__, __LINE__, #expr, got_, want_); \
            ++failures;                                                                              \
        }                                                                                            \
    } while (0)

// 256-byte aligned dummy buffers (never dereferenced by the checks)
alignas(256) static unsigned char pool[4096];
static void* P(size_t off) { return pool + off; }
static float* F(size_t off) { return reinterpret_cast<float*>(pool + off); }
static int32_t* I(size_t off) { return reinterpret_cast<int32_t*>(pool + off); }

// one message buffer per call, heap-allocated at exactly `cap` bytes; cap 0: none
struct Msg {
    char* p = nullptr;
    size_t cap = 0;
    explicit Msg(size_t c) : cap(c) { p = c ? static_cast<char*>(malloc(c)) : nullptr; }
    ~Msg() { free(p); }
};

static constexpr int64_t kTop = int64_t(1) << 30;

static q8_lora good(int64_t n) {
    q8_lora lo{};
    lo.a = P(0);
    lo.b = P(256);
    lo.adapter = I(512);
    lo.section_rows[0] = n;
    lo.type = Q8_LORA_BF16;
    lo.n_adapters = 3;
    lo.rank = 16;
    lo.n_sections = 1;
    return lo;
}

template <class Change>
static q8_lora with(int64_t n, Change&& change) {
    q8_lora lo = good(n);
    change(lo);
    return lo;
}

static void lora_cases(size_t cap) {
    Msg m(cap);
    const int64_t n = 64;
    auto check = [&](const q8_lora& lo, int64_t rows = 2, int64_t nn = 64) { return check_lora(&lo, nn, rows, m.p, m.cap); };
    EXPECT(check(good(n)), Q8_OK);
    EXPECT(check_lora(nullptr, n, 2, m.p, m.cap), Q8_ERR_NULL);
    for (int32_t t : {INT32_MIN, -1, 3, INT32_MAX}) EXPECT(check(with(n, [&](q8_lora& l) { l.type = t; })), Q8_ERR_SHAPE);
    for (int32_t c : {INT32_MIN, -1, 257, INT32_MAX})
        EXPECT(check(with(n, [&](q8_lora& l) { l.n_adapters = c; })), Q8_ERR_SHAPE);
    EXPECT(check(with(n, [](q8_lora& l) { l.n_adapters = 256; })), Q8_OK);
    for (int32_t r : {INT32_MIN, -8, 0, 4, 12, 257, 264, INT32_MAX})
        EXPECT(check(with(n, [&](q8_lora& l) { l.rank = r; })), Q8_ERR_SHAPE);
    EXPECT(check(with(n, [](q8_lora& l) { l.rank = 8; })), Q8_OK);
    EXPECT(check(with(n, [](q8_lora& l) { l.rank = 256; })), Q8_OK);
    for (int32_t s : {INT32_MIN, -1, 0, 5, INT32_MAX})
        EXPECT(check(with(n, [&](q8_lora& l) { l.n_sections = s; })), Q8_ERR_SHAPE);
    EXPECT(check(with(n, [](q8_lora& l) { l.n_sections = 4; })), Q8_OK);  // three empty ones
    EXPECT(check(with(n, [](q8_lora& l) { l.section_rows[0] = 63; })), Q8_ERR_SHAPE);
    EXPECT(check(with(n, [](q8_lora& l) { l.n_sections = 2; l.section_rows[0] = -1; l.section_rows[1] = 65; })), Q8_ERR_SHAPE);
    EXPECT(check(with(n, [](q8_lora& l) {
               l.n_sections = 4;
               for (auto& r : l.section_rows) r = INT64_MAX;
           })), Q8_ERR_SHAPE);
    EXPECT(check(with(n, [](q8_lora& l) { l.section_rows[0] = INT64_MIN; })), Q8_ERR_SHAPE);
    // four sections of the largest matrix: their sum does not overflow
    EXPECT(check(with(kTop, [](q8_lora& l) {
               l.n_sections = 4;
               for (auto& r : l.section_rows) r = kTop;
           }), 2, kTop), Q8_ERR_SHAPE);
    for (int q = 0; q < 3; ++q)
        EXPECT(check(with(n, [&](q8_lora& l) { (q == 0 ? l.a : q == 1 ? l.b : *(const void**)&l.adapter) = nullptr; })),
               Q8_ERR_NULL);
    EXPECT(check(with(n, [](q8_lora& l) { l.a = P(8); })), Q8_ERR_ALIGN);
    EXPECT(check(with(n, [](q8_lora& l) { l.b = P(2); })), Q8_ERR_ALIGN);
    EXPECT(check(with(n, [](q8_lora& l) { l.adapter = reinterpret_cast<int32_t*>(pool + 1); })), Q8_ERR_ALIGN);
    EXPECT(check(with(n, [](q8_lora& l) { l.ranks = reinterpret_cast<int32_t*>(pool + 2); })), Q8_ERR_ALIGN);
    EXPECT(check(with(n, [](q8_lora& l) { l.scale = reinterpret_cast<float*>(pool + 3); })), Q8_ERR_ALIGN);
    // nothing to correct: no pointers needed
    auto bare = [](q8_lora& l) { l.a = l.b = nullptr; l.adapter = nullptr; };
    EXPECT(check(with(n, bare), 0), Q8_OK);
    EXPECT(check(with(n, [&](q8_lora& l) { bare(l); l.n_adapters = 0; })), Q8_OK);
    EXPECT(check(with(0, bare), 2, 0), Q8_OK);
}

static void add_cases(size_t cap) {
    Msg m(cap);
    const int64_t n = 64, k = 256;
    const q8_lora lo = good(n), top = good(kTop);
    EXPECT(check_lora_add(F(0), n, n, F(0), 2, k, k, &lo, F(0), n, n, m.p, m.cap), Q8_OK);
    EXPECT(check_lora_add(F(0), n, n, F(0), 2, k, k, &lo, F(0), n / 2, n / 2, m.p, m.cap), Q8_OK);
    EXPECT(check_lora_add(F(0), kTop, 2 * kTop, F(0), int64_t(1) << 22, kTop, kTop, &top, F(0), kTop, kTop, m.p, m.cap), Q8_OK);
    EXPECT(check_lora_add(F(0), n, n, F(0), (int64_t(1) << 22) + 1, k, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_SHAPE);
    for (int64_t bad : {INT64_MIN, int64_t(-1), kTop + 1, INT64_MAX}) {
        EXPECT(check_lora_add(F(0), bad, n, F(0), 2, k, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_SHAPE);
        EXPECT(check_lora_add(F(0), n, n, F(0), bad, k, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_SHAPE);
        EXPECT(check_lora_add(F(0), n, n, F(0), 2, bad, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_SHAPE);
        EXPECT(check_lora_add(F(0), n, n, F(0), 2, k, bad, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_SHAPE);
        EXPECT(check_lora_add(F(0), n, n, F(0), 2, k, k, &lo, F(0), n, bad, m.p, m.cap), Q8_ERR_SHAPE);
    }
    for (int64_t bad : {INT64_MIN, int64_t(-1), n - 1, 2 * kTop + 1, INT64_MAX})
        EXPECT(check_lora_add(F(0), n, bad, F(0), 2, k, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_SHAPE);
    EXPECT(check_lora_add(F(0), n, n, F(0), 2, k, k - 4, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_SHAPE);
    EXPECT(check_lora_add(F(0), n, n, F(0), 2, 128, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_SHAPE);
    EXPECT(check_lora_add(nullptr, n, n, F(0), 2, k, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_NULL);
    EXPECT(check_lora_add(F(0), n, n, nullptr, 2, k, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_NULL);
    EXPECT(check_lora_add(F(0), n, n, F(0), 2, k, k, &lo, nullptr, n, n, m.p, m.cap), Q8_ERR_NULL);
    EXPECT(check_lora_add(F(0), n, n, F(0), 2, k, k, nullptr, F(0), n, n, m.p, m.cap), Q8_ERR_NULL);
    EXPECT(check_lora_add(F(0), n, n, F(4), 2, k, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_ALIGN);
    EXPECT(check_lora_add(F(0), n, n, F(0), 2, k, k + 2, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_ALIGN);
    EXPECT(check_lora_add(F(4), n, n + 1, F(0), 2, k, k, &lo, F(8), n, n + 3, m.p, m.cap), Q8_OK);
    EXPECT(check_lora_add(reinterpret_cast<float*>(pool + 2), n, n, F(0), 2, k, k, &lo, F(0), n, n, m.p, m.cap), Q8_ERR_ALIGN);
    EXPECT(check_lora_add(nullptr, n, n, nullptr, 0, k, k, &lo, nullptr, n, n, m.p, m.cap), Q8_OK);
}

static void moe_layer_cases(size_t cap) {
    Msg m(cap);
    const int64_t E = 128, FF = 768, H = 2048, M = 16;
    const size_t need = moe_layer_workspace_layout(M, 8, E, FF, H).total;
    auto call = [&](int64_t e = 128, int64_t f = 768, int64_t h = 2048, int64_t rows = 16, int32_t k = 8, float top_p = 1.0f,
                    const float* wr = F(0), const void* ws = P(0), size_t size = SIZE_MAX) {
        return check_moe_layer(wr, P(0), P(256), e, f, h, F(0), rows, h > 0 && h <= kTop ? h : 2048, k, top_p, F(0),
                               h > 0 && h <= kTop ? h : 2048, ws, size, m.p, m.cap);
    };
    EXPECT(call(), Q8_OK);
    EXPECT(call(E, FF, H, M, 8, 1.0f, F(0), P(0), need), Q8_OK);
    EXPECT(call(E, FF, H, M, 8, 1.0f, F(0), P(0), need - 1), Q8_ERR_WORKSPACE);
    EXPECT(call(E, FF, H, M, 8, 1.0f, F(0), nullptr), Q8_ERR_WORKSPACE);
    EXPECT(call(E, FF, H, M, 8, 1.0f, F(0), P(16)), Q8_ERR_ALIGN);
    EXPECT(call(E, FF, H, M, 8, 1.0f, nullptr), Q8_ERR_NULL);
    EXPECT(call(E, FF, H, M, 8, 1.0f, F(8)), Q8_ERR_ALIGN);
    for (float p : {0.0f, -1.0f, 1.5f, __builtin_nanf(""), __builtin_inff()}) EXPECT(call(E, FF, H, M, 8, p), Q8_ERR_SHAPE);
    for (int64_t bad : {INT64_MIN, int64_t(-1), int64_t(0), int64_t(257), INT64_MAX}) EXPECT(call(bad), Q8_ERR_SHAPE);
    for (int64_t bad : {INT64_MIN, int64_t(0), int64_t(100), int64_t(16640), INT64_MAX}) {
        EXPECT(call(E, bad), Q8_ERR_SHAPE);
        EXPECT(call(E, FF, bad), Q8_ERR_SHAPE);
    }
    for (int64_t bad : {INT64_MIN, int64_t(-1), int64_t(1) << 22, INT64_MAX}) EXPECT(call(E, FF, H, bad), Q8_ERR_SHAPE);
    for (int32_t bad : {INT32_MIN, 0, 129, INT32_MAX}) EXPECT(call(E, FF, H, M, bad), Q8_ERR_SHAPE);
    EXPECT(call(256, 16384, 16384, int64_t(1) << 16, 256), Q8_OK);
    EXPECT(call(E, FF, H, 0, 8, 1.0f, nullptr, nullptr, 0), Q8_OK);
}

template <size_t N>
static void ascending(const size_t (&off)[N], const char* what) {
    for (size_t i = 0; i < N; ++i)
        if (off[i] % 256 || (i && off[i] < off[i - 1])) {
            fprintf(stderr, "%s: region %zu at %zu\n", what, i, off[i]);
            ++failures;
        }
}
static void at_least(size_t have, size_t need, const char* what) {
    if (have < need) {
        fprintf(stderr, "%s: %zu bytes, needs %zu\n", what, have, need);
        ++failures;
    }
}

static void layouts() {
    for (int64_t m : {int64_t(0), int64_t(1), int64_t(47), int64_t(48), int64_t(255), int64_t(256), int64_t(2049), int64_t(1) << 22})
        for (int32_t rank : {8, 256})
            for (int32_t ns : {1, 4}) {
                const size_t cols = size_t(rank) * ns, tiles = m < kLoraTiledRows ? 0 : size_t(lora_max_tiles(m, 256));
                const LoraWorkspace L = lora_workspace_layout(m, ns, rank, 1000);
                ascending({L.u_off, L.split_off, L.sorted_off, L.tiles_off, L.count_off, L.base_off, L.total}, "adapters");
                at_least(L.split_off - L.u_off, 4 * size_t(lora_parts(m)) * size_t(m) * cols, "u");
                at_least(L.sorted_off - L.split_off, tiles * 3 * (cols / 8) * 64 * 16, "split u");
                at_least(L.tiles_off - L.sorted_off, 4 * size_t(m), "sorted rows");
                at_least(L.count_off - L.tiles_off, 16 * tiles, "tiles");
                at_least(L.total - L.base_off, 1000, "base");
                // rows in bins of 1 and 65: every tile the sort can make
                int64_t worst = 0;
                for (int64_t left = m, b = 0; left > 0 && b < 257; ++b) {
                    const int64_t c = b == 256 ? left : left < 65 ? left : b % 2 ? 65 : 1;
                    worst += (c + 63) / 64;
                    left -= c;
                }
                at_least(size_t(lora_max_tiles(m, 256)), size_t(worst), "tiles of the sort");
            }
    for (int64_t m : {int64_t(2), int64_t(17), int64_t(255)})
        for (int64_t n : {int64_t(1), int64_t(33), int64_t(1) << 20})
            for (int64_t k : {int64_t(256), int64_t(4096), int64_t(4352), int64_t(16384)}) {
                if (!lora_uses_tiles(m, n, k)) continue;
                const LoraTilesWorkspace T = lora_tiles_workspace_layout(m, n, k);
                ascending({T.rows_off, T.dig_off, T.partial_off, T.arrived_off, T.total}, "tiles");
                at_least(T.dig_off, 16 * size_t(m), "row facts");
                at_least(T.partial_off - T.dig_off, 4 * size_t(m) * size_t(k), "digits");
                if (k <= kLoraTilesMaxRange) continue;
                const size_t tiles = size_t((n + 15) / 16);
                for (int ng : {1, 2, 4}) {
                    const size_t groups = size_t((m + 4 * ng - 1) / (4 * ng));
                    at_least(T.arrived_off - T.partial_off, 4 * groups * 6 * tiles * ng * 64, "ranges' sums");
                    at_least(T.total - T.arrived_off, 4 * groups * tiles, "ranges' counts");
                }
            }
    // which form: no product of accepted sizes overflows
    for (int64_t m : {int64_t(1), int64_t(48), int64_t(1) << 22})
        for (int64_t n : {int64_t(0), int64_t(64), kTop})
            for (int64_t k : {int64_t(256), kTop})
                for (int32_t type : {Q8_LORA_F32, Q8_LORA_BF16}) {
                    q8_lora lo = good(n);
                    lo.type = type;
                    lo.rank = 256;
                    lo.n_sections = 4;
                    lo.n_adapters = 256;
                    const __int128 bytes = (__int128)m * (4 * (__int128)k + n) * 256 * (type == Q8_LORA_F32 ? 4 : 2);
                    const __int128 threads =
                        (__int128)lora_max_tiles(m, 256) * (n / kLoraOuterColumns + 2 * Q8_LORA_MAX_SECTIONS + 1) * 256;
                    const bool want = m >= kLoraTiledRows && bytes >= kLoraTiledBytes && threads < ((__int128)1 << 32);
                    EXPECT(lora_uses_matrix_cores(lo, m, n, k), want);
                    EXPECT(lora_base_bytes(m, n, k) >= (lora_uses_tiles(m, n, k) ? 1u : 0u), true);
                }
    // where the byte limit lies, from both sides: 48 rows of 3,495,254 bytes are 160 MB
    q8_lora lo = good(64);
    lo.rank = 8;
    for (int64_t k = 218112; k <= 218880; k += 256)
        EXPECT(lora_uses_matrix_cores(lo, 48, 64, k), 48 * (k + 64) * 16 >= kLoraTiledBytes);
    for (int64_t m : {int64_t(1), int64_t(16), int64_t(128), int64_t(129), int64_t(1) << 16})
        for (int32_t k : {1, 8, 64, 65, 256})
            for (int64_t f : {int64_t(256), int64_t(6144), int64_t(6400), int64_t(16384)}) {
                const size_t pairs = size_t(m) * k;
                const MoeLayerWorkspace L = moe_layer_workspace_layout(m, k, 256, f, f);
                if (moe_layer_uses_tiles(m, k, 256, f, f)) {
                    ascending({L.logits_off, L.count_off, L.max_off, L.exps_off, L.dig_off, L.hidden_off, L.out_off, L.total}, "layer");
                    at_least(L.max_off - L.count_off, kLayerCounterBytes, "counters");
                    at_least(L.dig_off - L.exps_off, 4 * size_t(m), "exponents");
                    at_least(L.hidden_off - L.dig_off, 4 * size_t(m) * f, "digits");
                    at_least(L.out_off - L.hidden_off, 4 * pairs * f, "hidden rows");
                    at_least(L.total - L.out_off, 4 * pairs * f, "outputs");
                    // an expert's tokens in eights
                    at_least(kLayerMaxJobs, (pairs < 256 ? pairs : 256) + pairs / 8, "jobs");
                } else {
                    ascending({L.logits_off, L.idx_off, L.w_off, L.moe_off, L.total}, "layer");
                    at_least(L.total - L.moe_off, moe_workspace_layout(m, k, 256, f, f).total, "mixture");
                }
                at_least(L.max_off ? L.count_off : L.idx_off, 4 * size_t(m) * 256, "logits");
            }
}

int main() {
    for (size_t cap : {size_t(0), size_t(1), size_t(256)}) {
        lora_cases(cap);
        add_cases(cap);
        moe_layer_cases(cap);
    }
    layouts();
    if (failures) {
        fprintf(stderr, "%d validation mismatches\n", failures);
        return 1;
    }
    printf("validation checks: all cases as expected\n");
    return 0;
}
