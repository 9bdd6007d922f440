// Host-only check of the 8-bit floating-point calls' argument validation and workspace layout
// (q8_validate.h) under AddressSanitizer and UndefinedBehaviorSanitizer: accepted boundary
// values and each error path, with message buffers of exact size, of capacity 1, and absent.
// Built with g++ (no HIP).
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

alignas(256) static unsigned char pool[4096];  // never dereferenced by the checks
static void* P(size_t off) { return pool + off; }

struct Msg {  // heap-allocated at exactly `cap` bytes; cap 0: none
    char* p = nullptr;
    size_t cap = 0;
    explicit Msg(size_t c) : cap(c) { p = c ? static_cast<char*>(malloc(c)) : nullptr; }
    ~Msg() { free(p); }
};

static constexpr int64_t kBig = INT64_MAX, kSmall = INT64_MIN;

static q8_status linear(int64_t n, int parts, int64_t k, int64_t m, int32_t type, int64_t ldy, int64_t ldgu, size_t cap) {
    Msg msg(cap);
    return check_f8_linear(P(0), P(16), n, parts, k, P(32), P(48), m, P(64), type, ldy, parts == 2 ? P(80) : nullptr,
                           ldgu, msg.p, msg.cap);
}
static q8_status backward(int64_t n, int parts, int64_t k, int64_t m, int32_t type, int64_t ld, size_t ws, size_t cap) {
    Msg msg(cap);
    return check_f8_backward(P(0), P(16), n, parts, k, P(32), P(48), m, P(64), ld, P(80), type, ld, P(96), ld, P(112), ld,
                             P(256), ws, msg.p, msg.cap);
}

int main() {
    const int64_t ld = kMaxDim;
    for (size_t cap : {size_t(256), size_t(1), size_t(0)}) {
        for (int parts : {1, 2}) {
            EXPECT(linear(kF8MaxDim / parts, parts, 16, 1, Q8_F32, ld, ld, cap), Q8_OK);
            EXPECT(linear(1, parts, kF8MaxDim, int64_t(1) << 17, Q8_BF16, ld, ld, cap), Q8_OK);
            EXPECT(linear(16, parts, 16, kF8MaxRows, Q8_F16, ld, ld, cap), Q8_OK);
            EXPECT(linear(kF8MaxDim, parts, 16, kF8MaxRows, Q8_F16, ld, ld, cap), Q8_ERR_SHAPE);
            for (int64_t bad : {kBig, kSmall, int64_t(-1), kF8MaxDim + 1}) {
                EXPECT(linear(bad, parts, 16, 1, Q8_F32, ld, ld, cap), Q8_ERR_SHAPE);
                EXPECT(linear(16, parts, bad, 1, Q8_F32, ld, ld, cap), Q8_ERR_SHAPE);
                if (bad != kF8MaxDim + 1) EXPECT(linear(16, parts, 16, bad, Q8_F32, ld, ld, cap), Q8_ERR_SHAPE);
                EXPECT(backward(bad, parts, 16, 1, Q8_F32, ld, ~size_t(0), cap), Q8_ERR_SHAPE);
                EXPECT(backward(16, parts, bad, 1, Q8_F32, ld, ~size_t(0), cap), Q8_ERR_SHAPE);
            }
            for (int32_t bad : {-1, 3, INT32_MAX, INT32_MIN}) {
                EXPECT(linear(16, parts, 16, 1, bad, ld, ld, cap), Q8_ERR_SHAPE);
                EXPECT(backward(16, parts, 16, 1, bad, ld, ~size_t(0), cap), Q8_ERR_SHAPE);
            }
            for (int64_t bad : {kBig, kSmall, int64_t(15), ld + 1}) {
                EXPECT(linear(16, parts, 16, 1, Q8_F32, bad, ld, cap), Q8_ERR_SHAPE);
                EXPECT(backward(16, parts, 16, 1, Q8_F32, bad, ~size_t(0), cap), Q8_ERR_SHAPE);
            }
            for (int32_t type : {Q8_F32, Q8_F16, Q8_BF16}) {
                const size_t need = f8_backward_workspace_bytes(7, 21, parts, 144, type);
                EXPECT(need % 256, 0);
                EXPECT(backward(21, parts, 144, 7, type, ld, need, cap), Q8_OK);
                EXPECT(backward(21, parts, 144, 7, type, ld, need - 1, cap), Q8_ERR_WORKSPACE);
                const F8BackwardWorkspace w = f8_backward_layout(7, 21, parts, 144, type);
                EXPECT(w.ldd, 64 * parts);
                EXPECT(w.x_off >= w.d_off + size_t(2 * f8_terms(type) * 7) * size_t(w.ldd), 1);
                EXPECT(w.sums_off >= w.x_off + size_t(2 * f8_terms(type) * 64 * 144), 1);
                EXPECT(w.total >= w.sums_off, 1);
                // ranges are whole and leave room for their sums
                for (int64_t m : {int64_t(0), int64_t(1), int64_t(64), int64_t(77), int64_t(1000), int64_t(1) << 14})
                    for (int64_t n : {int64_t(0), int64_t(1), int64_t(300), int64_t(2001), int64_t(1) << 15})
                        for (int64_t k : {int64_t(16), int64_t(1040), int64_t(1) << 14}) {
                            const F8GradPlan dx = f8_dx_plan(m, n, parts, k, type), dw = f8_dw_plan(m, n, parts, k, type);
                            const F8BackwardWorkspace l = f8_backward_layout(m, n, parts, k, type);
                            EXPECT(dx.ranges >= 1 && dx.ranges <= kF8MaxRanges && (!dx.big || dx.ranges == 1), 1);
                            EXPECT(dw.ranges >= 1 && dw.ranges <= kF8MaxRanges && (!dw.big || dw.ranges == 1), 1);
                            if (dx.ranges > 1) EXPECT(l.total - l.sums_off >= size_t(4 * dx.ranges * m * k), 1);
                            if (dw.ranges > 1) EXPECT(l.total - l.sums_off >= size_t(4 * dw.ranges * parts * n * k), 1);
                            if (dx.ranges > 1) EXPECT(l.dw_sums_off - l.sums_off >= size_t(4 * dx.ranges * m * k), 1);
                            if (dw.ranges > 1) EXPECT(l.total - l.dw_sums_off >= size_t(4 * dw.ranges * parts * n * k), 1);
                        }
                // the largest sizes stay within 64 bits
                EXPECT(f8_backward_workspace_bytes(int64_t(1) << 17, kF8MaxDim / parts, parts, int64_t(1) << 17, type) >
                           (size_t(1) << 38), 1);
            }
            EXPECT(f8_backward_workspace_bytes(kBig, 16, parts, 16, Q8_F32), 0);
            EXPECT(f8_backward_workspace_bytes(1, kBig, parts, 16, Q8_F32), 0);
            EXPECT(f8_backward_workspace_bytes(1, 16, parts, kSmall, Q8_F32), 0);
        }
        EXPECT(linear(16, 2, 16, 1, Q8_F32, ld, 31, cap), Q8_ERR_SHAPE);
        for (int64_t rows : {int64_t(0), int64_t(1), kF8MaxDim}) {
            Msg msg(cap);
            EXPECT(check_f8_quantize(P(0), Q8_F16, rows, kF8MaxDim, 16, 24, P(16), P(32), msg.p, msg.cap), Q8_OK);
            EXPECT(check_f8_quantize(P(0), Q8_F16, rows + kF8MaxDim + 1, kF8MaxDim, 16, 24, P(16), P(32), msg.p, msg.cap),
                   Q8_ERR_SHAPE);
        }
        Msg msg(cap);
        EXPECT(check_f8_quantize(P(0), Q8_F16, kBig, kF8MaxRows, 16, 24, P(16), P(32), msg.p, msg.cap), Q8_ERR_SHAPE);
        EXPECT(check_f8_quantize(P(0), Q8_F16, 1, kF8MaxDim, 16, 20, P(16), P(32), msg.p, msg.cap), Q8_ERR_ALIGN);
        EXPECT(check_f8_quantize(nullptr, Q8_F16, 1, kF8MaxDim, 16, 24, P(16), P(32), msg.p, msg.cap), Q8_ERR_NULL);
        EXPECT(check_f8_quantize(P(0), Q8_F16, 1, kF8MaxDim, 16, 24, P(8), P(32), msg.p, msg.cap), Q8_ERR_ALIGN);
    }
    if (failures) return 1;
    puts("all cases as expected");
    return 0;
}
