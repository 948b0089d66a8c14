// lru_norm_driver.cpp -- calls the gated linear recurrent layer's and the norms'
// entry points of include/gdn.h with arguments the host checks refuse, and their
// size queries with the smallest and largest sizes, in a host build of the library
// with AddressSanitizer and UndefinedBehaviorSanitizer.  Nothing reaches a device:
// each refused call returns before any HIP call.  Test infrastructure:
// tests/test_sanitizers_lru_norm.py builds and runs it.
// Exit status 0: every call returned the status expected of it.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "gdn.h"

namespace {
int failures = 0;
void expect(const char* what, int got, int want) {
    if (got != want) {
        std::fprintf(stderr, "%s: status %d, expected %d\n", what, got, want);
        ++failures;
    }
}
void expect_size(const char* what, size_t got, bool nonzero) {
    if ((got != 0) != nonzero) {
        std::fprintf(stderr, "%s: size %zu\n", what, got);
        ++failures;
    }
}
// Operands far apart, never dereferenced.
void* at(int k) { return reinterpret_cast<void*>(static_cast<uintptr_t>(k + 1) << 44); }
float* fa(int k) { return static_cast<float*>(at(k)); }
int32_t* ia(int k) { return static_cast<int32_t*>(at(k)); }

gdn_status prefill(const gdn_lru_dims& d, const gdn_lru_pitches* p, int T, void* y, size_t ws) {
    return gdn_lru_prefill(&d, p, fa(0), T, at(1), at(2), at(3), fa(4), at(5), ia(6), y, fa(8), ia(9), at(10), ws, nullptr);
}
gdn_status backward(const gdn_lru_dims& d, const gdn_lru_pitches* p, int T, void* dx, size_t ws) {
    return gdn_lru_backward(&d, p, p, T, at(1), at(2), at(3), fa(4), at(5), ia(6), fa(7), at(8), fa(9), dx, at(11), at(12), at(13),
                            fa(14), fa(15), ia(16), at(17), ws, nullptr);
}
}  // namespace

int main() {
    const gdn_lru_dims good{3, 264, GDN_BF16}, least{1, 8, GDN_F32}, widest{1, GDN_LRU_MAX_WIDTH, GDN_F32};
    for (const gdn_lru_dims* d : {&good, &least, &widest}) {
        expect_size("state", gdn_lru_state_bytes(d), true);
        for (int T : {1, 32, 33, 256, 257, 5000, 100000}) {
            expect_size("saved", gdn_lru_saved_bytes(d, T), true);
            expect_size("backward ws", gdn_lru_backward_workspace_bytes(d, T), true);
        }
        for (int T : {0, -1, INT_MIN, INT_MAX, GDN_LRU_MAX_TOKENS + 1}) {
            expect_size("saved", gdn_lru_saved_bytes(d, T), false);
            expect_size("prefill ws", gdn_lru_prefill_workspace_bytes(d, T), false);
            expect_size("backward ws", gdn_lru_backward_workspace_bytes(d, T), false);
            expect("T", prefill(*d, nullptr, T, at(7), SIZE_MAX), GDN_ERR_SHAPE);
            expect("T back", backward(*d, nullptr, T, at(10), SIZE_MAX), GDN_ERR_SHAPE);
        }
    }
    expect_size("longest", gdn_lru_prefill_workspace_bytes(&good, GDN_LRU_MAX_TOKENS), true);
    expect_size("longest back", gdn_lru_backward_workspace_bytes(&good, GDN_LRU_MAX_TOKENS), true);
    for (int field = 0; field < 3; ++field)
        for (int v : {INT_MIN, -1, 0, 7, 8, 1 << 30, INT_MAX}) {
            gdn_lru_dims d = good;
            (&d.batch)[field] = v;
            const bool ok = (field == 0 && (v == 7 || v == 8)) || (field == 1 && v == 8) || (field == 2 && v == 0);
            expect_size("dims", gdn_lru_state_bytes(&d), ok);
            if (!ok)
                expect("dims token", gdn_lru_decode_token(&d, nullptr, fa(0), at(1), at(2), at(3), fa(4), at(5), at(6), nullptr),
                       field == 2 ? GDN_ERR_DTYPE : GDN_ERR_SHAPE);
        }
    for (int64_t v : {INT64_MIN, INT64_C(-8), INT64_C(8), INT64_C(260), INT64_C(1) << 21, INT64_MAX}) {
        const gdn_lru_pitches p{0, v, 0, 0, 0};
        expect("pitch", prefill(good, &p, 100, at(7), SIZE_MAX), GDN_ERR_SHAPE);
        expect("pitch back", backward(good, &p, 100, at(10), SIZE_MAX), GDN_ERR_SHAPE);
    }
    // the largest pitch and the longest rows: spans of the overlap check stay within 64 bits
    const gdn_lru_pitches wide{1 << 20, 1 << 20, 1 << 20, 1 << 20, 1 << 20};
    expect("spans", prefill(least, &wide, GDN_LRU_MAX_TOKENS, at(1), SIZE_MAX), GDN_ERR_ALIAS);
    expect("spans back", backward(least, &wide, GDN_LRU_MAX_TOKENS, at(3), SIZE_MAX), GDN_ERR_ALIAS);
    expect("no workspace", prefill(good, nullptr, 1000, at(7), 1), GDN_ERR_WORKSPACE);
    expect("no workspace back", backward(good, nullptr, 1000, at(10), 1), GDN_ERR_WORKSPACE);
    expect("null", gdn_lru_prefill(nullptr, nullptr, nullptr, 1, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                   nullptr, nullptr, nullptr, 0, nullptr), GDN_ERR_NULL);

    for (int64_t rows : {INT64_MIN, INT64_C(-1), INT64_C(0), INT64_C(1) << 31, INT64_MAX}) {
        expect_size("norm ws", gdn_residual_norm_backward_workspace_bytes(rows, 64), false);
        expect_size("gated ws", gdn_gated_norm_backward_workspace_bytes(rows, 2, 64), false);
        expect("rows", gdn_residual_norm(rows, 64, GDN_F32, GDN_F32, 1e-6f, at(0), at(1), nullptr, nullptr, fa(2), at(3), at(4),
                                         nullptr), GDN_ERR_SHAPE);
        expect("gated rows", gdn_gated_norm(rows, 2, 64, GDN_F32, GDN_F32, 0, 1e-6f, at(0), at(1), 0, fa(2), at(3), nullptr),
               GDN_ERR_SHAPE);
    }
    for (int W : {INT_MIN, -8, 0, 4, GDN_NORM_MAX_WIDTH + 8, INT_MAX}) {
        expect_size("norm W", gdn_residual_norm_backward_workspace_bytes(10, W), false);
        expect_size("gated D", gdn_gated_norm_backward_workspace_bytes(10, 1, W), false);
        expect_size("gated H", gdn_gated_norm_backward_workspace_bytes(10, W > 0 ? INT_MAX : W, 8), false);
    }
    for (int W : {8, 1000, GDN_NORM_MAX_WIDTH})
        for (int64_t rows : {INT64_C(1), INT64_C(300), INT64_C(0x7FFFFFFF)}) {
            expect_size("norm ws", gdn_residual_norm_backward_workspace_bytes(rows, W), true);
            expect_size("gated ws", gdn_gated_norm_backward_workspace_bytes(rows, 1, W), true);
        }
    expect_size("many heads", gdn_gated_norm_backward_workspace_bytes(3, 65536, 8), true);
    for (float eps : {0.0f, -1.0f, 1e-42f, static_cast<float>(NAN), static_cast<float>(INFINITY)})
        expect("eps", gdn_residual_norm(4, 64, GDN_F32, GDN_F32, eps, at(0), at(1), nullptr, nullptr, fa(2), at(3), at(4), nullptr),
               GDN_ERR_SHAPE);
    // the largest spans
    expect("span", gdn_residual_norm(0x7FFFFFFF, GDN_NORM_MAX_WIDTH, GDN_F32, GDN_F32, 1e-6f, at(0), at(1), nullptr, nullptr, fa(2),
                                     at(3), at(1), nullptr), GDN_ERR_ALIAS);
    for (int64_t pitch : {INT64_MIN, INT64_C(-8), INT64_C(120), INT64_C(132), INT64_MAX, INT64_C(1) << 55})
        expect("gated pitch", gdn_gated_norm(4, 2, 64, GDN_F32, GDN_F32, 0, 1e-6f, at(0), at(1), pitch, fa(2), at(3), nullptr),
               GDN_ERR_SHAPE);
    expect("gated span", gdn_gated_norm(0x3FFFFFFF, 1, 64, GDN_F32, GDN_F32, 0, 1e-6f, at(0), at(1), INT64_C(1) << 25, fa(2), at(1),
                                        nullptr), GDN_ERR_ALIAS);
    if (failures == 0)
        std::puts("every call refused as expected");
    return failures != 0;
}
