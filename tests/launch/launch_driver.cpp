// launch_driver.cpp -- calls entry points of include/gdn.h at the ends of the sizes
// that their checks accept, and looks at what each would launch: this program's own
// hipLaunchKernel takes the runtime's place, records the grid and launches nothing.
// Operands are addresses that nothing dereferences.  Test infrastructure:
// tests/test_launch_sizes.py builds it against libgdn.so and runs it.
//
//   launch_driver lru|norms      exit status 0: every launch fits
//
// A launch counts fewer than 2^32 threads along each dimension, workgroups have at
// most 1,024, and y and z at most 65,535 workgroups.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "gdn.h"

namespace {
struct Dim3 {
    uint32_t x, y, z;
};
Dim3 pushed_grid, pushed_block;
size_t pushed_shared;
void* pushed_stream;

int launches, failures;
uint64_t largest;
char what[160];

void expect_launched(gdn_status got) {
    if (got == GDN_OK && launches > 0)
        return;
    std::fprintf(stderr, "%s: status %d after %d launches\n", what, got, launches);
    ++failures;
}

// Operands far apart, never dereferenced.
void* at(int k) { return reinterpret_cast<void*>(static_cast<uintptr_t>(k + 1) << 48); }
float* fa(int k) { return static_cast<float*>(at(k)); }
int32_t* ia(int k) { return static_cast<int32_t*>(at(k)); }

int lru() {
    int cases = 0;
    for (int act : {GDN_F32, GDN_BF16})
        for (int W : {8, 64, 72, 128, 136, 192, 200, 256, 264, 320, 4096, GDN_LRU_MAX_WIDTH})
            for (int T : {1, 31, 32, 33, 63, 64, 65, 128, 129, 256, 257, 4096, 65537, GDN_LRU_MAX_TOKENS})
                for (int64_t share : {1, 2, 3, 4, 64, 4096, 1 << 20}) {
                    // the most sequences that are taken, and parts of them
                    const int64_t each = static_cast<int64_t>((W + 63) / 64) * ((T + 63) / 64);
                    const int64_t B = ((1ll << 23) - 1) / each / share;
                    if (B < 1)
                        continue;
                    const gdn_lru_dims d{static_cast<int32_t>(B), W, act};
                    ++cases;
                    std::snprintf(what, sizeof what, "prefill , %lld sequences of %d tokens of %d channels, type %d",
                                  static_cast<long long>(B), T, W, act);
                    launches = 0;
                    expect_launched(gdn_lru_prefill(&d, nullptr, fa(0), T, at(1), at(2), at(3), fa(4), at(5), ia(6), at(7),
                                                    fa(8), ia(9), at(10), SIZE_MAX, nullptr));
                    std::memcpy(what, "gradient", 8);
                    launches = 0;
                    expect_launched(gdn_lru_backward(&d, nullptr, nullptr, T, at(1), at(2), at(3), fa(4), at(5), ia(6), fa(7),
                                                     at(8), fa(9), at(10), at(11), at(12), at(13), fa(14), fa(15), ia(16),
                                                     at(17), SIZE_MAX, nullptr));
                    if (T > 1)
                        continue;
                    std::memcpy(what, "token   ", 8);
                    launches = 0;
                    expect_launched(gdn_lru_decode_token(&d, nullptr, fa(0), at(1), at(2), at(3), fa(4), at(5), at(6), nullptr));
                }
    return cases;
}

int norms() {
    int cases = 0;
    struct Types {
        int act, other;
    };
    for (const Types t : {Types{GDN_F32, GDN_F32}, Types{GDN_BF16, GDN_F32}, Types{GDN_BF16, GDN_BF16}})
        for (int64_t rows : {INT64_C(1), INT64_C(2), INT64_C(1000), INT64_C(1) << 20, INT64_C(0x7FFFFFFF)})
            for (int D : {8, 64, 72, 256, 264, 1024, 4096, 8192, GDN_NORM_MAX_WIDTH}) {
                ++cases;
                std::snprintf(what, sizeof what, "residual norm, %lld rows of %d, types %d and %d", static_cast<long long>(rows), D,
                              t.act, t.other);
                launches = 0;
                expect_launched(gdn_residual_norm(rows, D, t.act, t.other, 1e-6f, at(0), at(1), fa(2), fa(3), fa(4), at(5), at(6),
                                                  nullptr));
                launches = 0;
                expect_launched(gdn_residual_norm_backward(rows, D, t.act, t.other, 1e-6f, at(0), at(1), fa(2), fa(3), fa(4), at(5),
                                                           at(6), at(7), at(8), fa(9), fa(10), fa(11), at(12), SIZE_MAX, nullptr));
                for (int H : {1, 3, 64, 1000, 32767, 65535, 65536})
                    for (int flags : {0, GDN_WEIGHT_PER_HEAD}) {
                        if (rows * H >= 1ll << 31 || static_cast<int64_t>(H) * D >= 1ll << 30)
                            continue;
                        std::snprintf(what, sizeof what, "gated norm, %lld rows of %d x %d, types %d and %d, flags %d",
                                      static_cast<long long>(rows), H, D, t.act, t.other, flags);
                        launches = 0;
                        expect_launched(gdn_gated_norm(rows, H, D, t.other, t.act, flags, 1e-6f, at(0), at(1), 0, fa(2), at(3),
                                                       nullptr));
                        launches = 0;
                        expect_launched(gdn_gated_norm_backward(rows, H, D, t.other, t.act, flags, 1e-6f, at(0), at(1), 0, fa(2),
                                                                at(3), at(4), at(5), 0, fa(6), at(7), SIZE_MAX, nullptr));
                    }
            }
    return cases;
}
}  // namespace

extern "C" {
int __hipPushCallConfiguration(Dim3 grid, Dim3 block, size_t shared, void* stream) {
    pushed_grid = grid, pushed_block = block, pushed_shared = shared, pushed_stream = stream;
    return 0;
}
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* shared, void** stream) {
    *grid = pushed_grid, *block = pushed_block, *shared = pushed_shared, *stream = pushed_stream;
    return 0;
}
int hipLaunchKernel(const void*, Dim3 grid, Dim3 block, void**, size_t, void*) {
    ++launches;
    const uint64_t x = static_cast<uint64_t>(grid.x) * block.x;
    largest = largest > x ? largest : x;
    const uint32_t threads = block.x * block.y * block.z;
    if (!grid.x || !grid.y || !grid.z || x >> 32 || grid.y > 65535 || grid.z > 65535 || !threads || threads > 1024) {
        std::fprintf(stderr, "%s: a launch of %u x %u x %u workgroups of %u threads\n", what, grid.x, grid.y, grid.z, threads);
        ++failures;
    }
    return 0;
}
int hipGetLastError() { return 0; }
}

int main(int argc, char** argv) {
    const char* which = argc > 1 ? argv[1] : "";
    const int cases = !std::strcmp(which, "lru") ? lru() : !std::strcmp(which, "norms") ? norms() : 0;
    std::printf("%d cases, at most %llu threads\n", cases, static_cast<unsigned long long>(largest));
    if (cases && !failures)
        std::puts("every launch fits");
    return !cases || failures;
}
