// ssm_beam_driver.cpp -- calls the state space and beam search entry points of
// include/gdn.h with arguments the host checks refuse, and their size queries
// with the smallest and largest sizes, in a host build of the library with
// AddressSanitizer and UndefinedBehaviorSanitizer.  Nothing reaches a device:
// each refused call returns before any HIP call.  Test infrastructure:
// tests/test_sanitizers_ssm_beam.py builds and runs it.
// Exit status 0: every call returned the status expected of it.
#include <climits>
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
}  // namespace

int main() {
    const gdn_ssm_dims good{2, 48, 16, 128, 128, 4, GDN_BF16}, tiny{1, 1, 1, 32, 32, 4, GDN_F32};
    void* f = reinterpret_cast<void*>(0x1000);   // never dereferenced
    void* g = reinterpret_cast<void*>(0x40000000);
    void* mis = reinterpret_cast<void*>(0x1004);
    float* ff = static_cast<float*>(f);
    int32_t* fi = static_cast<int32_t*>(f);

    for (const gdn_ssm_dims* d : {&good, &tiny}) {
        expect_size("channels", gdn_ssm_conv_channels(d), true);
        expect_size("state", gdn_ssm_state_bytes(d), true);
        expect_size("tail", gdn_ssm_conv_tail_bytes(d), true);
        for (int T : {1, 16, 17, 64, 65, 4097, GDN_SSM_MAX_TOKENS})
            expect_size("prefill ws", gdn_ssm_prefill_workspace_bytes(d, T), true);
        for (int T : {0, -1, INT_MIN, INT_MAX})
            expect_size("prefill ws", gdn_ssm_prefill_workspace_bytes(d, T), false);
    }
    // every field at its ends
    for (int field = 0; field < 7; ++field)
        for (int v : {INT_MIN, -1, 0, 3, 48, 1 << 30, INT_MAX}) {
            gdn_ssm_dims d = good;
            (&d.batch)[field] = v;
            const bool ok = (field == 0 && (v == 3 || v == 48)) || (field == 1 && v == 48) ||
                            (field == 2 && (v == 3 || v == 48)) || (field == 6 && v == 0);
            expect_size("dims", gdn_ssm_state_bytes(&d), ok);
            expect_size("dims ws", gdn_ssm_prefill_workspace_bytes(&d, 100), ok);
            if (!ok)
                expect("dims token",
                       gdn_ssm_decode_token(&d, ff, f, g, f, f, f, ff, ff, ff, ff, f, f, nullptr),
                       field == 6 ? GDN_ERR_DTYPE : GDN_ERR_SHAPE);
        }
    gdn_ssm_dims wide{1 << 20, 1, 1, 128, 32, 4, GDN_F32};   // 16 GB of states, the largest product of sizes
    expect_size("wide", gdn_ssm_prefill_workspace_bytes(&wide, GDN_SSM_MAX_TOKENS), true);
    wide.batch = 1 << 21;
    expect_size("too wide", gdn_ssm_state_bytes(&wide), false);

    expect("null dims", gdn_ssm_decode_token(nullptr, ff, f, g, f, f, f, ff, ff, ff, ff, f, f, nullptr), GDN_ERR_NULL);
    expect("null x", gdn_ssm_decode_token(&good, ff, f, g, f, f, nullptr, ff, ff, ff, ff, f, f, nullptr), GDN_ERR_NULL);
    expect("align z", gdn_ssm_decode_token(&good, ff, f, g, f, f, f, ff, ff, ff, ff, mis, f, nullptr), GDN_ERR_ALIGN);
    expect("alias", gdn_ssm_decode_token(&good, ff, f, f, f, f, f, ff, ff, ff, ff, f, f, nullptr), GDN_ERR_ALIAS);
    const size_t need = gdn_ssm_prefill_workspace_bytes(&good, 100);
    auto prefill = [&](int T, const int32_t* lengths, void* ws, size_t bytes) {
        return gdn_ssm_prefill(&good, ff, f, f, f, T, f, ff, ff, ff, ff, f, lengths, f, nullptr, ws, bytes, nullptr);
    };
    expect("T", prefill(0, nullptr, f, need), GDN_ERR_SHAPE);
    expect("T", prefill(INT_MAX, nullptr, f, need), GDN_ERR_SHAPE);
    expect("lengths", prefill(100, static_cast<int32_t*>(mis), f, need), GDN_ERR_ALIGN);
    expect("short ws", prefill(100, nullptr, f, need - 1), GDN_ERR_WORKSPACE);
    expect("no ws", prefill(100, nullptr, nullptr, need), GDN_ERR_WORKSPACE);
    expect("ws", prefill(100, nullptr, reinterpret_cast<void*>(0x1080), need), GDN_ERR_ALIGN);

    expect_size("select ws", gdn_beam_select_workspace_bytes(1, 1, 1, 1), true);
    expect_size("select ws", gdn_beam_select_workspace_bytes(1 << 15, 32, (1 << 26) - 1, 64), true);
    for (int v : {INT_MIN, -1, 0, INT_MAX}) {
        expect_size("select ws", gdn_beam_select_workspace_bytes(v, 4, 1000, 8), false);
        expect_size("select ws", gdn_beam_select_workspace_bytes(2, v, 1000, 8), false);
        expect_size("select ws", gdn_beam_select_workspace_bytes(2, 4, v, 8), false);
        expect_size("select ws", gdn_beam_select_workspace_bytes(2, 4, 1000, v), false);
    }
    const size_t sel = gdn_beam_select_workspace_bytes(2, 4, 1000, 8);
    auto select = [&](int64_t pitch, int eos, int S, float* out, size_t bytes) {
        return gdn_beam_select(2, 4, 1000, pitch, GDN_BF16, f, ff, static_cast<uint8_t*>(f), eos, S, out, fi, fi, g,
                               bytes, nullptr);
    };
    expect("pitch", select(999, 0, 8, static_cast<float*>(g), sel), GDN_ERR_SHAPE);
    expect("pitch", select(INT64_MAX, 0, 8, static_cast<float*>(g), sel), GDN_ERR_SHAPE);
    expect("pitch", select(INT64_MIN, 0, 8, static_cast<float*>(g), sel), GDN_ERR_SHAPE);
    expect("eos", select(1000, INT_MAX, 8, static_cast<float*>(g), sel), GDN_ERR_INDEX);
    expect("ws", select(1000, 0, 8, static_cast<float*>(g), sel - 1), GDN_ERR_WORKSPACE);
    expect("overlap", select(1000, 0, 8, ff, sel), GDN_ERR_ALIAS);

    for (int K : {INT_MIN, -1, 0, 3, 33, INT_MAX})
        expect("beams", gdn_ssm_beam_reorder(&good, K, ff, f, fi, nullptr, nullptr), GDN_ERR_SHAPE);
    expect("parent", gdn_ssm_beam_reorder(&good, 2, ff, f, nullptr, nullptr, nullptr), GDN_ERR_NULL);
    const gdn_dims gd{4, 16, 48, 128, 128, 4, GDN_BF16};
    expect("beams", gdn_beam_reorder(&gd, 3, ff, f, fi, nullptr, nullptr), GDN_ERR_SHAPE);
    expect("state", gdn_beam_reorder(&gd, 2, static_cast<float*>(mis), f, fi, nullptr, nullptr), GDN_ERR_ALIGN);
    const gdn_dims most{INT_MAX, 16, 48, 128, 128, 4, GDN_BF16};
    expect("most", gdn_beam_reorder(&most, 1, ff, f, fi, nullptr, nullptr), GDN_ERR_SHAPE);

    if (failures)
        return 1;
    std::printf("every call refused as expected\n");
    return 0;
}
