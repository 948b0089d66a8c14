// gdn_api.hip -- the C ABI declared in include/gdn.h: argument checks, then
// launches on the caller's stream.  Nothing here allocates, synchronises or
// keeps state between calls.
//
// Shapes are refused loudly rather than run wrongly (the CPU page's account of
// a hard-coded head width that silently corrupted memory ends with the engine
// refusing unsupported head sizes outright).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gdn.h"
#include "gdn_launch.hpp"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Validates dims and fills the kernel geometry.
gdn_status check_dims(const gdn_dims* d, gdn::Geo& g) {
    if (!d)
        return GDN_ERR_NULL;
    if (d->act_dtype != GDN_F32 && d->act_dtype != GDN_BF16)
        return GDN_ERR_DTYPE;
    if (d->batch < 1 || d->num_k_heads < 1 || d->num_v_heads < 1 || d->num_v_heads % d->num_k_heads != 0 ||
        d->head_k_dim != d->head_v_dim || (d->head_k_dim != 32 && d->head_k_dim != 128) || d->conv_width != 4)
        return GDN_ERR_SHAPE;
    const int64_t C = 2ll * d->num_k_heads * d->head_k_dim + static_cast<int64_t>(d->num_v_heads) * d->head_v_dim;
    // Kernel index arithmetic keeps per-sequence channel and head offsets in 32 bits.
    if (C > (1ll << 24) || static_cast<int64_t>(d->batch) * d->num_v_heads > (1ll << 24))
        return GDN_ERR_SHAPE;
    g.B = d->batch;
    g.Hk = d->num_k_heads;
    g.Hv = d->num_v_heads;
    g.D = d->head_k_dim;
    g.C = static_cast<int>(C);
    g.bf16 = d->act_dtype == GDN_BF16;
    return GDN_OK;
}

gdn_status ptrs_ok(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!p)
            return GDN_ERR_NULL;
    for (const void* p : ps)
        if (!aligned16(p))
            return GDN_ERR_ALIGN;
    return GDN_OK;
}

gdn_status launched(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// ws_optional: the UT-form calls accept a NULL workspace (the one-launch form).
gdn_status tree_verify_args(const gdn_dims* d, gdn::Geo& g, std::initializer_list<const void*> ptrs, int32_t n_nodes,
                            const int32_t* tree_status, const void* workspace, size_t workspace_bytes,
                            bool ws_optional = false) {
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK && (g.B > GDN_MAX_TREE_BATCH || g.Hv / g.Hk > 64))
        st = GDN_ERR_SHAPE;
    if (st == GDN_OK)
        st = ptrs_ok(ptrs);
    if (st == GDN_OK && tree_status && !aligned16(tree_status))
        st = GDN_ERR_ALIGN;
    if (st == GDN_OK && (n_nodes < 1 || n_nodes > GDN_MAX_TREE_NODES))
        st = GDN_ERR_TREE;
    if (st != GDN_OK)
        return st;
    if (ws_optional && !workspace)
        return GDN_OK;
    if (!workspace || workspace_bytes < gdn::tree_ws_bytes(g.B, n_nodes, g.Hk, g.Hv, g.D))
        return GDN_ERR_WORKSPACE;
    return aligned16(workspace) ? GDN_OK : GDN_ERR_ALIGN;
}

gdn_status check_ssm_dims(const gdn_ssm_dims* d, gdn::SsmGeo& g) {
    if (!d)
        return GDN_ERR_NULL;
    if (d->act_dtype != GDN_F32 && d->act_dtype != GDN_BF16)
        return GDN_ERR_DTYPE;
    if (d->batch < 1 || d->num_heads < 1 || d->num_groups < 1 || d->num_heads % d->num_groups != 0 ||
        (d->head_dim != 32 && d->head_dim != 64 && d->head_dim != 128) ||
        (d->state_dim != 32 && d->state_dim != 64 && d->state_dim != 128 && d->state_dim != 256) ||
        d->conv_width != 4)
        return GDN_ERR_SHAPE;
    const int64_t C = static_cast<int64_t>(d->num_heads) * d->head_dim + 2ll * d->num_groups * d->state_dim;
    // A chunk of 64 rows is addressed by 32-bit byte offsets, and a launch counts 2^32 threads: 16 per state row.
    if (C > (1ll << 22) || static_cast<int64_t>(d->batch) * d->num_heads * d->head_dim >= (1ll << 28))
        return GDN_ERR_SHAPE;
    g = {d->batch, d->num_heads, d->num_groups, d->head_dim, d->state_dim, static_cast<int>(C),
         d->act_dtype == GDN_BF16};
    return GDN_OK;
}

size_t ssm_tail_bytes(const gdn::SsmGeo& g) { return static_cast<size_t>(g.B) * g.C * 4 * (g.bf16 ? 2 : 4); }

gdn_status aligned_or_null(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned16(p))
            return GDN_ERR_ALIGN;
    return GDN_OK;
}

bool beam_sizes_ok(int32_t batch, int32_t beams, int32_t vocab, int32_t select) {
    return batch >= 1 && beams >= 1 && beams <= GDN_MAX_BEAMS && vocab >= 1 &&
           static_cast<int64_t>(beams) * vocab < (1ll << 31) && select >= 1 && select <= GDN_MAX_BEAM_SELECT &&
           select <= static_cast<int64_t>(beams) * vocab && static_cast<int64_t>(batch) * beams <= (1ll << 20);
}

// An operand as the alias check sees it: `rows` rows of `bytes` bytes, `pitch` bytes apart.
struct Span {
    const void* p;
    int64_t rows, bytes, pitch;
};

bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p)
        return false;
    const int64_t pa = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p)),
                  pb = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p));
    const int64_t ea = pa + (a.rows - 1) * a.pitch + a.bytes, eb = pb + (b.rows - 1) * b.pitch + b.bytes;
    if (pa >= eb || pb >= ea)
        return false;
    if (a.pitch != b.pitch)
        return true;
    // rows of one pitch may lie between each other's
    int64_t d = (pb - pa) % a.pitch;
    d = d < 0 ? d + a.pitch : d;
    return d < a.bytes || a.pitch - d < b.bytes;
}

// Whether an output overlaps an input or another output.
bool any_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (overlap(*o, i))
                return true;
        for (const Span* u = o + 1; u != outs.end(); ++u)
            if (overlap(*o, *u))
                return true;
    }
    return false;
}

gdn_status lru_pitch(const gdn_lru_pitches* q, int W, gdn::Pitches& p) {
    const int64_t w = W;
    p = {w, w, w, w, w};
    if (!q)
        return GDN_OK;
    const int64_t in[5] = {q->x, q->r, q->i, q->z, q->y};
    int64_t* const out[5] = {&p.x, &p.r, &p.i, &p.z, &p.y};
    for (int k = 0; k < 5; ++k) {
        if (in[k] == 0)
            continue;
        // a tile of rows is addressed by 32-bit byte offsets
        if (in[k] < w || in[k] % 8 != 0 || in[k] > (1 << 20))
            return GDN_ERR_SHAPE;
        *out[k] = in[k];
    }
    return GDN_OK;
}

gdn_status check_lru(const gdn_lru_dims* d, const gdn_lru_pitches* pitch, int64_t T, gdn::LruGeo& g) {
    if (!d)
        return GDN_ERR_NULL;
    if (d->act_dtype != GDN_F32 && d->act_dtype != GDN_BF16)
        return GDN_ERR_DTYPE;
    if (d->batch < 1 || d->width < 8 || d->width % 8 != 0 || d->width > GDN_LRU_MAX_WIDTH || T < 1 ||
        T > GDN_LRU_MAX_TOKENS)
        return GDN_ERR_SHAPE;
    // a launch counts 2^32 threads, and narrow tiles of 512 take 64 channels and at least 64 tokens (fewer
    // channels or tokens only where all of a sequence's are in it); wide tiles are taken where they are no more
    if (static_cast<int64_t>(d->batch) * ((d->width + 63) / 64) * ((T + 63) / 64) >= (1ll << 23))
        return GDN_ERR_SHAPE;
    g.B = d->batch;
    g.W = d->width;
    g.bf16 = d->act_dtype == GDN_BF16;
    return lru_pitch(pitch, g.W, g.p);
}

Span lru_rows(const gdn::LruGeo& g, const void* p, int64_t T, int64_t pitch) {
    const int64_t e = g.bf16 ? 2 : 4;
    return {p, g.B * T, g.W * e, pitch * e};
}
Span dense(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }

bool act_ok(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }

gdn_status norm_sizes(int64_t rows, int32_t H, int32_t D, int32_t act, int32_t other, float eps) {
    if (!act_ok(act) || !act_ok(other) || (other != GDN_F32 && other != act))
        return GDN_ERR_DTYPE;
    if (rows < 1 || rows >= (1ll << 31) || H < 1 || H > 65536 || rows * H >= (1ll << 31) || D < 8 || D % 8 != 0 ||
        D > GDN_NORM_MAX_WIDTH || !(eps >= 1.17549435e-38f) || !(eps <= 3.402823466e38f))
        return GDN_ERR_SHAPE;
    return GDN_OK;
}

gdn_status workspace_ok(const void* workspace, size_t have, size_t need) {
    if (need == 0)
        return GDN_OK;
    if (!workspace || have < need)
        return GDN_ERR_WORKSPACE;
    return reinterpret_cast<uintptr_t>(workspace) & 255u ? GDN_ERR_ALIGN : GDN_OK;
}

}  // namespace

extern "C" {

int gdn_abi_version(void) { return GDN_ABI_VERSION; }

const char* gdn_status_str(int status) {
    switch (status) {
        case GDN_OK: return "ok";
        case GDN_ERR_NULL: return "a required pointer is NULL";
        case GDN_ERR_SHAPE: return "unsupported or inconsistent shape";
        case GDN_ERR_DTYPE: return "unsupported activation dtype";
        case GDN_ERR_ALIGN: return "pointer not 16-byte aligned";
        case GDN_ERR_TREE: return "malformed draft tree or path";
        case GDN_ERR_WORKSPACE: return "workspace missing or too small";
        case GDN_ERR_HIP: return "HIP launch failed";
        case GDN_ERR_ALIAS: return "buffers that must be distinct overlap";
        case GDN_ERR_SIGNATURE: return "snapshot of another layer shape or format";
        case GDN_ERR_INDEX: return "sequence index out of range or repeated";
        case GDN_ERR_SELF_CHECK: return "self-check: verify or commit rows differ from decode";
        default: return "unknown status";
    }
}

size_t gdn_conv_channels(const gdn_dims* d) {
    gdn::Geo g;
    return check_dims(d, g) == GDN_OK ? static_cast<size_t>(g.C) : 0;
}

size_t gdn_state_bytes(const gdn_dims* d) {
    gdn::Geo g;
    if (check_dims(d, g) != GDN_OK)
        return 0;
    return static_cast<size_t>(g.B) * g.Hv * g.D * g.D * sizeof(float);
}

size_t gdn_conv_tail_bytes(const gdn_dims* d) {
    gdn::Geo g;
    if (check_dims(d, g) != GDN_OK)
        return 0;
    return static_cast<size_t>(g.B) * g.C * 4 * (g.bf16 ? 2 : 4);
}

gdn_status gdn_conv_update(const gdn_dims* d, const void* x, void* conv_tail, const void* conv_w, float* y,
                           void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK)
        st = ptrs_ok({x, conv_tail, conv_w, y});
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_conv_update(g, x, conv_tail, conv_w, y, as_stream(stream)));
}

gdn_status gdn_decode_step(const gdn_dims* d, float* state, const float* y, const float* a, const float* b,
                           float* o, void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK)
        st = ptrs_ok({state, y, a, b, o});
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_decode(g, state, y, a, b, o, as_stream(stream)));
}

gdn_status gdn_decode_token(const gdn_dims* d, float* state, const void* conv_tail_in, void* conv_tail_out,
                            const void* conv_w, const void* x, const float* a, const float* b, float* o,
                            void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK)
        st = ptrs_ok({state, conv_tail_in, conv_tail_out, conv_w, x, a, b, o});
    if (st != GDN_OK)
        return st;
    const size_t tail_bytes = static_cast<size_t>(g.B) * g.C * 4 * (g.bf16 ? 2 : 4);
    const uintptr_t ti = reinterpret_cast<uintptr_t>(conv_tail_in), to = reinterpret_cast<uintptr_t>(conv_tail_out);
    if (ti < to + tail_bytes && to < ti + tail_bytes)
        return GDN_ERR_ALIAS;
    return launched(gdn::launch_token(g, state, conv_tail_in, conv_tail_out, conv_w, x, a, b, o, as_stream(stream)));
}

gdn_status gdn_kda_decode_step(const gdn_dims* d, float* state, const float* y, const float* a, const float* b,
                               float* o, void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK)
        st = ptrs_ok({state, y, a, b, o});
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_kda_decode(g, state, y, a, b, o, as_stream(stream)));
}

gdn_status gdn_kda_decode_token(const gdn_dims* d, float* state, const void* conv_tail_in, void* conv_tail_out,
                                const void* conv_w, const void* x, const float* a, const float* b, float* o,
                                void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK)
        st = ptrs_ok({state, conv_tail_in, conv_tail_out, conv_w, x, a, b, o});
    if (st != GDN_OK)
        return st;
    const size_t tail_bytes = static_cast<size_t>(g.B) * g.C * 4 * (g.bf16 ? 2 : 4);
    const uintptr_t ti = reinterpret_cast<uintptr_t>(conv_tail_in), to = reinterpret_cast<uintptr_t>(conv_tail_out);
    if (ti < to + tail_bytes && to < ti + tail_bytes)
        return GDN_ERR_ALIAS;
    return launched(
        gdn::launch_kda_token(g, state, conv_tail_in, conv_tail_out, conv_w, x, a, b, o, as_stream(stream)));
}

gdn_status gdn_tree_tables(int32_t n_nodes, const int32_t* parent, int32_t* depth, int32_t* order,
                           int32_t* tree_status, void* stream) {
    if (n_nodes < 1 || n_nodes > GDN_MAX_TREE_NODES)
        return GDN_ERR_TREE;
    const gdn_status st = ptrs_ok({parent, depth, order, tree_status});
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_tree_tables(n_nodes, parent, depth, order, tree_status, as_stream(stream)));
}

size_t gdn_tree_workspace_bytes(const gdn_dims* d, int32_t n_nodes) {
    gdn::Geo g;
    if (check_dims(d, g) != GDN_OK || n_nodes < 1 || n_nodes > GDN_MAX_TREE_NODES)
        return 0;
    return gdn::tree_ws_bytes(g.B, n_nodes, g.Hk, g.Hv, g.D);
}

gdn_status gdn_tree_verify(const gdn_dims* d, const float* state_ckpt, const void* conv_tail, const void* conv_w,
                           int32_t n_nodes, const int32_t* parent, const void* x, const float* a, const float* b,
                           float* o, int32_t* tree_status, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::Geo g;
    const gdn_status st = tree_verify_args(d, g, {state_ckpt, conv_tail, conv_w, parent, x, a, b, o}, n_nodes,
                                           tree_status, workspace, workspace_bytes);
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_tree_verify(g, state_ckpt, conv_tail, conv_w, n_nodes, parent, x, a, b, o,
                                            tree_status, workspace, as_stream(stream)));
}

gdn_status gdn_tree_verify_ut(const gdn_dims* d, const float* state_ckpt, const void* conv_tail, const void* conv_w,
                              int32_t n_nodes, const int32_t* parent, const void* x, const float* a, const float* b,
                              float* o, int32_t* tree_status, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::Geo g;
    const gdn_status st = tree_verify_args(d, g, {state_ckpt, conv_tail, conv_w, parent, x, a, b, o}, n_nodes,
                                           tree_status, workspace, workspace_bytes, true);
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_tree_verify_ut(g, state_ckpt, conv_tail, conv_w, n_nodes, parent, x, a, b, o,
                                               tree_status, workspace, as_stream(stream)));
}

gdn_status gdn_commit_path(const gdn_dims* d, float* state, void* conv_tail, const void* conv_w, int32_t n_nodes,
                           const int32_t* parent, const void* x, const float* a, const float* b, int32_t path_len,
                           const int32_t* path, float* o, int32_t* tree_status, void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK && (g.B > GDN_MAX_TREE_BATCH || g.Hv / g.Hk > 64))
        st = GDN_ERR_SHAPE;
    if (st == GDN_OK)
        st = ptrs_ok({state, conv_tail, conv_w, parent, x, a, b, path});
    if (st == GDN_OK && ((o && !aligned16(o)) || (tree_status && !aligned16(tree_status))))
        st = GDN_ERR_ALIGN;
    if (st == GDN_OK && (n_nodes < 1 || n_nodes > GDN_MAX_TREE_NODES || path_len < 1 ||
                         path_len > GDN_MAX_TREE_DEPTH || path_len > n_nodes))
        st = GDN_ERR_TREE;
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_commit(g, state, conv_tail, conv_w, n_nodes, parent, x, a, b, path_len, path, o,
                                       tree_status, nullptr, as_stream(stream)));
}

gdn_status gdn_commit_path_prepared(const gdn_dims* d, float* state, void* conv_tail, int32_t n_nodes,
                                    const int32_t* parent, const void* x, int32_t path_len, const int32_t* path,
                                    float* o, int32_t* tree_status, const void* workspace, size_t workspace_bytes,
                                    void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK && (g.B > GDN_MAX_TREE_BATCH || g.Hv / g.Hk > 64))
        st = GDN_ERR_SHAPE;
    if (st == GDN_OK)
        st = ptrs_ok({state, conv_tail, parent, x, path});
    if (st == GDN_OK && ((o && !aligned16(o)) || (tree_status && !aligned16(tree_status))))
        st = GDN_ERR_ALIGN;
    if (st == GDN_OK && (n_nodes < 1 || n_nodes > GDN_MAX_TREE_NODES || path_len < 1 ||
                         path_len > GDN_MAX_TREE_DEPTH || path_len > n_nodes))
        st = GDN_ERR_TREE;
    if (st != GDN_OK)
        return st;
    if (!workspace || workspace_bytes < gdn::tree_ws_bytes(g.B, n_nodes, g.Hk, g.Hv, g.D))
        return GDN_ERR_WORKSPACE;
    if (!aligned16(workspace))
        return GDN_ERR_ALIGN;
    return launched(gdn::launch_commit(g, state, conv_tail, nullptr, n_nodes, parent, x, nullptr, nullptr, path_len,
                                       path, o, tree_status, const_cast<void*>(workspace), as_stream(stream)));
}

size_t gdn_block_workspace_bytes(const gdn_dims* d, int32_t k) {
    gdn::Geo g;
    if (check_dims(d, g) != GDN_OK || k < 1 || k > GDN_MAX_TREE_NODES)
        return 0;
    return gdn::tree_ws_bytes(g.B, k, g.Hk, g.Hv, g.D);
}

}  // extern "C"

namespace {

gdn_status block_args(const gdn_dims* d, gdn::Geo& g, std::initializer_list<const void*> ptrs, int32_t k,
                      const void* o, const int32_t* status, const void* workspace, size_t workspace_bytes,
                      bool ws_optional = false) {
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK && (g.B > GDN_MAX_TREE_BATCH || g.Hv / g.Hk > 64))
        st = GDN_ERR_SHAPE;
    if (st == GDN_OK)
        st = ptrs_ok(ptrs);
    if (st == GDN_OK && ((o && !aligned16(o)) || (status && !aligned16(status))))
        st = GDN_ERR_ALIGN;
    if (st == GDN_OK && (k < 1 || k > GDN_MAX_TREE_NODES))
        st = GDN_ERR_SHAPE;
    if (st != GDN_OK)
        return st;
    if (ws_optional && !workspace)
        return GDN_OK;
    if (!workspace || workspace_bytes < gdn::tree_ws_bytes(g.B, k, g.Hk, g.Hv, g.D))
        return GDN_ERR_WORKSPACE;
    return aligned16(workspace) ? GDN_OK : GDN_ERR_ALIGN;
}

}  // namespace

extern "C" {

gdn_status gdn_block_verify(const gdn_dims* d, const float* state_ckpt, const void* conv_tail, const void* conv_w,
                            int32_t k, const void* x, const float* a, const float* b, float* o, void* workspace,
                            size_t workspace_bytes, void* stream) {
    gdn::Geo g;
    const gdn_status st = block_args(d, g, {state_ckpt, conv_tail, conv_w, x, a, b, o}, k, o, nullptr, workspace,
                                     workspace_bytes);
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_block(g, false, const_cast<float*>(state_ckpt), const_cast<void*>(conv_tail),
                                      conv_w, k, x, a, b, nullptr, o, nullptr, workspace, false,
                                      as_stream(stream)));
}

gdn_status gdn_block_verify_ut(const gdn_dims* d, const float* state_ckpt, const void* conv_tail, const void* conv_w,
                               int32_t k, const void* x, const float* a, const float* b, float* o, void* workspace,
                               size_t workspace_bytes, void* stream) {
    gdn::Geo g;
    const gdn_status st = block_args(d, g, {state_ckpt, conv_tail, conv_w, x, a, b, o}, k, o, nullptr, workspace,
                                     workspace_bytes, true);
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_tree_verify_ut(g, state_ckpt, conv_tail, conv_w, k, nullptr, x, a, b, o, nullptr,
                                               workspace, as_stream(stream)));
}

gdn_status gdn_block_commit(const gdn_dims* d, float* state, void* conv_tail, const void* conv_w, int32_t k,
                            const void* x, const float* a, const float* b, const int32_t* accepted, float* o,
                            int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::Geo g;
    const gdn_status st = block_args(d, g, {state, conv_tail, conv_w, x, a, b, accepted}, k, o, status, workspace,
                                     workspace_bytes);
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_block(g, true, state, conv_tail, conv_w, k, x, a, b, accepted, o, status, workspace,
                                      false, as_stream(stream)));
}

gdn_status gdn_block_commit_prepared(const gdn_dims* d, float* state, void* conv_tail, int32_t k, const void* x,
                                     const int32_t* accepted, float* o, int32_t* status, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    gdn::Geo g;
    const gdn_status st = block_args(d, g, {state, conv_tail, x, accepted}, k, o, status, workspace, workspace_bytes);
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_block(g, true, state, conv_tail, nullptr, k, x, nullptr, nullptr, accepted, o, status,
                                      workspace, true, as_stream(stream)));
}

uint64_t gdn_state_signature(const gdn_dims* d) {
    gdn::Geo g;
    return check_dims(d, g) == GDN_OK ? gdn::state_signature(g) : 0;
}

size_t gdn_snapshot_bytes(const gdn_dims* d, int32_t count) {
    gdn::Geo g;
    if (check_dims(d, g) != GDN_OK || count < 1 || count > GDN_MAX_TREE_BATCH)
        return 0;
    return gdn::snapshot_bytes(g, count);
}

}  // extern "C"

namespace {

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

gdn_status snapshot_args(const gdn_dims* d, gdn::Geo& g, const void* state, const void* tail, int32_t count,
                         const int32_t* seqs, const void* blob, size_t blob_bytes, const int32_t* status) {
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK && g.B > GDN_MAX_TREE_BATCH)
        st = GDN_ERR_SHAPE;
    if (st == GDN_OK)
        st = ptrs_ok({state, tail, seqs, blob, status});
    if (st == GDN_OK && (reinterpret_cast<uintptr_t>(blob) & 255u))
        st = GDN_ERR_ALIGN;
    if (st == GDN_OK && (count < 1 || count > GDN_MAX_TREE_BATCH))
        st = GDN_ERR_SHAPE;
    if (st != GDN_OK)
        return st;
    const size_t need = gdn::snapshot_bytes(g, count);
    if (blob_bytes < need)
        return GDN_ERR_WORKSPACE;
    const size_t sb = static_cast<size_t>(g.B) * g.Hv * g.D * g.D * 4;
    const size_t tb = static_cast<size_t>(g.B) * g.C * 4 * (g.bf16 ? 2 : 4);
    if (overlaps(blob, need, state, sb) || overlaps(blob, need, tail, tb))
        return GDN_ERR_ALIAS;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_snapshot(const gdn_dims* d, const float* state, const void* conv_tail, int32_t count,
                        const int32_t* seqs, void* blob, size_t blob_bytes, int32_t* status, void* stream) {
    gdn::Geo g;
    const gdn_status st = snapshot_args(d, g, state, conv_tail, count, seqs, blob, blob_bytes, status);
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_snapshot(g, false, const_cast<float*>(state), const_cast<void*>(conv_tail), count,
                                         seqs, blob, status, as_stream(stream)));
}

gdn_status gdn_restore(const gdn_dims* d, float* state, void* conv_tail, int32_t count, const int32_t* seqs,
                       const void* blob, size_t blob_bytes, int32_t* status, void* stream) {
    gdn::Geo g;
    const gdn_status st = snapshot_args(d, g, state, conv_tail, count, seqs, blob, blob_bytes, status);
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_snapshot(g, true, state, conv_tail, count, seqs, const_cast<void*>(blob), status,
                                         as_stream(stream)));
}

size_t gdn_prefill_workspace_bytes(const gdn_dims* d, int32_t T) {
    gdn::Geo g;
    if (check_dims(d, g) != GDN_OK || T < 1)
        return 0;
    return gdn::prefill_workspace_bytes(g, T);
}

gdn_status gdn_prefill_chunked(const gdn_dims* d, float* state, void* conv_tail, const void* conv_w, int32_t T,
                               const void* x, const float* a, const float* b, float* o, void* workspace,
                               size_t workspace_bytes, void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK)
        st = ptrs_ok({state, conv_tail, conv_w, x, a, b, o});
    if (st == GDN_OK && (T < 1 || g.D != 128 || g.Hv / g.Hk > 8))
        st = GDN_ERR_SHAPE;
    if (st == GDN_OK && static_cast<int64_t>(g.B) * T * g.C >= (1ll << 40))
        st = GDN_ERR_SHAPE;
    if (st != GDN_OK)
        return st;
    const size_t need = gdn::prefill_workspace_bytes(g, T);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return GDN_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace))
        return GDN_ERR_ALIGN;
    return launched(gdn::launch_prefill(g, state, conv_tail, conv_w, T, x, a, b, o, workspace, as_stream(stream)));
}

size_t gdn_self_check_workspace_bytes(const gdn_dims* d) {
    gdn::Geo g;
    if (check_dims(d, g) != GDN_OK || g.Hv / g.Hk > 64)
        return 0;
    return gdn::self_check_ws_bytes(g);
}

gdn_status gdn_self_check(const gdn_dims* d, uint32_t seed, int32_t flags, void* workspace, size_t workspace_bytes,
                          int32_t* result, void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK && g.Hv / g.Hk > 64)
        st = GDN_ERR_SHAPE;
    if (st == GDN_OK)
        st = ptrs_ok({result});
    if (st == GDN_OK && (flags & ~GDN_SELF_CHECK_PERTURB))
        st = GDN_ERR_SHAPE;
    if (st != GDN_OK)
        return st;
    if (!workspace || workspace_bytes < gdn::self_check_ws_bytes(g))
        return GDN_ERR_WORKSPACE;
    if (!aligned16(workspace))
        return GDN_ERR_ALIGN;
    return launched(gdn::launch_self_check(g, workspace, seed, flags & GDN_SELF_CHECK_PERTURB, result,
                                           as_stream(stream)));
}

gdn_status gdn_tree_verify_ut_noalloc(const gdn_dims* d, const float* state_ckpt, const void* conv_tail,
                                      const void* conv_w, int32_t n_nodes, const int32_t* parent, const void* x,
                                      const float* a, const float* b, float* o, int32_t* tree_status, void* stream) {
    gdn::Geo g;
    gdn_status st = check_dims(d, g);
    if (st == GDN_OK && (g.B > GDN_MAX_TREE_BATCH || g.Hv / g.Hk > 64))
        st = GDN_ERR_SHAPE;
    if (st == GDN_OK)
        st = ptrs_ok({state_ckpt, conv_tail, conv_w, parent, x, a, b, o});
    if (st == GDN_OK && tree_status && !aligned16(tree_status))
        st = GDN_ERR_ALIGN;
    if (st == GDN_OK && (n_nodes < 1 || n_nodes > GDN_MAX_TREE_NODES))
        st = GDN_ERR_TREE;
    if (st != GDN_OK)
        return st;
    if (gdn::tree_ws_bytes(g.B, n_nodes, g.Hk, g.Hv, g.D) > GDN_NOALLOC_SCRATCH_BYTES)
        return GDN_ERR_WORKSPACE;
    void* ws = nullptr;
    if (gdn::noalloc_scratch(&ws) != hipSuccess)
        return GDN_ERR_HIP;
    return launched(gdn::launch_tree_verify_ut(g, state_ckpt, conv_tail, conv_w, n_nodes, parent, x, a, b, o,
                                               tree_status, ws, as_stream(stream)));
}

size_t gdn_ssm_conv_channels(const gdn_ssm_dims* d) {
    gdn::SsmGeo g;
    return check_ssm_dims(d, g) == GDN_OK ? static_cast<size_t>(g.C) : 0;
}

size_t gdn_ssm_state_bytes(const gdn_ssm_dims* d) {
    gdn::SsmGeo g;
    return check_ssm_dims(d, g) == GDN_OK ? static_cast<size_t>(g.B) * g.H * g.P * g.N * sizeof(float) : 0;
}

size_t gdn_ssm_conv_tail_bytes(const gdn_ssm_dims* d) {
    gdn::SsmGeo g;
    return check_ssm_dims(d, g) == GDN_OK ? ssm_tail_bytes(g) : 0;
}

gdn_status gdn_ssm_decode_token(const gdn_ssm_dims* d, float* state, const void* conv_tail_in, void* conv_tail_out,
                                const void* conv_w, const void* conv_bias, const void* x, const float* dt,
                                const float* dt_bias, const float* A, const float* D, const void* z, void* y,
                                void* stream) {
    gdn::SsmGeo g;
    gdn_status st = check_ssm_dims(d, g);
    if (st == GDN_OK)
        st = ptrs_ok({state, conv_tail_in, conv_tail_out, conv_w, x, dt, A, y});
    if (st == GDN_OK)
        st = aligned_or_null({conv_bias, dt_bias, D, z});
    if (st != GDN_OK)
        return st;
    const uintptr_t ti = reinterpret_cast<uintptr_t>(conv_tail_in), to = reinterpret_cast<uintptr_t>(conv_tail_out);
    if (ti < to + ssm_tail_bytes(g) && to < ti + ssm_tail_bytes(g))
        return GDN_ERR_ALIAS;
    const gdn::SsmArgs a{state, conv_tail_in, conv_w, conv_bias, conv_tail_out, x, dt, dt_bias, A, D, z, y};
    return launched(gdn::launch_ssm_token(g, a, as_stream(stream)));
}

size_t gdn_ssm_prefill_workspace_bytes(const gdn_ssm_dims* d, int32_t T) {
    gdn::SsmGeo g;
    if (check_ssm_dims(d, g) != GDN_OK || T < 1 || T > GDN_SSM_MAX_TOKENS)
        return 0;
    return gdn::ssm_prefill_ws_bytes(g, T);
}

gdn_status gdn_ssm_prefill(const gdn_ssm_dims* d, float* state, void* conv_tail, const void* conv_w,
                           const void* conv_bias, int32_t T, const void* x, const float* dt, const float* dt_bias,
                           const float* A, const float* D, const void* z, const int32_t* lengths, void* y,
                           int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::SsmGeo g;
    gdn_status st = check_ssm_dims(d, g);
    if (st == GDN_OK && (T < 1 || T > GDN_SSM_MAX_TOKENS))
        st = GDN_ERR_SHAPE;
    if (st == GDN_OK)
        st = ptrs_ok({state, conv_tail, conv_w, x, dt, A, y});
    if (st == GDN_OK)
        st = aligned_or_null({conv_bias, dt_bias, D, z, lengths, status});
    if (st != GDN_OK)
        return st;
    if (!workspace || workspace_bytes < gdn::ssm_prefill_ws_bytes(g, T))
        return GDN_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return GDN_ERR_ALIGN;
    const gdn::SsmArgs a{state, conv_tail, conv_w, conv_bias, conv_tail, x, dt, dt_bias, A, D, z, y};
    return launched(gdn::launch_ssm_prefill(g, a, T, lengths, status, workspace, as_stream(stream)));
}

size_t gdn_beam_select_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t select) {
    return beam_sizes_ok(batch, beams, vocab, select) ? gdn::beam_select_ws_bytes(batch, beams, vocab, select) : 0;
}

gdn_status gdn_beam_select(int32_t batch, int32_t beams, int32_t vocab, int64_t vocab_pitch, int32_t act_dtype,
                           const void* logits, const float* scores, const uint8_t* finished, int32_t eos,
                           int32_t select, float* out_scores, int32_t* parent, int32_t* token, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (act_dtype != GDN_F32 && act_dtype != GDN_BF16)
        return GDN_ERR_DTYPE;
    // a pitch of 2^40 elements is far beyond any memory and keeps every offset within 64 bits
    if (!beam_sizes_ok(batch, beams, vocab, select) || vocab_pitch < vocab || vocab_pitch > (1ll << 40))
        return GDN_ERR_SHAPE;
    if (!logits)
        return GDN_ERR_NULL;
    gdn_status st = ptrs_ok({scores, out_scores, parent, token});
    if (st == GDN_OK && ((reinterpret_cast<uintptr_t>(logits) & (act_dtype == GDN_BF16 ? 1u : 3u)) ||
                         !aligned16(finished)))
        st = GDN_ERR_ALIGN;
    if (st == GDN_OK && finished && (eos < 0 || eos >= vocab))
        st = GDN_ERR_INDEX;
    if (st != GDN_OK)
        return st;
    if (!workspace || workspace_bytes < gdn::beam_select_ws_bytes(batch, beams, vocab, select))
        return GDN_ERR_WORKSPACE;
    if (!aligned16(workspace))
        return GDN_ERR_ALIGN;
    // in place a workgroup replaces the scores that it alone has read; any other overlap is a race
    const uintptr_t si = reinterpret_cast<uintptr_t>(scores), so = reinterpret_cast<uintptr_t>(out_scores);
    const uintptr_t in_bytes = 4ull * batch * beams, out_bytes = 4ull * batch * select;
    if (si < so + out_bytes && so < si + in_bytes && !(si == so && select == beams))
        return GDN_ERR_ALIAS;
    const gdn::BeamGeo g{batch, beams, vocab, select, vocab_pitch, act_dtype == GDN_BF16};
    return launched(gdn::launch_beam_select(g, logits, scores, finished, eos, out_scores, parent, token, workspace,
                                            as_stream(stream)));
}

static gdn_status beam_reorder(int32_t batch, int32_t beams, int64_t state_bytes, int64_t tail_bytes, float* state,
                               void* conv_tail, const int32_t* parent, int32_t* status, void* stream) {
    if (beams < 1 || beams > GDN_MAX_BEAMS || batch % beams != 0)
        return GDN_ERR_SHAPE;
    // one workgroup per 4 KB of a sequence and group; a launch counts 2^32 threads
    if ((state_bytes + tail_bytes + 4095) / 4096 * (batch / beams) >= (1ll << 24))
        return GDN_ERR_SHAPE;
    gdn_status st = ptrs_ok({state, conv_tail, parent});
    if (st == GDN_OK)
        st = aligned_or_null({status});
    if (st != GDN_OK)
        return st;
    return launched(gdn::launch_beam_reorder(batch / beams, beams, state_bytes, tail_bytes, state, conv_tail, parent,
                                             status, as_stream(stream)));
}

gdn_status gdn_beam_reorder(const gdn_dims* d, int32_t beams, float* state, void* conv_tail, const int32_t* parent,
                            int32_t* status, void* stream) {
    gdn::Geo g;
    const gdn_status st = check_dims(d, g);
    if (st != GDN_OK)
        return st;
    return beam_reorder(g.B, beams, static_cast<int64_t>(g.Hv) * g.D * g.D * 4,
                        static_cast<int64_t>(g.C) * 4 * (g.bf16 ? 2 : 4), state, conv_tail, parent, status, stream);
}

gdn_status gdn_ssm_beam_reorder(const gdn_ssm_dims* d, int32_t beams, float* state, void* conv_tail,
                                const int32_t* parent, int32_t* status, void* stream) {
    gdn::SsmGeo g;
    const gdn_status st = check_ssm_dims(d, g);
    if (st != GDN_OK)
        return st;
    return beam_reorder(g.B, beams, static_cast<int64_t>(g.H) * g.P * g.N * 4,
                        static_cast<int64_t>(g.C) * 4 * (g.bf16 ? 2 : 4), state, conv_tail, parent, status, stream);
}

size_t gdn_lru_state_bytes(const gdn_lru_dims* d) {
    gdn::LruGeo g;
    return check_lru(d, nullptr, 1, g) == GDN_OK ? static_cast<size_t>(g.B) * g.W * sizeof(float) : 0;
}

gdn_status gdn_lru_decode_token(const gdn_lru_dims* d, const gdn_lru_pitches* pitch, float* state, const void* x,
                                const void* r, const void* i, const float* A, const void* z, void* y, void* stream) {
    gdn::LruGeo g;
    gdn_status st = check_lru(d, pitch, 1, g);
    if (st == GDN_OK)
        st = ptrs_ok({state, x, r, i, A, y});
    if (st == GDN_OK)
        st = aligned_or_null({z});
    if (st != GDN_OK)
        return st;
    if (any_overlap({lru_rows(g, y, 1, g.p.y), dense(state, 4ll * g.B * g.W)},
                    {lru_rows(g, x, 1, g.p.x), lru_rows(g, r, 1, g.p.r), lru_rows(g, i, 1, g.p.i),
                     lru_rows(g, z, 1, g.p.z), dense(A, 4ll * g.W)}))
        return GDN_ERR_ALIAS;
    return launched(gdn::launch_lru_token(g, {state, x, r, i, A, z, y}, as_stream(stream)));
}

size_t gdn_lru_prefill_workspace_bytes(const gdn_lru_dims* d, int32_t T) {
    gdn::LruGeo g;
    return check_lru(d, nullptr, T, g) == GDN_OK ? gdn::lru_prefill_ws_bytes(g, T) : 0;
}

size_t gdn_lru_saved_bytes(const gdn_lru_dims* d, int32_t T) {
    gdn::LruGeo g;
    return check_lru(d, nullptr, T, g) == GDN_OK ? gdn::lru_saved_bytes(g, T) : 0;
}

gdn_status gdn_lru_prefill(const gdn_lru_dims* d, const gdn_lru_pitches* pitch, float* state, int32_t T, const void* x,
                           const void* r, const void* i, const float* A, const void* z, const int32_t* lengths,
                           void* y, float* saved, int32_t* status, void* workspace, size_t workspace_bytes,
                           void* stream) {
    gdn::LruGeo g;
    gdn_status st = check_lru(d, pitch, T, g);
    if (st == GDN_OK)
        st = ptrs_ok({state, x, r, i, A, y});
    if (st == GDN_OK)
        st = aligned_or_null({z, lengths, saved, status});
    if (st != GDN_OK)
        return st;
    const size_t need = gdn::lru_prefill_ws_bytes(g, T);
    st = workspace_ok(workspace, workspace_bytes, need);
    if (st != GDN_OK)
        return st;
    const Span ws = dense(need ? workspace : nullptr, static_cast<int64_t>(need));
    if (any_overlap({lru_rows(g, y, T, g.p.y), dense(state, 4ll * g.B * g.W),
                     dense(saved, static_cast<int64_t>(gdn::lru_saved_bytes(g, T))), dense(status, 4ll * g.B), ws},
                    {lru_rows(g, x, T, g.p.x), lru_rows(g, r, T, g.p.r), lru_rows(g, i, T, g.p.i),
                     lru_rows(g, z, T, g.p.z), dense(A, 4ll * g.W), dense(lengths, 4ll * g.B)}))
        return GDN_ERR_ALIAS;
    return launched(gdn::launch_lru_prefill(g, {state, x, r, i, A, z, y}, T, lengths, saved, status, workspace,
                                            as_stream(stream)));
}

size_t gdn_lru_backward_workspace_bytes(const gdn_lru_dims* d, int32_t T) {
    gdn::LruGeo g;
    return check_lru(d, nullptr, T, g) == GDN_OK ? gdn::lru_backward_ws_bytes(g, T) : 0;
}

gdn_status gdn_lru_backward(const gdn_lru_dims* d, const gdn_lru_pitches* pitch, const gdn_lru_pitches* grad_pitch,
                            int32_t T, const void* x, const void* r, const void* i, const float* A, const void* z,
                            const int32_t* lengths, const float* saved, const void* dy, const float* dstate, void* dx,
                            void* dr, void* di, void* dz, float* dA, float* dstate0, int32_t* status, void* workspace,
                            size_t workspace_bytes, void* stream) {
    gdn::LruGeo g;
    gdn_status st = check_lru(d, pitch, T, g);
    if (st == GDN_OK)
        st = lru_pitch(grad_pitch, g.W, g.gp);
    if (st == GDN_OK)
        st = ptrs_ok({x, r, i, A, saved, dy, dx, dr, di, dA});
    if (st == GDN_OK && (z == nullptr) != (dz == nullptr))
        st = GDN_ERR_NULL;
    if (st == GDN_OK)
        st = aligned_or_null({z, dz, lengths, dstate, dstate0, status});
    if (st != GDN_OK)
        return st;
    const size_t need = gdn::lru_backward_ws_bytes(g, T);
    st = workspace_ok(workspace, workspace_bytes, need);
    if (st != GDN_OK)
        return st;
    const int64_t rows4 = 4ll * g.B * g.W;
    const Span in_x = lru_rows(g, x, T, g.p.x), in_r = lru_rows(g, r, T, g.p.r), in_i = lru_rows(g, i, T, g.p.i),
               in_z = lru_rows(g, z, T, g.p.z), in_dy = lru_rows(g, dy, T, g.p.y), in_A = dense(A, 4ll * g.W),
               in_len = dense(lengths, 4ll * g.B),
               in_saved = dense(saved, static_cast<int64_t>(gdn::lru_saved_bytes(g, T)));
    // dstate0 may be dstate itself: a channel's first is read before its last is written
    if (any_overlap({lru_rows(g, dx, T, g.gp.x), lru_rows(g, dr, T, g.gp.r), lru_rows(g, di, T, g.gp.i),
                     lru_rows(g, dz, T, g.gp.z), dense(dA, 4ll * g.W), dense(dstate0, rows4), dense(status, 4ll * g.B),
                     dense(workspace, static_cast<int64_t>(need))},
                    {in_x, in_r, in_i, in_z, in_dy, in_A, in_len, in_saved, dense(dstate == dstate0 ? nullptr : dstate, rows4)}))
        return GDN_ERR_ALIAS;
    return launched(gdn::launch_lru_backward(g, {x, r, i, A, z, saved, dy, dstate, dx, dr, di, dz, dA, dstate0}, T,
                                             lengths, status, workspace, as_stream(stream)));
}

gdn_status gdn_residual_norm(int64_t rows, int32_t W, int32_t act_dtype, int32_t res_dtype, float eps,
                             const void* residual, const void* delta, const float* scale, const float* w_post,
                             const float* w, void* out, void* y, void* stream) {
    gdn_status st = norm_sizes(rows, 1, W, act_dtype, res_dtype, eps);
    if (st == GDN_OK)
        st = ptrs_ok({residual, w, y});
    if (st == GDN_OK && ((delta == nullptr) != (out == nullptr) || (!delta && (scale || w_post))))
        st = GDN_ERR_NULL;
    if (st == GDN_OK)
        st = aligned_or_null({delta, scale, w_post, out});
    if (st != GDN_OK)
        return st;
    const bool act16 = act_dtype == GDN_BF16, res16 = res_dtype == GDN_BF16;
    const int64_t n = rows * W, na = n * (act16 ? 2 : 4), nr = n * (res16 ? 2 : 4);
    if (any_overlap({dense(out, nr), dense(y, na)},
                    {dense(out == residual ? nullptr : residual, nr), dense(delta, na), dense(scale, 4ll * W),
                     dense(w_post, 4ll * W), dense(w, 4ll * W)}) ||
        overlap(dense(y, na), dense(residual, nr)))
        return GDN_ERR_ALIAS;
    return launched(gdn::launch_residual_norm({rows, W, act16, res16, eps, residual, delta, scale, w_post, w, out, y},
                                              as_stream(stream)));
}

size_t gdn_residual_norm_backward_workspace_bytes(int64_t rows, int32_t W) {
    return norm_sizes(rows, 1, W, GDN_F32, GDN_F32, 1.0f) == GDN_OK ? gdn::residual_norm_back_ws_bytes(rows, W) : 0;
}

gdn_status gdn_residual_norm_backward(int64_t rows, int32_t W, int32_t act_dtype, int32_t res_dtype, float eps,
                                      const void* out, const void* delta, const float* scale, const float* w_post,
                                      const float* w, const void* dy, const void* ds, void* dresidual, void* ddelta,
                                      float* dw, float* dscale, float* dw_post, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    gdn_status st = norm_sizes(rows, 1, W, act_dtype, res_dtype, eps);
    if (st == GDN_OK)
        st = ptrs_ok({out, w, dy, dresidual, dw});
    if (st == GDN_OK && ((delta == nullptr) != (ddelta == nullptr) || (scale == nullptr) != (dscale == nullptr) ||
                         (w_post == nullptr) != (dw_post == nullptr) || (!delta && (scale || w_post))))
        st = GDN_ERR_NULL;
    if (st == GDN_OK)
        st = aligned_or_null({delta, scale, w_post, ds, ddelta, dscale, dw_post});
    if (st != GDN_OK)
        return st;
    const size_t need = gdn::residual_norm_back_ws_bytes(rows, W);
    st = workspace_ok(workspace, workspace_bytes, need);
    if (st != GDN_OK)
        return st;
    const bool act16 = act_dtype == GDN_BF16, res16 = res_dtype == GDN_BF16;
    const int64_t n = rows * W, na = n * (act16 ? 2 : 4), nr = n * (res16 ? 2 : 4), nw = 4ll * W;
    if (any_overlap({dense(dresidual, nr), dense(ddelta, na), dense(dw, nw), dense(dscale, nw), dense(dw_post, nw),
                     dense(workspace, static_cast<int64_t>(need))},
                    {dense(out, nr), dense(delta, na), dense(scale, nw), dense(w_post, nw), dense(w, nw),
                     dense(dy, na), dense(ds == dresidual ? nullptr : ds, nr)}))
        return GDN_ERR_ALIAS;
    return launched(gdn::launch_residual_norm_backward({rows, W, act16, res16, eps, out, delta, scale, w_post, w, dy,
                                                        ds, dresidual, ddelta, dw, dscale, dw_post},
                                                       workspace, as_stream(stream)));
}

static gdn_status gated_sizes(int64_t rows, int32_t H, int32_t D, int32_t o_dtype, int32_t act_dtype, int32_t flags,
                              float eps, int64_t& z_pitch) {
    const gdn_status st = norm_sizes(rows, H, D, act_dtype, o_dtype, eps);
    if (st != GDN_OK)
        return st;
    const int64_t row = static_cast<int64_t>(H) * D;
    if (z_pitch == 0)
        z_pitch = row;
    // weights are counted in 32 bits, and offsets of z stay within 64
    if ((flags & ~(GDN_GATE_FIRST | GDN_WEIGHT_PER_HEAD)) || row >= (1ll << 30) || z_pitch < row || z_pitch % 8 != 0 ||
        z_pitch > (1ll << 56) / rows)
        return GDN_ERR_SHAPE;
    return GDN_OK;
}

gdn_status gdn_gated_norm(int64_t rows, int32_t H, int32_t D, int32_t o_dtype, int32_t act_dtype, int32_t flags,
                          float eps, const void* o, const void* z, int64_t z_pitch, const float* w, void* y,
                          void* stream) {
    gdn_status st = gated_sizes(rows, H, D, o_dtype, act_dtype, flags, eps, z_pitch);
    if (st == GDN_OK)
        st = ptrs_ok({o, z, w, y});
    if (st != GDN_OK)
        return st;
    const bool o16 = o_dtype == GDN_BF16, act16 = act_dtype == GDN_BF16, each = flags & GDN_WEIGHT_PER_HEAD;
    const int64_t row = static_cast<int64_t>(H) * D, ea = act16 ? 2 : 4;
    const int64_t nw = 4ll * D * (each ? H : 1);
    if (any_overlap({dense(y, rows * row * ea)}, {dense(o, rows * row * (o16 ? 2 : 4)), dense(w, nw)}) ||
        overlap({y, rows, row * ea, row * ea}, {z, rows, row * ea, z_pitch * ea}))
        return GDN_ERR_ALIAS;
    return launched(gdn::launch_gated_norm(
        {rows, H, D, o16, act16, each, (flags & GDN_GATE_FIRST) != 0, eps, z_pitch, o, z, w, y}, as_stream(stream)));
}

size_t gdn_gated_norm_backward_workspace_bytes(int64_t rows, int32_t H, int32_t D) {
    int64_t pitch = 0;
    return gated_sizes(rows, H, D, GDN_F32, GDN_F32, 0, 1.0f, pitch) == GDN_OK
               ? gdn::gated_norm_back_ws_bytes(rows, H, D) : 0;
}

gdn_status gdn_gated_norm_backward(int64_t rows, int32_t H, int32_t D, int32_t o_dtype, int32_t act_dtype,
                                   int32_t flags, float eps, const void* o, const void* z, int64_t z_pitch,
                                   const float* w, const void* dy, void* do_, void* dz, int64_t dz_pitch, float* dw,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status st = gated_sizes(rows, H, D, o_dtype, act_dtype, flags, eps, z_pitch);
    if (st == GDN_OK)
        st = gated_sizes(rows, H, D, o_dtype, act_dtype, flags, eps, dz_pitch);
    if (st == GDN_OK)
        st = ptrs_ok({o, z, w, dy, do_, dz, dw});
    if (st != GDN_OK)
        return st;
    const size_t need = gdn::gated_norm_back_ws_bytes(rows, H, D);
    st = workspace_ok(workspace, workspace_bytes, need);
    if (st != GDN_OK)
        return st;
    const bool o16 = o_dtype == GDN_BF16, act16 = act_dtype == GDN_BF16, each = flags & GDN_WEIGHT_PER_HEAD;
    const int64_t row = static_cast<int64_t>(H) * D, ea = act16 ? 2 : 4, no = rows * row * (o16 ? 2 : 4);
    const int64_t nw = 4ll * D * (each ? H : 1);
    if (any_overlap({dense(do_, no), {dz, rows, row * ea, dz_pitch * ea}, dense(dw, nw),
                     dense(workspace, static_cast<int64_t>(need))},
                    {dense(o, no), {z, rows, row * ea, z_pitch * ea}, dense(w, nw), dense(dy, rows * row * ea)}))
        return GDN_ERR_ALIAS;
    return launched(gdn::launch_gated_norm_backward(
        {rows, H, D, o16, act16, each, (flags & GDN_GATE_FIRST) != 0, eps, z_pitch, o, z, w, nullptr},
        {dy, do_, dz, dz_pitch, dw}, workspace, as_stream(stream)));
}

}  // extern "C"
