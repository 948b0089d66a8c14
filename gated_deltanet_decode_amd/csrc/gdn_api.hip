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

}  // extern "C"
