"""Python binding of libgdn, the HIP library of the Gated DeltaNet recurrent
mixer for MI355X (gfx950).  The C ABI is include/gdn.h; this module only
marshals torch tensors (device memory) and streams into those calls and
checks that each tensor has the size, dtype and device the call expects, so
that a mistake in Python raises here instead of reaching a kernel.

Every computation runs in the HIP library.  If libgdn.so is missing this
module raises on import: there is no other path.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

__all__ = [
    "GdnError", "Dims", "dims", "conv_channels", "state_bytes", "conv_tail_bytes",
    "prefill_workspace_bytes", "tree_workspace_bytes", "block_workspace_bytes", "snapshot_bytes",
    "conv_update", "decode_step", "decode_token", "kda_decode_step", "kda_decode_token", "tree_verify",
    "tree_verify_ut", "commit_path",
    "commit_path_prepared",
    "tree_tables", "block_verify", "block_verify_ut", "block_commit", "block_commit_prepared", "state_signature", "snapshot", "restore", "prefill_chunked",
    "self_check_workspace_bytes", "self_check", "SELF_CHECK_PERTURB", "tree_verify_ut_noalloc",
    "NOALLOC_SCRATCH_BYTES",
    "SsmDims", "ssm_dims", "ssm_conv_channels", "ssm_state_bytes", "ssm_conv_tail_bytes", "ssm_decode_token",
    "ssm_prefill_workspace_bytes", "ssm_prefill", "SSM_MAX_TOKENS",
    "beam_select_workspace_bytes", "beam_select", "beam_reorder", "MAX_BEAMS", "MAX_BEAM_SELECT",
    "LruDims", "lru_dims", "lru_state_bytes", "lru_decode_token", "lru_prefill_workspace_bytes", "lru_saved_bytes",
    "lru_prefill", "lru_backward_workspace_bytes", "lru_backward", "LRU_MAX_WIDTH", "LRU_MAX_TOKENS",
    "residual_norm", "residual_norm_backward_workspace_bytes", "residual_norm_backward", "gated_norm",
    "gated_norm_backward_workspace_bytes", "gated_norm_backward", "NORM_MAX_WIDTH",
    "LIB_PATH", "MAX_TREE_NODES", "MAX_TREE_DEPTH", "PREFILL_CHUNK", "PREFILL_SEGMENT", "F32", "BF16",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")
MAX_TREE_NODES = 32
MAX_TREE_DEPTH = 8
PREFILL_CHUNK = 64
PREFILL_SEGMENT = 4096   # tokens per group of prefill launches; the workspace stops growing here
F32, BF16 = 0, 1
SELF_CHECK_PERTURB = 1
NOALLOC_SCRATCH_BYTES = 16 << 20
SSM_MAX_TOKENS = 1 << 22
MAX_BEAMS = 32
MAX_BEAM_SELECT = 64
LRU_MAX_WIDTH = 1 << 18
LRU_MAX_TOKENS = 1 << 22
NORM_MAX_WIDTH = 16384
_GATE_FIRST, _WEIGHT_PER_HEAD = 1, 2
_STATUS_TREE = 5

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python gated_deltanet_decode_amd/build.py`")

_lib = C.CDLL(LIB_PATH)


class Dims(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("batch", "num_k_heads", "num_v_heads", "head_k_dim",
                                         "head_v_dim", "conv_width", "act_dtype")]

    @property
    def C(self) -> int:
        return 2 * self.num_k_heads * self.head_k_dim + self.num_v_heads * self.head_v_dim

    @property
    def act_torch(self):
        return torch.bfloat16 if self.act_dtype == BF16 else torch.float32


def dims(batch, num_k_heads, num_v_heads, head_k_dim, head_v_dim, conv_width=4, act="bf16") -> Dims:
    return Dims(batch, num_k_heads, num_v_heads, head_k_dim, head_v_dim, conv_width,
                BF16 if act in ("bf16", BF16, torch.bfloat16) else F32)


class SsmDims(C.Structure):
    """A selective state space layer (gdn_ssm_dims)."""
    _fields_ = [(n, C.c_int32) for n in ("batch", "num_heads", "num_groups", "head_dim", "state_dim", "conv_width",
                                         "act_dtype")]

    @property
    def C(self) -> int:
        return self.num_heads * self.head_dim + 2 * self.num_groups * self.state_dim

    @property
    def act_torch(self):
        return torch.bfloat16 if self.act_dtype == BF16 else torch.float32


def ssm_dims(batch, num_heads, num_groups, head_dim, state_dim, conv_width=4, act="bf16") -> SsmDims:
    return SsmDims(batch, num_heads, num_groups, head_dim, state_dim, conv_width,
                   BF16 if act in ("bf16", BF16, torch.bfloat16) else F32)


class LruDims(C.Structure):
    """A gated linear recurrent layer (gdn_lru_dims)."""
    _fields_ = [(n, C.c_int32) for n in ("batch", "width", "act_dtype")]

    @property
    def act_torch(self):
        return torch.bfloat16 if self.act_dtype == BF16 else torch.float32


def lru_dims(batch, width, act="bf16") -> LruDims:
    return LruDims(batch, width, BF16 if act in ("bf16", BF16, torch.bfloat16) else F32)


class _LruPitches(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("x", "r", "i", "z", "y")]


_P = C.c_void_p
_L = C.POINTER(LruDims)
_LP = C.POINTER(_LruPitches)
_M = C.POINTER(SsmDims)
_D = C.POINTER(Dims)
_I = C.c_int32
_sig = {
    "gdn_abi_version": ([], C.c_int),
    "gdn_status_str": ([C.c_int], C.c_char_p),
    "gdn_conv_channels": ([_D], C.c_size_t),
    "gdn_state_bytes": ([_D], C.c_size_t),
    "gdn_conv_tail_bytes": ([_D], C.c_size_t),
    "gdn_prefill_workspace_bytes": ([_D, _I], C.c_size_t),
    "gdn_conv_update": ([_D, _P, _P, _P, _P, _P], C.c_int),
    "gdn_decode_step": ([_D, _P, _P, _P, _P, _P, _P], C.c_int),
    "gdn_decode_token": ([_D, _P, _P, _P, _P, _P, _P, _P, _P, _P], C.c_int),
    "gdn_kda_decode_step": ([_D, _P, _P, _P, _P, _P, _P], C.c_int),
    "gdn_kda_decode_token": ([_D, _P, _P, _P, _P, _P, _P, _P, _P, _P], C.c_int),
    "gdn_tree_workspace_bytes": ([_D, _I], C.c_size_t),
    "gdn_tree_verify": ([_D, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P], C.c_int),
    "gdn_tree_verify_ut": ([_D, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P], C.c_int),
    "gdn_commit_path": ([_D, _P, _P, _P, _I, _P, _P, _P, _P, _I, _P, _P, _P, _P], C.c_int),
    "gdn_block_commit_prepared": ([_D, _P, _P, _I, _P, _P, _P, _P, _P, C.c_size_t, _P], C.c_int),
    "gdn_commit_path_prepared": ([_D, _P, _P, _I, _P, _P, _I, _P, _P, _P, _P, C.c_size_t, _P], C.c_int),
    "gdn_tree_tables": ([_I, _P, _P, _P, _P, _P], C.c_int),
    "gdn_prefill_chunked": ([_D, _P, _P, _P, _I, _P, _P, _P, _P, _P, C.c_size_t, _P], C.c_int),
    "gdn_block_workspace_bytes": ([_D, _I], C.c_size_t),
    "gdn_block_verify": ([_D, _P, _P, _P, _I, _P, _P, _P, _P, _P, C.c_size_t, _P], C.c_int),
    "gdn_block_verify_ut": ([_D, _P, _P, _P, _I, _P, _P, _P, _P, _P, C.c_size_t, _P], C.c_int),
    "gdn_block_commit": ([_D, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P], C.c_int),
    "gdn_state_signature": ([_D], C.c_uint64),
    "gdn_snapshot_bytes": ([_D, _I], C.c_size_t),
    "gdn_snapshot": ([_D, _P, _P, _I, _P, _P, C.c_size_t, _P, _P], C.c_int),
    "gdn_restore": ([_D, _P, _P, _I, _P, _P, C.c_size_t, _P, _P], C.c_int),
    "gdn_self_check_workspace_bytes": ([_D], C.c_size_t),
    "gdn_self_check": ([_D, C.c_uint32, _I, _P, C.c_size_t, _P, _P], C.c_int),
    "gdn_tree_verify_ut_noalloc": ([_D, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P], C.c_int),
    "gdn_ssm_conv_channels": ([_M], C.c_size_t),
    "gdn_ssm_state_bytes": ([_M], C.c_size_t),
    "gdn_ssm_conv_tail_bytes": ([_M], C.c_size_t),
    "gdn_ssm_decode_token": ([_M] + [_P] * 13, C.c_int),
    "gdn_ssm_prefill_workspace_bytes": ([_M, _I], C.c_size_t),
    "gdn_ssm_prefill": ([_M, _P, _P, _P, _P, _I] + [_P] * 10 + [C.c_size_t, _P], C.c_int),
    "gdn_beam_select_workspace_bytes": ([_I] * 4, C.c_size_t),
    "gdn_beam_select": ([_I, _I, _I, C.c_int64, _I, _P, _P, _P, _I, _I, _P, _P, _P, _P, C.c_size_t, _P], C.c_int),
    "gdn_beam_reorder": ([_D, _I, _P, _P, _P, _P, _P], C.c_int),
    "gdn_ssm_beam_reorder": ([_M, _I, _P, _P, _P, _P, _P], C.c_int),
    "gdn_lru_state_bytes": ([_L], C.c_size_t),
    "gdn_lru_decode_token": ([_L, _LP] + [_P] * 8, C.c_int),
    "gdn_lru_prefill_workspace_bytes": ([_L, _I], C.c_size_t),
    "gdn_lru_saved_bytes": ([_L, _I], C.c_size_t),
    "gdn_lru_prefill": ([_L, _LP, _P, _I] + [_P] * 10 + [C.c_size_t, _P], C.c_int),
    "gdn_lru_backward_workspace_bytes": ([_L, _I], C.c_size_t),
    "gdn_lru_backward": ([_L, _LP, _LP, _I] + [_P] * 17 + [C.c_size_t, _P], C.c_int),
    "gdn_residual_norm": ([C.c_int64, _I, _I, _I, C.c_float] + [_P] * 8, C.c_int),
    "gdn_residual_norm_backward_workspace_bytes": ([C.c_int64, _I], C.c_size_t),
    "gdn_residual_norm_backward": ([C.c_int64, _I, _I, _I, C.c_float] + [_P] * 13 + [C.c_size_t, _P], C.c_int),
    "gdn_gated_norm": ([C.c_int64] + [_I] * 5 + [C.c_float, _P, _P, C.c_int64, _P, _P, _P], C.c_int),
    "gdn_gated_norm_backward_workspace_bytes": ([C.c_int64, _I, _I], C.c_size_t),
    "gdn_gated_norm_backward": ([C.c_int64] + [_I] * 5 + [C.c_float, _P, _P, C.c_int64, _P, _P, _P, _P, C.c_int64, _P,
                                                         _P, C.c_size_t, _P], C.c_int),
}
for _name, (_args, _res) in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res


class GdnError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call}: {_lib.gdn_status_str(status).decode()} (status {status})")
        self.status = status


def _check(status: int, call: str) -> None:
    if status != 0:
        raise GdnError(status, call)


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _t(t: torch.Tensor, name: str, dtype, numel: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _opt(t, name, dtype, numel):
    return None if t is None else _t(t, name, dtype, numel)


def conv_channels(d: Dims) -> int:
    return _lib.gdn_conv_channels(C.byref(d))


def state_bytes(d: Dims) -> int:
    return _lib.gdn_state_bytes(C.byref(d))


def conv_tail_bytes(d: Dims) -> int:
    return _lib.gdn_conv_tail_bytes(C.byref(d))


def prefill_workspace_bytes(d: Dims, T: int) -> int:
    return _lib.gdn_prefill_workspace_bytes(C.byref(d), T)


def conv_update(d: Dims, x, tail, w, y, stream=None) -> None:
    B, Cc = d.batch, d.C
    _check(_lib.gdn_conv_update(C.byref(d), _t(x, "x", d.act_torch, B * Cc),
                                _t(tail, "conv_tail", d.act_torch, B * Cc * 4),
                                _t(w, "conv_w", d.act_torch, Cc * 4),
                                _t(y, "y", torch.float32, B * Cc), _stream(stream)), "gdn_conv_update")


def decode_step(d: Dims, state, y, a, b, o, stream=None) -> None:
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    _check(_lib.gdn_decode_step(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                                _t(y, "y", torch.float32, B * Cc), _t(a, "a", torch.float32, B * Hv),
                                _t(b, "b", torch.float32, B * Hv), _t(o, "o", torch.float32, B * Hv * dv),
                                _stream(stream)), "gdn_decode_step")


def decode_token(d: Dims, state, tail_in, tail_out, w, x, a, b, o, stream=None) -> None:
    """conv_update + decode_step in one launch; the tail goes from tail_in to tail_out."""
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    _check(_lib.gdn_decode_token(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                                 _t(tail_in, "conv_tail_in", d.act_torch, B * Cc * 4),
                                 _t(tail_out, "conv_tail_out", d.act_torch, B * Cc * 4),
                                 _t(w, "conv_w", d.act_torch, Cc * 4), _t(x, "x", d.act_torch, B * Cc),
                                 _t(a, "a", torch.float32, B * Hv), _t(b, "b", torch.float32, B * Hv),
                                 _t(o, "o", torch.float32, B * Hv * dv), _stream(stream)), "gdn_decode_token")


def kda_decode_step(d: Dims, state, y, a, b, o, stream=None) -> None:
    """decode_step with the per-channel forget gate: a is [B][Hv][dk]."""
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    _check(_lib.gdn_kda_decode_step(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                                    _t(y, "y", torch.float32, B * Cc), _t(a, "a", torch.float32, B * Hv * dk),
                                    _t(b, "b", torch.float32, B * Hv), _t(o, "o", torch.float32, B * Hv * dv),
                                    _stream(stream)), "gdn_kda_decode_step")


def kda_decode_token(d: Dims, state, tail_in, tail_out, w, x, a, b, o, stream=None) -> None:
    """decode_token with the per-channel forget gate: a is [B][Hv][dk]."""
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    _check(_lib.gdn_kda_decode_token(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                                     _t(tail_in, "conv_tail_in", d.act_torch, B * Cc * 4),
                                     _t(tail_out, "conv_tail_out", d.act_torch, B * Cc * 4),
                                     _t(w, "conv_w", d.act_torch, Cc * 4), _t(x, "x", d.act_torch, B * Cc),
                                     _t(a, "a", torch.float32, B * Hv * dk), _t(b, "b", torch.float32, B * Hv),
                                     _t(o, "o", torch.float32, B * Hv * dv), _stream(stream)),
           "gdn_kda_decode_token")


def tree_workspace_bytes(d: Dims, n_nodes: int) -> int:
    return _lib.gdn_tree_workspace_bytes(C.byref(d), n_nodes)


def tree_verify(d: Dims, state, tail, w, parent, x, a, b, o, status=None, workspace=None, stream=None) -> None:
    """One tree of n nodes per sequence: parent [B][n]; workspace: a device byte tensor of at
    least tree_workspace_bytes(d, n) bytes; status [B] or None."""
    _tree_verify("gdn_tree_verify", d, state, tail, w, parent, x, a, b, o, status, workspace, stream)


def tree_verify_ut(d: Dims, state, tail, w, parent, x, a, b, o, status=None, workspace=None, stream=None) -> None:
    """tree_verify in the UT form (one read of each checkpoint, MFMA products); outputs equal
    decode's to rounding rather than bit for bit.  workspace None: one launch that prepares
    nothing for commit_path_prepared; with a workspace, as tree_verify."""
    _tree_verify("gdn_tree_verify_ut", d, state, tail, w, parent, x, a, b, o, status, workspace, stream,
                 optional=True)


def _tree_verify(name, d, state, tail, w, parent, x, a, b, o, status, workspace, stream, optional=False) -> None:
    B = d.batch
    if parent.numel() % B:
        raise ValueError("parent must be [B][n_nodes]")
    n = parent.numel() // B
    Hv, dk, dv, Cc = d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    if workspace is None and optional:
        ws_ptr, ws_bytes = None, 0
    else:
        ws_ptr, ws_bytes = _blob(workspace, tree_workspace_bytes(d, n), "workspace")
    _check(getattr(_lib, name)(C.byref(d), _t(state, "state_ckpt", torch.float32, B * Hv * dv * dk),
                               _t(tail, "conv_tail", d.act_torch, B * Cc * 4), _t(w, "conv_w", d.act_torch, Cc * 4),
                               n, _t(parent, "parent", torch.int32, B * n), _t(x, "x", d.act_torch, B * n * Cc),
                               _t(a, "a", torch.float32, B * n * Hv), _t(b, "b", torch.float32, B * n * Hv),
                               _t(o, "o", torch.float32, B * n * Hv * dv), _opt(status, "tree_status", torch.int32, B),
                               ws_ptr, ws_bytes, _stream(stream)), name)


def commit_path(d: Dims, state, tail, w, parent, x, a, b, path, o=None, status=None, stream=None) -> None:
    """path [B][L]: each row root first, -1 after its end; o [B][L][Hv][dv] or None; status [B] or None."""
    B = d.batch
    if parent.numel() % B or path.numel() % B:
        raise ValueError("parent must be [B][n_nodes] and path [B][path_len]")
    n, L = parent.numel() // B, path.numel() // B
    Hv, dk, dv, Cc = d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    _check(_lib.gdn_commit_path(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                                _t(tail, "conv_tail", d.act_torch, B * Cc * 4), _t(w, "conv_w", d.act_torch, Cc * 4),
                                n, _t(parent, "parent", torch.int32, B * n), _t(x, "x", d.act_torch, B * n * Cc),
                                _t(a, "a", torch.float32, B * n * Hv), _t(b, "b", torch.float32, B * n * Hv),
                                L, _t(path, "path", torch.int32, B * L), _opt(o, "o", torch.float32, B * L * Hv * dv),
                                _opt(status, "tree_status", torch.int32, B), _stream(stream)), "gdn_commit_path")


def commit_path_prepared(d: Dims, state, tail, parent, x, path, workspace, o=None, status=None,
                         stream=None) -> None:
    """commit_path for the trees just verified with `workspace` (tree_verify or
    tree_verify_ut on the same inputs): the path's operands are read from it."""
    B = d.batch
    if parent.numel() % B or path.numel() % B:
        raise ValueError("parent must be [B][n_nodes] and path [B][path_len]")
    n, L = parent.numel() // B, path.numel() // B
    Hv, dk, dv, Cc = d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    if workspace is None or workspace.device.type != "cuda" or not workspace.is_contiguous():
        raise ValueError("commit_path_prepared needs the verify's contiguous device workspace tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(_lib.gdn_commit_path_prepared(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                                         _t(tail, "conv_tail", d.act_torch, B * Cc * 4), n,
                                         _t(parent, "parent", torch.int32, B * n), _t(x, "x", d.act_torch, B * n * Cc),
                                         L, _t(path, "path", torch.int32, B * L),
                                         _opt(o, "o", torch.float32, B * L * Hv * dv),
                                         _opt(status, "tree_status", torch.int32, B), workspace.data_ptr(), ws_bytes,
                                         _stream(stream)), "gdn_commit_path_prepared")


def tree_tables(parent, depth, order, status, stream=None) -> None:
    n = parent.numel()
    _check(_lib.gdn_tree_tables(n, _t(parent, "parent", torch.int32, n), _t(depth, "depth", torch.int32, n),
                                _t(order, "order", torch.int32, n), _t(status, "tree_status", torch.int32, 1),
                                _stream(stream)), "gdn_tree_tables")


def block_workspace_bytes(d: Dims, k: int) -> int:
    return _lib.gdn_block_workspace_bytes(C.byref(d), k)


def _block_common(d, x, workspace, optional=False):
    B, Cc = d.batch, d.C
    if x.numel() % (B * Cc):
        raise ValueError("x must be [B][k][C]")
    k = x.numel() // (B * Cc)
    if workspace is None and optional:
        return k, None, 0
    ptr, nbytes = _blob(workspace, block_workspace_bytes(d, k), "workspace")
    return k, ptr, nbytes


def block_verify(d: Dims, state, tail, w, x, a, b, o, workspace, stream=None) -> None:
    """A block of k tokens per sequence: x [B][k][C], a, b [B][k][Hv], o [B][k][Hv][dv]."""
    _block_verify("gdn_block_verify", d, state, tail, w, x, a, b, o, workspace, stream)


def block_verify_ut(d: Dims, state, tail, w, x, a, b, o, workspace=None, stream=None) -> None:
    """block_verify in the UT form; outputs equal decode's to rounding.  workspace None: one
    launch that prepares nothing for block_commit_prepared."""
    _block_verify("gdn_block_verify_ut", d, state, tail, w, x, a, b, o, workspace, stream, optional=True)


def _block_verify(name, d, state, tail, w, x, a, b, o, workspace, stream, optional=False) -> None:
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    k, ptr, nbytes = _block_common(d, x, workspace, optional)
    _check(getattr(_lib, name)(C.byref(d), _t(state, "state_ckpt", torch.float32, B * Hv * dv * dk),
                               _t(tail, "conv_tail", d.act_torch, B * Cc * 4), _t(w, "conv_w", d.act_torch, Cc * 4),
                               k, _t(x, "x", d.act_torch, B * k * Cc), _t(a, "a", torch.float32, B * k * Hv),
                               _t(b, "b", torch.float32, B * k * Hv), _t(o, "o", torch.float32, B * k * Hv * dv),
                               ptr, nbytes, _stream(stream)), name)


def block_commit(d: Dims, state, tail, w, x, a, b, accepted, o=None, status=None, workspace=None,
                 stream=None) -> None:
    """Advance each sequence by its first accepted[seq] (int32 [B], device) block tokens."""
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    k, ptr, nbytes = _block_common(d, x, workspace)
    _check(_lib.gdn_block_commit(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                                 _t(tail, "conv_tail", d.act_torch, B * Cc * 4), _t(w, "conv_w", d.act_torch, Cc * 4),
                                 k, _t(x, "x", d.act_torch, B * k * Cc), _t(a, "a", torch.float32, B * k * Hv),
                                 _t(b, "b", torch.float32, B * k * Hv), _t(accepted, "accepted", torch.int32, B),
                                 _opt(o, "o", torch.float32, B * k * Hv * dv), _opt(status, "status", torch.int32, B),
                                 ptr, nbytes, _stream(stream)), "gdn_block_commit")


def block_commit_prepared(d: Dims, state, tail, x, accepted, workspace, o=None, status=None, stream=None) -> None:
    """block_commit for the blocks just verified with `workspace` (block_verify or
    block_verify_ut on the same inputs): the operands are read from it."""
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    k, ptr, nbytes = _block_common(d, x, workspace)
    _check(_lib.gdn_block_commit_prepared(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                                          _t(tail, "conv_tail", d.act_torch, B * Cc * 4), k,
                                          _t(x, "x", d.act_torch, B * k * Cc), _t(accepted, "accepted", torch.int32, B),
                                          _opt(o, "o", torch.float32, B * k * Hv * dv),
                                          _opt(status, "status", torch.int32, B), ptr, nbytes, _stream(stream)),
           "gdn_block_commit_prepared")


def state_signature(d: Dims) -> int:
    return _lib.gdn_state_signature(C.byref(d))


def snapshot_bytes(d: Dims, count: int) -> int:
    return _lib.gdn_snapshot_bytes(C.byref(d), count)


def _blob(blob, need, name):
    if not isinstance(blob, torch.Tensor) or blob.device.type != "cuda" or not blob.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor")
    nbytes = blob.numel() * blob.element_size()
    if nbytes < need:
        raise ValueError(f"{name} of {nbytes} bytes, need {need}")
    return blob.data_ptr(), nbytes


def snapshot(d: Dims, state, tail, seqs, blob, status, stream=None) -> None:
    """Copy sequences seqs [count] (int32, device) of (state, tail) into blob (device bytes of at
    least snapshot_bytes(d, count)); status [1] int32 (device) receives the outcome."""
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    n = seqs.numel()
    ptr, nbytes = _blob(blob, snapshot_bytes(d, n), "blob")
    _check(_lib.gdn_snapshot(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                             _t(tail, "conv_tail", d.act_torch, B * Cc * 4), n, _t(seqs, "seqs", torch.int32, n),
                             ptr, nbytes, _t(status, "status", torch.int32, 1), _stream(stream)), "gdn_snapshot")


def restore(d: Dims, state, tail, seqs, blob, status, stream=None) -> None:
    """Copy blob slots 0..count-1 into sequences seqs [count] (distinct) of (state, tail)."""
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    n = seqs.numel()
    ptr, nbytes = _blob(blob, snapshot_bytes(d, n), "blob")
    _check(_lib.gdn_restore(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                            _t(tail, "conv_tail", d.act_torch, B * Cc * 4), n, _t(seqs, "seqs", torch.int32, n),
                            ptr, nbytes, _t(status, "status", torch.int32, 1), _stream(stream)), "gdn_restore")


def prefill_chunked(d: Dims, state, tail, w, x, a, b, o, workspace=None, stream=None) -> None:
    B, Hv, dk, dv, Cc = d.batch, d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    if x.numel() % (B * Cc):
        raise ValueError("x must be [B][T][C]")
    T = x.numel() // (B * Cc)
    need = prefill_workspace_bytes(d, T)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if workspace.device.type != "cuda" or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if ws_bytes < need:
        raise ValueError(f"workspace of {ws_bytes} bytes, need {need}")
    _check(_lib.gdn_prefill_chunked(C.byref(d), _t(state, "state", torch.float32, B * Hv * dv * dk),
                                    _t(tail, "conv_tail", d.act_torch, B * Cc * 4),
                                    _t(w, "conv_w", d.act_torch, Cc * 4), T, _t(x, "x", d.act_torch, B * T * Cc),
                                    _t(a, "a", torch.float32, B * T * Hv), _t(b, "b", torch.float32, B * T * Hv),
                                    _t(o, "o", torch.float32, B * T * Hv * dv), ws_ptr, ws_bytes, _stream(stream)),
           "gdn_prefill_chunked")


def self_check_workspace_bytes(d: Dims) -> int:
    return _lib.gdn_self_check_workspace_bytes(C.byref(d))


def self_check(d: Dims, result, workspace, seed: int = 0x5EED, flags: int = 0, stream=None) -> None:
    """Queue the load-time self-check for d's layer shape; result [4] int32 (device) receives
    the verdict: result[0] == 0 when verify and commit rows equal decode's bit for bit."""
    ptr, nbytes = _blob(workspace, self_check_workspace_bytes(d), "workspace")
    _check(_lib.gdn_self_check(C.byref(d), seed & 0xFFFFFFFF, flags, ptr, nbytes,
                               _t(result, "result", torch.int32, 4), _stream(stream)), "gdn_self_check")


def tree_verify_ut_noalloc(d: Dims, state, tail, w, parent, x, a, b, o, status=None, stream=None) -> None:
    """tree_verify_ut with no workspace argument: the library's per-GPU scratch array
    (NOALLOC_SCRATCH_BYTES) holds the prepared operands; calls on one GPU must not overlap."""
    B = d.batch
    if parent.numel() % B:
        raise ValueError("parent must be [B][n_nodes]")
    n = parent.numel() // B
    Hv, dk, dv, Cc = d.num_v_heads, d.head_k_dim, d.head_v_dim, d.C
    _check(_lib.gdn_tree_verify_ut_noalloc(C.byref(d), _t(state, "state_ckpt", torch.float32, B * Hv * dv * dk),
                                           _t(tail, "conv_tail", d.act_torch, B * Cc * 4),
                                           _t(w, "conv_w", d.act_torch, Cc * 4), n,
                                           _t(parent, "parent", torch.int32, B * n),
                                           _t(x, "x", d.act_torch, B * n * Cc), _t(a, "a", torch.float32, B * n * Hv),
                                           _t(b, "b", torch.float32, B * n * Hv),
                                           _t(o, "o", torch.float32, B * n * Hv * dv),
                                           _opt(status, "tree_status", torch.int32, B), _stream(stream)),
           "gdn_tree_verify_ut_noalloc")


# ------------------------------------------------ selective state space layers
#
# These calls are made once per layer and token, so their checks take one pass
# of cheap queries per tensor; a tensor that fails them goes through _t, which
# says what is wrong with it.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # the handle without a Stream object around it


def _p(t, name, dtype, numel, dev):
    """Address of a contiguous tensor of numel elements on device dev, the current one."""
    try:
        if t.get_device() == dev and t.dtype is dtype and t.numel() == numel and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _t(t, name, dtype, numel)
    raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")


def _here(stream):
    """(current device, stream handle); a launch goes to the current device."""
    dev = torch.cuda.current_device()
    if stream is not None:
        return dev, _stream(stream)
    return dev, _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream


def _ws(workspace, need, dev):
    ptr, nbytes = _blob(workspace, need, "workspace")
    if workspace.get_device() != dev:
        raise ValueError(f"workspace is on {workspace.device}, but the current device is cuda:{dev}")
    return ptr, nbytes


def ssm_conv_channels(d: SsmDims) -> int:
    return _lib.gdn_ssm_conv_channels(C.byref(d))


def ssm_state_bytes(d: SsmDims) -> int:
    return _lib.gdn_ssm_state_bytes(C.byref(d))


def ssm_conv_tail_bytes(d: SsmDims) -> int:
    return _lib.gdn_ssm_conv_tail_bytes(C.byref(d))


def ssm_decode_token(d: SsmDims, state, tail_in, tail_out, w, x, dt, A, y, conv_bias=None, dt_bias=None, D=None,
                     z=None, stream=None) -> None:
    """One token of a selective state space layer: x [B][C], dt [B][H], y and z [B][H][P];
    the tail goes from tail_in to tail_out."""
    B, H, P, act = d.batch, d.num_heads, d.head_dim, torch.bfloat16 if d.act_dtype == BF16 else torch.float32
    HP, f32 = H * P, torch.float32
    Cc = HP + 2 * d.num_groups * d.state_dim
    dev, s = _here(stream)
    _check(_lib.gdn_ssm_decode_token(C.byref(d), _p(state, "state", f32, B * HP * d.state_dim, dev),
                                     _p(tail_in, "conv_tail_in", act, B * Cc * 4, dev),
                                     _p(tail_out, "conv_tail_out", act, B * Cc * 4, dev),
                                     _p(w, "conv_w", act, Cc * 4, dev),
                                     None if conv_bias is None else _p(conv_bias, "conv_bias", act, Cc, dev),
                                     _p(x, "x", act, B * Cc, dev), _p(dt, "dt", f32, B * H, dev),
                                     None if dt_bias is None else _p(dt_bias, "dt_bias", f32, H, dev),
                                     _p(A, "A", f32, H, dev), None if D is None else _p(D, "D", f32, H, dev),
                                     None if z is None else _p(z, "z", act, B * HP, dev), _p(y, "y", act, B * HP, dev),
                                     s), "gdn_ssm_decode_token")


def ssm_prefill_workspace_bytes(d: SsmDims, T: int) -> int:
    return _lib.gdn_ssm_prefill_workspace_bytes(C.byref(d), T)


def ssm_prefill(d: SsmDims, state, tail, w, x, dt, A, y, workspace, conv_bias=None, dt_bias=None, D=None, z=None,
                lengths=None, status=None, stream=None) -> None:
    """Prompts of a selective state space layer: x [B][T][C], dt [B][T][H], y and z [B][T][H][P];
    state and tail in place.  lengths [B] (int32, device): tokens of each sequence, None for T.
    workspace: a device byte tensor of at least ssm_prefill_workspace_bytes(d, T) bytes."""
    B, H, P, act = d.batch, d.num_heads, d.head_dim, torch.bfloat16 if d.act_dtype == BF16 else torch.float32
    HP, f32 = H * P, torch.float32
    Cc = HP + 2 * d.num_groups * d.state_dim
    if B < 1 or Cc < 1:
        raise GdnError(2, "gdn_ssm_prefill")
    if not isinstance(x, torch.Tensor) or not x.numel() or x.numel() % (B * Cc):
        raise ValueError("x must be [B][T][C]")
    T = x.numel() // (B * Cc)
    dev, s = _here(stream)
    ptr, nbytes = _ws(workspace, _lib.gdn_ssm_prefill_workspace_bytes(C.byref(d), T), dev)
    _check(_lib.gdn_ssm_prefill(C.byref(d), _p(state, "state", f32, B * HP * d.state_dim, dev),
                                _p(tail, "conv_tail", act, B * Cc * 4, dev), _p(w, "conv_w", act, Cc * 4, dev),
                                None if conv_bias is None else _p(conv_bias, "conv_bias", act, Cc, dev), T,
                                _p(x, "x", act, B * T * Cc, dev), _p(dt, "dt", f32, B * T * H, dev),
                                None if dt_bias is None else _p(dt_bias, "dt_bias", f32, H, dev),
                                _p(A, "A", f32, H, dev), None if D is None else _p(D, "D", f32, H, dev),
                                None if z is None else _p(z, "z", act, B * T * HP, dev),
                                None if lengths is None else _p(lengths, "lengths", torch.int32, B, dev),
                                _p(y, "y", act, B * T * HP, dev),
                                None if status is None else _p(status, "status", torch.int32, B, dev), ptr, nbytes, s),
           "gdn_ssm_prefill")


# ------------------------------------------------ beam search over recurrent states

def beam_select_workspace_bytes(batch: int, beams: int, vocab: int, select: int) -> int:
    return _lib.gdn_beam_select_workspace_bytes(batch, beams, vocab, select)


def beam_select(logits, scores, out_scores, parent, token, workspace, finished=None, eos=0, stream=None) -> None:
    """The S best continuations of each sequence's K beams: logits [B][K][V] (bf16 or fp32; the
    rows may be a slice of wider ones), scores [B][K]; out_scores, parent, token [B][S].
    finished [B][K] (bool): beams that have ended, whose one candidate is eos at their own score."""
    if not isinstance(logits, torch.Tensor) or logits.device.type != "cuda" or logits.dim() != 3:
        raise ValueError("logits must be a device tensor [B][K][V]")
    if logits.dtype is torch.bfloat16:
        act = BF16
    elif logits.dtype is torch.float32:
        act = F32
    else:
        raise ValueError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    B, K, V = logits.shape
    if V == 0 or B == 0 or K == 0:
        raise ValueError("logits must not be empty")
    # strides of dimensions of one entry say nothing
    sb, sk, sv = logits.stride()
    pitch = sk if K > 1 else sb if B > 1 else V
    if (V > 1 and sv != 1) or (K > 1 and B > 1 and sb != K * pitch) or pitch < V:
        raise ValueError("logits must have contiguous entries and rows at one pitch of at least V")
    if not isinstance(out_scores, torch.Tensor) or out_scores.numel() % B:
        raise ValueError("out_scores must be [B][S]")
    S = out_scores.numel() // B
    if B * K >= 1 << 31 or K * V >= 1 << 31 or S >= 1 << 31:   # C's integers would wrap
        raise GdnError(2, "gdn_beam_select")
    dev, s = _here(stream)
    if logits.get_device() != dev:
        raise ValueError(f"logits is on {logits.device}, but the current device is cuda:{dev}")
    ptr, nbytes = _ws(workspace, _lib.gdn_beam_select_workspace_bytes(B, K, V, S), dev)
    fin = None
    if finished is not None:
        byte = getattr(finished, "dtype", None) is torch.uint8
        fin = _p(finished, "finished", torch.uint8 if byte else torch.bool, B * K, dev)
    _check(_lib.gdn_beam_select(B, K, V, pitch, act, logits.data_ptr(), _p(scores, "scores", torch.float32, B * K, dev),
                                fin, eos, S, _p(out_scores, "out_scores", torch.float32, B * S, dev),
                                _p(parent, "parent", torch.int32, B * S, dev),
                                _p(token, "token", torch.int32, B * S, dev), ptr, nbytes, s), "gdn_beam_select")


def beam_reorder(d, state, tail, parent, status=None, stream=None) -> None:
    """Move the beams' states and conv tails in place: parent [groups][beams] (int32), groups * beams
    == d.batch; sequence g*beams + k takes what g*beams + parent[g][k] had.  d: Dims or SsmDims."""
    if not isinstance(parent, torch.Tensor) or parent.dim() != 2 or parent.numel() != d.batch:
        raise ValueError("parent must be [groups][beams] with groups * beams == batch")
    groups, beams = parent.shape
    dev, s = _here(stream)
    if isinstance(d, SsmDims):
        f, name, n = _lib.gdn_ssm_beam_reorder, "gdn_ssm_beam_reorder", d.num_heads * d.head_dim * d.state_dim
    else:
        f, name, n = _lib.gdn_beam_reorder, "gdn_beam_reorder", d.num_v_heads * d.head_v_dim * d.head_k_dim
    _check(f(C.byref(d), beams, _p(state, "state", torch.float32, d.batch * n, dev),
             _p(tail, "conv_tail", d.act_torch, d.batch * d.C * 4, dev), _p(parent, "parent", torch.int32, d.batch, dev),
             None if status is None else _p(status, "status", torch.int32, groups, dev), s), name)


# ------------------------------------------------ gated linear recurrent layers

def _rows(t, name, dtype, lead, W, dev):
    """(address, pitch) of rows of W contiguous values that follow each other at one pitch, lead of
    them in all; pitch 0 for a contiguous tensor alone, since the library takes 0 for "rows next to
    each other": one row many times over (a stride of 0) has no pitch.  A slice of a wider
    projection's output is one."""
    try:
        if t.get_device() == dev and t.dtype is dtype and t.numel() == lead * W:
            if t.is_contiguous():
                return t.data_ptr(), 0
            shape, strides = t.shape, t.stride()
            n = len(shape)
            if shape[-1] == W and strides[-1] == 1:
                pitch = 0
                if n == 2 or (n == 3 and shape[0] == 1):
                    pitch = strides[-2]
                elif n == 3 and shape[1] > 1:
                    pitch = strides[1] if strides[0] == shape[1] * strides[1] else 0
                else:
                    span = 1                # rows of the dimensions behind this one
                    for m, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
                        if m == 1:
                            continue
                        pitch = pitch or s
                        if not s or s != pitch * span:
                            pitch = 0
                            break
                        span *= m
                if pitch:
                    return t.data_ptr(), pitch
            raise ValueError(f"{name} must have contiguous rows of {W} at one pitch")
    except AttributeError:
        pass
    return _p(t, name, dtype, lead * W, dev), 0


def _pitches(x, r, i, z, y):
    return C.byref(_LruPitches(x, r, i, z, y)) if x or r or i or z or y else None


def lru_state_bytes(d: LruDims) -> int:
    return _lib.gdn_lru_state_bytes(C.byref(d))


def lru_decode_token(d: LruDims, state, x, r, i, A, y, z=None, stream=None) -> None:
    """One token of a gated linear recurrent layer: x, r, i, y and z [B][W], state [B][W] in place."""
    B, W, f32 = d.batch, d.width, torch.float32
    act = torch.bfloat16 if d.act_dtype == BF16 else f32
    dev, s = _here(stream)
    xp, px = _rows(x, "x", act, B, W, dev)
    rp, pr = _rows(r, "r", act, B, W, dev)
    ip, pi = _rows(i, "i", act, B, W, dev)
    zp, pz = (None, 0) if z is None else _rows(z, "z", act, B, W, dev)
    yp, py = _rows(y, "y", act, B, W, dev)
    _check(_lib.gdn_lru_decode_token(C.byref(d), _pitches(px, pr, pi, pz, py), _p(state, "state", f32, B * W, dev), xp, rp,
                                     ip, _p(A, "A", f32, W, dev), zp, yp, s), "gdn_lru_decode_token")


def lru_prefill_workspace_bytes(d: LruDims, T: int) -> int:
    return _lib.gdn_lru_prefill_workspace_bytes(C.byref(d), T)


def lru_saved_bytes(d: LruDims, T: int) -> int:
    return _lib.gdn_lru_saved_bytes(C.byref(d), T)


def _lru_tokens(d, x, call):
    if d.batch < 1 or d.width < 1:
        raise GdnError(2, call)
    if not isinstance(x, torch.Tensor) or not x.numel() or x.numel() % (d.batch * d.width):
        raise ValueError("x must be [B][T][W]")
    T = x.numel() // (d.batch * d.width)
    if T >= 1 << 31:   # C's integers would wrap
        raise GdnError(2, call)
    return T


def _room(buf, name, need, dev):
    """Address and bytes of a device buffer of at least need bytes; None serves where none are needed."""
    if buf is None and need == 0:
        return None, 0
    try:
        if buf.get_device() == dev and buf.is_contiguous() and buf.nbytes >= need:
            return buf.data_ptr(), buf.nbytes
    except AttributeError:
        pass
    _blob(buf, need, name)   # says what is wrong
    raise ValueError(f"{name} is on {buf.device}, but the current device is cuda:{dev}")


def lru_prefill(d: LruDims, state, x, r, i, A, y, workspace, z=None, lengths=None, saved=None, status=None,
                stream=None) -> None:
    """Prompts of a gated linear recurrent layer, or a training step's forward pass: x, r, i, y and z
    [B][T][W] (slices of wider rows are taken as they are; rows that `expand` repeats are refused),
    state [B][W] in place.  lengths [B] (int32, device): tokens of each sequence, None for T.  saved:
    a device byte tensor of at least lru_saved_bytes(d, T) bytes for lru_backward.  workspace: one of
    at least lru_prefill_workspace_bytes(d, T) bytes (None where that is 0)."""
    T = _lru_tokens(d, x, "gdn_lru_prefill")
    B, W, f32 = d.batch, d.width, torch.float32
    act = torch.bfloat16 if d.act_dtype == BF16 else f32
    dev, s = _here(stream)
    n = B * T
    xp, px = _rows(x, "x", act, n, W, dev)
    rp, pr = _rows(r, "r", act, n, W, dev)
    ip, pi = _rows(i, "i", act, n, W, dev)
    zp, pz = (None, 0) if z is None else _rows(z, "z", act, n, W, dev)
    yp, py = _rows(y, "y", act, n, W, dev)
    ws, nbytes = _room(workspace, "workspace", 0, dev)   # the library knows what it needs
    keep = None if saved is None else _room(saved, "saved", _lib.gdn_lru_saved_bytes(C.byref(d), T), dev)[0]
    _check(_lib.gdn_lru_prefill(C.byref(d), _pitches(px, pr, pi, pz, py), _p(state, "state", f32, B * W, dev), T, xp, rp, ip,
                                _p(A, "A", f32, W, dev), zp,
                                None if lengths is None else _p(lengths, "lengths", torch.int32, B, dev), yp, keep,
                                None if status is None else _p(status, "status", torch.int32, B, dev), ws, nbytes, s),
           "gdn_lru_prefill")


def lru_backward_workspace_bytes(d: LruDims, T: int) -> int:
    return _lib.gdn_lru_backward_workspace_bytes(C.byref(d), T)


def lru_backward(d: LruDims, x, r, i, A, dy, saved, dx, dr, di, dA, workspace, z=None, dz=None, dstate=None,
                 dstate0=None, lengths=None, status=None, stream=None) -> None:
    """Gradients of lru_prefill: from dy [B][T][W] and dstate [B][W] (None: 0) to dx, dr, di, dz, dA [W]
    and dstate0 [B][W].  x, r, i, A, z and lengths as the forward pass had them, saved as it left it;
    rows behind a sequence's end have gradients of 0."""
    T = _lru_tokens(d, x, "gdn_lru_backward")
    B, W, act, f32 = d.batch, d.width, d.act_torch, torch.float32
    dev, s = _here(stream)
    n = B * T
    row = lambda t, name: (None, 0) if t is None and name in ("z", "dz") else _rows(t, name, act, n, W, dev)
    (xp, px), (rp, pr), (ip, pi), (zp, pz), (yp, py) = (row(x, "x"), row(r, "r"), row(i, "i"), row(z, "z"), row(dy, "dy"))
    (xg, gx), (rg, gr), (ig, gi), (zg, gz) = row(dx, "dx"), row(dr, "dr"), row(di, "di"), row(dz, "dz")
    ws, nbytes = _room(workspace, "workspace", _lib.gdn_lru_backward_workspace_bytes(C.byref(d), T), dev)
    _check(_lib.gdn_lru_backward(C.byref(d), _pitches(px, pr, pi, pz, py), _pitches(gx, gr, gi, gz, 0), T, xp, rp, ip,
                                 _p(A, "A", f32, W, dev), zp,
                                 None if lengths is None else _p(lengths, "lengths", torch.int32, B, dev),
                                 _room(saved, "saved", _lib.gdn_lru_saved_bytes(C.byref(d), T), dev)[0], yp,
                                 None if dstate is None else _p(dstate, "dstate", f32, B * W, dev), xg, rg, ig, zg,
                                 _p(dA, "dA", f32, W, dev),
                                 None if dstate0 is None else _p(dstate0, "dstate0", f32, B * W, dev),
                                 None if status is None else _p(status, "status", torch.int32, B, dev), ws, nbytes, s),
           "gdn_lru_backward")


# ------------------------------------------------ the norms around a block

def _kind(t, name):
    dtype = getattr(t, "dtype", None)
    if dtype is torch.bfloat16:
        return BF16
    if dtype is torch.float32:
        return F32
    raise ValueError(f"{name} must be a bfloat16 or float32 device tensor")


def _width(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() < 1 or not t.numel():
        raise ValueError(f"{name} must be [rows][W]")
    W = t.shape[-1]
    if W >= 1 << 31:   # C's integers would wrap
        raise ValueError(f"{name} has rows of {W}")
    return W, t.numel() // W


def residual_norm(residual, delta, w, out, y, scale=None, w_post=None, eps=1e-6, stream=None) -> None:
    """The residual sum behind a block and the norm before the next: out = residual + scale * n with n =
    delta, or its RMS norm times w_post; y = RMS norm of out times w.  residual, out [rows][W] (fp32, or
    delta's and y's type; out may be residual); w, scale, w_post [W] fp32.  delta and out None: the norm
    of residual alone."""
    W, rows = _width(residual, "residual")
    res, act = _kind(residual, "residual"), _kind(y, "y")
    dev, s = _here(stream)
    n, f32, rt, at = rows * W, torch.float32, residual.dtype, y.dtype
    _check(_lib.gdn_residual_norm(rows, W, act, res, eps, _p(residual, "residual", rt, n, dev),
                                  None if delta is None else _p(delta, "delta", at, n, dev),
                                  None if scale is None else _p(scale, "scale", f32, W, dev),
                                  None if w_post is None else _p(w_post, "w_post", f32, W, dev), _p(w, "w", f32, W, dev),
                                  None if out is None else _p(out, "out", rt, n, dev), _p(y, "y", at, n, dev), s),
           "gdn_residual_norm")


def residual_norm_backward_workspace_bytes(rows: int, W: int) -> int:
    return _lib.gdn_residual_norm_backward_workspace_bytes(rows, W)


def residual_norm_backward(out, delta, w, dy, dresidual, ddelta, dw, workspace, ds=None, scale=None, w_post=None,
                           dscale=None, dw_post=None, eps=1e-6, stream=None) -> None:
    """Gradients of residual_norm: out as it left it (where delta is None, the residual), dy [rows][W], ds
    the gradient that reaches out from elsewhere (None: 0).  dresidual may be ds."""
    W, rows = _width(out, "out")
    res, act = _kind(out, "out"), _kind(dy, "dy")
    dev, s = _here(stream)
    n, f32, rt, at = rows * W, torch.float32, out.dtype, dy.dtype
    ws, nbytes = _room(workspace, "workspace", _lib.gdn_residual_norm_backward_workspace_bytes(rows, W), dev)
    opt = lambda t, name, dtype, k: None if t is None else _p(t, name, dtype, k, dev)
    _check(_lib.gdn_residual_norm_backward(rows, W, act, res, eps, _p(out, "out", rt, n, dev), opt(delta, "delta", at, n),
                                           opt(scale, "scale", f32, W), opt(w_post, "w_post", f32, W),
                                           _p(w, "w", f32, W, dev), _p(dy, "dy", at, n, dev), opt(ds, "ds", rt, n),
                                           _p(dresidual, "dresidual", rt, n, dev), opt(ddelta, "ddelta", at, n),
                                           _p(dw, "dw", f32, W, dev), opt(dscale, "dscale", f32, W),
                                           opt(dw_post, "dw_post", f32, W), ws, nbytes, s), "gdn_residual_norm_backward")


def _heads(o, w, gate_first):
    if not isinstance(o, torch.Tensor) or o.dim() < 2 or not o.numel():
        raise ValueError("o must be [rows][H][D]")
    H, D = o.shape[-2:]
    if H * D >= 1 << 31:   # C's integers would wrap
        raise ValueError(f"o has rows of {H} x {D}")
    each = isinstance(w, torch.Tensor) and w.numel() != D
    return o.numel() // (H * D), H, D, (_GATE_FIRST if gate_first else 0) | (_WEIGHT_PER_HEAD if each else 0), D * (H if each else 1)


def _head_rows(t, name, dtype, rows, H, D, dev):
    """_rows over the heads' H * D values; the heads of a row lie next to each other."""
    if not isinstance(t, torch.Tensor) or t.is_contiguous():
        return _p(t, name, dtype, rows * H * D, dev), 0
    shape, strides = t.shape, t.stride()
    if len(shape) < 2 or shape[-2:] != (H, D) or strides[-1] != 1 or (H > 1 and strides[-2] != D):
        raise ValueError(f"{name} must be [rows][H][D] with contiguous rows at one pitch")
    if len(shape) == 3 and t.get_device() == dev and t.dtype is dtype and shape[0] == rows and strides[0]:
        return t.data_ptr(), strides[0]
    return _rows(t.flatten(-2), name, dtype, rows, H * D, dev)


def gated_norm(o, z, w, y, eps=1e-6, gate_first=False, stream=None) -> None:
    """The norm of a mixer's output with its gate: y = RMS norm of o over each head's D values, times w
    and SiLU(z); with gate_first the norm is of o * SiLU(z).  o [rows][H][D] (fp32, or z's and y's
    type); z [rows][H][D], its rows may be a slice of wider ones; w [D] or [H][D] fp32."""
    rows, H, D, flags, nw = _heads(o, w, gate_first)
    ok, act = _kind(o, "o"), _kind(y, "y")
    dev, s = _here(stream)
    n, at = rows * H * D, y.dtype
    zp, pz = _head_rows(z, "z", at, rows, H, D, dev)
    _check(_lib.gdn_gated_norm(rows, H, D, ok, act, flags, eps, _p(o, "o", o.dtype, n, dev), zp, pz,
                               _p(w, "w", torch.float32, nw, dev), _p(y, "y", at, n, dev), s), "gdn_gated_norm")


def gated_norm_backward_workspace_bytes(rows: int, H: int, D: int) -> int:
    return _lib.gdn_gated_norm_backward_workspace_bytes(rows, H, D)


def gated_norm_backward(o, z, w, dy, do, dz, dw, workspace, eps=1e-6, gate_first=False, stream=None) -> None:
    """Gradients of gated_norm: do has o's type, dz z's (its rows may be a slice), dw w's shape."""
    rows, H, D, flags, nw = _heads(o, w, gate_first)
    ok, act = _kind(o, "o"), _kind(dy, "dy")
    dev, s = _here(stream)
    n, at, f32 = rows * H * D, dy.dtype, torch.float32
    zp, pz = _head_rows(z, "z", at, rows, H, D, dev)
    zg, gz = _head_rows(dz, "dz", at, rows, H, D, dev)
    ws, nbytes = _room(workspace, "workspace", _lib.gdn_gated_norm_backward_workspace_bytes(rows, H, D), dev)
    _check(_lib.gdn_gated_norm_backward(rows, H, D, ok, act, flags, eps, _p(o, "o", o.dtype, n, dev), zp, pz,
                                        _p(w, "w", f32, nw, dev), _p(dy, "dy", at, n, dev),
                                        _p(do, "do", o.dtype, n, dev), zg, gz, _p(dw, "dw", f32, nw, dev), ws, nbytes, s),
           "gdn_gated_norm_backward")
