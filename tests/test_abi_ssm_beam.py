"""CPU: the selective state space and beam search calls refuse bad arguments
before they touch a device, and the binding refuses bad tensors."""
import ctypes as C

import pytest
import torch

from tests.test_abi import Dims, lib, mk  # noqa: F401  (lib is a fixture)

P = C.c_void_p
F = 0x1000          # non-null, aligned, never touched


class SsmDims(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("batch", "num_heads", "num_groups", "head_dim", "state_dim", "conv_width",
                                         "act_dtype")]


def sd(**kw):
    d = dict(batch=2, num_heads=48, num_groups=16, head_dim=128, state_dim=128, conv_width=4, act_dtype=1)
    d.update(kw)
    return SsmDims(*[d[n] for n, _ in SsmDims._fields_])


BAD = [(dict(batch=0), 2), (dict(num_heads=0), 2), (dict(num_groups=0), 2), (dict(num_heads=47), 2),
       (dict(head_dim=48), 2), (dict(head_dim=256), 2), (dict(state_dim=16), 2), (dict(state_dim=512), 2),
       (dict(conv_width=3), 2), (dict(act_dtype=2), 3), (dict(batch=1 << 20), 2),
       (dict(num_heads=1 << 20, num_groups=1), 2)]


def test_sizes(lib):  # noqa: F811
    for f in ("gdn_ssm_conv_channels", "gdn_ssm_state_bytes", "gdn_ssm_conv_tail_bytes"):
        getattr(lib, f).restype = C.c_size_t
    d = sd()
    assert lib.gdn_ssm_conv_channels(C.byref(d)) == 10240
    assert lib.gdn_ssm_state_bytes(C.byref(d)) == 2 * 48 * 128 * 128 * 4
    assert lib.gdn_ssm_conv_tail_bytes(C.byref(d)) == 2 * 10240 * 4 * 2
    for kw, _ in BAD:
        bad = sd(**kw)
        for f in ("gdn_ssm_conv_channels", "gdn_ssm_state_bytes", "gdn_ssm_conv_tail_bytes"):
            assert getattr(lib, f)(C.byref(bad)) == 0


def test_token_refusals(lib):  # noqa: F811
    lib.gdn_ssm_decode_token.argtypes = [C.POINTER(SsmDims)] + [P] * 13

    def call(d=None, **kw):
        names = ["state", "tin", "tout", "w", "bias", "x", "dt", "dtb", "A", "D", "z", "y"]
        a = {n: F for n in names}
        a["tout"] = 0x10000000
        a.update(kw)
        return lib.gdn_ssm_decode_token(C.byref(sd() if d is None else d), *[a[n] for n in names], None)
    for kw, want in BAD:
        assert call(sd(**kw)) == want
    for n in ("state", "tin", "tout", "w", "x", "dt", "A", "y"):
        assert call(**{n: None}) == 1
    for n in ("state", "tout", "w", "bias", "x", "dt", "dtb", "A", "D", "z", "y"):
        assert call(**{n: F + 8}) == 4
    assert call(tout=F) == 8
    assert call(tout=F + 2 * 10240 * 8 - 16) == 8


def test_prefill_refusals(lib):  # noqa: F811
    lib.gdn_ssm_prefill_workspace_bytes.restype = C.c_size_t
    lib.gdn_ssm_prefill_workspace_bytes.argtypes = [C.POINTER(SsmDims), C.c_int32]
    lib.gdn_ssm_prefill.argtypes = [C.POINTER(SsmDims)] + [P] * 4 + [C.c_int32] + [P] * 10 + [C.c_size_t, P]
    need = lib.gdn_ssm_prefill_workspace_bytes(C.byref(sd()), 100)
    assert need > 0

    def call(d=None, T=100, ws=F, nbytes=need, **kw):
        names = ["state", "tail", "w", "bias", "x", "dt", "dtb", "A", "D", "z", "lengths", "y", "status"]
        a = {n: F for n in names}
        a.update(kw)
        v = [a[n] for n in names]
        return lib.gdn_ssm_prefill(C.byref(sd() if d is None else d), *v[:4], T, *v[4:], ws, nbytes, None)
    for kw, want in BAD:
        assert lib.gdn_ssm_prefill_workspace_bytes(C.byref(sd(**kw)), 100) == 0
        assert call(sd(**kw)) == want
    for T in (0, -1, (1 << 22) + 1):
        assert lib.gdn_ssm_prefill_workspace_bytes(C.byref(sd()), T) == 0
        assert call(T=T) == 2
    for n in ("state", "tail", "w", "x", "dt", "A", "y"):
        assert call(**{n: None}) == 1
    for n in ("state", "bias", "lengths", "status", "z"):
        assert call(**{n: F + 4}) == 4
    assert call(ws=None) == 6
    assert call(nbytes=need - 1) == 6
    assert call(ws=F + 16) == 4


def test_select_refusals(lib):  # noqa: F811
    lib.gdn_beam_select_workspace_bytes.restype = C.c_size_t
    lib.gdn_beam_select.argtypes = ([C.c_int32] * 3 + [C.c_int64, C.c_int32, P, P, P, C.c_int32, C.c_int32]
                                    + [P] * 4 + [C.c_size_t, P])
    need = lib.gdn_beam_select_workspace_bytes(2, 4, 1000, 8)
    assert need > 0

    def call(B=2, K=4, V=1000, pitch=1000, act=1, logits=F, scores=F, fin=F, eos=2, S=8, o=F, p=F, t=F, ws=F,
             nbytes=need):
        return lib.gdn_beam_select(B, K, V, pitch, act, logits, scores, fin, eos, S, o, p, t, ws, nbytes, None)
    for kw in (dict(B=0), dict(K=0), dict(K=33), dict(V=0), dict(S=0), dict(S=65), dict(K=1, V=3, pitch=3, S=4),
               dict(pitch=999), dict(K=32, V=1 << 26, pitch=1 << 26), dict(B=1 << 19), dict(pitch=1 << 41)):
        assert call(**kw) == 2, kw
    assert lib.gdn_beam_select_workspace_bytes(1, 1, 3, 4) == 0
    assert call(act=2) == 3
    for n in ("logits", "scores", "o", "p", "t"):
        assert call(**{n: None}) == 1
    assert call(logits=F + 1) == 4 and call(logits=F + 2, act=0) == 4 and call(scores=F + 4) == 4
    assert call(fin=F + 1) == 4 and call(t=F + 8) == 4
    assert call(eos=-1) == 10 and call(eos=1000) == 10
    assert call(ws=None) == 6 and call(nbytes=need - 1) == 6 and call(ws=F + 8) == 4


def test_reorder_refusals(lib):  # noqa: F811
    lib.gdn_beam_reorder.argtypes = [C.POINTER(Dims), C.c_int32] + [P] * 5
    lib.gdn_ssm_beam_reorder.argtypes = [C.POINTER(SsmDims), C.c_int32] + [P] * 5
    for f, good, bad in ((lib.gdn_beam_reorder, mk(batch=8), mk(batch=8, num_v_heads=47)),
                         (lib.gdn_ssm_beam_reorder, sd(batch=8), sd(batch=8, state_dim=48))):
        call = lambda d, K=4, s=F, t=F, p=F, st=None: f(C.byref(d), K, s, t, p, st, None)
        assert call(bad) == 2
        for K in (0, 3, 33, -4):
            assert call(good, K) == 2
        for kw in (dict(s=None), dict(t=None), dict(p=None)):
            assert call(good, **kw) == 1
        for kw in (dict(s=F + 8), dict(t=F + 8), dict(p=F + 4), dict(st=F + 4)):
            assert call(good, **kw) == 4
        assert f(None, 4, F, F, F, None, None) == 1


def test_more_than_a_grid_holds(lib):  # noqa: F811
    """States of more workgroups than a launch can count are refused, not cut short."""
    lib.gdn_ssm_state_bytes.restype = C.c_size_t
    for kw in (dict(batch=1 << 22, num_heads=1, num_groups=1, head_dim=64), dict(batch=1 << 15, num_heads=64,
                                                                                  num_groups=1, head_dim=128)):
        assert lib.gdn_ssm_state_bytes(C.byref(sd(state_dim=32, **kw))) == 0
        kw["batch"] -= 1
        assert lib.gdn_ssm_state_bytes(C.byref(sd(state_dim=32, **kw))) > 0
    lib.gdn_ssm_beam_reorder.argtypes = [C.POINTER(SsmDims), C.c_int32] + [P] * 5
    d = sd(batch=1 << 16, num_heads=32, num_groups=1, head_dim=64, state_dim=128)     # 64 GB and the tails
    assert lib.gdn_ssm_beam_reorder(C.byref(d), 1, F, F, F, None, None) == 2
    assert lib.gdn_ssm_beam_reorder(C.byref(d), 4, F, F, F + 4, None, None) == 4      # a quarter of the groups: only the pointer


def test_scores_that_overlap(lib):  # noqa: F811
    """out_scores may be scores itself where as many are selected as there are beams, and nothing else of it."""
    lib.gdn_beam_select_workspace_bytes.restype = C.c_size_t
    lib.gdn_beam_select.argtypes = ([C.c_int32] * 3 + [C.c_int64, C.c_int32, P, P, P, C.c_int32, C.c_int32]
                                    + [P] * 4 + [C.c_size_t, P])
    call = lambda S, o: lib.gdn_beam_select(8, 4, 1000, 1000, 1, F, F, None, 0, S, o, 0x100000, 0x200000, 0x300000,
                                            1 << 30, None)
    assert call(5, F) == 8 and call(3, F) == 8
    assert call(4, F + 16) == 8 and call(4, F - 16) == 8 and call(4, F + 112) == 8


def test_binding_refuses_host_tensors():
    import gated_deltanet_decode_amd as gdn
    with pytest.raises(ValueError, match="device tensor"):
        gdn.beam_select(torch.zeros(1, 2, 8), None, None, None, None, None)
    with pytest.raises(ValueError, match="parent"):
        gdn.beam_reorder(gdn.ssm_dims(6, 4, 1, 32, 32), None, None, torch.zeros(2, 2, dtype=torch.int32))
