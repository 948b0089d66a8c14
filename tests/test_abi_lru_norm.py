"""CPU: the gated linear recurrent layer's calls and the norms' refuse bad arguments
before they touch a device, and the binding refuses bad tensors."""
import ctypes as C
import random

import pytest
import torch

from tests.test_abi import lib  # noqa: F401  (a fixture)

P, I64, I32 = C.c_void_p, C.c_int64, C.c_int32
STEP = 0x100000000           # between operands that are never touched


class LruDims(C.Structure):
    _fields_ = [(n, I32) for n in ("batch", "width", "act_dtype")]


class Pitches(C.Structure):
    _fields_ = [(n, I64) for n in ("x", "r", "i", "z", "y")]


def ld(batch=2, width=256, act_dtype=1):
    return LruDims(batch, width, act_dtype)


BAD = [(dict(batch=0), 2), (dict(batch=-1), 2), (dict(width=0), 2), (dict(width=4), 2), (dict(width=252), 2),
       (dict(width=(1 << 18) + 8), 2), (dict(act_dtype=2), 3), (dict(act_dtype=-1), 3), (dict(batch=1 << 23), 2)]
BAD_PITCH = [dict(x=248), dict(r=260), dict(i=(1 << 20) + 8), dict(z=-256), dict(y=8)]


class Call:
    """A call by its operands' names, each at an address of its own."""

    def __init__(self, f, names, argtypes, build):
        self.f, self.names, self.build = f, names, build
        f.argtypes = argtypes

    def __call__(self, **kw):
        a = {n: (k + 1) * STEP for k, n in enumerate(self.names)}
        a.update(kw)
        return self.f(*self.build(a))


@pytest.fixture
def token(lib):  # noqa: F811
    names = ["state", "x", "r", "i", "A", "z", "y"]
    return Call(lib.gdn_lru_decode_token, names, [P, P] + [P] * 8,
                lambda a: [C.byref(a.get("d", ld())), a.get("p"), *[a[n] for n in names], None])


@pytest.fixture
def prefill(lib):  # noqa: F811
    names = ["state", "x", "r", "i", "A", "z", "lengths", "y", "saved", "status", "ws"]
    lib.gdn_lru_prefill_workspace_bytes.restype = C.c_size_t
    return Call(lib.gdn_lru_prefill, names, [P, P, P, I32] + [P] * 10 + [C.c_size_t, P],
                lambda a: [C.byref(a.get("d", ld())), a.get("p"), a["state"], a.get("T", 1000),
                           *[a[n] for n in names[1:]], a.get("n", 1 << 30), None])


@pytest.fixture
def backward(lib):  # noqa: F811
    names = ["x", "r", "i", "A", "z", "lengths", "saved", "dy", "dstate", "dx", "dr", "di", "dz", "dA", "dstate0", "status", "ws"]
    return Call(lib.gdn_lru_backward, names, [P, P, P, I32] + [P] * 17 + [C.c_size_t, P],
                lambda a: [C.byref(a.get("d", ld())), a.get("p"), a.get("g"), a.get("T", 1000), *[a[n] for n in names],
                           a.get("n", 1 << 30), None])


def test_layer_refusals(lib, token, prefill, backward):  # noqa: F811
    for f in (lib.gdn_lru_state_bytes, lib.gdn_lru_saved_bytes, lib.gdn_lru_prefill_workspace_bytes,
              lib.gdn_lru_backward_workspace_bytes):
        f.restype = C.c_size_t
    assert lib.gdn_lru_state_bytes(C.byref(ld())) == 2 * 256 * 4
    for kw, want in BAD:
        for call in (token, prefill, backward):
            assert call(d=ld(**kw)) == want, kw
        assert lib.gdn_lru_state_bytes(C.byref(ld(**kw))) == 0
        for f in (lib.gdn_lru_saved_bytes, lib.gdn_lru_prefill_workspace_bytes, lib.gdn_lru_backward_workspace_bytes):
            assert f(C.byref(ld(**kw)), 1000) == 0
    for kw in BAD_PITCH:
        p = C.byref(Pitches(**kw))
        for call in (token, prefill, backward):
            assert call(p=p) == 2, kw
    for kw in BAD_PITCH[:4]:
        assert backward(g=C.byref(Pitches(**kw))) == 2, kw
    for T in (0, -1, (1 << 22) + 1):
        assert prefill(T=T) == 2 and backward(T=T) == 2
        assert lib.gdn_lru_saved_bytes(C.byref(ld()), T) == 0
    for call, names in ((token, token.names[:5] + ["y"]), (prefill, ["state", "x", "r", "i", "A", "y"]),
                        (backward, ["x", "r", "i", "A", "saved", "dy", "dx", "dr", "di", "dA"])):
        for n in names:
            assert call(**{n: None}) == 1, n
    for call in (token, prefill, backward):
        for n in call.names:
            if n != "ws":
                assert call(**{n: STEP * 40 + 8}) == 4, n
    assert backward(z=None) == 1 and backward(dz=None) == 1        # both or neither
    for call in (prefill, backward):
        assert call(ws=None) == 6 and call(n=16) == 6 and call(ws=STEP * 30 + 16) == 4
    assert prefill(T=50, ws=None, y=None) == 1                      # a short prompt needs no workspace: only the pointer
    assert lib.gdn_lru_prefill_workspace_bytes(C.byref(ld()), 50) == 0


def test_operands_that_overlap(token, prefill, backward):
    row = 256 * 2
    for call in (token, prefill):
        assert call(y=1 * STEP) == 8                                # the state
        for n in ("x", "r", "i", "z"):
            at = (call.names.index(n) + 1) * STEP
            assert call(y=at) == 8 and call(y=at + row // 2) == 8, n
    assert prefill(saved=STEP * 2 + 32) == 8 and prefill(status=STEP * 7) == 8 and prefill(ws=STEP * 2) == 8
    at = {n: (k + 1) * STEP for k, n in enumerate(backward.names)}
    for n in ("x", "r", "i", "z", "dy", "A", "lengths", "saved", "dr", "di", "dz", "dA"):
        assert backward(dx=at[n]) == 8, n
    assert backward(dA=at["A"]) == 8 and backward(dstate0=at["dstate"] + 16) == 8 and backward(ws=at["dy"]) == 8
    # rows between each other's are apart, rows that touch are not
    p = C.byref(Pitches(r=512, i=512))
    assert backward(p=p, g=p, dr=STEP * 50, di=STEP * 50 + row - 16) == 8
    assert backward(p=p, g=p, dr=STEP * 50, di=STEP * 50 + row, dA=None) == 1     # past the alias check's operands: only the pointer


def test_workspace_sizes_grow_with_every_argument(lib):  # noqa: F811
    fs = [lib.gdn_lru_prefill_workspace_bytes, lib.gdn_lru_backward_workspace_bytes, lib.gdn_lru_saved_bytes]
    for f in fs:
        f.restype = C.c_size_t
        f.argtypes = [P, I32]
    r = random.Random(2)
    seen = set()
    for _ in range(20000):
        a = [r.choice([1, 2, 3, 8, 16, 40, 200]), 8 * int(10 ** r.uniform(0, 3)), int(10 ** r.uniform(0, 4.5))]
        b = list(a)
        k = r.randrange(3)
        b[k] = b[k] + (8 * r.choice([1, 3, 8, 16, 100]) if k == 1 else r.choice([1, 2, 7, 31, 32, 64, 500]))
        for act in (0, 1):
            if not fs[2](C.byref(ld(b[0], b[1], act)), b[2]):       # beyond what a launch can count
                continue
            for f in fs:
                lo, hi = f(C.byref(ld(a[0], a[1], act)), a[2]), f(C.byref(ld(b[0], b[1], act)), b[2])
                assert lo <= hi, (a, b, act)
                seen.add((f is fs[0], lo == 0))
    assert (True, True) in seen and (True, False) in seen
    g, h = lib.gdn_residual_norm_backward_workspace_bytes, lib.gdn_gated_norm_backward_workspace_bytes
    g.restype = h.restype = C.c_size_t
    g.argtypes, h.argtypes = [I64, I32], [I64, I32, I32]
    for W in (8, 64, 264, 1024, 4096, 5120, 16384):
        got = [g(n, W) for n in (1, 2, 3, 255, 256, 257, 1000, 5000, 1 << 20)]
        assert got[0] > 0 and got == sorted(got)
        for H in (1, 3, 48):
            got = [h(n, H, W) for n in (1, 2, 3, 255, 256, 257, 1000, 5000, 1 << 20)]
            assert got[0] > 0 and got == sorted(got)


def test_residual_norm_refusals(lib):  # noqa: F811
    names = ["residual", "delta", "scale", "post", "w", "out", "y"]
    f = Call(lib.gdn_residual_norm, names, [I64, I32, I32, I32, C.c_float] + [P] * 8,
             lambda a: [a.get("rows", 4), a.get("W", 64), a.get("act", 1), a.get("res", 1), a.get("eps", 1e-6),
                        *[a[n] for n in names], None])
    gn = ["out", "delta", "scale", "post", "w", "dy", "ds", "dres", "ddelta", "dw", "dscale", "dpost", "ws"]
    g = Call(lib.gdn_residual_norm_backward, gn, [I64, I32, I32, I32, C.c_float] + [P] * 13 + [C.c_size_t, P],
             lambda a: [a.get("rows", 4), a.get("W", 64), a.get("act", 1), a.get("res", 1), a.get("eps", 1e-6),
                        *[a[n] for n in gn], a.get("n", 1 << 30), None])
    for call in (f, g):
        for kw in (dict(rows=0), dict(rows=-1), dict(rows=1 << 31), dict(W=0), dict(W=4), dict(W=60), dict(W=16392),
                   dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-39), dict(eps=float("nan")), dict(eps=float("inf"))):
            assert call(**kw) == 2, kw
        assert call(act=2) == 3 and call(res=2) == 3 and call(act=0, res=1) == 3
        for n in call.names:
            if n != "ws":
                assert call(**{n: STEP * 40 + 4}) == 4, n
    for n in ("residual", "w", "y", "delta", "out"):
        assert f(**{n: None}) == 1, n
    for n in ("out", "w", "dy", "dres", "dw", "delta", "ddelta", "scale", "dscale", "post", "dpost"):
        assert g(**{n: None}) == 1, n
    assert g(ws=None) == 6 and g(n=8) == 6 and g(ws=STEP * 40 + 16) == 4
    at = {n: (k + 1) * STEP for k, n in enumerate(names)}
    assert f(y=at["residual"]) == 8 and f(y=at["delta"]) == 8 and f(out=at["residual"] + 16) == 8 and f(out=at["y"]) == 8
    at = {n: (k + 1) * STEP for k, n in enumerate(gn)}
    assert g(dres=at["out"]) == 8 and g(dres=at["ds"] + 16) == 8 and g(ddelta=at["dy"]) == 8 and g(dw=at["w"]) == 8


def test_gated_norm_refusals(lib):  # noqa: F811
    names = ["o", "z", "w", "y"]
    head = [I64, I32, I32, I32, I32, I32, C.c_float, P, P, I64]
    pick = lambda a: [a.get("rows", 4), a.get("H", 3), a.get("D", 64), a.get("odt", 0), a.get("act", 1), a.get("flags", 0),
                      a.get("eps", 1e-6), a["o"], a["z"], a.get("pitch", 0), a["w"]]
    f = Call(lib.gdn_gated_norm, names, head + [P, P, P], lambda a: [*pick(a), a["y"], None])
    gn = ["o", "z", "w", "dy", "do", "dz", "dw", "ws"]
    g = Call(lib.gdn_gated_norm_backward, gn, head + [P, P, P, P, I64, P, P, C.c_size_t, P],
             lambda a: [*pick(a), a["dy"], a["do"], a["dz"], a.get("dpitch", 0), a["dw"], a["ws"], a.get("n", 1 << 30), None])
    for call in (f, g):
        for kw in (dict(rows=0), dict(H=0), dict(H=65537), dict(D=0), dict(D=12), dict(D=16392), dict(rows=1 << 30, H=2),
                   dict(flags=4), dict(flags=-1), dict(eps=0.0), dict(pitch=184), dict(pitch=196), dict(pitch=-8),
                   dict(pitch=1 << 55), dict(H=65536, D=16384)):
            assert call(**kw) == 2, kw
        assert call(act=2) == 3 and call(odt=5) == 3 and call(odt=1, act=0) == 3
        for n in call.names:
            if n != "ws":
                assert call(**{n: None}) == 1, n
                assert call(**{n: STEP * 40 + 8}) == 4, n
    assert g(dpitch=184) == 2
    assert g(ws=None) == 6 and g(n=8) == 6 and g(ws=STEP * 40 + 16) == 4
    at = {n: (k + 1) * STEP for k, n in enumerate(gn)}
    assert f(y=1 * STEP) == 8 and f(y=2 * STEP) == 8 and f(y=3 * STEP) == 8
    assert g(dz=at["z"]) == 8 and g(do=at["o"]) == 8 and g(dw=at["w"]) == 8 and g(do=at["dz"]) == 8


def test_binding_refusals():
    import gated_deltanet_decode_amd as gdn
    with pytest.raises(gdn.GdnError):
        gdn.lru_prefill(gdn.lru_dims(0, 64), None, torch.zeros(1, 2, 64), None, None, None, None, None)
    with pytest.raises(ValueError, match="x must be"):
        gdn.lru_prefill(gdn.lru_dims(2, 64), None, torch.zeros(3, 63), None, None, None, None, None)
    with pytest.raises(ValueError, match="x must be"):
        gdn.lru_backward(gdn.lru_dims(2, 64), None, None, None, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="residual must be"):
        gdn.residual_norm(torch.zeros(0, 8), None, None, None, None)
    with pytest.raises(ValueError, match="y must be a bfloat16 or float32"):
        gdn.residual_norm(torch.zeros(2, 8), None, None, None, torch.zeros(2, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="o must be"):
        gdn.gated_norm(torch.zeros(8), None, None, None)
    with pytest.raises(ValueError, match="out must be"):
        gdn.residual_norm_backward(None, None, None, None, None, None, None, None)


def test_pitch_of_a_slice():
    """The binding finds the one pitch of a slice's rows, and refuses slices without one."""
    import gated_deltanet_decode_amd as gdn

    class Dev(torch.Tensor):      # a host tensor that says it is on device 0
        def get_device(self):
            return 0
    wide = torch.zeros(4, 6, 64).as_subclass(Dev)
    rows = lambda t, lead, W: gdn._rows(t, "x", torch.float32, lead, W, 0)[1]
    assert rows(wide, 24, 64) == 0
    assert rows(wide[..., 16:32], 24, 16) == 64
    assert rows(wide[1:2, :, :16], 6, 16) == 64
    assert rows(wide[:, :1, :16], 4, 16) == 6 * 64
    assert rows(wide[:, 0, :16], 4, 16) == 6 * 64
    assert rows(wide[:1, :1, :16], 1, 16) in (0, 64)
    assert rows(wide.view(2, 2, 6, 64)[..., :8], 24, 8) == 64
    for t, lead, W in ((wide[:, :3, :16], 12, 16), (wide.transpose(0, 1)[..., :16], 24, 16), (wide[..., ::2], 24, 32)):
        with pytest.raises(ValueError, match="one pitch"):
            rows(t, lead, W)
