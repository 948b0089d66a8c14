"""Operands whose rows are one row many times over (`expand`, a stride of 0) have no pitch:
the binding refuses them as inputs and as outputs, on the host and before any launch.
A constant gate is given as rows of its own."""
import pytest
import torch

import gated_deltanet_decode_amd as gdn


class Dev(torch.Tensor):
    """A host tensor that says it is on device 0."""
    def get_device(self):
        return 0


def zeros(*shape):
    return torch.zeros(*shape).as_subclass(Dev)


def rows(t, lead, W):
    return gdn._rows(t, "x", torch.float32, lead, W, 0)[1]


def heads(t, n, H, D):
    return gdn._head_rows(t, "z", torch.float32, n, H, D, 0)[1]


@pytest.mark.parametrize("of,to", [
    ((64,), (5, 64)), ((1, 64), (4, 64)), ((64,), (2, 3, 64)), ((1, 1, 64), (4, 6, 64)), ((1, 1, 64), (1, 6, 64)),
    ((1, 1, 64), (6, 1, 64)), ((1, 6, 64), (4, 6, 64)), ((4, 1, 64), (4, 6, 64)), ((1, 1, 1, 64), (2, 3, 4, 64)),
    ((2, 1, 1, 64), (2, 3, 4, 64)), ((1, 3, 1, 64), (2, 3, 4, 64)), ((1, 1, 4, 64), (2, 3, 4, 64)),
    ((2, 3, 1, 64), (2, 3, 4, 64)), ((6, 1), (6, 64)),
])
def test_rows_that_repeat_have_no_pitch(of, to):
    t = zeros(*of).expand(*to)
    with pytest.raises(ValueError, match="one pitch"):
        rows(t, t.numel() // 64, 64)
    wide = zeros(*of[:-1], 128)[..., :of[-1]].expand(*to)      # the same of a slice
    with pytest.raises(ValueError, match="one pitch"):
        rows(wide, t.numel() // 64, 64)


@pytest.mark.parametrize("of,to", [
    ((3, 16), (5, 3, 16)), ((1, 3, 16), (5, 3, 16)), ((1, 1, 16), (5, 1, 16)), ((1, 1, 16), (5, 3, 16)), ((5, 1, 16), (5, 3, 16)),
    ((1, 1, 3, 16), (2, 5, 3, 16)), ((2, 1, 3, 16), (2, 5, 3, 16)), ((1, 5, 3, 16), (2, 5, 3, 16)), ((5, 3, 1), (5, 3, 16)),
])
def test_heads_that_repeat_have_no_pitch(of, to):
    t = zeros(*of).expand(*to)
    with pytest.raises(ValueError, match="one pitch"):
        heads(t, t.numel() // (to[-2] * to[-1]), to[-2], to[-1])


def test_a_stride_of_0_over_one_row_says_nothing():
    one = torch.as_strided(torch.zeros(6 * 64), (1, 6, 64), (0, 64, 1)).as_subclass(Dev)
    assert rows(one, 6, 64) == 0
    part = torch.as_strided(torch.zeros(6 * 128), (1, 6, 64), (0, 128, 1)).as_subclass(Dev)
    assert rows(part, 6, 64) == 128
    assert rows(torch.as_strided(torch.zeros(6 * 128), (6, 1, 64), (128, 0, 1)).as_subclass(Dev), 6, 64) == 128
    assert rows(torch.as_strided(torch.zeros(6 * 128), (3, 1, 2, 64), (256, 0, 128, 1)).as_subclass(Dev), 6, 64) == 128
    assert heads(torch.as_strided(torch.zeros(5 * 64), (5, 1, 16), (64, 0, 1)).as_subclass(Dev), 5, 1, 16) == 64


B, T, W, H = 4, 6, 64, 4


def calls():
    """(name, function, operands that take rows at a pitch): each call of the binding that has any."""
    d = gdn.lru_dims(B, W, "f32")
    state, A = zeros(B, W), zeros(W)
    full = lambda *lead: {k: zeros(*lead, W) for k in ("x", "r", "i", "z", "y", "dy", "dx", "dr", "di", "dz")}
    t, p = full(B), full(B, T)
    buf = zeros(1 << 20)
    g = {k: zeros(B, H, W // H) for k in ("o", "z", "y", "dy", "do", "dz")}
    w = zeros(W // H)
    return [
        ("token", lambda a: gdn.lru_decode_token(d, state, a["x"], a["r"], a["i"], A, a["y"], z=a["z"]), t, "xrizy"),
        ("prefill", lambda a: gdn.lru_prefill(d, state, a["x"], a["r"], a["i"], A, a["y"], buf, z=a["z"], saved=buf), p, "xrizy"),
        ("backward", lambda a: gdn.lru_backward(d, a["x"], a["r"], a["i"], A, a["dy"], buf, a["dx"], a["dr"], a["di"], A, buf,
                                                z=a["z"], dz=a["dz"]), p, ["x", "r", "i", "z", "dy", "dx", "dr", "di", "dz"]),
        ("gated", lambda a: gdn.gated_norm(a["o"], a["z"], w, a["y"]), g, ["o", "z", "y"]),
        ("gated_backward", lambda a: gdn.gated_norm_backward(a["o"], a["z"], w, a["dy"], a["do"], a["dz"], w, buf), g,
         ["o", "z", "dy", "do", "dz"]),
    ]


@pytest.mark.parametrize("which", range(5))
def test_no_call_takes_repeated_rows(which, monkeypatch):
    """Inputs and outputs alike, and nothing reaches the library."""
    class Closed:
        def __getattr__(self, name):
            def call(*args):
                assert name.endswith("_bytes"), f"{name} was called"
                return 1
            return call
    name, call, operands, names = calls()[which]
    monkeypatch.setattr(gdn, "_here", lambda stream: (0, 0))
    monkeypatch.setattr(gdn, "_lib", Closed())
    for n in names:
        t = operands[n]
        for lead in {t.shape[:1], t.shape[:-2] if len(t.shape) > 2 else t.shape[:1]}:
            one = zeros(*[1] * len(lead), *t.shape[len(lead):])
            with pytest.raises(ValueError):
                call({**operands, n: one.expand(t.shape)})
        with pytest.raises(ValueError):
            call({**operands, n: zeros(t.shape[-1]).expand(t.shape)})


@pytest.mark.gpu
def test_device_operands_that_repeat():
    """The same on a device: nothing is written; a constant gate as rows of its own is taken."""
    d = gdn.lru_dims(B, W, "f32")
    full = lambda *s: torch.randn(*s, device="cuda")
    x, r, i, z, A, state = full(B, T, W), full(B, T, W), full(B, T, W), full(B, T, W), -torch.rand(W, device="cuda"), full(B, W)
    y, before = torch.full_like(x, 7.0), state.clone()
    for kw in (dict(r=full(W).expand(B, T, W)), dict(i=full(B, 1, W).expand(B, T, W)), dict(z=full(1, T, W).expand(B, T, W)),
               dict(x=full(1, 1, W).expand(B, T, W)), dict(y=full(W).expand(B, T, W))):
        a = {**dict(x=x, r=r, i=i, z=z, y=y), **kw}
        with pytest.raises(ValueError, match="one pitch"):
            gdn.lru_prefill(d, state, a["x"], a["r"], a["i"], A, a["y"], None, z=a["z"])
    o, w, out = full(B, H, 16), full(16), torch.full((B, H, 16), 7.0, device="cuda")
    with pytest.raises(ValueError, match="one pitch"):
        gdn.gated_norm(o, full(H, 16).expand(B, H, 16), w, out)
    torch.cuda.synchronize()
    assert torch.equal(state, before) and (y == 7.0).all() and (out == 7.0).all()
    gate = full(W)
    gdn.lru_prefill(d, state, x, gate.expand(B, T, W).contiguous(), i, A, y, None, z=z)
    s2 = before.clone()
    y2 = torch.empty(B, W, device="cuda")
    for t in range(T):
        gdn.lru_decode_token(d, s2, x[:, t], gate.expand(B, W).contiguous(), i[:, t], A, y2, z=z[:, t])
        # sums of at most 7 terms of magnitude below 8 each, gates within 10 half steps
        assert (y2 - y[:, t]).abs().max() < 7 * 8 * 20 * 2.0 ** -24 * z.abs().max()
