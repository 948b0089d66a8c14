"""CPU: the 64-bit gradients that the GPU tests compare with, against central
differences of the 64-bit forward forms; and the layer against a hand-worked step."""
import math

import numpy as np
import pytest

from tests import lru_reference as lr


def differences(loss, arrays, grads, seed=0, picks=12, h=1e-5):
    r = np.random.default_rng(seed)
    for name, a in arrays.items():
        for _ in range(picks):
            at = tuple(r.integers(0, n) for n in a.shape)
            was = a[at]
            a[at] = was + h
            up = loss()
            a[at] = was - h
            down = loss()
            a[at] = was
            want = (up - down) / (2 * h)
            # the difference itself is off by h^2/6 of a third derivative and by rounding over 2h
            assert abs(grads[name][at] - want) < 1e-6 * max(1, abs(want)), (name, at)


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("lengths", [None, [5, 0, 3]])
def test_layer_gradients(gate, lengths):
    i = lr.make(1, 3, 5, 8, False, gate)
    i = {k: v.astype(np.float64) if isinstance(v, np.ndarray) else v for k, v in i.items()}
    out, _ = lr.grad(i, lengths)

    def loss():
        f = lr.run(i, lengths)
        return np.nansum(f["y"] * i["dy"]) + (f["state"] * i["dstate"]).sum()
    names = {"x": "dx", "r": "dr", "i": "di", "A": "dA", "state": "dstate0", **({"z": "dz"} if gate else {})}
    differences(loss, {g: i[k] for k, g in names.items()}, out)


def test_layer_by_hand():
    i = dict(B=1, T=1, W=1, bf16=False, state=np.array([[2.0]]), A=np.array([-math.log(4)]), x=np.array([[[3.0]]]),
             r=np.zeros((1, 1, 1)), i=np.zeros((1, 1, 1)), z=np.zeros((1, 1, 1)))
    f = lr.run(i)
    # a = 4^(-1/2), m = sqrt(1 - 1/4), gate 1/2
    assert abs(f["state"][0, 0] - (1.0 + math.sqrt(0.75) * 1.5)) < 1e-14
    assert f["y"][0, 0, 0] == 0.0
    i["A"] = np.array([5.0])               # a rate above 0 is 0: the state stays, nothing enters
    assert lr.run(i)["state"][0, 0] == 2.0


@pytest.mark.parametrize("scale", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("delta", [True, False])
def test_residual_norm_gradients(delta, scale, post):
    if not delta and (scale or post):
        return
    r = np.random.default_rng(3)
    W = 8
    a = {k: r.standard_normal((4, W)) for k in ("residual", "delta", "dy", "ds")}
    a |= {k: 1 + 0.3 * r.standard_normal(W) for k in ("w", "scale", "post")}
    opt = lambda k, on: a[k] if on else None
    args = lambda: dict(scale=opt("scale", scale), post=opt("post", post))

    def loss():
        out, _ = lr.residual_norm(a["residual"], opt("delta", delta), a["w"], **args())
        return (lr.norm_of(out, a["w"])[0] * a["dy"]).sum() + (out * a["ds"]).sum()
    out, _ = lr.residual_norm(a["residual"], opt("delta", delta), a["w"], **args())
    g, _ = lr.residual_norm_grad(out, opt("delta", delta), a["w"], a["dy"], a["ds"], **args())
    names = {"dresidual": "residual", "dw": "w"}
    if delta:
        names |= {"ddelta": "delta", **({"dscale": "scale"} if scale else {}), **({"dw_post": "post"} if post else {})}
    differences(loss, {k: a[v] for k, v in names.items()}, g)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("shared", [True, False])
def test_gated_norm_gradients(first, shared):
    r = np.random.default_rng(4)
    H, D = 3, 8
    a = {k: r.standard_normal((4, H, D)) for k in ("o", "z", "dy")}
    a["w"] = 1 + 0.3 * r.standard_normal(D if shared else (H, D))
    loss = lambda: (lr.gated_norm(a["o"], a["z"], a["w"], first)[0] * a["dy"]).sum()
    g, _ = lr.gated_norm_grad(a["o"], a["z"], a["w"], a["dy"], first, shared=shared)
    differences(loss, {"do": a["o"], "dz": a["z"], "dw": a["w"]}, g)
