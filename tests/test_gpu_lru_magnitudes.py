"""GPU: the recurrent layer far from 1: large and small states that decay through many tokens, and infinities."""
import numpy as np
import pytest
import torch

from tests import lru_reference as lr
from tests.test_gpu_lru import Layer, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1e-30, 1e12, 1e30])
@pytest.mark.parametrize("B,T,W", [(2, 40, 64), (2, 700, 72), (16, 300, 1032)])
@pytest.mark.parametrize("empty", [True, False])
def test_states_that_decay(B, T, W, size, empty):
    """A product of decays below 2^-126 may count as 0: what it multiplies is a state, no larger than the first one
    and the terms behind it together, once for a lane's tokens, a wave's, a tile's and the tiles' looked at."""
    i = lr.make(5, B, T, W, False)
    i["state"] = (i["state"] * size).astype(np.float32)
    i["dstate"] = (i["dstate"] * size).astype(np.float32)
    i["A"][::2] *= 12                                    # a channel of two forgets within some tokens
    if empty:
        i["x"][:, 3:-3], i["dy"][:, 3:-3] = 0, 0
    m = Layer(i)
    m.prefill(saved=True)
    f = lr.run(i)
    # what is lost of a state in all tokens behind it
    lost = 4 * lr.TINY * f["mag"].max(1)
    near(m.state, f["state"], f["es"] + lost, "state")
    z = np.abs(i["z"]) if i["z"] is not None else 1.0
    near(m.y, f["y"], f["ey"] + lost[:, None] * z, "y")
    m.backward()
    want, tol = lr.grad(i, None, f)
    most = np.abs(i["dstate"]) + np.abs(i["dy"] * i["z"]).sum(1)
    near(m.dstate0, want["dstate0"], tol["dstate0"] + 4 * lr.TINY * most, "dstate0")
    # dx = G m g with m and g at most 1
    near(m.dx, want["dx"], tol["dx"] + 4 * lr.TINY * most[:, None], "dx")


@pytest.mark.parametrize("where", ["state", "x"])
def test_infinities_stay_in_their_channel(where):
    """Not finite from its token on, in its channel alone."""
    i = lr.make(54, 2, 400, 64, False, gate=False)
    m = Layer(i)
    if where == "state":
        m.state[1, 9] = float("inf")
    else:
        m.x[1, 130, 9] = float("inf")
    m.prefill()
    torch.cuda.synchronize()
    bad = ~torch.isfinite(m.y).cpu()
    want = torch.zeros_like(bad)
    want[1, 0 if where == "state" else 130:, 9] = True
    assert torch.equal(bad, want)
    assert torch.equal(~torch.isfinite(m.state).cpu(), want[:, -1])
