"""GPU: rows of large values, and of small ones beside a small eps.  A row's norm is right for every mean square that fp32 holds, however many values
the row has: the sum of the squares, up to 16,384 times the mean, may be beyond fp32."""
import numpy as np
import pytest
import torch

from tests import lru_reference as lr
from tests.test_gpu_lru import dev
from tests.test_gpu_norms import TYPES, Gated, Residual

pytestmark = pytest.mark.gpu
# mean squares of some 4e34 and 2e37: 16,384 squares of the first and a few of the second pass 3.4e38
SIZES = [1e17, 2e18]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("W", [16, 64, 520, 4104, 8200, 16384])
@pytest.mark.parametrize("act,res", TYPES)
def test_residual_norm(W, size, act, res):
    m = Residual(W, 5, W, act, res, post=W != 520, size=size, ds=False)
    with np.errstate(over="ignore"):      # the reference's sums are of 64 bits
        m.forward()
        m.check()
        m.backward()
        m.check_grads()
    assert (m.y.float().abs().amax(1) > 0.1).all()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("H,D", [(3, 16), (3, 128), (2, 4096), (1, 8200), (1, 16384)])
@pytest.mark.parametrize("act,o", TYPES)
@pytest.mark.parametrize("first", [True, False])
def test_gated_norm(H, D, size, act, o, first):
    m = Gated(D, 5, H, D, act, o, first, False)
    big = m.n["o"].astype(np.float64) * (2 * size / 0.5)
    m.n["o"] = lr.bf16_round(big) if o == "bf16" else big.astype(np.float32)
    m.t["o"] = dev(m.n["o"], o == "bf16")
    m.run()
    m.check()


@pytest.mark.parametrize("eps", [1.2e-38, 1e-31, 1e-20])
@pytest.mark.parametrize("W", [128, 16384])
def test_small_rows_beside_a_small_eps(eps, W):
    """Mean squares around the smallest eps keep their digits, as they do around any."""
    import gated_deltanet_decode_amd as gdn
    r = np.random.default_rng(W)
    # powers of two of the root of eps: squares from far below eps to far above it
    x = (r.standard_normal((9, W)) * np.sqrt(eps) * 2.0 ** np.arange(-12, 15, 3)[:, None]).astype(np.float32)
    w, y = dev(np.ones(W)), torch.empty(9, W, device="cuda")
    gdn.residual_norm(dev(x), None, w, None, y, eps=eps)
    v = x.astype(np.float64)
    want = v * lr.rms(v, float(np.float32(eps)))
    got = y.double().cpu().numpy()
    # a square below 2^-126 is off by half a step of 2^-149: W of them by 2^-150 each of their mean, half of it in
    # the root, beside an eps of at least 2^-126
    tol = (lr.norm_error(0) + 3 * lr.U + 0.5 * 2.0 ** -150 / eps) * np.abs(want) + lr.TINY
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("W", [8, 64, 128, 256, 1024, 8200])
def test_large_rows_beside_ordinary_ones(W):
    """A row that is summed again changes nothing of its neighbours', which share its wave or follow in its workgroup;
    infinite and NaN values reach their own row alone."""
    a, b = (Residual(W, 300, W, "bf16", "bf16") for _ in range(2))
    huge = torch.arange(300) % 7 == 3
    for k in ("residual", "delta"):
        b.t[k][huge] *= 2.0 ** 60
    b.t["residual"][5, 3], b.t["residual"][12, W - 1] = float("inf"), float("nan")
    ga, gb = (Gated(W, 300, 2, W, "bf16", "f32", True, False) for _ in range(2))
    gb.t["o"][huge] *= 2.0 ** 61
    gb.t["o"][5, 0, 3], gb.t["o"][12, 1, W - 1] = float("inf"), float("nan")
    for m in (a, b):
        m.forward()
        m.backward()
    for m in (ga, gb):
        m.run()
    torch.cuda.synchronize()
    rest = ~huge
    rest[5] = rest[12] = False
    for k in ("out", "y", "dres", "ddelta"):
        assert torch.equal(getattr(a, k)[rest], getattr(b, k)[rest]), k
    for k in ("y", "do", "dz"):
        assert torch.equal(getattr(ga, k)[rest], getattr(gb, k)[rest]), k
    assert (b.y[huge].float().abs().amax(1) > 0.1).all() and (gb.y[huge].float().abs().amax((1, 2)) > 1e-3).all()
    assert torch.isnan(b.y[12]).all() and torch.isnan(gb.y[12, 1]).all() and torch.isfinite(gb.y[12, 0]).all()
    assert torch.isfinite(gb.y[5, 1]).all()
