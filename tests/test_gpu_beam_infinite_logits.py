"""GPU: beam selection where +inf, which counts as the largest finite fp32
value, stands beside the largest finite bf16 value, which is smaller."""
import numpy as np
import pytest

from tests import ssm_reference as sr
from tests.test_gpu_beam import INF, gpu_select

pytestmark = pytest.mark.gpu
MAX16 = 3.3895313892515355e38


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("S", [1, 2, 5, 40])
@pytest.mark.parametrize("many", [3, 60, 400])
def test_infinite_beside_the_largest_finite(many, S, bf16):
    """`many` of the largest finite value before a few infinite ones, in every span of the row."""
    r = np.random.default_rng(many + S)
    V = 4096
    lg = r.standard_normal((2, 2, V))
    for s in range(0, V, 1024):
        lg[:, :, s + 3 + 2 * np.arange(many)] = MAX16
        lg[0, :, s + 900] = INF
        lg[1, 1, s + 1000:s + 1010] = INF
    scores = -r.random((2, 2)).astype(np.float32)
    logits = (np.where(np.isfinite(lg), sr.bf16_round(lg), lg) if bf16 else lg).astype(np.float32)
    want = sr.select(logits, scores, S)
    got = gpu_select(logits, scores, S, bf16=bf16)
    for b in range(2):
        # An ordinary logit l beside a largest of M = 3.4e38 has the value l - M, which is -M in 64 bits for any
        # |l| < 2^74 (half their spacing at M): the definition in 64 bits orders only the values above that.
        n = int((want[0][b] > -2e38).sum())
        assert n >= min(S, 8)
        assert np.array_equal(got[1][b, :n], want[1][b, :n]) and np.array_equal(got[2][b, :n], want[2][b, :n])
        assert np.allclose(got[0][b], want[0][b], rtol=2.0 ** -23, atol=2.0 ** -18)
        assert len(set(zip(got[1][b], got[2][b]))) == S
