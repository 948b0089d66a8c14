"""GPU: beam selection where a row holds about as many 16-byte groups of logits
as are selected, and masks empty whole groups: the bound that the scan starts
from then lies among the masked logits."""
import numpy as np
import pytest

from tests import ssm_reference as sr
from tests.test_gpu_beam import INF, check, gpu_select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("K", [1, 3])
@pytest.mark.parametrize("S", [1, 2, 16, 64])
def test_masked_groups(S, K, bf16):
    """One group masked, all but one, every one, and single entries of each; rows of exactly S groups and a few more."""
    E = 8 if bf16 else 4
    r = np.random.default_rng(S + K)
    for V in range(E * S, E * S + E):
        for bad in (-INF, np.nan):
            lg = r.standard_normal((6, K, V))
            lg[0, :, :E] = bad                                 # the first group
            lg[1, :, E * (S - 1):E * S] = bad                  # the last whole one
            lg[2, 0, :E * S] = bad                             # every group of one beam
            lg[3, :, E:] = bad                                 # all but the first
            lg[4] = bad                                        # nothing left
            lg[5, :, ::2] = bad                                # half of each
            check(lg, -r.random((6, K)), min(S, K * V), bf16=bf16)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_masked_groups_of_rows_off_their_alignment(off):
    """Rows that start within 16 bytes, so that the groups do too."""
    r = np.random.default_rng(off)
    for S in (2, 16, 64):
        V = 4 * S + 3
        lg = r.standard_normal((2, 3, V))
        lg[:, :, 4:8] = -INF
        lg[1, 1, :] = -INF
        check(lg, -r.random((2, 3)), S, pitch=V + off)


def test_nothing_but_masked_logits_in_many_spans():
    """Long rows of masked logits with a few live ones, S above and below their number."""
    r = np.random.default_rng(3)
    for bf16 in (False, True):
        lg = np.full((2, 2, 40007), -INF, np.float32)
        lg[:, :, [5, 9001, 39999]] = r.standard_normal((2, 2, 3))
        for S in (1, 3, 6, 40):
            check(lg, -r.random((2, 2)), S, bf16=bf16)


def test_every_output_is_written():
    """With one beam whose logits are all masked but for a few in one group."""
    lg = np.full((1, 1, 64), -INF, np.float32)
    lg[0, 0, 4:8] = [1, 2, 3, 4]
    val, par, tok = gpu_select(lg, np.zeros((1, 1)), 16)
    want = sr.select(lg, np.zeros((1, 1), np.float32), 16)
    assert (par == 0).all() and np.array_equal(tok, want[2])
    assert tok[0, :4].tolist() == [7, 6, 5, 4] and tok[0, 4:].tolist() == [0, 1, 2, 3, *range(8, 16)]
