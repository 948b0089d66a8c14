"""CPU: the 64-bit reference of the selective state space layer and of beam
selection, pinned by closed forms and hand-worked cases."""
import numpy as np
import pytest

from tests import ssm_reference as sr


def test_bf16_rounding_is_to_nearest_even():
    one = np.float32(1)
    assert sr.bf16_round(np.array([1 + 2.0 ** -8], np.float32))[0] == one                # tie, even below
    assert sr.bf16_round(np.array([1 + 3 * 2.0 ** -8], np.float32))[0] == one + 2.0 ** -6  # tie, even above
    assert sr.bf16_round(np.array([1 + 2.0 ** -8 + 2.0 ** -16], np.float32))[0] == one + 2.0 ** -7


def test_one_entry_by_hand():
    """One head of one row and entry, no bias: two tokens worked out by hand."""
    i = dict(B=1, T=2, H=1, G=1, P=1, N=1, C=3, bf16=False, state=np.full((1, 1, 1, 1), 2.0), tail=np.zeros((1, 3, 4)),
             w=np.tile(np.array([0, 0, 0, 1.0]), (3, 1)), conv_bias=None, x=np.array([[[1.0, 2.0, 3.0], [0, 1.0, 1.0]]]),
             dt=np.array([[[0.0], [0.0]]]), dt_bias=None, A=np.array([-1.0]), D=np.array([0.5]), z=None)
    y, state, tail = sr.run(i)
    s = lambda v: v / (1 + np.exp(-v))
    d = np.log(2)                                      # softplus(0); the decay is exp(-log 2) = 1/2
    S1 = 0.5 * 2 + d * s(1) * s(2)
    S2 = 0.5 * S1
    assert y[0, 0, 0, 0] == pytest.approx(S1 * s(3) + 0.5 * s(1), rel=1e-14)
    assert y[0, 1, 0, 0] == pytest.approx(S2 * s(1), rel=1e-14)
    assert state[0, 0, 0, 0] == pytest.approx(S2, rel=1e-14)
    assert tail[0, 0].tolist() == [0, 0, 1, 0]


def test_chunk_form_is_the_same_algebra():
    """y and state of 37 tokens from the closed form: S_T = sum_t exp(sum_{s>t} a_s) d_t x_t B_t^T."""
    i = sr.make(3, 1, 37, 4, 2, 32, 32, False, gate=False)
    y, state, _ = sr.run(i)
    rows = np.concatenate([i["tail"][0].T[1:], i["x"][0]], 0).astype(np.float64)
    u = sum(rows[j:j + 37] * i["w"][:, j] for j in range(4)) + i["conv_bias"]
    u = u / (1 + np.exp(-u))
    d = np.logaddexp(0, i["dt"][0].astype(np.float64) + i["dt_bias"])
    cum = np.cumsum(d * i["A"], 0)
    for h in range(4):
        g = h // 2
        x = u[:, h * 32:(h + 1) * 32]
        Bm, Cm = u[:, 128 + g * 32:160 + g * 32], u[:, 192 + g * 32:224 + g * 32]
        L = np.tril(np.exp(np.minimum(cum[:, None, h] - cum[None, :, h], 0)))
        yy = (L * (Cm @ Bm.T)) @ (d[:, h:h + 1] * x) + np.exp(cum[:, h:h + 1]) * (Cm @ i["state"][0, h].T.astype(float))
        SS = np.exp(cum[-1, h]) * i["state"][0, h] + (np.exp(cum[-1, h] - cum[:, h:h + 1]) * d[:, h:h + 1] * x).T @ Bm
        assert np.allclose(yy + i["D"][h] * x, y[0, :, h], rtol=1e-11, atol=1e-12)
        assert np.allclose(SS, state[0, h], rtol=1e-11, atol=1e-12)


def test_select_by_hand():
    lg = np.log(np.array([[[0.5, 0.25, 0.25], [0.125, 0.125, 0.75]]]))
    val, par, tok = sr.select(lg, np.log(np.array([[0.5, 1.0]])), 4)
    # 0.25, 0.125, 0.125 | 0.125, 0.125, 0.75
    assert list(zip(par[0], tok[0])) == [(1, 2), (0, 0), (0, 1), (0, 2)]
    assert np.allclose(np.exp(val[0]), [0.75, 0.25, 0.125, 0.125])
    val, par, tok = sr.select(lg, np.log(np.array([[0.5, 1.0]])), 5, finished=np.array([[0, 1]]), eos=1)
    assert list(zip(par[0], tok[0])) == [(1, 1), (0, 0), (0, 1), (0, 2), (1, 0)]
    assert val[0, 0] == 0 and val[0, 4] == -np.inf
