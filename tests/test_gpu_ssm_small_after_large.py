"""GPU: state space prompts whose small values follow large ones within a chunk
of 64 tokens: a long step that wipes the state, with and without an input of its
own, and an entering state that decays away.  Every state row and every output
is held to its own terms, so that nothing large elsewhere hides it.

Taps are (0, 0, 0, 1) without a bias, so that conv outputs are SiLU(x) and have
no cancellation of their own.  With u = 2^-24 and magnitudes (the same
recurrence over absolute values) S~ of a state entry and y~ of an output:

State.  An entry's terms err by 8 u each for x and B, 12 u for the fp16 parts and
the product that they leave out, and for a decay of 2^-c by 4 u of the steps, u of
the rate and u of the rounded sum, 6 u c ln 2: 250 u for c = 60, the most of any
row here that is not zero.  A chunk's products are added to an accumulator 12
times: 120 u over the ten chunks that a term may last.  Parts below fp16's range
are off by 2^-25 beside a row's largest of 2^8.  So each entry is held to
400 u of its row's largest S~.
Outputs.  fp32: the same, C's 8 u and the sums' 64 u: 500 u of y~.  bf16: half a
step, 2^-8 of |y|, and fp16 operands: C, B and G cut (2^-10 each), M.G, x, X'
and the state rounded (2^-11 each, X' twice), the decays' high part alone
(2^-11): 6 * 2^-10 of y~.  And beside the chunk's largest product Z = N |C_t|
max_j(d_j |B_j|) max_j |x_j| (largest entries over the chunk's tokens j) what is
below fp16's range: 2^-24 of it in fp32, 2^-16 in bf16, whose steps are fp16
numbers in one scale per chunk.
"""
import numpy as np
import pytest

from tests import ssm_reference as sr
from tests.test_gpu_ssm import Layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def reference(i):
    """(y, state, y~, S~, Z) in 64 bits, token by token; taps (0, 0, 0, 1), no bias, no gate."""
    B, T, H, G, P, N = (i[k] for k in ("B", "T", "H", "G", "P", "N"))
    u = i["x"].astype(np.float64)
    u = u / (1 + np.exp(-u))
    grp = np.arange(H) // (H // G)
    x = u[..., :H * P].reshape(B, T, H, P)
    Bm = u[..., H * P:H * P + G * N].reshape(B, T, G, N)[:, :, grp]
    Cm = u[..., H * P + G * N:].reshape(B, T, G, N)[:, :, grp]
    d = np.logaddexp(0, i["dt"].astype(np.float64))
    a = np.exp(d * np.minimum(i["A"].astype(np.float64), 0))
    D = i["D"].astype(np.float64)[:, None]
    S = i["state"].astype(np.float64)
    Sm = np.abs(S)
    y, ym, Z = (np.zeros((B, T, H, P)) for _ in range(3))
    dB = d * np.abs(Bm).max(-1)
    for t in range(T):
        inc = (d[:, t, :, None] * x[:, t])[..., None] * Bm[:, t, :, None, :]
        S = a[:, t, :, None, None] * S + inc
        Sm = a[:, t, :, None, None] * Sm + np.abs(inc)
        y[:, t] = (S * Cm[:, t, :, None, :]).sum(-1) + D * x[:, t]
        ym[:, t] = (Sm * np.abs(Cm[:, t, :, None, :])).sum(-1) + np.abs(D * x[:, t])
        c = slice(t // 64 * 64, t // 64 * 64 + 64)
        Z[:, t] = N * np.abs(Cm[:, t]).max(-1)[..., None] * dB[:, c].max(1)[..., None] * np.abs(x[:, c]).max(1)
    return y, S, ym, Sm, Z


def quiet(seed, T, H, G, P, N, bf16, steps):
    """Two sequences with plain taps, steps of about `steps` and A = -8 or -16."""
    i = sr.make(seed, 2, T, H, G, P, N, bf16, gate=False)
    i["w"][:] = [0, 0, 0, 1]
    i["conv_bias"] = i["dt_bias"] = None
    i["dt"] = np.log(np.expm1(steps * np.random.default_rng(seed).uniform(0.5, 1.5, i["dt"].shape))).astype(np.float32)
    i["A"] = np.resize(np.array([-8.0, -16.0], np.float32), H)
    return i


def raw_step(d):
    return np.log(np.expm1(d)).astype(np.float32)


def run(i, copies):
    """The prompts, each `copies` times over (enough to fill the chip takes the form of one segment)."""
    y, S, ym, Sm, Z = reference(i)
    tile = lambda v: np.tile(v, (copies,) + (1,) * (v.ndim - 1))
    m = Layer({**i, "B": 2 * copies, **{k: tile(i[k]) for k in ("state", "tail", "x", "dt")}})
    m.prefill()
    got_S = m.state.cpu().numpy().astype(np.float64).reshape(copies, *S.shape)
    got_y = m.y.float().cpu().numpy().astype(np.float64).reshape(copies, *y.shape)
    lim = 400 * U * Sm.max(-1, keepdims=True)
    worst = (np.abs(got_S - S) / lim).max()
    assert worst <= 1, f"state: {worst:.3g} times the bound"
    lim = 2.0 ** -8 * np.abs(y) + 6 * 2.0 ** -10 * ym + 2.0 ** -16 * Z if i["bf16"] else 500 * U * ym + U * Z
    worst = (np.abs(got_y - y) / (lim + 1e-37)).max()
    assert worst <= 1, f"outputs: {worst:.3g} times the bound"


# name, T, H, G, P, N, copies of the two sequences
FORMS = [("segments", 270, 6, 2, 64, 64, 1), ("segments_n128_p128", 400, 4, 2, 128, 128, 1),
         ("segments_n256", 270, 3, 1, 32, 256, 1), ("one_segment", 200, 64, 2, 64, 32, 8),
         ("one_segment_n128", 140, 64, 1, 64, 128, 8), ("one_segment_n256", 140, 64, 1, 64, 256, 4)]
forms = pytest.mark.parametrize("T,H,G,P,N,copies", [f[1:] for f in FORMS], ids=[f[0] for f in FORMS])
types = pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])


@types
@forms
def test_a_wipe_without_an_input(T, H, G, P, N, copies, bf16):
    """A chunk's last token decays the state by 2^-6 to 2^-40 and has x = 0, and so have all that follow: what they
    put out is carried over the wipe."""
    i = quiet(1, T, H, G, P, N, bf16, 0.003)
    bits = np.resize(np.array([6, 18.5, 20.5, 22.5, 25.5, 40]), H)
    i["dt"][:, 63] = raw_step(bits * np.log(2) / -i["A"])
    i["x"][:, 63:, :H * P] = 0
    run(i, copies)


@types
@forms
def test_an_entering_state_behind_a_wipe(T, H, G, P, N, copies, bf16):
    """No inputs at all, and a step that decays the entering state by 2^-6 to 2^-40 within the first chunk."""
    i = quiet(5, T, H, G, P, N, bf16, 0.003)
    bits = np.resize(np.array([6, 18.5, 20.5, 22.5, 25.5, 40]), H)
    i["dt"][:, 5] = raw_step(bits * np.log(2) / -i["A"])
    i["x"][..., :H * P] = 0
    run(i, copies)


@types
@forms
@pytest.mark.parametrize("at", [5, 63])
def test_a_long_step(T, H, G, P, N, copies, bf16, at):
    """A step of 5e4 with its input, of which later decays leave nothing."""
    i = quiet(2, T, H, G, P, N, bf16, 0.1)
    i["dt"][:, at] = 5e4
    i["dt"][:, -40] = 3e4
    run(i, copies)


@types
@forms
@pytest.mark.parametrize("size", [1e3, 1e6])
def test_a_large_state_that_decays_away(T, H, G, P, N, copies, bf16, size):
    i = quiet(3, T, H, G, P, N, bf16, 0.1)
    i["state"] *= size
    run(i, copies)


@types
@forms
def test_inputs_far_apart(T, H, G, P, N, copies, bf16):
    """Channels of very different sizes, and steps that fall by 2^12 within a chunk."""
    i = quiet(4, T, H, G, P, N, bf16, 0.1)
    i["dt"][:, 20::64] = raw_step(2.0 ** -12)
    i["x"][..., :H * P:3] *= 2.0 ** -10
    i["x"][..., 1:H * P:3] *= 2.0 ** 7
    run(i, copies)
