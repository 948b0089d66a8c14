"""GPU: the selective state space layer, token by token and over prompts,
against the 64-bit reference.

Tolerances, normwise (largest difference over the largest value), from a count
of roundings u = 2^-24: a conv output takes at most 8 (taps, exp2, reciprocal,
product), a step size 4, a decay weight exp(c_i - c_j) at most 64 u |c| exp(-|c|)
<= 24 u, operands split into two fp16 parts 4 u each: about 44 u of the terms'
absolute sum.  With random signs that sum is at most about 8 times the result's
largest value over the sizes used here, so state and fp32 outputs are held to
352 u = 2.1e-5.  A bf16 output adds half a step, 2^-8, and its chunk products
take fp16 operands (three roundings of 2^-12 relative, again times 8 at most):
2^-8 + 2^-9 = 5.9e-3.  Tails are copies and compared exactly.
"""
import numpy as np
import pytest
import torch

from tests import ssm_reference as sr
from tests.conftest import normwise

pytestmark = pytest.mark.gpu
TOL32, TOL16 = 2.1e-5, 5.9e-3

# name, H, G, P, N, bf16
LAYERS = [("p32n32_f32", 4, 2, 32, 32, False), ("p64n128_bf16", 6, 2, 64, 128, True),
          ("p64n64_g1_bf16", 5, 1, 64, 64, True), ("p128n128_bf16", 3, 3, 128, 128, True),
          ("p32n256_f32", 3, 1, 32, 256, False), ("p128n256_bf16", 2, 1, 128, 256, True),
          ("p64n32_f32", 3, 1, 64, 32, False), ("p64n128_f32", 4, 1, 64, 128, False),
          ("p128n64_f32", 2, 2, 128, 64, False)]
IDS = [c[0] for c in LAYERS]


def act(a, bf16):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(
        torch.bfloat16 if bf16 else torch.float32)


class Layer:
    def __init__(self, i):
        import gated_deltanet_decode_amd as gdn
        self.gdn, self.i = gdn, i
        bf = i["bf16"]
        self.d = gdn.ssm_dims(i["B"], i["H"], i["G"], i["P"], i["N"], 4, "bf16" if bf else "f32")
        f = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
        self.state, self.tail = f(i["state"]), act(i["tail"], bf)
        self.w, self.x = act(i["w"], bf), act(i["x"], bf)
        self.opt = dict(conv_bias=act(i["conv_bias"], bf), dt_bias=f(i["dt_bias"]), D=f(i["D"]))
        self.dt, self.A, self.z = f(i["dt"]), f(i["A"]), act(i["z"], bf)
        self.y = torch.full((i["B"], i["T"], i["H"], i["P"]), 7.0, device="cuda", dtype=self.d.act_torch)

    def tokens(self, t0, t1):
        other = torch.full_like(self.tail, 9.0)
        for t in range(t0, t1):
            c = lambda a: None if a is None else a[:, t].clone(memory_format=torch.contiguous_format)   # 16-byte aligned
            y = torch.empty_like(self.y[:, t]).contiguous()
            self.gdn.ssm_decode_token(self.d, self.state, self.tail, other, self.w, c(self.x), c(self.dt), self.A, y,
                                      z=c(self.z), **self.opt)
            self.y[:, t] = y
            self.tail, other = other, self.tail

    def prefill(self, lengths=None, status=None, ws=None, stream=None):
        T = self.i["T"]
        need = self.gdn.ssm_prefill_workspace_bytes(self.d, T)
        if ws is None:
            ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        self.gdn.ssm_prefill(self.d, self.state, self.tail, self.w, self.x, self.dt, self.A, self.y, ws, z=self.z,
                             lengths=lengths, status=status, stream=stream, **self.opt)
        return ws

    def check(self, lengths=None, what=""):
        torch.cuda.synchronize()
        y, state, tail = sr.run(self.i, lengths)
        assert normwise(self.state.cpu().numpy(), state) < TOL32, what
        assert np.array_equal(self.tail.float().cpu().numpy(), tail.astype(np.float32)), what
        got = self.y.float().cpu().numpy()
        live = ~np.isnan(y)
        assert (got[~live] == 7.0).all(), f"{what}: rows behind a sequence's end were written"
        if live.any():
            assert normwise(got[live], y[live]) < (TOL16 if self.i["bf16"] else TOL32), what


@pytest.mark.parametrize("name,H,G,P,N,bf16", LAYERS, ids=IDS)
@pytest.mark.parametrize("B", [1, 3])
def test_tokens(name, H, G, P, N, bf16, B):
    m = Layer(sr.make(11, B, 7, H, G, P, N, bf16))
    m.tokens(0, 7)
    m.check(what=name)


@pytest.mark.parametrize("P,N,H", [(32, 64, 40), (64, 64, 40), (128, 128, 33), (32, 128, 40), (64, 32, 40), (64, 256, 33)])
@pytest.mark.parametrize("bf16", [True, False])
def test_tokens_of_many_heads(P, N, H, bf16):
    """More (sequence, head) pairs than fill the chip: wider workgroups."""
    m = Layer(sr.make(12, 16, 3, H, 1, P, N, bf16))
    m.tokens(0, 3)
    m.check()


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 64, 65, 200])
@pytest.mark.parametrize("name,H,G,P,N,bf16", LAYERS, ids=IDS)
def test_prefill(name, H, G, P, N, bf16, T):
    m = Layer(sr.make(20 + T, 2, T, H, G, P, N, bf16, gate=T % 2 == 0))
    m.prefill()
    m.check(what=f"{name} T={T}")


@pytest.mark.parametrize("T", [7, 8, 9, 15, 16, 17, 33, 129, 500])
@pytest.mark.parametrize("H,G,P,N,bf16", [(4, 2, 32, 256, True), (2, 1, 128, 32, True), (6, 3, 64, 64, False),
                                          (2, 2, 128, 128, False)])
def test_prefill_around_its_forms(H, G, P, N, bf16, T):
    """Lengths on both sides of the token walk's end, and with one and several segments."""
    m = Layer(sr.make(220 + T, 2, T, H, G, P, N, bf16))
    m.prefill()
    m.check(what=f"T={T}")


@pytest.mark.parametrize("bf16", [True, False])
def test_prefill_of_a_batch_that_fills_the_chip(bf16):
    """Enough sequences and heads for one segment of many chunks each, with ragged ends."""
    i = sr.make(230, 16, 200, 64, 2, 64, 32, bf16)
    m = Layer(i)
    m.prefill()
    m.check()
    lengths = np.random.default_rng(1).integers(0, 201, 16).astype(np.int32)
    m = Layer(i)
    m.prefill(torch.from_numpy(lengths).cuda())
    m.check(lengths)


def test_prefill_of_sets_that_do_not_divide_by_the_xcds():
    """3 sequences x 23 segments: 69 sets of heads over eight XCDs."""
    m = Layer(sr.make(231, 3, 2944, 2, 1, 32, 32, True, gate=False))
    m.prefill()
    m.check()


@pytest.mark.parametrize("bf16", [True, False])
def test_prefill_many_chunks(bf16):
    """Long enough for several segments of chunks per sequence, with an odd end."""
    m = Layer(sr.make(5, 1, 1500, 2, 1, 64, 128, bf16, gate=False))
    m.prefill()
    m.check()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("H,G,P,N", [(66, 33, 32, 32), (33, 1, 64, 64), (65, 1, 32, 32), (24, 2, 64, 256), (68, 1, 32, 64)])
def test_prefill_of_segments_that_fill_the_chip(H, G, P, N, bf16):
    """Long prompts with one, two and four heads to a workgroup."""
    m = Layer(sr.make(33, 2, 2100, H, G, P, N, bf16))
    lengths = np.array([2100, 1801], np.int32)
    m.prefill(lengths=torch.from_numpy(lengths).cuda())
    m.check(lengths)


@pytest.mark.parametrize("name,H,G,P,N,bf16", LAYERS, ids=IDS)
def test_prefill_then_tokens(name, H, G, P, N, bf16):
    """A prompt, then decode: both continue from the same state and tail as the reference's one run."""
    i = sr.make(31, 2, 75, H, G, P, N, bf16)
    m = Layer(i)
    whole = dict(i)
    part = {**i, "T": 71, "x": i["x"][:, :71], "dt": i["dt"][:, :71], "z": i["z"][:, :71]}
    p = Layer(part)
    p.prefill()
    m.state, m.tail = p.state, p.tail
    m.y[:, :71] = p.y
    m.tokens(71, 75)
    m.i = whole
    m.check()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
def test_ragged_lengths(bf16, P, N):
    """Lengths 0, 1, chunk edges and T; a bad length leaves its sequence alone; what lies behind a
    sequence's end (NaN here) reaches nothing."""
    lengths = np.array([0, 1, 3, 63, 64, 65, 130, 150, 151, -1, 400], np.int32)
    i = sr.make(41, len(lengths), 150, 3, 1, P, N, bf16)
    m = Layer(i)
    for b, n in enumerate(lengths):
        for a in (m.x, m.dt, m.z):
            a[b, max(0, n):] = float("nan")
    st = torch.full((len(lengths),), -5, dtype=torch.int32, device="cuda")
    m.prefill(torch.from_numpy(lengths).cuda(), st)
    torch.cuda.synchronize()
    bad = (lengths < 0) | (lengths > 150)
    assert st.cpu().tolist() == [10 if b else 0 for b in bad]
    m.check(np.where(bad, 0, lengths))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T", [1, 40, 150])
def test_without_optional_operands(bf16, T):
    i = sr.make(51, 2, T, 4, 2, 64, 64, bf16, gate=False)
    i.update(conv_bias=None, dt_bias=None, D=None)
    m = Layer(i)
    m.prefill()
    m.check()
    m = Layer(i)
    m.tokens(0, min(T, 5))
    short = {**i, "T": min(T, 5)}
    m.i, m.y = short, m.y[:, :min(T, 5)]
    m.check()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("scale", [1e-4, 300.0])
def test_scales_of_the_activations(bf16, scale):
    """Activations far from one: SiLU passes large ones through, so x, B and C reach about scale."""
    m = Layer(sr.make(61, 1, 100, 2, 1, 64, 128, bf16, scale=scale, gate=False))
    m.prefill()
    m.check()


def test_large_values_stay_finite():
    """bf16 activations of 1e5 (beyond fp16's range), states of 1e8."""
    m = Layer(sr.make(62, 1, 80, 2, 1, 64, 64, True, scale=1e5, gate=False, state_scale=1e8))
    m.prefill()
    m.check()


@pytest.mark.parametrize("bf16", [True, False])
def test_strong_and_absent_decay(bf16):
    """Decays that vanish within a token, that never decay (A = 0), and a positive A (taken as 0)."""
    i = sr.make(71, 2, 130, 4, 1, 64, 64, bf16, gate=False)
    i["A"] = np.array([-1e4, 0.0, 2.0, -0.5], np.float32)
    m = Layer(i)
    m.prefill()
    m.check()
    m = Layer(i)
    m.tokens(0, 130)
    m.check()


def test_step_sizes_at_the_ends_of_softplus():
    i = sr.make(72, 1, 70, 2, 1, 64, 64, False, gate=False)
    i["dt_bias"] = None
    i["dt"][0, ::3] = -200.0        # softplus underflows to 0: state and output pass through
    i["dt"][0, 1::3] = 30.0
    m = Layer(i)
    m.prefill()
    m.check()


@pytest.mark.parametrize("bf16", [True, False])
def test_a_token_that_wipes_the_state(bf16):
    """A step so long that the sums of decays grow past what their differences may be rounded by."""
    i = sr.make(73, 1, 130, 2, 1, 64, 64, bf16, gate=False)
    i["A"] = np.array([-8.0, -2.0], np.float32)
    i["dt"][0, 5], i["dt"][0, 70] = 5e4, 3e4
    m = Layer(i)
    m.prefill()
    m.check()


@pytest.mark.parametrize("T", [1, 5, 100])
@pytest.mark.parametrize("bf16", [True, False])
def test_a_broken_decay_shows(bf16, T):
    """A NaN in A: that head's state and outputs are NaN, the other heads' as ever."""
    i = sr.make(74, 1, T, 3, 1, 64, 64, bf16)
    i["A"][1] = np.nan
    y, state, _ = sr.run(i)
    for by_token in (True, False):
        m = Layer(i)
        if by_token:
            m.tokens(0, min(T, 5))
        else:
            m.prefill()
        torch.cuda.synchronize()
        n = min(T, 5) if by_token else T
        assert torch.isnan(m.state[:, 1]).all() and torch.isnan(m.y[:, :n, 1]).all()
        got = m.y.float().cpu().numpy()[:, :n, [0, 2]]
        assert normwise(got, y[:, :n, [0, 2]]) < (TOL16 if bf16 else TOL32)
        if not by_token:
            assert normwise(m.state.cpu().numpy()[:, [0, 2]], state[:, [0, 2]]) < TOL32


def test_a_sequence_does_not_depend_on_its_batch():
    """Bit for bit the same sequence alone in a batch of three copies (same grid rule per call)."""
    i = sr.make(81, 3, 100, 4, 1, 64, 128, True)
    for k in ("state", "tail", "x", "dt", "z"):
        i[k][1] = i[k][0]
    m = Layer(i)
    m.prefill()
    torch.cuda.synchronize()
    assert torch.equal(m.state[0], m.state[1]) and torch.equal(m.y[0], m.y[1]) and torch.equal(m.tail[0], m.tail[1])


def test_repeats_are_bitwise_equal_and_two_streams_do_not_mix():
    i = sr.make(82, 2, 300, 4, 1, 64, 128, True)
    j = sr.make(83, 2, 300, 4, 1, 64, 128, True)
    a, b = Layer(i), Layer(i)
    a.prefill()
    b.prefill()
    c, e = Layer(i), Layer(j)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        c.prefill()
    with torch.cuda.stream(s2):
        e.prefill()
    torch.cuda.synchronize()
    for o in (b, c):
        assert torch.equal(a.state, o.state) and torch.equal(a.y, o.y) and torch.equal(a.tail, o.tail)
    e.check()


@pytest.mark.parametrize("P,N,bf16", [(64, 128, True), (128, 256, False)])
def test_graph_of_prefill_and_tokens(P, N, bf16):
    """One captured prefill and two tokens, replayed three times with eager resets in between."""
    i = sr.make(84, 2, 200, 3, 1, P, N, bf16)
    m = Layer(i)
    ws = torch.empty(m.gdn.ssm_prefill_workspace_bytes(m.d, 200), dtype=torch.uint8, device="cuda")
    start = [m.state.clone(), m.tail.clone()]
    xt, dt, zt = m.x[:, 5].contiguous(), m.dt[:, 5].contiguous(), m.z[:, 5].contiguous()
    t2, yt = torch.empty_like(m.tail), torch.empty_like(m.y[:, 0]).contiguous()
    tail1 = m.tail

    def work():
        m.gdn.ssm_prefill(m.d, m.state, tail1, m.w, m.x, m.dt, m.A, m.y, ws, z=m.z, **m.opt)
        m.gdn.ssm_decode_token(m.d, m.state, tail1, t2, m.w, xt, dt, m.A, yt, z=zt, **m.opt)
        m.gdn.ssm_decode_token(m.d, m.state, t2, tail1, m.w, xt, dt, m.A, yt, z=zt, **m.opt)
    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in (m.state, tail1, m.y, yt)]

    def reset():
        m.state.copy_(start[0])
        tail1.copy_(start[1])
        m.y.fill_(7.0)
        yt.fill_(0)
        ws.fill_(0xAB)
        torch.cuda.synchronize()
    reset()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for _ in range(3):
        reset()
        g.replay()
        torch.cuda.synchronize()
        for got, w in zip((m.state, tail1, m.y, yt), want):
            assert torch.equal(got, w)


def test_refuses_short_and_foreign_tensors():
    m = Layer(sr.make(91, 2, 10, 2, 1, 64, 64, True))
    with pytest.raises(ValueError, match="workspace"):
        m.prefill(ws=torch.empty(1, dtype=torch.uint8, device="cuda"))
    ok = m.dt
    m.dt = ok[:, :5].contiguous()
    with pytest.raises(ValueError, match="dt"):
        m.prefill()
    m.dt, m.A = ok, m.A.double()
    with pytest.raises(ValueError, match="A must be"):
        m.prefill()
    with pytest.raises(m.gdn.GdnError):
        m.gdn.ssm_decode_token(m.d, m.state, m.tail, m.tail, m.w, m.x[:, 0].contiguous(), ok[:, 0].contiguous(),
                               m.A.float(), m.y[:, 0].contiguous())
