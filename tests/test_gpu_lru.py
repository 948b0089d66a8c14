"""GPU: the gated linear recurrent layer, token by token, over prompts, and its
gradient, against the 64-bit reference.  Every value is held to the bound that
the reference carries beside it (its own terms, counted in half steps of fp32 and
of the output's type)."""
import numpy as np
import pytest
import torch

from tests import lru_reference as lr

pytestmark = pytest.mark.gpu
HELD = 7.0      # what outputs hold before a call


def dev(a, bf16=False):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(
        torch.bfloat16 if bf16 else torch.float32)


def near(got, want, tol, what):
    got = got.detach().float().cpu().numpy().astype(np.float64)
    live = ~np.isnan(want)
    off = np.abs(got[live] - want[live]) - tol[live]
    assert not (off > 0).any() and not np.isnan(got[live]).any(), (
        f"{what}: off by {np.abs(got[live] - want[live])[np.argmax(off)]:.3e} where {tol[live][np.argmax(off)]:.3e} is allowed")
    return got[~live]


class Layer:
    def __init__(self, i, packed=False):
        import gated_deltanet_decode_amd as gdn
        self.gdn, self.i = gdn, i
        bf, W = i["bf16"], i["W"]
        self.d = gdn.lru_dims(i["B"], W, "bf16" if bf else "f32")
        self.state, self.A = dev(i["state"]), dev(i["A"])
        self.x, self.r, self.i_, self.z = (dev(i[k], bf) for k in ("x", "r", "i", "z"))
        new = lambda n=1: torch.full((i["B"], i["T"], n * W), HELD, device="cuda", dtype=self.d.act_torch)
        self.y, self.dx, self.dr, self.di = new(), new(), new(), new()
        self.dz = new() if i["z"] is not None else None
        if packed:   # r | i | x | z in one projection's rows, and their gradients in another's
            both = new(4)
            for k, t in enumerate((self.r, self.i_, self.x, self.z)):
                if t is not None:
                    both[..., k * W:(k + 1) * W] = t
            self.r, self.i_, self.x = (both[..., k * W:(k + 1) * W] for k in range(3))
            if self.z is not None:
                self.z = both[..., 3 * W:]
            grads = new(4)
            self.dr, self.di, self.dx = (grads[..., k * W:(k + 1) * W] for k in range(3))
            if self.dz is not None:
                self.dz = grads[..., 3 * W:]
            wide = new(2)
            self.y = wide[..., W:]
            self.held = [(wide, W)]
        self.dA = torch.full((W,), HELD, device="cuda")
        self.dstate0 = torch.full((i["B"], W), HELD, device="cuda")

    def ws(self, n):
        return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") if n else None

    def prefill(self, lengths=None, saved=False, status=None, stream=None):
        T = self.i["T"]
        self.saved = self.ws(self.gdn.lru_saved_bytes(self.d, T)) if saved else None
        w = self.ws(self.gdn.lru_prefill_workspace_bytes(self.d, T))
        self.gdn.lru_prefill(self.d, self.state, self.x, self.r, self.i_, self.A, self.y, w, z=self.z, lengths=lengths,
                             saved=self.saved, status=status, stream=stream)

    def backward(self, lengths=None, status=None, dstate=True, stream=None):
        w = self.ws(self.gdn.lru_backward_workspace_bytes(self.d, self.i["T"]))
        dy = torch.full_like(self.x, HELD).contiguous()
        dy.copy_(dev(self.i["dy"], self.i["bf16"]))
        if lengths is not None:
            for b, n in enumerate(lengths.tolist()):
                dy[b, max(0, n):] = float("nan")
        self.gdn.lru_backward(self.d, self.x, self.r, self.i_, self.A, dy, self.saved, self.dx, self.dr, self.di, self.dA, w,
                              z=self.z, dz=self.dz, dstate=dev(self.i["dstate"]) if dstate else None, dstate0=self.dstate0,
                              lengths=lengths, status=status, stream=stream)

    def check(self, lengths=None, what="", ref=None):
        torch.cuda.synchronize()
        f = lr.run(self.i, lengths) if ref is None else ref
        near(self.state, f["state"], f["es"], what + " state")
        held = near(self.y, f["y"], f["ey"], what + " y")
        assert (held == HELD).all(), f"{what}: rows behind a sequence's end were written"
        return f

    def check_grads(self, f, lengths=None, what=""):
        torch.cuda.synchronize()
        want, tol = lr.grad(self.i, lengths, f)
        for k in want:
            near(getattr(self, k), want[k], tol[k], f"{what} {k}")


SIZES = [(8, 1), (40, 3), (64, 2), (72, 1), (200, 3)]


@pytest.mark.parametrize("W,B", SIZES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("packed", [True, False])
def test_tokens(W, B, bf16, packed):
    i = lr.make(1, B, 6, W, bf16, gate=W != 40)
    m = Layer(i, packed)
    for t in range(6):
        at = lambda v: None if v is None else v[:, t] if packed else v[:, t].contiguous().clone()
        y = m.y[:, t] if packed else torch.empty(B, W, device="cuda", dtype=m.d.act_torch)
        m.gdn.lru_decode_token(m.d, m.state, at(m.x), at(m.r), at(m.i_), m.A, y, z=at(m.z))
        if not packed:
            m.y[:, t] = y
    m.check(what=f"W={W}")


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 512, 513, 1030])
@pytest.mark.parametrize("bf16", [True, False])
def test_prefill_and_gradient(T, bf16):
    W, B = SIZES[T % len(SIZES)]
    m = Layer(lr.make(100 + T, B, T, W, bf16, gate=T % 3 != 0), packed=T % 2 == 0)
    m.prefill(saved=True)
    f = m.check(what=f"T={T}")
    m.backward(dstate=True)
    m.check_grads(f, what=f"T={T}")


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("gate", [True, False])
def test_many_segments(bf16, gate):
    """Long enough that many tiles of one sequence run side by side; batches and widths beside it."""
    m = Layer(lr.make(7, 2, 3000, 136, bf16, gate))
    m.prefill(saved=True)
    f = m.check()
    m.backward()
    m.check_grads(f)


@pytest.mark.parametrize("B,T,W", [(16, 128, 2056), (16, 100, 2056), (40, 33, 1032), (70, 32, 2056), (6, 300, 2056), (3, 1100, 1032),
                                   (24, 129, 1544)])
@pytest.mark.parametrize("bf16", [True, False])
def test_batches_that_fill_the_chip(B, T, W, bf16):
    """Enough channels and sequences for the wide tiles, on both sides of their lengths."""
    m = Layer(lr.make(9, B, T, W, bf16, gate=T != 100))
    m.prefill(saved=True)
    f = m.check()
    m.backward()
    m.check_grads(f)


@pytest.mark.parametrize("bf16", [True, False])
def test_no_saved_states_and_no_gradient_of_the_state(bf16):
    i = lr.make(8, 2, 300, 64, bf16)
    m = Layer(i)
    m.prefill()
    f = m.check()
    m = Layer({**i, "dstate": np.zeros_like(i["dstate"])})
    m.prefill(saved=True)
    m.backward(dstate=False)
    m.check_grads(f)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("packed", [True, False])
def test_ragged_lengths(bf16, packed):
    """Lengths 0, 1, tile edges and T; a bad length leaves its sequence alone; what lies behind a
    sequence's end (NaN here) reaches nothing, and its gradients are 0."""
    lengths = np.array([0, 1, 3, 127, 128, 129, 255, 256, 257, 511, 600, -1, 601, 2 ** 31 - 1], np.int32)
    i = lr.make(41, len(lengths), 600, 72, bf16)
    good = [b for b, n in enumerate(lengths) if 0 <= n <= 600]
    m = Layer(i, packed)
    for b, n in enumerate(lengths):
        for a in (m.x, m.r, m.i_, m.z):
            a[b, max(0, n):] = float("nan")
    ld = torch.from_numpy(lengths).cuda()
    st = torch.full((len(lengths),), -5, dtype=torch.int32, device="cuda")
    before = m.state.clone()
    m.prefill(ld, saved=True, status=st)
    sub = {k: (v[good] if isinstance(v, np.ndarray) and k != "A" else v) for k, v in i.items()}
    sub["B"] = len(good)
    ok = lengths[good]
    f = lr.run(sub, ok)
    torch.cuda.synchronize()
    assert st.tolist() == [0 if b in good else 10 for b in range(len(lengths))]
    bad = [b for b in range(len(lengths)) if b not in good]
    assert torch.equal(m.state[bad], before[bad]) and (m.y[bad].float() == HELD).all()
    near(m.state[good], f["state"], f["es"], "state")
    assert (near(m.y[good], f["y"], f["ey"], "y") == HELD).all()
    st.fill_(-5)
    m.backward(ld, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0 if b in good else 10 for b in range(len(lengths))]
    want, tol = lr.grad(sub, ok, f)
    for k in ("dx", "dr", "di", "dz", "dstate0"):
        g = getattr(m, k)
        near(g[good], want[k], tol[k], k)
        assert (g[bad].float() == HELD).all(), k
    near(m.dA, want["dA"], tol["dA"], "dA")


def test_prefill_then_tokens_and_prefill_in_parts():
    i = lr.make(31, 2, 400, 64, False)
    m = Layer(i)
    cut = [0, 300, 301, 397, 400]
    for a, b in zip(cut, cut[1:]):
        p = Layer({**i, "T": b - a, **{k: i[k][:, a:b] for k in ("x", "r", "i", "z", "dy")}})
        p.state = m.state
        if b - a == 3:
            for t in range(3):
                at = lambda v: v[:, t].contiguous().clone()
                y = torch.empty(2, 64, device="cuda")
                p.gdn.lru_decode_token(p.d, p.state, at(p.x), at(p.r), at(p.i_), p.A, y, z=at(p.z))
                p.y[:, t] = y
        else:
            p.prefill()
        m.y[:, a:b] = p.y
    m.check()


def test_a_prompt_of_one_token_is_the_token_bit_for_bit():
    i = lr.make(32, 5, 1, 200, False)
    m, n = Layer(i), Layer(i)
    m.prefill()
    n.gdn.lru_decode_token(n.d, n.state, n.x, n.r, n.i_, n.A, n.y, z=n.z)
    torch.cuda.synchronize()
    assert torch.equal(m.state, n.state) and torch.equal(m.y, n.y)


@pytest.mark.parametrize("bf16", [True, False])
def test_extreme_gates(bf16):
    """Gates far open and shut, rates of 0, above 0, tiny and large: every value stays within its bound."""
    i = lr.make(51, 2, 260, 64, bf16)
    r = np.random.default_rng(2)
    pick = lambda *v: lr.bf16_round(r.choice(v, (2, 260, 64)))
    i["r"], i["i"], i["z"] = pick(-90, -30, -8, 0, 8, 30, 80), pick(-60, -20, 0, 15, 90), pick(-80, -20, 0, 25)
    i["A"] = r.choice([0.0, 3.0, -1e-6, -0.01, -1.0, -8.0, -60.0], 64).astype(np.float32)
    m = Layer(i)
    m.prefill(saved=True)
    f = m.check()
    m.backward()
    # a shut gate's 1/m meets 0 gradients of r: bounded by the terms, which the reference counts
    m.check_grads(f)


def test_infinite_gate_inputs_are_their_limits():
    i = lr.make(52, 1, 140, 64, False, gate=False)
    j = {**i, "r": i["r"].copy(), "i": i["i"].copy()}
    i["r"][0, 5], i["r"][0, 70], i["i"][0, 9] = np.inf, -np.inf, np.inf
    j["r"][0, 5], j["r"][0, 70], j["i"][0, 9] = 200, -200, 200
    m, n = Layer(i), Layer(j)
    for a in (m, n):
        a.prefill(saved=True)
        a.backward()
    torch.cuda.synchronize()
    for k in ("y", "state", "dx", "dr", "di", "dA", "dstate0"):
        assert torch.equal(getattr(m, k), getattr(n, k)), k


@pytest.mark.parametrize("t", [0, 4, 127, 128, 300])
def test_nan_reaches_its_channel_from_its_token_on(t):
    i = lr.make(53, 1, 400, 64, False)
    m = Layer(i)
    m.x[0, t, 11] = float("nan")
    m.prefill()
    torch.cuda.synchronize()
    nan = torch.isnan(m.y[0]).cpu()
    want = torch.zeros_like(nan)
    want[t:, 11] = True
    assert torch.equal(nan, want)


def test_equal_inputs_give_equal_bits_and_gradients_on_another_stream():
    i = lr.make(61, 3, 700, 200, True)
    a, b = Layer(i), Layer(i)
    a.prefill(saved=True)
    a.backward()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b.prefill(saved=True)
        b.backward()
    s.synchronize()
    for k in ("y", "state", "dx", "dr", "di", "dz", "dA", "dstate0"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k


def test_gradient_of_the_state_in_place():
    i = lr.make(62, 2, 500, 64, False)
    a, b = Layer(i), Layer(i)
    for m in (a, b):
        m.prefill(saved=True)
    a.backward()
    g = dev(i["dstate"])
    w = b.ws(b.gdn.lru_backward_workspace_bytes(b.d, 500))
    b.gdn.lru_backward(b.d, b.x, b.r, b.i_, b.A, dev(i["dy"]), b.saved, b.dx, b.dr, b.di, b.dA, w, z=b.z, dz=b.dz, dstate=g,
                       dstate0=g)
    torch.cuda.synchronize()
    assert torch.equal(g, a.dstate0) and torch.equal(b.dx, a.dx)


def test_captured_calls_share_a_workspace():
    """Two graphs on one workspace, replayed in turn with eager work between, give the eager results every time."""
    i = lr.make(63, 2, 600, 136, True)
    eager = Layer(i)
    eager.prefill(saved=True)
    eager.backward()
    torch.cuda.synchronize()
    m = Layer(i)
    m.prefill(saved=True)
    m.backward()
    first = dev(i["state"])
    n = max(m.gdn.lru_prefill_workspace_bytes(m.d, 600), m.gdn.lru_backward_workspace_bytes(m.d, 600))
    w, dy, g = m.ws(n), dev(i["dy"], True), dev(i["dstate"])
    torch.cuda.synchronize()
    fwd, bwd = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(fwd):
        m.state.copy_(first)
        m.gdn.lru_prefill(m.d, m.state, m.x, m.r, m.i_, m.A, m.y, w, z=m.z, saved=m.saved)
    with torch.cuda.graph(bwd):
        m.gdn.lru_backward(m.d, m.x, m.r, m.i_, m.A, dy, m.saved, m.dx, m.dr, m.di, m.dA, w, z=m.z, dz=m.dz, dstate=g,
                           dstate0=m.dstate0)
    for _ in range(4):
        for t in (m.y, m.dx, m.dr, m.di, m.dz, m.dA, m.dstate0, m.saved, w):
            t.zero_()
        torch.cuda.synchronize()
        fwd.replay()
        (m.y.float() * 2).sum().item()
        bwd.replay()
        torch.cuda.synchronize()
        for k in ("y", "state", "dx", "dr", "di", "dz", "dA", "dstate0"):
            assert torch.equal(getattr(m, k), getattr(eager, k)), k


def test_rows_whose_offsets_pass_32_bits():
    """Rows 1 MB apart (2^20 bf16 elements, the largest pitch): 2,600 of them reach beyond 2^32 bytes and 2^31 elements."""
    T, W = 2600, 64
    i = lr.make(71, 1, T, W, True)
    m = Layer(i)
    wide = torch.empty(1, T, 1 << 20, dtype=torch.bfloat16, device="cuda")
    for k, name in enumerate(("x", "r", "i_", "z")):
        part = wide[..., k * W:(k + 1) * W]
        part.copy_(getattr(m, name))
        setattr(m, name, part)
    m.y = wide[..., 4 * W:5 * W]
    m.dx, m.dr, m.di, m.dz = (wide[..., k * W:(k + 1) * W] for k in range(5, 9))
    m.prefill(saved=True)
    f = m.check()
    m.backward()
    m.check_grads(f)


def test_two_prompts_at_once():
    """Chained calls on two streams, each with a workspace of its own, several times over: both end as they do alone."""
    i, j = lr.make(81, 4, 2000, 264, True), lr.make(82, 2, 3100, 520, False)
    want = [Layer(i), Layer(j)]
    for m in want:
        m.prefill(saved=True)
        m.backward()
    torch.cuda.synchronize()
    got, streams = [Layer(i), Layer(j)], [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [m.ws(max(m.gdn.lru_prefill_workspace_bytes(m.d, m.i["T"]), m.gdn.lru_backward_workspace_bytes(m.d, m.i["T"]))) for m in got]
    first, dy = [m.state.clone() for m in got], [dev(m.i["dy"], m.i["bf16"]) for m in got]
    g = [dev(m.i["dstate"]) for m in got]
    saved = [m.ws(m.gdn.lru_saved_bytes(m.d, m.i["T"])) for m in got]
    torch.cuda.synchronize()
    for _ in range(6):
        for k, m in enumerate(got):
            with torch.cuda.stream(streams[k]):
                m.state.copy_(first[k])
                m.gdn.lru_prefill(m.d, m.state, m.x, m.r, m.i_, m.A, m.y, ws[k], z=m.z, saved=saved[k])
                m.gdn.lru_backward(m.d, m.x, m.r, m.i_, m.A, dy[k], saved[k], m.dx, m.dr, m.di, m.dA, ws[k], z=m.z, dz=m.dz,
                                   dstate=g[k], dstate0=m.dstate0)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for k in ("y", "state", "dx", "dr", "di", "dz", "dA", "dstate0"):
            assert torch.equal(getattr(a, k), getattr(b, k)), k


def test_more_sequences_than_a_grid_is_high():
    """70,000 sequences of 8 channels: tokens, and prompts of two tokens."""
    i = lr.make(83, 70000, 2, 8, True)
    m, n = Layer(i), Layer(i)
    m.prefill(saved=True)
    for t in range(2):
        at = lambda v: v[:, t].contiguous().clone()
        y = torch.empty(70000, 8, device="cuda", dtype=torch.bfloat16)
        n.gdn.lru_decode_token(n.d, n.state, at(n.x), at(n.r), at(n.i_), n.A, y, z=at(n.z))
        n.y[:, t] = y
    torch.cuda.synchronize()
    # both are within 100 u of values below 8, and round a bf16 half a step of a value below 12 each at most
    assert (m.state - n.state).abs().max() < 5e-5 and (m.y.float() - n.y.float()).abs().max() < 0.1
    f = lr.run({**i, "B": 3, **{k: i[k][-3:] for k in ("x", "r", "i", "z", "dy", "state", "dstate")}})
    near(n.state[-3:], f["state"], f["es"], "state")
    near(m.y[-3:], f["y"], f["ey"], "y")


def test_device_operands_that_do_not_fit():
    """Wrong types, sizes, strides, devices and workspaces raise before anything is launched."""
    i = lr.make(91, 2, 300, 64, True)
    m = Layer(i)
    g, T = m.gdn, 300
    w = m.ws(g.lru_backward_workspace_bytes(m.d, T))
    saved = m.ws(g.lru_saved_bytes(m.d, T))
    ok = dict(x=m.x, r=m.r, i=m.i_, A=m.A, y=m.y, state=m.state, z=m.z, saved=saved, workspace=w, lengths=None)
    before = {k: v.clone() for k, v in ok.items() if v is not None}

    def call(**kw):
        a = {**ok, **kw}
        g.lru_prefill(m.d, a["state"], a["x"], a["r"], a["i"], a["A"], a["y"], a["workspace"], z=a["z"], lengths=a["lengths"],
                      saved=a["saved"])
    wide = torch.zeros(2, T, 128, dtype=torch.bfloat16, device="cuda")
    for kw, err in ((dict(r=m.r.float()), ValueError), (dict(r=m.r[:, :100]), ValueError), (dict(r=m.r.cpu()), ValueError),
                    (dict(r=wide[..., ::2]), ValueError), (dict(i=wide[..., 4:68]), g.GdnError), (dict(A=m.A[:32]), ValueError),
                    (dict(state=m.state.double()), ValueError), (dict(z=m.z.float()), ValueError), (dict(saved=saved[:-4]), ValueError),
                    (dict(workspace=None), g.GdnError), (dict(workspace=w[:256]), g.GdnError), (dict(workspace=w[16:]), g.GdnError),
                    (dict(workspace=w.cpu()), ValueError), (dict(lengths=torch.zeros(2, device="cuda")), ValueError),
                    (dict(y=m.x), g.GdnError), (dict(y=None), TypeError)):
        with pytest.raises(err):
            call(**kw)
    torch.cuda.synchronize()
    for k, v in before.items():
        assert torch.equal(v, ok[k]), k


@pytest.mark.parametrize("bf16", [True, False])
def test_ragged_lengths_of_wide_tiles(bf16):
    """The same where the batch is large enough for the wide tiles (32 and 128 tokens), with ends on and beside their edges."""
    lengths = np.array([0, 1, 31, 32, 33, 63, 64, 96, 127, 128, 129, 255, 256, 512, 599, 600], np.int32)
    i = lr.make(92, 16, 600, 2056, bf16, gate=bf16)
    m = Layer(i)
    for b, n in enumerate(lengths):
        for a in (m.x, m.r, m.i_, m.z):
            if a is not None:
                a[b, n:] = float("nan")
    ld = torch.from_numpy(lengths).cuda()
    m.prefill(ld, saved=True)
    f = m.check(lengths)
    m.backward(ld)
    m.check_grads(f, lengths)


@pytest.mark.parametrize("bf16", [True, False])
def test_a_long_narrow_sequence(bf16):
    """One sequence of few channels: chains of 157 and 313 tiles, each link waited for."""
    m = Layer(lr.make(93, 1, 20011, 8, bf16))
    m.prefill(saved=True)
    f = m.check()
    m.backward()
    m.check_grads(f)
