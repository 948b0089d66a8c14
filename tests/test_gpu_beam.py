"""GPU: beam search's selection against its definition in 64 bits (indices
exactly, values to fp32 rounding), and the in-place move of beams' states
against plain indexing (bit for bit)."""
import numpy as np
import pytest
import torch

from tests import ssm_reference as sr

pytestmark = pytest.mark.gpu
INF = float("inf")


def gpu_select(logits, scores, S, finished=None, eos=0, bf16=False, pitch=None):
    import gated_deltanet_decode_amd as gdn
    B, K, V = logits.shape
    t = torch.from_numpy(logits).cuda().to(torch.bfloat16 if bf16 else torch.float32)
    if pitch is not None:
        wide = torch.full((B, K, pitch), INF, device="cuda", dtype=t.dtype)    # +inf outside: must not be read in
        wide[..., :V] = t
        t = wide[..., :V]
    val = torch.full((B, S), 7.0, device="cuda")
    par = torch.full((B, S), -7, dtype=torch.int32, device="cuda")
    tok = torch.full((B, S), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((gdn.beam_select_workspace_bytes(B, K, V, S),), 0xFF, dtype=torch.uint8, device="cuda")
    fin = None if finished is None else torch.from_numpy(finished.astype(bool)).cuda()
    gdn.beam_select(t, torch.from_numpy(scores.astype(np.float32)).cuda(), val, par, tok, ws, finished=fin, eos=eos)
    torch.cuda.synchronize()
    return val.cpu().numpy(), par.cpu().numpy(), tok.cpu().numpy()


def check(logits, scores, S, finished=None, eos=0, bf16=False, pitch=None):
    logits = logits.astype(np.float32)
    if bf16:
        with np.errstate(all="ignore"):
            logits = np.where(np.isfinite(logits), sr.bf16_round(logits), logits).astype(np.float32)
    scores = scores.astype(np.float32)
    with np.errstate(all="ignore"):
        want = sr.select(logits, scores, S, finished, eos)
    got = gpu_select(logits, scores, S, finished, eos, bf16, pitch)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])
    live = np.isfinite(want[0])
    assert np.array_equal(got[0][~live], want[0][~live].astype(np.float32))
    # log of a sum of fp32 exponentials (each within 2 u of its argument's rounding, here below 64 u |l|) and one
    # rounding on output: 2^-18 absolute plus 2^-23 relative
    assert np.all(np.abs(got[0][live] - want[0][live]) <= 2.0 ** -18 + 2.0 ** -23 * np.abs(want[0][live]))


SIZES = [(1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (1, 4, 64, 64), (3, 2, 1000, 4), (2, 5, 4099, 10), (1, 32, 777, 64),
         (1, 1, 50021, 1), (2, 3, 70001, 6), (5, 7, 2048, 14), (40, 8, 1500, 16)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,K,V,S", SIZES)
def test_select(B, K, V, S, bf16):
    r = np.random.default_rng(B * 1000 + V)
    check(r.standard_normal((B, K, V)) * 2.5, -8 * r.random((B, K)), S, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("pitch", [1001, 1003, 1024])
def test_rows_at_a_pitch(pitch, bf16):
    r = np.random.default_rng(pitch)
    check(r.standard_normal((2, 3, 1000)), -r.random((2, 3)), 6, bf16=bf16, pitch=pitch)


@pytest.mark.parametrize("bf16", [True, False])
def test_every_order_and_ties(bf16):
    """Logits that rise (every one enters the list), that fall, that are all equal, and few distinct values."""
    V = 3000
    rise = np.linspace(-5, 5, V)
    rows = np.stack([rise, rise[::-1], np.zeros(V), np.round(np.random.default_rng(1).standard_normal(V))])
    for k in range(4):
        for S in (1, 9, 64):
            check(np.tile(rows[k], (2, 3, 1)), np.array([[-1.0, -1.0, -1.0], [-3.0, -2.0, -1.0]]), S, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
def test_long_spans_in_every_order(bf16):
    """Rows enough for four long spans each: buffers fill and are cut again and again."""
    B, K, V = 256, 4, 12000
    r = np.random.default_rng(2)
    for row in (np.linspace(-5, 5, V), np.linspace(5, -5, V), np.zeros(V) - 3, r.integers(0, 5, V) * 0.5):
        lg = np.ascontiguousarray(np.broadcast_to(row, (B, K, V)), dtype=np.float32)
        check(lg, -r.random((B, K)), 24, bf16=bf16)
    lg = np.full((B, K, V), -INF, np.float32)              # all but a few tokens masked
    lg[:, :, r.integers(0, V, 5)] = r.standard_normal(5)
    check(lg, -r.random((B, K)), 12, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
def test_masked_and_broken_logits(bf16):
    r = np.random.default_rng(5)
    V = 1030
    lg = r.standard_normal((6, 3, V))
    lg[0, :, 10:] = -INF                      # few candidates left
    lg[1, 1] = -INF                           # a row that the mask leaves empty
    lg[2, :, ::2] = np.nan
    lg[3, :] = -INF                           # nothing at all
    lg[4, 2, 5] = INF
    lg[4, 2, 900] = INF
    lg[5, 0] = np.finfo(np.float32).min if not bf16 else -3.3895313892515355e38
    for S in (1, 12, 64):
        check(lg, -r.random((6, 3)), S, bf16=bf16)


@pytest.mark.parametrize("V", [3, 64, 65, 900])
def test_first_step_and_finished_beams(V):
    r = np.random.default_rng(V)
    lg, sc = r.standard_normal((5, 4, V)), -r.random((5, 4))
    S = min(16, 4 * V)
    sc[0, 1:] = -INF                          # the first step: one beam exists
    sc[1] = -INF
    sc[2, 1] = np.nan
    fin = r.random((5, 4)) < 0.5
    fin[3] = True
    fin[4] = False
    for eos in (0, 2, V - 1):
        check(lg, sc, S, finished=fin, eos=eos)
        check(lg, sc, S, finished=fin, eos=eos, bf16=True)


def test_every_kind_of_nan_is_masked():
    """Quiet and signalling NaNs of either sign, in both types."""
    import gated_deltanet_decode_amd as gdn
    r = np.random.default_rng(11)
    V = 700
    for bf16, bad in ((True, [0x7FC0, 0xFFC0, 0x7F81, 0xFF81, 0x7FFF, 0xFFFF]),
                      (False, [0x7FC00000, 0xFFC00000, 0x7F800001, 0xFF800001, 0x7FFFFFFF, 0xFFFFFFFF])):
        clean = sr.bf16_round(r.standard_normal((1, 2, V)))
        masked = clean.copy()
        masked[:, :, ::3] = np.nan
        bits = (clean.view(np.uint32) >> 16).astype(np.uint16) if bf16 else clean.view(np.uint32).copy()
        bits[:, :, ::3] = np.resize(np.array(bad, bits.dtype), bits[:, :, ::3].shape)
        t = torch.from_numpy(bits.view(np.int16 if bf16 else np.int32)).cuda().view(
            torch.bfloat16 if bf16 else torch.float32)
        sc = np.array([[-0.5, -0.25]], np.float32)
        val, par, tok = (torch.zeros(1, 9, device="cuda", dtype=d) for d in (torch.float32, torch.int32, torch.int32))
        ws = torch.empty(gdn.beam_select_workspace_bytes(1, 2, V, 9), dtype=torch.uint8, device="cuda")
        gdn.beam_select(t, torch.from_numpy(sc).cuda(), val, par, tok, ws)
        torch.cuda.synchronize()
        want = sr.select(masked, sc, 9)
        assert np.array_equal(par.cpu().numpy(), want[1]) and np.array_equal(tok.cpu().numpy(), want[2])
        assert np.allclose(val.cpu().numpy(), want[0], rtol=2.0 ** -23, atol=2.0 ** -18)


def test_select_is_captured_and_replayed():
    import gated_deltanet_decode_amd as gdn
    r = np.random.default_rng(9)
    B, K, V, S = 2, 4, 9000, 8
    sets = [(r.standard_normal((B, K, V)).astype(np.float32), -r.random((B, K)).astype(np.float32)) for _ in range(3)]
    lg, sc = torch.empty(B, K, V, device="cuda"), torch.empty(B, K, device="cuda")
    val, par, tok = (torch.zeros(B, S, device="cuda", dtype=d) for d in (torch.float32, torch.int32, torch.int32))
    ws = torch.empty(gdn.beam_select_workspace_bytes(B, K, V, S), dtype=torch.uint8, device="cuda")
    lg.copy_(torch.from_numpy(sets[0][0]))
    sc.copy_(torch.from_numpy(sets[0][1]))
    gdn.beam_select(lg, sc, val, par, tok, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.beam_select(lg, sc, val, par, tok, ws)
    for l, s in sets:
        lg.copy_(torch.from_numpy(l))
        sc.copy_(torch.from_numpy(s))
        ws.fill_(0x11)
        g.replay()
        torch.cuda.synchronize()
        want = sr.select(l, s, S)
        assert np.array_equal(par.cpu().numpy(), want[1]) and np.array_equal(tok.cpu().numpy(), want[2])


def test_scores_in_place():
    """With as many selected as there are beams the scores may be replaced where they are."""
    import gated_deltanet_decode_amd as gdn
    r = np.random.default_rng(31)
    B, K, V = 6, 5, 3000
    logits = r.standard_normal((B, K, V)).astype(np.float32)
    scores = (-8 * r.random((B, K))).astype(np.float32)
    want = gpu_select(logits, scores, K)
    t, sc = torch.from_numpy(logits).cuda(), torch.from_numpy(scores).cuda()
    par, tok = (torch.empty(B, K, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(gdn.beam_select_workspace_bytes(B, K, V, K), dtype=torch.uint8, device="cuda")
    gdn.beam_select(t, sc, sc, par, tok, ws)
    for a, b in zip(want, (sc, par, tok)):
        assert np.array_equal(a, b.cpu().numpy())
    with pytest.raises(RuntimeError):
        gdn.beam_select(t, sc, sc.view(-1)[:B * 4].view(B, 4), par[:, :4].contiguous(), tok[:, :4].contiguous(), ws)


def test_refuses_a_vocabulary_beyond_32_bits():
    import gated_deltanet_decode_amd as gdn
    V = (1 << 32) + 64
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 9 GB")
    t = torch.empty(1, 1, V, dtype=torch.bfloat16, device="cuda")
    sc, par = torch.zeros(1, 1, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises((RuntimeError, ValueError)):
        gdn.beam_select(t, sc, sc.clone(), par, par.clone(), ws)


def test_select_refusals():
    import gated_deltanet_decode_amd as gdn
    lg = torch.zeros(2, 3, 100, device="cuda")
    out = (torch.zeros(2, 6, device="cuda"), torch.zeros(2, 6, dtype=torch.int32, device="cuda"),
           torch.zeros(2, 6, dtype=torch.int32, device="cuda"))
    ws = torch.empty(gdn.beam_select_workspace_bytes(2, 3, 100, 6), dtype=torch.uint8, device="cuda")
    sc = torch.zeros(2, 3, device="cuda")
    with pytest.raises(ValueError, match="pitch"):
        gdn.beam_select(lg.transpose(0, 1).contiguous().transpose(0, 1), sc, *out, ws)
    with pytest.raises(ValueError, match="pitch"):
        gdn.beam_select(torch.zeros(2, 3, 200, device="cuda")[..., ::2], sc, *out, ws)
    with pytest.raises(ValueError):
        gdn.beam_select(lg.half(), sc, *out, ws)
    with pytest.raises(ValueError, match="scores"):
        gdn.beam_select(lg, sc[:1], *out, ws)
    with pytest.raises(gdn.GdnError):
        gdn.beam_select(lg, sc, *out, ws, finished=torch.zeros(2, 3, dtype=torch.bool, device="cuda"), eos=100)


# ------------------------------------------------------------------ reorder

def layer(kind, batch, bf16=True, H=3, P=64, N=128, G=1):
    import gated_deltanet_decode_amd as gdn
    a = "bf16" if bf16 else "f32"
    d = gdn.dims(batch, 2, 4, 32, 32, 4, a) if kind == "gdn" else gdn.ssm_dims(batch, H, G, P, N, 4, a)
    g = torch.Generator(device="cuda").manual_seed(batch)
    n = gdn.state_bytes(d) // 4 if kind == "gdn" else gdn.ssm_state_bytes(d) // 4
    state = torch.randn(batch, n // batch, generator=g, device="cuda")
    tail = torch.randn(batch, d.C * 4, generator=g, device="cuda").to(d.act_torch)
    return d, state, tail


@pytest.mark.parametrize("kind", ["gdn", "ssm"])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,K", [(1, 1), (1, 2), (3, 4), (2, 5), (4, 8), (2, 13), (1, 16), (2, 17), (1, 32)])
def test_reorder(kind, bf16, B, K):
    import gated_deltanet_decode_amd as gdn
    d, state, tail = layer(kind, B * K, bf16)
    r = np.random.default_rng(K)
    for parents in (r.integers(0, K, (B, K)), np.stack([r.permutation(K) for _ in range(B)]),
                    np.tile(np.arange(K), (B, 1)), np.full((B, K), K - 1), np.tile(np.roll(np.arange(K), 1), (B, 1))):
        par = torch.from_numpy(parents.astype(np.int32)).cuda()
        flat = (par.long() + torch.arange(B, device="cuda")[:, None] * K).reshape(-1)
        want = state[flat], tail[flat]
        st = torch.full((B,), -3, dtype=torch.int32, device="cuda")
        gdn.beam_reorder(d, state, tail, par, st)
        torch.cuda.synchronize()
        assert st.cpu().tolist() == [0] * B
        assert torch.equal(state, want[0]) and torch.equal(tail, want[1])


def test_reorder_leaves_a_bad_group_alone():
    import gated_deltanet_decode_amd as gdn
    d, state, tail = layer("ssm", 12)
    par = torch.tensor([[1, 0, 0, 3], [0, 4, 2, 2], [-1, 0, 0, 0]], dtype=torch.int32, device="cuda")
    s0, t0 = state.clone(), tail.clone()
    st = torch.full((3,), -3, dtype=torch.int32, device="cuda")
    gdn.beam_reorder(d, state, tail, par, st)
    gdn.beam_reorder(d, *[a.clone() for a in (state, tail)], par)            # no status word wanted
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0, 10, 10]
    assert torch.equal(state[4:], s0[4:]) and torch.equal(tail[4:], t0[4:])
    assert torch.equal(state[:4], s0[[1, 0, 0, 3]]) and torch.equal(tail[:4], t0[[1, 0, 0, 3]])


def test_reorder_refusals():
    import gated_deltanet_decode_amd as gdn
    d, state, tail = layer("ssm", 6)
    with pytest.raises(ValueError, match="parent"):
        gdn.beam_reorder(d, state, tail, torch.zeros(2, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="parent must be torch.int32"):
        gdn.beam_reorder(d, state, tail, torch.zeros(2, 3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="state"):
        gdn.beam_reorder(d, state[:5], tail, torch.zeros(2, 3, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ together

def test_beam_search_over_a_hybrid_stack():
    """A GDN layer and a selective state space layer under beam search: prompt, then steps of decode, selection
    and reordering, against beams that each replay their own tokens from the prompt."""
    import gated_deltanet_decode_amd as gdn
    B, K, V, T, steps = 2, 3, 97, 70, 5
    n = B * K
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    sd, gd = gdn.ssm_dims(n, 2, 1, 32, 64, 4, "f32"), gdn.dims(n, 1, 2, 32, 32, 4, "f32")
    sw, gw, A = rnd(sd.C, 4) * 0.5, rnd(gd.C, 4) * 0.5, -torch.rand(2, generator=g, device="cuda") * 4
    embed_s, embed_g, head = rnd(V, sd.C), rnd(V, gd.C), rnd(128, V)
    dts, ga, gb = rnd(V, 2), rnd(V, 2), rnd(V, 2)
    prompt = torch.randint(0, V, (B, 1, T), generator=g, device="cuda").expand(B, K, T).reshape(n, T)

    class Stack:
        def __init__(self, count):
            self.n = count
            self.sd, self.gd = gdn.ssm_dims(count, 2, 1, 32, 64, 4, "f32"), gdn.dims(count, 1, 2, 32, 32, 4, "f32")
            z = lambda *s: torch.zeros(*s, device="cuda")
            self.ss, self.st, self.so = z(count, 2, 32, 64), z(count, sd.C, 4), z(count, sd.C, 4)
            self.gs, self.gt, self.go = z(count, 2, 32, 32), z(count, gd.C, 4), z(count, gd.C, 4)
            self.ys, self.yg = z(count, 2, 32), z(count, 2, 32)

        def token(self, tok):
            tok = tok.reshape(-1).long()
            gdn.ssm_decode_token(self.sd, self.ss, self.st, self.so, sw, embed_s[tok], dts[tok], A, self.ys)
            self.st, self.so = self.so, self.st
            gdn.decode_token(self.gd, self.gs, self.gt, self.go, gw, embed_g[tok], ga[tok], gb[tok], self.yg)
            self.gt, self.go = self.go, self.gt
            return torch.cat([self.ys.reshape(self.n, -1), self.yg.reshape(self.n, -1)], 1) @ head * 0.3

    s = Stack(n)
    y = torch.empty(n, T, 2, 32, device="cuda")
    ws = torch.empty(gdn.ssm_prefill_workspace_bytes(sd, T - 1), dtype=torch.uint8, device="cuda")
    gdn.ssm_prefill(sd, s.ss, s.st, sw, embed_s[prompt[:, :-1]].contiguous(), dts[prompt[:, :-1]].contiguous(), A,
                    y[:, :T - 1].contiguous(), ws)
    for t in range(T - 1):
        tok = prompt[:, t]
        gdn.decode_token(gd, s.gs, s.gt, s.go, gw, embed_g[tok], ga[tok], gb[tok], s.yg)
        s.gt, s.go = s.go, s.gt
    logits = s.token(prompt[:, -1])
    scores = torch.full((B, K), -INF, device="cuda")
    scores[:, 0] = 0
    out, par, tok = (torch.zeros(B, K, device="cuda", dtype=d) for d in (torch.float32, torch.int32, torch.int32))
    wsel = torch.empty(gdn.beam_select_workspace_bytes(B, K, V, K), dtype=torch.uint8, device="cuda")
    history = torch.zeros(B, K, 0, dtype=torch.long, device="cuda")
    for _ in range(steps):
        gdn.beam_select(logits.view(B, K, V), scores, out, par, tok, wsel)
        gdn.beam_reorder(s.sd, s.ss, s.st, par)
        gdn.beam_reorder(s.gd, s.gs, s.gt, par)
        history = torch.cat([history.gather(1, par.long()[..., None].expand(-1, -1, history.shape[2])),
                             tok.long()[..., None]], 2)
        scores = out.clone()
        logits = s.token(tok)
    torch.cuda.synchronize()
    assert torch.isfinite(scores).all()
    # each surviving beam's tokens, replayed one by one from the empty state
    r = Stack(n)
    tokens = torch.cat([prompt, history.reshape(n, steps)], 1)
    total = torch.zeros(n, device="cuda", dtype=torch.float64)
    for t in range(T + steps):
        if t >= T:
            total += torch.log_softmax(lg.double(), -1).gather(1, tokens[:, t:t + 1])[:, 0]
        lg = r.token(tokens[:, t])
    torch.cuda.synchronize()
    rel = lambda a, b: float((a - b).abs().max() / b.abs().max())
    assert rel(s.ss, r.ss) < 2.1e-5                          # the prompt went through the prefill call
    assert torch.equal(s.gs, r.gs) and torch.equal(s.gt, r.gt) and torch.equal(s.st, r.st)
    # a logit is a 128-term product of outputs within 2.1e-5 of their largest, times 0.3 and weights of about one:
    # 0.3 * 128 * 4 * 2.1e-5 at most, per step
    assert float((scores.reshape(-1).double() - total).abs().max()) < steps * 2 * 0.3 * 128 * 4 * 2.1e-5
    best = scores.sort(dim=1, descending=True).values
    assert torch.equal(best, scores)
