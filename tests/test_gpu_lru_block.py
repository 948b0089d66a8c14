"""GPU: the operators in a row, as a model uses them: a recurrent block behind its
norms, trained against a 64-bit plain form with automatic differentiation, and a
hybrid stack (delta rule, then gated linear recurrence) decoded token by token
against its own prompt.

The blocks run in fp32.  A product over 64 to 128 values rounds each output by at
most 128 u of its terms, the operators by less; over the three products and five
operators that a value passes, with sums about 8 times their results, errors stay
below 8 * 1000 u = 5e-4 of the largest value.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TOL = 5e-4


def worst(got, want):
    want = want.detach().double().cpu()
    return ((got.detach().double().cpu() - want).abs().max() / want.abs().max()).item()


class Block:
    """norm -> x, r, i, z by one product -> recurrence -> norm and gate -> product -> sum and norm."""

    def __init__(self, seed, B, T, W, H):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
        self.B, self.T, self.W, self.H, self.D = B, T, W, H, W // H
        self.p = dict(w1=1 + 0.1 * n(W), win=n(W, 5 * W) / W ** 0.5, A=-torch.rand(W, generator=g, dtype=torch.float64),
                      wg=1 + 0.1 * n(self.D), wout=n(W, W) / W ** 0.5, scale=1 + 0.1 * n(W), post=1 + 0.1 * n(W), w2=1 + 0.1 * n(W))
        self.s, self.state, self.c, self.cs = n(B, T, W), n(B, W), n(B, T, W), n(B, T, W)

    def plain(self, lengths):
        """(y, stream, state, gradients) in 64 bits on the host."""
        p = {k: v.clone().requires_grad_(True) for k, v in self.p.items()}
        s, h0 = self.s.clone().requires_grad_(True), self.state.clone().requires_grad_(True)
        rms = lambda v: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)
        q = rms(s) * p["w1"] @ p["win"]
        x, r, i, z, gate = q.split(self.W, -1)
        la = torch.clamp(p["A"], max=0) * torch.sigmoid(r)
        a, v = torch.exp(la), torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i) * x
        rows, ends = [], []
        for b in range(self.B):
            h, path = h0[b], []
            for t in range(self.T):
                if t < lengths[b]:
                    h = a[b, t] * h + v[b, t]
                path.append(h * (z[b, t] * torch.sigmoid(z[b, t])) if t < lengths[b] else torch.zeros_like(h))
            rows.append(torch.stack(path))
            ends.append(h)
        o = torch.stack(rows).unflatten(-1, (self.H, self.D))
        gate = gate.unflatten(-1, (self.H, self.D))
        m = (rms(o) * p["wg"] * gate * torch.sigmoid(gate)).flatten(-2) @ p["wout"]
        out = s + p["scale"] * (rms(m) * p["post"])
        y = rms(out) * p["w2"]
        ((y * self.c).sum() + (out * self.cs).sum()).backward()
        return y, out, torch.stack(ends), {**{k: v.grad for k, v in p.items()}, "s": s.grad, "state": h0.grad}

    def run(self, lengths):
        import gated_deltanet_decode_amd as gdn
        B, T, W, H, D = self.B, self.T, self.W, self.H, self.D
        dev = lambda t: t.float().cuda()
        p, s, state = {k: dev(v) for k, v in self.p.items()}, dev(self.s), dev(self.state)
        new = lambda *sh: torch.zeros(*sh, device="cuda")
        ws = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        d, ln = gdn.lru_dims(B, W, "f32"), torch.tensor(lengths, dtype=torch.int32, device="cuda")
        n1 = new(B, T, W)
        gdn.residual_norm(s, None, p["w1"], None, n1)
        q = n1 @ p["win"]
        x, r, i, z, gate = q.split(W, -1)              # slices of one product's rows, used as they are
        o, saved, hT = new(B, T, W), ws(gdn.lru_saved_bytes(d, T)), state.clone()
        w = ws(max(gdn.lru_prefill_workspace_bytes(d, T), gdn.lru_backward_workspace_bytes(d, T)))
        gdn.lru_prefill(d, hT, x, r, i, p["A"], o, w, z=z, lengths=ln, saved=saved)
        heads = lambda t: t.reshape(B * T, W).unflatten(1, (H, D)) if t.is_contiguous() else t.flatten(0, 1).unflatten(1, (H, D))
        gn = new(B * T, H, D)
        gdn.gated_norm(heads(o), heads(gate), p["wg"], gn)
        m = gn.view(B, T, W) @ p["wout"]
        out, y = new(B, T, W), new(B, T, W)
        gdn.residual_norm(s, m, p["w2"], out, y, scale=p["scale"], w_post=p["post"])
        # and back
        g = {k: torch.zeros_like(v) for k, v in p.items()}
        dm, ds, dc = new(B, T, W), dev(self.cs), dev(self.c)
        wn = ws(max(gdn.residual_norm_backward_workspace_bytes(B * T, W), gdn.gated_norm_backward_workspace_bytes(B * T, H, D)))
        gdn.residual_norm_backward(out, m, p["w2"], dc, ds, dm, g["w2"], wn, ds=ds, scale=p["scale"], w_post=p["post"],
                                   dscale=g["scale"], dw_post=g["post"])
        g["wout"] = gn.view(B * T, W).t() @ dm.view(B * T, W)
        dgn, do, dq = (dm.view(B * T, W) @ p["wout"].t()).view(B * T, H, D), new(B * T, H, D), new(B, T, 5 * W)
        dx, dr, di, dz, dgate = dq.split(W, -1)
        gdn.gated_norm_backward(heads(o), heads(gate), p["wg"], dgn, do, heads(dgate), g["wg"], wn)
        dstate = new(B, W)
        gdn.lru_backward(d, x, r, i, p["A"], do.view(B, T, W), saved, dx, dr, di, g["A"], w, z=z, dz=dz, dstate0=dstate, lengths=ln)
        g["win"] = n1.view(B * T, W).t() @ dq.view(B * T, 5 * W)
        dn1 = dq @ p["win"].t()
        gdn.residual_norm_backward(s, None, p["w1"], dn1, ds, None, g["w1"], wn, ds=ds)
        torch.cuda.synchronize()
        return y, out, hT, {**g, "s": ds, "state": dstate}


@pytest.mark.parametrize("lengths", [[70, 70], [33, 0], [1, 70]])
def test_a_block_trains_as_its_formulas(lengths):
    b = Block(1, 2, 70, 64, 4)
    want, got = b.plain(lengths), b.run(lengths)
    for name, a, c in zip(("y", "stream", "state"), got, want):
        assert worst(a, c) < TOL, name
    for k, c in want[3].items():
        assert worst(got[3][k], c) < TOL, k


def test_a_hybrid_stack_decodes_as_its_prompt():
    """A delta-rule layer (4 heads of 32), its gated norm, a product, the residual norm, and a recurrent
    layer: 20 tokens one by one; the norms' and the recurrence's part also over the whole prompt."""
    import gated_deltanet_decode_amd as gdn
    B, T, W = 3, 20, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    d, dl = gdn.dims(B, 4, 4, 32, 32, 4, "f32"), gdn.lru_dims(B, W, "f32")
    S, w = n(B, 4, 32, 32) * 0.1, n(d.C, 4) * 0.5
    tails = [n(B, d.C, 4), torch.empty(B, d.C, 4, device="cuda")]
    xs, a, b = n(T, B, d.C), n(T, B, 4), n(T, B, 4)
    zs, wg, wo = n(T, B, 4, 32), 1 + 0.1 * n(32), n(W, W) / W ** 0.5
    wr, wp, A = 1 + 0.1 * n(W), n(W, 4 * W) / W ** 0.5, -torch.rand(W, device="cuda", generator=g)
    res, h = n(T, B, W), n(B, W)
    h0 = h.clone()
    new = lambda *s: torch.empty(*s, device="cuda")
    os_, ys, outs = new(T, B, 4, 32), new(T, B, W), new(T, B, W)
    for t in range(T):
        gdn.decode_token(d, S, tails[t % 2], tails[1 - t % 2], w, xs[t], a[t], b[t], os_[t])
        gn, out, nx = new(B, 4, 32), new(B, W), new(B, W)
        gdn.gated_norm(os_[t], zs[t], wg, gn)
        gdn.residual_norm(res[t], gn.view(B, W) @ wo, wr, out, nx)
        q = nx @ wp
        x, r, i, z = q.split(W, -1)
        gdn.lru_decode_token(dl, h, x, r, i, A, ys[t], z=z)
        outs[t] = out
    # the same norms and recurrence over the prompt, sequences first
    o = os_.transpose(0, 1).contiguous().view(B * T, 4, 32)
    gn, out, nx = new(B * T, 4, 32), new(B * T, W), new(B * T, W)
    gdn.gated_norm(o, zs.transpose(0, 1).contiguous().view(B * T, 4, 32), wg, gn)
    gdn.residual_norm(res.transpose(0, 1).contiguous().view(B * T, W), gn.view(B * T, W) @ wo, wr, out, nx)
    x, r, i, z = (nx @ wp).view(B, T, 4 * W).split(W, -1)
    y, hp = new(B, T, W), h0.clone()
    gdn.lru_prefill(dl, hp, x, r, i, A, y, None, z=z)
    torch.cuda.synchronize()
    assert worst(out.view(B, T, W), outs.transpose(0, 1)) < TOL
    assert worst(y, ys.transpose(0, 1)) < TOL and worst(hp, h) < TOL
    assert np.isfinite(y.cpu().numpy()).all()
