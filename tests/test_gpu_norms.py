"""GPU: the residual norm and the gated norm, and their gradients, against the
64-bit reference, each value held to the bound that the reference gives for its
own terms (half steps of fp32 along the sums, and of the output's type)."""
import numpy as np
import pytest
import torch

from tests import lru_reference as lr
from tests.test_gpu_lru import dev, near

pytestmark = pytest.mark.gpu
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]      # activations, stream (or mixer output)


def arr(r, bf16, *shape, scale=1.0):
    a = r.standard_normal(shape) * scale
    return lr.bf16_round(a) if bf16 else a.astype(np.float32)


def rounded(want, tol, bf16):
    return want, lr.stored(want, tol, bf16)


class Residual:
    def __init__(self, seed, rows, W, act, res, scale=True, post=True, delta=True, ds=True, size=1.0):
        import gated_deltanet_decode_amd as gdn
        self.gdn, self.a16, self.r16 = gdn, act == "bf16", res == "bf16"
        r = np.random.default_rng(seed)
        self.n = n = dict(residual=arr(r, self.r16, rows, W, scale=2 * size), delta=arr(r, self.a16, rows, W, scale=size) if delta else None,
                          dy=arr(r, self.a16, rows, W), ds=arr(r, self.r16, rows, W) if ds else None,
                          w=arr(r, False, W) + 1, scale=arr(r, False, W) if scale and delta else None,
                          post=arr(r, False, W) + 1 if post and delta else None)
        kind = dict(residual=self.r16, delta=self.a16, dy=self.a16, ds=self.r16)
        self.t = {k: dev(v, kind.get(k, False)) for k, v in n.items()}
        new = lambda b: torch.full((rows, W), 7.0, device="cuda", dtype=torch.bfloat16 if b else torch.float32)
        self.out = new(self.r16) if delta else None
        self.y, self.dres, self.ddelta = new(self.a16), new(self.r16), new(self.a16) if delta else None
        col = lambda on: torch.full((W,), 7.0, device="cuda") if on is not None else None
        self.dw, self.dscale, self.dpost = col(0), col(n["scale"]), col(n["post"])
        self.rows, self.W = rows, W

    def forward(self, out=None):
        t = self.t
        self.gdn.residual_norm(t["residual"], t["delta"], t["w"], self.out if out is None else out, self.y, scale=t["scale"],
                               w_post=t["post"])

    def backward(self, dres=None):
        t = self.t
        ws = torch.full((self.gdn.residual_norm_backward_workspace_bytes(self.rows, self.W),), 0xA5, dtype=torch.uint8, device="cuda")
        stream = t["residual"] if self.out is None else self.out
        self.gdn.residual_norm_backward(stream, t["delta"], t["w"], t["dy"], self.dres if dres is None else dres, self.ddelta, self.dw,
                                        ws, ds=t["ds"], scale=t["scale"], w_post=t["post"], dscale=self.dscale, dw_post=self.dpost)

    def check(self):
        torch.cuda.synchronize()
        n = self.n
        want, tol = lr.residual_norm(n["residual"], n["delta"], n["w"], n["scale"], n["post"])
        stream = want
        if self.out is not None:
            near(self.out, *rounded(want, tol, self.r16), "out")
            stream = self.out.float().cpu().numpy()            # y is the norm of the stream as it is stored
        near(self.y, *rounded(*lr.norm_of(stream, n["w"]), self.a16), "y")
        self.stream = stream

    def check_grads(self):
        torch.cuda.synchronize()
        n = self.n
        want, tol = lr.residual_norm_grad(self.stream, n["delta"], n["w"], n["dy"], n["ds"], n["scale"], n["post"])
        got = dict(dresidual=(self.dres, self.r16), ddelta=(self.ddelta, self.a16), dw=(self.dw, False),
                   dscale=(self.dscale, False), dw_post=(self.dpost, False))
        for k in want:
            near(got[k][0], *rounded(want[k], tol[k], got[k][1]), k)


WIDTHS = [8, 16, 24, 64, 104, 128, 256, 264, 512, 520, 1000, 1024, 2048, 4096, 5120, 8200, 16384]


@pytest.mark.parametrize("W", WIDTHS)
@pytest.mark.parametrize("act,res", TYPES)
def test_residual_norm(W, act, res):
    m = Residual(W, 5, W, act, res, scale=W % 3 != 0, post=W % 16 == 0)
    m.forward()
    m.check()
    m.backward()
    m.check_grads()


@pytest.mark.parametrize("rows", [1, 2, 3, 511, 512, 513, 1500])
@pytest.mark.parametrize("W", [40, 1096])
def test_rows(rows, W):
    """Around the number of workgroups that share the weights' sums, and beyond it."""
    m = Residual(rows, rows, W, "bf16", "f32")
    m.forward()
    m.check()
    m.backward()
    m.check_grads()


@pytest.mark.parametrize("W", [48, 2048])
@pytest.mark.parametrize("scale,post,delta,ds", [(False, False, True, False), (True, False, True, True), (False, True, True, False),
                                                 (False, False, False, True), (False, False, False, False)])
@pytest.mark.parametrize("act,res", TYPES)
def test_optional_operands(W, scale, post, delta, ds, act, res):
    m = Residual(3, 9, W, act, res, scale, post, delta, ds)
    m.forward()
    m.check()
    m.backward()
    m.check_grads()


@pytest.mark.parametrize("act,res", TYPES)
def test_in_place(act, res):
    """The stream may be replaced, and its gradient too: the same bits."""
    a, b = Residual(4, 70, 136, act, res), Residual(4, 70, 136, act, res)
    a.forward()
    a.backward()
    b.forward(out=b.t["residual"])
    b.out = b.t["residual"]
    b.backward(dres=b.t["ds"])
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.y, b.y) and torch.equal(a.dres, b.t["ds"])
    for k in ("ddelta", "dw", "dscale", "dpost"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k


@pytest.mark.parametrize("size", [1e-12, 1e-3, 1e8])
def test_magnitudes(size):
    """Rows far below eps and rows of large values."""
    m = Residual(5, 6, 128, "f32", "f32", size=size, ds=False)
    m.forward()
    m.check()
    m.backward()
    m.check_grads()


def test_rows_of_zeros():
    m = Residual(6, 3, 64, "bf16", "bf16")
    for k in ("residual", "delta"):
        m.n[k][1] = 0
        m.t[k][1] = 0
    m.forward()
    m.check()
    m.backward()
    m.check_grads()
    assert (m.y[1] == 0).all()


class Gated:
    def __init__(self, seed, rows, H, D, act, o, first, each, pitch=0):
        import gated_deltanet_decode_amd as gdn
        self.gdn, self.a16, self.o16, self.first, self.each = gdn, act == "bf16", o == "bf16", first, each
        r = np.random.default_rng(seed)
        self.n = dict(o=arr(r, self.o16, rows, H, D, scale=0.5), z=arr(r, self.a16, rows, H, D), dy=arr(r, self.a16, rows, H, D),
                      w=arr(r, False, H, D) + 1 if each else arr(r, False, D) + 1)
        kind = dict(o=self.o16, z=self.a16, dy=self.a16, w=False)
        self.t = {k: dev(v, kind[k]) for k, v in self.n.items()}
        new = lambda b, n=H * D: torch.full((rows, n), 7.0, device="cuda", dtype=torch.bfloat16 if b else torch.float32)
        self.y, self.do = new(self.a16).view(rows, H, D), new(self.o16).view(rows, H, D)
        self.wide = [new(self.a16, H * D + pitch), new(self.a16, H * D + pitch)]
        part = [w[:, pitch:].unflatten(1, (H, D)) for w in self.wide]
        part[0].copy_(self.t["z"])
        self.t["z"], self.dz = part
        self.pitch = pitch
        self.dw = torch.full_like(self.t["w"], 7.0)
        self.rows, self.H, self.D = rows, H, D

    def run(self):
        t = self.t
        self.gdn.gated_norm(t["o"], t["z"], t["w"], self.y, gate_first=self.first)
        ws = torch.full((self.gdn.gated_norm_backward_workspace_bytes(self.rows, self.H, self.D),), 0xA5, dtype=torch.uint8, device="cuda")
        self.gdn.gated_norm_backward(t["o"], t["z"], t["w"], t["dy"], self.do, self.dz, self.dw, ws, gate_first=self.first)

    def check(self):
        torch.cuda.synchronize()
        n = self.n
        near(self.y, *rounded(*lr.gated_norm(n["o"], n["z"], n["w"], self.first), self.a16), "y")
        want, tol = lr.gated_norm_grad(n["o"], n["z"], n["w"], n["dy"], self.first, shared=not self.each)
        for k, got, b in (("do", self.do, self.o16), ("dz", self.dz, self.a16), ("dw", self.dw, False)):
            near(got, *rounded(want[k], tol[k], b), k)
        if self.pitch:
            assert (self.wide[1][:, :self.pitch].float() == 7.0).all()


@pytest.mark.parametrize("D", [8, 16, 32, 40, 64, 96, 128, 256, 264, 512, 520, 1024, 4096, 6000, 16384])
@pytest.mark.parametrize("act,o", TYPES)
@pytest.mark.parametrize("first", [True, False])
def test_gated_norm(D, act, o, first):
    H = 1 if D > 4000 else 3
    m = Gated(D, 5, H, D, act, o, first, each=D % 3 == 0, pitch=8 * (D % 5))
    m.run()
    m.check()


@pytest.mark.parametrize("each", [True, False])
@pytest.mark.parametrize("rows,H,D", [(1, 1, 128), (1, 48, 128), (3, 7, 64), (700, 48, 32), (1500, 2, 520), (90, 300, 16), (2, 9000, 8),
                                      (2, 600, 520)])
def test_rows_and_heads(rows, H, D, each):
    """Fewer and more heads and rows than teams that share the weights' sums."""
    m = Gated(rows + H, rows, H, D, "bf16", "f32", False, each, pitch=16)
    m.run()
    m.check()


@pytest.mark.parametrize("first", [True, False])
def test_extreme_gates(first):
    m = Gated(9, 4, 3, 64, "f32", "f32", first, False)
    z = np.random.default_rng(1).choice([-120.0, -30.0, 0.0, 40.0, 120.0], m.n["z"].shape).astype(np.float32)
    m.n["z"] = z
    m.t["z"].copy_(dev(z))
    m.run()
    m.check()


def test_norms_on_another_stream_and_captured():
    a, b = Residual(11, 300, 1096, "bf16", "f32"), Gated(12, 300, 5, 96, "bf16", "f32", False, True)
    ws = torch.empty(max(a.gdn.residual_norm_backward_workspace_bytes(300, 1096), a.gdn.gated_norm_backward_workspace_bytes(300, 5, 96)),
                     dtype=torch.uint8, device="cuda")

    def all_calls():
        a.forward()
        t = a.t
        a.gdn.residual_norm_backward(a.out, t["delta"], t["w"], t["dy"], a.dres, a.ddelta, a.dw, ws, ds=t["ds"], scale=t["scale"],
                                     w_post=t["post"], dscale=a.dscale, dw_post=a.dpost)
        t = b.t
        b.gdn.gated_norm(t["o"], t["z"], t["w"], b.y)
        b.gdn.gated_norm_backward(t["o"], t["z"], t["w"], t["dy"], b.do, b.dz, b.dw, ws)
    outs = [a.out, a.y, a.dres, a.ddelta, a.dw, a.dscale, a.dpost, b.y, b.do, b.dz, b.dw]
    all_calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for t in outs:
            t.zero_()
        all_calls()
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        all_calls()
    for _ in range(3):
        for t in outs:
            t.zero_()
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_elements_beyond_32_bits():
    """More than 2^31 elements and 2^32 bytes: the last rows of a stream, of heads and of a gate at a pitch."""
    import gated_deltanet_decode_amd as gdn
    rows, W = 131200, 16384
    r = np.random.default_rng(13)
    res = torch.empty(rows, W, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    y, w = torch.empty_like(res), dev(arr(r, False, W) + 1)
    last = arr(r, True, 1, W)
    res[-1:] = dev(last, True)
    gdn.residual_norm(res, None, w, None, y)
    near(y[-1:], *rounded(*lr.norm_of(last, w.cpu().numpy()), True), "last row")
    one = lr.norm_of(np.ones((1, W)), w.cpu().numpy())
    near(y[:1], *rounded(*one, True), "first row")
    o, z, wh = res.view(rows, 128, 128), y.view(rows, 128, 128), dev(arr(r, False, 128) + 1)
    out = torch.empty_like(o)
    n = (last.reshape(1, 128, 128), y[-1:].float().cpu().numpy().reshape(1, 128, 128), wh.cpu().numpy())
    gdn.gated_norm(o, z, wh, out)
    near(out[-1:], *rounded(*lr.gated_norm(*n), True), "last heads")


@pytest.mark.parametrize("W", [4104, 5120, 8200])
def test_many_wide_rows(W):
    """bf16 rows of more than 512 units of 8, enough of them that a lane takes two units."""
    m = Residual(21, 1030, W, "bf16", "bf16")
    m.forward()
    m.check()
    g = Gated(22, 520, 2, W, "bf16", "bf16", W == 5120, False, pitch=8)
    g.run()
    g.check()
