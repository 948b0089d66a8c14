"""GPU: the norms at the ends of their sizes."""
import pytest
import torch

from tests import lru_reference as lr
from tests.test_gpu_norms import Gated, Residual

pytestmark = pytest.mark.gpu
KINDS, TIMES = 41, 3200      # 131,200 rows of 16,384 values: 2^31 elements and 2^32 bytes of bf16 and more


def same(got, want, what):
    assert (got.view(TIMES, *want.shape) == want).all(), what


def sums_near(got, small, mag, what):
    """A weight's gradient over TIMES as many rows: off by a half step of its terms for each of some 131,200 / 256
    rows that a workgroup adds and 16 parts of 256 that a lane adds, and by the small call's own error."""
    off = (got.double() - TIMES * small.double()).abs()
    assert (off <= (131200 / 256 + 16 + 16 + 200) * lr.U * TIMES * mag.double().abs()).all(), what


def test_residual_norm_beyond_32_bits():
    """Stream, block output and every gradient: rows far into each array are those of a call of 41 rows, bit for bit."""
    import gated_deltanet_decode_amd as gdn
    W = 16384
    m = Residual(3, KINDS, W, "bf16", "f32")
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    t = {k: v.repeat(TIMES, 1) for k, v in m.t.items() if v.dim() == 2}
    out, dres = torch.empty_like(t["residual"]), torch.empty_like(t["residual"])
    y, ddelta = torch.empty_like(t["delta"]), torch.empty_like(t["delta"])
    dw, dscale, dpost = (torch.full((W,), 7.0, device="cuda") for _ in range(3))
    ws = torch.empty(gdn.residual_norm_backward_workspace_bytes(KINDS * TIMES, W), dtype=torch.uint8, device="cuda")
    gdn.residual_norm(t["residual"], t["delta"], m.t["w"], out, y, scale=m.t["scale"], w_post=m.t["post"])
    gdn.residual_norm_backward(out, t["delta"], m.t["w"], t["dy"], dres, ddelta, dw, ws, ds=t["ds"], scale=m.t["scale"],
                               w_post=m.t["post"], dscale=dscale, dw_post=dpost)
    torch.cuda.synchronize()
    for got, want, what in ((out, m.out, "out"), (y, m.y, "y"), (dres, m.dres, "dresidual"), (ddelta, m.ddelta, "ddelta")):
        same(got, want, what)
    # the sums' terms by magnitude: |dy y / w| for dw, and the same of the other two
    q = 1 / torch.sqrt((m.out * m.out).mean(-1, keepdim=True) + 1e-6)
    d = m.t["delta"].float()
    dn = d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-6)
    sums_near(dw, m.dw, (m.t["dy"].float() * m.out * q).abs().sum(0), "dw")
    sums_near(dscale, m.dscale, (m.dres * dn * m.t["post"]).abs().sum(0), "dscale")
    sums_near(dpost, m.dpost, (m.dres * m.t["scale"] * dn).abs().sum(0), "dw_post")
    del t, out, dres, y, ddelta
    torch.cuda.empty_cache()


@pytest.mark.parametrize("first", [True, False])
def test_gated_norm_beyond_32_bits(first):
    import gated_deltanet_decode_amd as gdn
    H, D = 128, 128
    m = Gated(4, KINDS, H, D, "bf16", "f32", first, False)
    m.run()
    torch.cuda.synchronize()
    wide = torch.zeros(KINDS * TIMES, 2 * H * D, dtype=torch.bfloat16, device="cuda")      # z behind others in wider rows, and dz
    z, grad = (w[:, H * D:].unflatten(1, (H, D)) for w in (wide, torch.zeros_like(wide)))
    z.view(TIMES, KINDS, H, D).copy_(m.t["z"])
    o, dy = m.t["o"].repeat(TIMES, 1, 1), m.t["dy"].repeat(TIMES, 1, 1)
    y, do, dw = torch.empty_like(dy), torch.empty_like(o), torch.full_like(m.t["w"], 7.0)
    ws = torch.empty(gdn.gated_norm_backward_workspace_bytes(KINDS * TIMES, H, D), dtype=torch.uint8, device="cuda")
    gdn.gated_norm(o, z, m.t["w"], y, gate_first=first)
    gdn.gated_norm_backward(o, z, m.t["w"], dy, do, grad, dw, ws, gate_first=first)
    torch.cuda.synchronize()
    for got, want, what in ((y, m.y, "y"), (do, m.do, "do"), (grad, m.dz, "dz")):
        same(got, want, what)
    zf = m.t["z"].float()
    gate = zf * torch.sigmoid(zf)
    u = m.t["o"] * gate if first else m.t["o"]
    n = u / torch.sqrt((u * u).mean(-1, keepdim=True) + 1e-6)
    mag = (m.t["dy"].float() * (1 if first else gate) * n).abs().sum((0, 1))
    # 768 workgroups of 8 teams walk 131,200 x 128 heads: some 2,734 rows each, then 8 teams and 48 parts a lane
    off = (dw.double() - TIMES * m.dw.double()).abs()
    assert (off <= (2734 + 8 + 48 + 16 + 200) * lr.U * TIMES * mag.double()).all()
    del wide, z, grad, o, dy, y, do
    torch.cuda.empty_cache()


def test_a_weight_for_each_of_many_wide_heads():
    """65,536 heads of 4,104, each with a weight of its own: more columns of weight gradients than a launch of one
    workgroup per 64 could count.  Heads of equal inputs have equal bits, those of a call of 16 heads."""
    import gated_deltanet_decode_amd as gdn
    H, D, n = 65536, 4104, 16
    r = torch.Generator(device="cuda").manual_seed(1)
    base = {k: torch.randn(1, n, D, device="cuda", generator=r).bfloat16() for k in ("o", "z", "dy")}
    w = 1 + 0.2 * torch.randn(n, D, device="cuda", generator=r)

    def run(t, w):
        rows, h, _ = t["o"].shape
        out = dict(y=torch.empty_like(t["o"]), do=torch.empty_like(t["o"]), dz=torch.empty_like(t["o"]), dw=torch.full_like(w, 7.0))
        ws = torch.empty(gdn.gated_norm_backward_workspace_bytes(rows, h, D), dtype=torch.uint8, device="cuda")
        gdn.gated_norm(t["o"], t["z"], w, out["y"])
        gdn.gated_norm_backward(t["o"], t["z"], w, t["dy"], out["do"], out["dz"], out["dw"], ws)
        torch.cuda.synchronize()
        return out
    want = run(base, w)
    wide = {k: v.repeat(1, H // n, 1) for k, v in base.items()}
    got = run(wide, w.repeat(H // n, 1))
    for k in ("y", "do", "dz"):
        assert (got[k].view(H // n, n, D) == want[k]).all(), k
    assert (got["dw"].view(H // n, n, D) == want["dw"]).all()
    del wide, got
    torch.cuda.empty_cache()
