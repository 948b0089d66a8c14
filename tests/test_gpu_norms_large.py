"""GPU: the norms at the ends of their sizes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


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
