"""GPU: the most sequences that a gradient takes, of channels that do not fill a wide
tile: one call over as many as a launch can count gives every sequence the bits that
it has in a call of three."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def grads(gdn, d, T, x, state, A, y, g, dA, dstate0):
    saved = torch.empty(gdn.lru_saved_bytes(d, T), dtype=torch.uint8, device="cuda")
    ws = torch.empty(max(gdn.lru_prefill_workspace_bytes(d, T), gdn.lru_backward_workspace_bytes(d, T)), dtype=torch.uint8,
                     device="cuda")
    gdn.lru_prefill(d, state, x, x, x, A, y, ws, saved=saved)
    gdn.lru_backward(d, x, x, x, A, x, saved, g[0], g[1], g[2], dA, ws, dstate0=dstate0)


# 4,194,306 sequences of one block of 64 channels, 2,097,153 of three: twice as many tiles
# of 32 tokens would be 2^23 workgroups of 512 threads and more
@pytest.mark.parametrize("B,W", [(3 * 1398102, 8), (3 * 699051, 136)])
def test_more_tiles_than_a_launch_counts(B, W):
    import gated_deltanet_decode_amd as gdn
    T, n = 33, B // 3
    r = torch.Generator(device="cuda").manual_seed(W)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=r)
    base, h0, A = rand(3, T, W).bfloat16(), rand(3, W), -torch.rand(W, device="cuda", generator=r)
    one = [torch.empty_like(base) for _ in range(4)]
    part, s1, d1 = torch.zeros(3, W, device="cuda"), h0.clone(), torch.empty(3, W, device="cuda")
    small = gdn.lru_dims(3, W)
    grads(gdn, small, T, base, s1, A, one[0], one[1:], torch.empty(W, device="cuda"), d1)
    for k in range(3):                                       # each sequence's own part of dA
        at = slice(k, k + 1)
        grads(gdn, gdn.lru_dims(1, W), T, base[at].contiguous(), h0[at].clone(), A, torch.empty_like(base[at]),
              [torch.empty_like(base[at]) for _ in range(3)], part[k], torch.empty(1, W, device="cuda"))
    torch.cuda.synchronize()
    print(f"B={B} W={W}: the large call", flush=True)
    x = torch.empty(B, T, W, dtype=torch.bfloat16, device="cuda")
    x.view(n, 3, T, W).copy_(base)
    state, dstate0, dA = torch.empty(B, W, device="cuda"), torch.empty(B, W, device="cuda"), torch.empty(W, device="cuda")
    state.view(n, 3, W).copy_(h0)
    all_ = [torch.empty_like(x) for _ in range(4)]
    grads(gdn, gdn.lru_dims(B, W), T, x, state, A, all_[0], all_[1:], dA, dstate0)
    torch.cuda.synchronize()
    for got, want in ((state, s1), (dstate0, d1), *zip(all_, one)):
        assert (got.view(n, 3, *want.shape[1:]) == want).all()
    # 16 lanes add every 16th of the tiles' parts one after the other, then the lanes; a sequence of 33
    # tokens has one or two parts, which round once more than their sum in a call of one sequence
    want, mag = part.double().sum(0) * n, part.double().abs().sum(0) * n
    print("dA", ((dA.double() - want).abs() / mag).max().item(), flush=True)
    assert ((dA.double() - want).abs() <= (B / 16 + 17 + 2) * U * mag).all()
    del x, all_
    torch.cuda.empty_cache()
