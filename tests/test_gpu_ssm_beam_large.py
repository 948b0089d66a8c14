"""GPU: the state space and beam search calls where offsets pass 32 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
GB = 1 << 30
U = 2.0 ** -24


def room(n):
    if torch.cuda.mem_get_info()[0] < n * GB:
        pytest.skip(f"needs {n} GB of device memory")


def test_a_prompt_beyond_32_bits():
    """600,000 tokens at once against the same in two calls: x and y hold more than 2^31 elements."""
    import gated_deltanet_decode_amd as gdn
    room(40)
    T, cut, H = 600_000, 590_011, 64
    d = gdn.ssm_dims(1, H, 1, 64, 64, 4, "bf16")
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(T, d.C, device="cuda", dtype=torch.bfloat16)
    for t in range(0, T, 50_000):
        x[t:t + 50_000] = torch.randn(50_000, d.C, device="cuda", generator=g).to(torch.bfloat16)
    assert x.numel() > 1 << 31
    dt = torch.randn(T, H, device="cuda", generator=g) - 3
    A = -1 - 8 * torch.rand(H, device="cuda", generator=g)
    w = (torch.randn(d.C, 4, device="cuda", generator=g) * 0.5).to(torch.bfloat16)
    ws = torch.empty(gdn.ssm_prefill_workspace_bytes(d, T), dtype=torch.uint8, device="cuda")
    zeros = lambda: (torch.zeros(1, H, 64, 64, device="cuda"), torch.zeros(1, d.C, 4, device="cuda", dtype=torch.bfloat16))
    S, tail = zeros()
    y = torch.empty(T, H, 64, device="cuda", dtype=torch.bfloat16)
    gdn.ssm_prefill(d, S, tail, w, x, dt, A, y, ws)
    S2, tail2 = zeros()
    rest = x[cut:].clone()
    y2 = torch.empty(T - cut, H, 64, device="cuda", dtype=torch.bfloat16)
    # the state that enters the second part depends on the last few thousand tokens before it only
    back = 6_000
    head = torch.empty(back, H, 64, device="cuda", dtype=torch.bfloat16)
    gdn.ssm_prefill(d, S2, tail2, w, x[cut - back:cut].clone(), dt[cut - back:cut].clone(), A, head, ws)
    gdn.ssm_prefill(d, S2, tail2, w, rest, dt[cut:].clone(), A, y2, ws)
    torch.cuda.synchronize()
    assert torch.equal(tail, tail2)
    rel = lambda a, b: float((a.float() - b.float()).abs().max() / b.float().abs().max())
    # each within 352 u of the exact state, and each output within 2^-8 + 2^-9 of it (as in test_gpu_ssm)
    assert rel(S, S2) < 2 * 352 * U
    assert rel(y[cut:], y2) < 2 * (2.0 ** -8 + 2.0 ** -9)
    assert rel(y[cut - 64:cut], head[-64:]) < 2 * (2.0 ** -8 + 2.0 ** -9)


def test_states_beyond_32_bits():
    """2,200 sequences of 4 MB: the last ones' token and move are those of a small batch."""
    import gated_deltanet_decode_amd as gdn
    room(24)
    B, K = 2200, 4
    mk = lambda b: gdn.ssm_dims(b, 64, 1, 128, 128, 4, "bf16")
    d, few = mk(B), mk(2 * K)
    g = torch.Generator(device="cuda").manual_seed(6)
    S = torch.empty(B, 64, 128, 128, device="cuda")
    assert S.numel() > 1 << 31
    for s in range(0, B, 100):
        S[s:s + 100] = torch.randn(100, 64, 128, 128, device="cuda", generator=g)
    bf = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
    tail, w, x = bf(B, d.C, 4), bf(d.C, 4), bf(B, d.C)
    dt, A = torch.randn(B, 64, device="cuda", generator=g) - 3, -torch.rand(64, device="cuda", generator=g)
    ends = torch.cat([torch.arange(K), torch.arange(B - K, B)]).cuda()
    S2, tail2 = S[ends].clone(), tail[ends].clone()
    out, out2 = torch.empty_like(tail), torch.empty_like(tail2)
    y, y2 = bf(B, 64, 128), bf(2 * K, 64, 128)
    gdn.ssm_decode_token(d, S, tail, out, w, x, dt, A, y)
    parent = torch.randint(0, K, (B // K, K), device="cuda", generator=g, dtype=torch.int32)
    gdn.beam_reorder(d, S, out, parent)
    for s in range(2 * K):   # one by one: few enough heads take narrower workgroups, the same arithmetic
        one = mk(1)
        o = torch.empty_like(tail2[s])
        gdn.ssm_decode_token(one, S2[s], tail2[s].clone(), o, w, x[ends[s]].clone(), dt[ends[s]].clone(), A, y2[s])
        out2[s] = o
    par2 = torch.cat([parent[:1], parent[-1:]])
    gdn.beam_reorder(few, S2, out2, par2)
    torch.cuda.synchronize()
    assert torch.equal(S[ends], S2) and torch.equal(out[ends], out2) and torch.equal(y[ends], y2)


def test_logits_beyond_32_bits():
    import gated_deltanet_decode_amd as gdn
    room(12)
    B, K, V, pitch = 64, 8, 1003, (1 << 23) + 5
    wide = torch.empty(B, K, pitch, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn(B, K, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)).to(torch.bfloat16)
    wide[..., :V] = logits
    scores = -torch.arange(B * K, device="cuda", dtype=torch.float32).view(B, K) / 64
    ws = torch.empty(gdn.beam_select_workspace_bytes(B, K, V, 8), dtype=torch.uint8, device="cuda")
    got = []
    for t in (wide[..., :V], logits):
        o = (torch.empty(B, 8, device="cuda"), *(torch.empty(B, 8, dtype=torch.int32, device="cuda") for _ in range(2)))
        gdn.beam_select(t, scores, *o, ws)
        got.append(o)
    torch.cuda.synchronize()
    assert torch.equal(got[0][1], got[1][1]) and torch.equal(got[0][2], got[1][2])
    # The rows start at other places within 16 bytes, so a row's fp32 sums are split over the lanes in another way:
    # each result is within 2^-18 plus 2^-23 of its size of the exact one (a sum of exponentials of |l| < 8 whose
    # terms are each within 2 u |l| + u and whose lane sums take at most log2 of the terms per lane in steps of u,
    # below 32 u = 2^-19 of the sum and so of its logarithm, and the output's rounding), and they are within twice that.
    a, b = got[0][0], got[1][0]
    assert ((a - b).abs() <= 2 * (2.0 ** -18 + 2.0 ** -23 * b.abs())).all()
