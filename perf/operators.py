"""Cases of the selective state space mixer and of beam search over recurrent
states: what is measured, the operators' plain forms, and their definition in
64 bits.

`own` False computes a case with elementary torch operations; `own` True makes
the library's calls.  An SSM layer's channels are x | B | C (H*P + 2*G*N); its
state is fp32 [B][H][P][N].
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 64
_workspace = None      # one per process, grown to the largest call, as a serving loop keeps it


def _act(case):
    return torch.bfloat16 if case["act"] == "bf16" else torch.float32


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one short chat turn through a small layer: launch latency counts
        dict(name="ssm_prefill_short", op="ssm_prefill", B=1, T=77, H=16, P=64, N=64, G=1, act="bf16", ragged=False, gate=False),
        # one long document through a 64-head layer with one B/C group
        dict(name="ssm_prefill_32k", op="ssm_prefill", B=1, T=32768, H=64, P=64, N=128, G=1, act="bf16", ragged=False, gate=False),
        # a padded batch of prompts of different lengths, heads of the 27B-class layer's width, gated output
        dict(name="ssm_prefill_ragged", op="ssm_prefill", B=8, T=2048, H=48, P=128, N=128, G=16, act="bf16", ragged=True, gate=True),
        # fp32 activations, odd length
        dict(name="ssm_prefill_f32", op="ssm_prefill", B=2, T=1003, H=32, P=64, N=128, G=8, act="f32", ragged=False, gate=True),
        # one decoded token, single stream: latency
        dict(name="ssm_token_b1", op="ssm_token", B=1, H=48, P=128, N=128, G=16, act="bf16", gate=True),
        # one decoded token for a full serving batch: the states stream from HBM
        dict(name="ssm_token_b64", op="ssm_token", B=64, H=48, P=128, N=128, G=16, act="bf16", gate=True),
        # odd batch, narrow heads with a wide state, fp32
        dict(name="ssm_token_f32", op="ssm_token", B=5, H=33, P=32, N=256, G=3, act="f32", gate=False),
        # one request with four beams
        dict(name="beam_select_b1", op="beam_select", B=1, K=4, V=32000, S=4, act="bf16", finished=False),
        # a serving batch, twice as many candidates as beams, some beams finished
        dict(name="beam_select_b64", op="beam_select", B=64, K=8, V=128000, S=16, act="bf16", finished=True),
        # odd vocabulary, fp32 logits
        dict(name="beam_select_f32", op="beam_select", B=7, K=5, V=50021, S=10, act="f32", finished=True),
        # eight requests of four beams: the states of one 27B-class GDN layer move
        dict(name="beam_reorder_gdn", op="beam_reorder", kind="gdn", B=8, K=4, H=48, P=128, N=128, G=16, act="bf16"),
        # one request of five beams over a small SSM layer: latency
        dict(name="beam_reorder_ssm", op="beam_reorder", kind="ssm", B=1, K=5, H=16, P=64, N=128, G=1, act="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ssm_prefill", "ssm_prefill", "ssm_token", "beam_select", "beam_reorder"])
    act = rng.choice(["bf16", "bf16", "f32"])
    if op == "beam_select":
        K = rng.randint(1, 16)
        V = _log_int(rng, 1000, 150000)
        B = _log_int(rng, 1, max(2, min(64, 60_000_000 // (K * V))))
        return dict(op=op, B=B, K=K, V=V, S=rng.choice([K, 2 * K, K + 1]), act=act, finished=rng.random() < 0.5)
    G = rng.choice([1, 1, 2, 4, 8])
    H = G * rng.randint(1, max(1, 64 // G))
    P, N = rng.choice([32, 64, 64, 128]), rng.choice([32, 64, 128, 128, 256])
    if op == "beam_reorder":
        kind = rng.choice(["gdn", "ssm"])
        if kind == "gdn":
            P = N = rng.choice([32, 128])
        K = rng.randint(2, 16)
        B = _log_int(rng, 1, max(2, min(64, 25_000_000 // (K * H * P * N))))
        return dict(op=op, kind=kind, B=B, K=K, H=H, P=P, N=N, G=G, act=act)
    if op == "ssm_token":
        B = _log_int(rng, 1, max(2, min(128, 48_000_000 // (H * P * N))))
        return dict(op=op, B=B, H=H, P=P, N=N, G=G, act=act, gate=rng.random() < 0.5)
    B = _log_int(rng, 1, 16)
    T = _log_int(rng, 1, max(64, min(20000, 5_000_000_000 // (H * P * N * B))))
    return dict(op=op, B=B, T=T, H=H, P=P, N=N, G=G, act=act, ragged=rng.random() < 0.5, gate=rng.random() < 0.5)


def _channels(c):
    return c["H"] * c["P"] + 2 * c["G"] * c["N"]


def work(case):
    c = case
    a = 2 if c["act"] == "bf16" else 4
    if c["op"] == "beam_select":
        return {"bytes": c["B"] * c["K"] * c["V"] * a + 12 * c["B"] * c["S"] + 4 * c["B"] * c["K"],
                "flops": 4 * c["B"] * c["K"] * c["V"]}
    C = _channels(c)                                       # the same count for both kinds of layer
    if c["op"] == "beam_reorder":
        K = c["K"]
        written = K - 1                                    # expected slots whose parent is another slot
        read = K * (1 - (1 - 1 / K) ** (K - 1))            # expected sources that some other slot takes
        return {"bytes": c["B"] * (read + written) * (4 * c["H"] * c["P"] * c["N"] + 4 * C * a), "flops": 0}
    B, H, P, N = c["B"], c["H"], c["P"], c["N"]
    weights = C * 4 * a + C * a + 12 * H
    tails = 2 * B * C * 4 * a
    state = 8 * B * H * P * N
    if c["op"] == "ssm_token":
        per = C * a + 4 * H + H * P * a * (2 if c["gate"] else 1)
        return {"bytes": state + tails + weights + B * per, "flops": 6 * B * H * P * N + 10 * B * C}
    tokens = B * c["T"] * (0.5 if c["ragged"] else 1.0)    # lengths are spread evenly over 0..T
    per = C * a + 4 * H + H * P * a * (2 if c["gate"] else 1)
    flops = H * (4 * P * N + CHUNK * P) + c["G"] * CHUNK * N + 12 * C
    return {"bytes": state + tails + weights + tokens * per, "flops": tokens * flops}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * scale


def prepare(case, seed):
    c, act = case, _act(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    B = c["B"]
    if c["op"] == "beam_select":
        K, V, S = c["K"], c["V"], c["S"]
        s["logits"] = torch.randn(B, K, V, generator=g, device=DEV).mul_(2.5).to(act)
        s["scores"] = -torch.rand(B, K, generator=g, device=DEV) * 8
        fin = torch.rand(B, K, generator=g, device=DEV) < 0.2
        s["finished"] = fin if c["finished"] else None
        s["eos"] = 2
        s["out"] = (torch.zeros(B, S, device=DEV), torch.zeros(B, S, dtype=torch.int32, device=DEV),
                    torch.zeros(B, S, dtype=torch.int32, device=DEV))
        return s
    H, P, N, C = c["H"], c["P"], c["N"], _channels(c)
    if c["op"] == "beam_reorder":
        K = c["K"]
        s["state"] = _normal(g, B * K, H, P, N)
        s["tail"] = _normal(g, B * K, C, 4).to(act)
        s["parent"] = torch.randint(0, K, (B, K), generator=g, device=DEV, dtype=torch.int32)
        return s
    s["state"] = _normal(g, B, H, P, N, scale=0.3)
    s["tail"] = _normal(g, B, C, 4).to(act)
    s["w"] = _normal(g, C, 4, scale=0.5).to(act)
    s["conv_bias"] = _normal(g, C, scale=0.1).to(act)
    s["A"] = -(1 + 15 * torch.rand(H, generator=g, device=DEV))
    dt0 = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(H, generator=g, device=DEV))   # 0.001 .. 0.1
    s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))                                            # softplus inverse
    s["D"] = 1 + _normal(g, H, scale=0.2)
    lead = (B,) if c["op"] == "ssm_token" else (B, c["T"])
    s["x"] = _normal(g, *lead, C).to(act)
    s["dt"] = _normal(g, *lead, H)
    s["z"] = _normal(g, *lead, H, P).to(act) if c["gate"] else None
    s["y"] = torch.zeros(*lead, H, P, device=DEV, dtype=act)
    if c["op"] == "ssm_token":
        s["tail_other"] = torch.zeros_like(s["tail"])
    else:
        s["lengths"] = (torch.randint(0, c["T"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
                        if c["ragged"] else None)
    return s


# ------------------------------------------------------------------ the library's calls

def _ws(nbytes):
    global _workspace
    if _workspace is None or _workspace.numel() < nbytes:
        _workspace = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    return _workspace


def _run_own(s):
    import gated_deltanet_decode_amd as gdn
    c = s["case"]
    if c["op"] == "beam_select":
        o = s["out"]
        ws = _ws(gdn.beam_select_workspace_bytes(c["B"], c["K"], c["V"], c["S"]))
        gdn.beam_select(s["logits"], s["scores"], o[0], o[1], o[2], ws, finished=s["finished"], eos=s["eos"])
        return o
    batch = c["B"] * c["K"] if c["op"] == "beam_reorder" else c["B"]
    if c["op"] == "beam_reorder" and c["kind"] == "gdn":
        d = gdn.dims(batch, c["G"], c["H"], c["N"], c["P"], 4, c["act"])
    else:
        d = gdn.ssm_dims(batch, c["H"], c["G"], c["P"], c["N"], 4, c["act"])
    if c["op"] == "beam_reorder":
        gdn.beam_reorder(d, s["state"], s["tail"], s["parent"])
        return s["state"], s["tail"]
    if c["op"] == "ssm_token":
        gdn.ssm_decode_token(d, s["state"], s["tail"], s["tail_other"], s["w"], s["x"], s["dt"], s["A"], s["y"],
                             conv_bias=s["conv_bias"], dt_bias=s["dt_bias"], D=s["D"], z=s["z"])
        s["tail"], s["tail_other"] = s["tail_other"], s["tail"]
        return s["y"], s["state"], s["tail"]
    ws = _ws(gdn.ssm_prefill_workspace_bytes(d, c["T"]))
    gdn.ssm_prefill(d, s["state"], s["tail"], s["w"], s["x"], s["dt"], s["A"], s["y"], ws, conv_bias=s["conv_bias"],
                    dt_bias=s["dt_bias"], D=s["D"], z=s["z"], lengths=s["lengths"])
    return s["y"], s["state"], s["tail"]


# ------------------------------------------------------------------ the plain forms

def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_select(s):
    c = s["case"]
    B, K, V, S = c["B"], c["K"], c["V"], c["S"]
    lg = s["logits"].double()
    m = lg.amax(-1, keepdim=True)
    cand = s["scores"].double().unsqueeze(-1) + ((lg - m) - torch.log(torch.exp(lg - m).sum(-1, keepdim=True)))
    if s["finished"] is not None:
        done = s["finished"].unsqueeze(-1)
        only = torch.full((V,), -math.inf, dtype=torch.float64, device=DEV)
        only[s["eos"]] = 0
        cand = torch.where(done, s["scores"].double().unsqueeze(-1) + only, cand)
    cand = cand.reshape(B, K * V)
    # values first, then the lowest index among equals: all candidates at or above the S-th value, in a stable order
    kth = torch.topk(cand, S, dim=-1).values[:, -1:]
    spare = min(K * V, 4 * S + 64)
    val, idx = torch.topk(torch.where(cand >= kth, cand, -math.inf), spare, dim=-1)
    by_index = torch.argsort(idx, dim=-1, stable=True)
    val, idx = val.gather(1, by_index), idx.gather(1, by_index)
    by_value = torch.argsort(val, dim=-1, descending=True, stable=True)[:, :S]
    val, idx = val.gather(1, by_value), idx.gather(1, by_value)
    return val.float(), (idx // V).int(), (idx % V).int()


def _plain_reorder(s):
    c = s["case"]
    flat = (s["parent"].long() + torch.arange(c["B"], device=DEV).unsqueeze(1) * c["K"]).reshape(-1)
    s["state"], s["tail"] = s["state"][flat], s["tail"][flat]
    return s["state"], s["tail"]


def _split(u, c):
    H, P, N, G = c["H"], c["P"], c["N"], c["G"]
    x, b, k = u.split([H * P, G * N, G * N], dim=-1)
    lead = u.shape[:-1]
    return x.reshape(*lead, H, P), b.reshape(*lead, G, N), k.reshape(*lead, G, N)


def _plain_token(s):
    c = s["case"]
    act = _act(c)
    tail = torch.cat([s["tail"][..., 1:], s["x"].unsqueeze(-1)], -1)
    u = _silu((tail.float() * s["w"].float()).sum(-1) + s["conv_bias"].float())
    x, b, k = _split(u, c)
    rep = c["H"] // c["G"]
    b, k = b.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    dt = _softplus(s["dt"] + s["dt_bias"])
    decay = torch.exp(dt * s["A"].clamp(max=0))
    state = s["state"] * decay[..., None, None] + (dt.unsqueeze(-1) * x).unsqueeze(-1) * b.unsqueeze(-2)
    y = (state * k.unsqueeze(-2)).sum(-1) + s["D"].unsqueeze(-1) * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"], s["tail"], s["y"] = state, tail, y.to(act)
    return s["y"], state, tail


def _plain_prefill(s):
    c = s["case"]
    act = _act(c)
    B, T, H, P, N, G = c["B"], c["T"], c["H"], c["P"], c["N"], c["G"]
    rep, Q = H // G, CHUNK
    nc = -(-T // Q)
    pad = nc * Q - T
    length = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=DEV)
    live = torch.arange(T, device=DEV) < length.unsqueeze(1)                       # [B, T]
    rows = torch.cat([s["tail"].transpose(1, 2), s["x"]], 1)                       # [B, 4 + T, C]
    r32, w = rows.float(), s["w"].float()
    u = _silu(r32[:, 1:T + 1] * w[:, 0] + r32[:, 2:T + 2] * w[:, 1] + r32[:, 3:T + 3] * w[:, 2]
              + r32[:, 4:] * w[:, 3] + s["conv_bias"].float())
    x, b, k = _split(u, c)
    dt = _softplus(s["dt"] + s["dt_bias"]) * live.unsqueeze(-1)
    da = dt * s["A"].clamp(max=0)
    skip = s["D"].unsqueeze(-1) * x
    xd = x * dt.unsqueeze(-1)
    fill = lambda v: torch.nn.functional.pad(v, (0, 0) * (v.dim() - 2) + (0, pad))  # noqa: E731
    xd = fill(xd).reshape(B, nc, Q, G, rep, P).permute(0, 1, 3, 4, 2, 5)           # [B, nc, G, rep, Q, P]
    b = fill(b).reshape(B, nc, Q, G, N).permute(0, 1, 3, 2, 4)                     # [B, nc, G, Q, N]
    k = fill(k).reshape(B, nc, Q, G, N).permute(0, 1, 3, 2, 4)
    da = fill(da).reshape(B, nc, Q, G, rep).permute(0, 1, 3, 4, 2)                 # [B, nc, G, rep, Q]
    cum = da.double().cumsum(-1)
    c32, total = cum.float(), cum[..., -1]
    causal = torch.ones(Q, Q, dtype=torch.bool, device=DEV).tril()
    L = torch.exp((c32.unsqueeze(-1) - c32.unsqueeze(-2)).masked_fill(~causal, -math.inf))
    gram = torch.matmul(k, b.transpose(-1, -2))                                     # [B, nc, G, Q, Q]
    y = torch.matmul(L * gram.unsqueeze(3), xd)                                     # inside the chunk
    # each chunk's own contribution to the state, then the states that enter the chunks
    wx = xd * torch.exp((total.unsqueeze(-1) - cum).float()).unsqueeze(-1)
    own_state = torch.matmul(wx.transpose(-1, -2), b.unsqueeze(3))                  # [B, nc, G, rep, P, N]
    first = s["state"].reshape(B, 1, G, rep, P, N)
    parts = torch.cat([first, own_state], 1).permute(0, 2, 3, 1, 4, 5).reshape(B, G, rep, nc + 1, P * N)
    upto = torch.cat([torch.zeros_like(total[:, :1]), total], 1).cumsum(1).permute(0, 2, 3, 1)   # [B, G, rep, nc + 1]
    tri = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=DEV).tril()
    carry = torch.exp((upto.unsqueeze(-1) - upto.unsqueeze(-2)).masked_fill(~tri, -math.inf).float())
    entering = torch.matmul(carry, parts).reshape(B, G, rep, nc + 1, P, N)
    ent = entering[:, :, :, :nc].permute(0, 3, 1, 2, 4, 5)                          # [B, nc, G, rep, P, N]
    y = y + torch.exp(c32).unsqueeze(-1) * torch.matmul(k.unsqueeze(3), ent.transpose(-1, -2))
    y = y.permute(0, 1, 4, 2, 3, 5).reshape(B, nc * Q, H, P)[:, :T] + skip
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["y"] = torch.where(live[..., None, None], y.to(act), s["y"])
    s["state"] = entering[:, :, :, nc].reshape(B, H, P, N).contiguous()
    last = length.unsqueeze(1) + torch.arange(4, device=DEV)                        # rows len .. len+3 of (tail ++ x)
    s["tail"] = rows.gather(1, last.unsqueeze(-1).expand(-1, -1, rows.shape[-1])).transpose(1, 2).contiguous()
    return s["y"], s["state"], s["tail"]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "ssm_prefill":
        return _plain_prefill(state)
    if op == "ssm_token":
        return _plain_token(state)
    if op == "beam_select":
        return _plain_select(state)
    return _plain_reorder(state)


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_select(s, c):
    V, S = c["V"], c["S"]
    values, parents, tokens = [], [], []
    for b in range(c["B"]):
        rows = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double()[:, None]
        if s["finished"] is not None:
            for k in range(c["K"]):
                if bool(s["finished"][b, k]):
                    rows[k] = -math.inf
                    rows[k, s["eos"]] = float(s["scores"][b, k])
        order = torch.sort(rows.reshape(-1), descending=True, stable=True)
        values.append(order.values[:S])
        parents.append((order.indices[:S] // V).int())
        tokens.append((order.indices[:S] % V).int())
    return torch.stack(values), torch.stack(parents), torch.stack(tokens)


def _exact_step(state, window, dt_raw, z, s, c):
    """The recurrence for one token: window [B, C, 4] raw inputs, oldest first."""
    H, P, N, G = c["H"], c["P"], c["N"], c["G"]
    f = window.double() * s["w"].double()
    u = f.sum(-1) + s["conv_bias"].double()
    u = u * torch.sigmoid(u)
    x = u[:, :H * P].reshape(-1, H, P)
    group = torch.arange(H, device=u.device) // (H // G)
    b = u[:, H * P:H * P + G * N].reshape(-1, G, N)[:, group]
    k = u[:, H * P + G * N:].reshape(-1, G, N)[:, group]
    raw = dt_raw.double() + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    state = torch.exp(dt * torch.clamp(s["A"].double(), max=0))[:, :, None, None] * state
    state = torch.addcmul(state, (dt[..., None] * x)[..., None], b[:, :, None, :])
    y = (state @ k[..., None])[..., 0] + s["D"].double()[:, None] * x
    if z is not None:
        z = z.double()
        y = y * (z * torch.sigmoid(z))
    return y, state


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "beam_select":
        return _exact_select(s, c)
    if c["op"] == "beam_reorder":
        state, tail = s["state"].clone(), s["tail"].clone()
        for b in range(c["B"]):
            for k, p in enumerate(s["parent"][b].tolist()):
                state[b * c["K"] + k] = s["state"][b * c["K"] + p]
                tail[b * c["K"] + k] = s["tail"][b * c["K"] + p]
        return state, tail
    state = s["state"].double()
    if c["op"] == "ssm_token":
        tail = torch.cat([s["tail"][..., 1:], s["x"][..., None]], -1)
        y, state = _exact_step(state, tail, s["dt"], s["z"], s, c)
        return y, state, tail
    if c["T"] * state.numel() > 2 ** 39:
        return None
    length = s["lengths"].tolist() if s["lengths"] is not None else [c["T"]] * c["B"]
    y, tail = s["y"].double(), s["tail"].clone()
    until = torch.tensor(length, device=state.device)
    ends = sorted(set(length))
    last = ends[-1]
    for t in range(last):
        window = torch.cat([tail[..., 1:], s["x"][:, t, :, None]], -1)
        z = s["z"][:, t] if s["z"] is not None else None
        yt, new = _exact_step(state, window, s["dt"][:, t], z, s, c)
        if t < ends[0]:
            y[:, t], state, tail = yt, new, window
        else:
            on = until > t
            y[:, t] = torch.where(on[:, None, None], yt, y[:, t])
            state = torch.where(on[:, None, None, None], new, state)
            tail = torch.where(on[:, None, None], window, tail)
    return y, state, tail
