"""Cases of the gated linear recurrent layer (prompts, training steps, single
tokens) and of the norms on either side of a recurrent mixer: what is measured,
the operators' plain forms, and their definition in 64 bits.

`own` False computes a case with elementary torch operations; `own` True makes
the library's calls.  A layer of W channels keeps a state of fp32 [B][W]; x and
the gate inputs r, i and z are [B][T][W], a token's [B][W].
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
_workspace = None      # one per process, grown to the largest call, as a program keeps it
_saved = None          # what a training forward leaves for its backward, the same way


def _act(case):
    return torch.bfloat16 if case["act"] == "bf16" else torch.float32


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoded token, single stream: launch latency counts
        dict(name="lru_token_b1", op="lru_token", B=1, W=5120, act="bf16", gate=True, packed=False),
        # one decoded token for a large serving batch; gate inputs are halves of one projection's rows
        dict(name="lru_token_b200", op="lru_token", B=200, W=4096, act="bf16", gate=True, packed=True),
        # one short chat turn
        dict(name="lru_prefill_short", op="lru_prefill", B=1, T=77, W=2560, act="bf16", ragged=False, gate=True, packed=False),
        # one long document
        dict(name="lru_prefill_32k", op="lru_prefill", B=1, T=32768, W=4096, act="bf16", ragged=False, gate=True, packed=True),
        # a padded batch of prompts of different lengths, fp32, no output gate
        dict(name="lru_prefill_ragged_f32", op="lru_prefill", B=8, T=2500, W=2560, act="f32", ragged=True, gate=False, packed=False),
        # a training step of one layer: forward and backward over a batch of sequences
        dict(name="lru_train", op="lru_train", B=4, T=4096, W=4096, act="bf16", ragged=False, gate=True, packed=True),
        # a small fp32 training step of odd lengths
        dict(name="lru_train_f32", op="lru_train", B=3, T=1003, W=1544, act="f32", ragged=True, gate=False, packed=False),
        # before a block, one token of each of 64 sequences: latency
        dict(name="residual_norm_b64", op="residual_norm", rows=64, W=5120, act="bf16", res="bf16", scale=False, post=False),
        # the same over a long prompt: an fp32 residual stream, the block's output normed and scaled before it is added
        dict(name="residual_norm_32k", op="residual_norm", rows=32768, W=5120, act="bf16", res="f32", scale=True, post=True),
        # a training step of that norm
        dict(name="residual_norm_train", op="residual_norm_train", rows=8192, W=4096, act="bf16", res="bf16", scale=True, post=True),
        # after a delta-rule mixer of 48 heads of 128, one token of each of 64 sequences: fp32 outputs, gate, bf16 for the projection
        dict(name="gated_norm_b64", op="gated_norm", rows=64, H=48, D=128, o="f32", act="bf16", first=False, per_head=False, packed=True),
        # a training step of that norm over 8,192 tokens
        dict(name="gated_norm_train", op="gated_norm_train", rows=8192, H=48, D=128, o="f32", act="bf16", first=False, per_head=False, packed=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["lru_prefill", "lru_prefill", "lru_train", "lru_token", "residual_norm", "residual_norm_train",
                     "gated_norm", "gated_norm_train"])
    act = rng.choice(["bf16", "bf16", "f32"])
    half = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("lru_prefill", "lru_train"):
        W = 8 * _log_int(rng, 16, 800)
        B = _log_int(rng, 1, 16)
        T = _log_int(rng, 1, max(64, min(20000, (60_000_000 if op == "lru_prefill" else 25_000_000) // (B * W))))
        return dict(op=op, B=B, T=T, W=W, act=act, ragged=half(), gate=half(), packed=half())
    if op == "lru_token":
        return dict(op=op, B=_log_int(rng, 1, 400), W=8 * _log_int(rng, 16, 1000), act=act, gate=half(), packed=half())
    if op in ("residual_norm", "residual_norm_train"):
        W = 8 * _log_int(rng, 16, 1500)
        rows = _log_int(rng, 1, max(64, min(30000, 40_000_000 // W)))
        return dict(op=op, rows=rows, W=W, act=act, res=rng.choice(["f32", act]), scale=half(), post=half())
    whole = rng.random() < 0.3                              # groups of channels, as wide as a state space layer's
    D = 8 * _log_int(rng, 40, 800) if whole else rng.choice([32, 64, 96, 128, 128, 256])
    H = rng.randint(1, 4) if whole else rng.randint(1, 64)
    rows = _log_int(rng, 1, max(64, min(30000, 40_000_000 // (H * D))))
    return dict(op=op, rows=rows, H=H, D=D, o=rng.choice(["f32", act]), act=act, first=half(), per_head=whole or half(),
                packed=half())


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    c = case
    a, op = _size(c["act"]), c["op"]
    if op.startswith("lru"):
        B, W, z = c["B"], c["W"], 1 if c["gate"] else 0
        edge = 8 * B * W + 4 * W                            # the state in and out, A
        if op == "lru_token":
            return {"bytes": edge + B * W * a * (4 + z), "flops": B * W * (22 + 5 * z)}
        n = B * c["T"] * W * (0.5 if c["ragged"] else 1.0)  # lengths are spread evenly over 0..T
        if op == "lru_prefill":
            return {"bytes": edge + n * a * (4 + z), "flops": n * (22 + 5 * z)}
        back = B * c["T"] * W * a * (3 + z)                 # gradients are written behind a sequence's end too
        return {"bytes": 2 * edge + 4 * W + n * a * (4 + z) + n * a * (4 + z) + back, "flops": n * (70 + 18 * z)}
    if op.startswith("residual"):
        n, r, W = c["rows"] * c["W"], _size(c["res"]), c["W"]
        fwd = n * (2 * r + 2 * a) + 4 * W * (1 + c["scale"] + c["post"])
        if op == "residual_norm":
            return {"bytes": fwd, "flops": n * (6 + c["scale"] + 4 * c["post"])}
        again = n * (r + 2 * a) + n * (2 * r + a)           # s, delta, dy; the residual's gradient in and out, ddelta
        return {"bytes": fwd + again + 8 * W * (1 + c["scale"] + c["post"]), "flops": n * (18 + 3 * c["scale"] + 14 * c["post"])}
    n, o = c["rows"] * c["H"] * c["D"], _size(c["o"])
    weights = 4 * c["D"] * (c["H"] if c["per_head"] else 1)
    fwd = n * (o + 2 * a) + weights
    if op == "gated_norm":
        return {"bytes": fwd, "flops": 10 * n}
    return {"bytes": fwd + n * (2 * o + 3 * a) + 2 * weights, "flops": 34 * n}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c, act = case, _act(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    s = {"case": c}
    if c["op"].startswith("lru"):
        B, W = c["B"], c["W"]
        lead = (B,) if c["op"] == "lru_token" else (B, c["T"])
        s["state"] = normal(B, W)
        # a channel whose gate r is fully open keeps 0.9^8 to 0.999^8 of its state a token, a half-open one their roots
        s["A"] = 8 * torch.log(0.9 + 0.099 * torch.rand(W, generator=g, device=DEV))
        if c["packed"]:                                     # both gates' inputs are one projection's output
            gates = normal(*lead, 2 * W).to(act)
            s["r"], s["i"] = gates[..., :W], gates[..., W:]
        else:
            s["r"], s["i"] = normal(*lead, W).to(act), normal(*lead, W).to(act)
        s["x"] = normal(*lead, W).to(act)
        s["z"] = normal(*lead, W).to(act) if c["gate"] else None
        s["y"] = torch.zeros(*lead, W, device=DEV, dtype=act)
        if c["op"] == "lru_token":
            return s
        s["lengths"] = (torch.randint(0, c["T"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
                        if c["ragged"] else None)
        if c["op"] == "lru_train":
            s["dy"], s["dstate"] = normal(*lead, W).to(act), normal(B, W)
            gates = torch.zeros(*lead, 2 * W, device=DEV, dtype=act)
            s["grads"] = {"dx": torch.zeros_like(s["y"]), "dr": gates[..., :W], "di": gates[..., W:],
                          "dA": torch.zeros(W, device=DEV), "dstate0": torch.zeros(B, W, device=DEV),
                          "dz": torch.zeros_like(s["y"]) if c["gate"] else None}
        return s
    weight = lambda *shape: 1 + 0.2 * normal(*shape)  # noqa: E731
    if c["op"].startswith("residual"):
        rows, W, res = c["rows"], c["W"], _dtype(c["res"])
        s["residual"] = (2 * normal(rows, W)).to(res)
        s["delta"] = normal(rows, W).to(act)
        s["w"] = weight(W)
        s["scale"] = 0.5 + 0.2 * normal(W) if c["scale"] else None
        s["w_post"] = weight(W) if c["post"] else None
        s["out"] = torch.zeros_like(s["residual"])
        s["y"] = torch.zeros(rows, W, device=DEV, dtype=act)
        if c["op"] == "residual_norm_train":
            s["dy"], s["ds"] = normal(rows, W).to(act), normal(rows, W).to(res)
            opt = lambda on: torch.zeros(W, device=DEV) if on else None  # noqa: E731
            s["grads"] = {"dresidual": torch.zeros_like(s["residual"]), "ddelta": torch.zeros_like(s["delta"]),
                          "dw": torch.zeros(W, device=DEV), "dscale": opt(c["scale"]), "dw_post": opt(c["post"])}
        return s
    rows, H, D = c["rows"], c["H"], c["D"]
    s["o"] = (0.5 * normal(rows, H, D)).to(_dtype(c["o"]))
    if c["packed"]:                                         # z lies behind the mixer's inputs in one projection's rows
        s["z"] = normal(rows, 2 * H * D).to(act)[:, H * D:].unflatten(1, (H, D))
    else:
        s["z"] = normal(rows, H, D).to(act)
    s["w"] = weight(H, D) if c["per_head"] else weight(D)
    s["y"] = torch.zeros(rows, H, D, device=DEV, dtype=act)
    if c["op"] == "gated_norm_train":
        s["dy"] = normal(rows, H, D).to(act)
        s["grads"] = {"do": torch.zeros_like(s["o"]), "dz": torch.zeros(rows, H, D, device=DEV, dtype=act),
                      "dw": torch.zeros_like(s["w"])}
    return s


# ------------------------------------------------------------------ the library's calls

def _ws(nbytes):
    global _workspace
    if _workspace is None or _workspace.numel() < nbytes:
        _workspace = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    return _workspace


def _keep(nbytes):
    global _saved
    if _saved is None or _saved.numel() < nbytes:
        _saved = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    return _saved


def _run_own(s):
    import gated_deltanet_decode_amd as gdn
    c, g = s["case"], s.get("grads")
    if c["op"].startswith("lru"):
        d = gdn.lru_dims(c["B"], c["W"], c["act"])
        if c["op"] == "lru_token":
            gdn.lru_decode_token(d, s["state"], s["x"], s["r"], s["i"], s["A"], s["y"], z=s["z"])
            return s["y"], s["state"]
        ws = _ws(gdn.lru_prefill_workspace_bytes(d, c["T"]))
        saved = _keep(gdn.lru_saved_bytes(d, c["T"])) if g else None
        gdn.lru_prefill(d, s["state"], s["x"], s["r"], s["i"], s["A"], s["y"], ws, z=s["z"], lengths=s["lengths"],
                        saved=saved)
        if not g:
            return s["y"], s["state"]
        ws = _ws(gdn.lru_backward_workspace_bytes(d, c["T"]))
        gdn.lru_backward(d, s["x"], s["r"], s["i"], s["A"], s["dy"], saved, g["dx"], g["dr"], g["di"], g["dA"], ws,
                         z=s["z"], dz=g["dz"], dstate=s["dstate"], dstate0=g["dstate0"], lengths=s["lengths"])
        return _outputs(s, "state")
    if c["op"].startswith("residual"):
        gdn.residual_norm(s["residual"], s["delta"], s["w"], s["out"], s["y"], scale=s["scale"], w_post=s["w_post"],
                          eps=EPS)
        if not g:
            return s["y"], s["out"]
        ws = _ws(gdn.residual_norm_backward_workspace_bytes(c["rows"], c["W"]))
        gdn.residual_norm_backward(s["out"], s["delta"], s["w"], s["dy"], g["dresidual"], g["ddelta"], g["dw"], ws,
                                   ds=s["ds"], scale=s["scale"], w_post=s["w_post"], dscale=g["dscale"],
                                   dw_post=g["dw_post"], eps=EPS)
        return _outputs(s, "out")
    gdn.gated_norm(s["o"], s["z"], s["w"], s["y"], eps=EPS, gate_first=c["first"])
    if not g:
        return s["y"]
    ws = _ws(gdn.gated_norm_backward_workspace_bytes(c["rows"], c["H"], c["D"]))
    gdn.gated_norm_backward(s["o"], s["z"], s["w"], s["dy"], g["do"], g["dz"], g["dw"], ws, eps=EPS,
                            gate_first=c["first"])
    return _outputs(s)


def _outputs(s, *more):
    return {"y": s["y"], **{k: s[k] for k in more}, **{k: v for k, v in s["grads"].items() if v is not None}}


# ------------------------------------------------------------------ the plain forms

def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _scan(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dimension 1 by doubling; both are replaced, b by h."""
    k = 1
    while k < a.shape[1]:
        b[:, k:] += a[:, k:] * b[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return b


def _plain_token(s):
    act = _act(s["case"])
    rate = s["A"].clamp(max=0)
    la = rate * _sigmoid(s["r"].float())
    h = torch.exp(la) * s["state"] + torch.sqrt(-torch.expm1(2 * la)) * _sigmoid(s["i"].float()) * s["x"].float()
    y = h
    if s["z"] is not None:
        z = s["z"].float()
        y = h * (z * _sigmoid(z))
    s["state"], s["y"] = h, y.to(act)
    return s["y"], s["state"]


def _plain_lru(s):
    c, act = s["case"], _act(s["case"])
    B, T = c["B"], c["T"]
    x, r, i = s["x"].float(), s["r"].float(), s["i"].float()
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(T, device=DEV) < s["lengths"].long().unsqueeze(1)).unsqueeze(-1)     # [B, T, 1]
    rate = s["A"].clamp(max=0)
    rho, gi = _sigmoid(r), _sigmoid(i)
    la = rate * rho
    a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    b = m * gi * x
    if live is not None:
        a, b = torch.where(live, a, 1.0), torch.where(live, b, 0.0)
    first = s["state"]
    b[:, 0] += a[:, 0] * first
    h = _scan(a.clone(), b)
    out = h
    if s["z"] is not None:
        z = s["z"].float()
        sz = _sigmoid(z)
        out = h * (z * sz)
    out = out.to(act)
    s["y"] = out if live is None else torch.where(live, out, s["y"])
    s["state"] = h[:, -1].clone()
    if c["op"] == "lru_prefill":
        return s["y"], s["state"]
    dy = s["dy"].float()
    dout = dy * (z * sz) if s["z"] is not None else dy
    if live is not None:
        dout = torch.where(live, dout, 0.0)
    # from the last token back: G[t] = dout[t] + a[t+1] G[t+1]
    step = torch.cat([torch.ones_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    e = dout.flip(1)
    e[:, 0] += s["dstate"]
    G = _scan(step, e).flip(1)
    before = torch.cat([first.unsqueeze(1), h[:, :-1]], 1)
    dla = G * (a * before - torch.where(m > 0, a * a / m, 0.0) * gi * x)
    grads = {"dx": G * m * gi, "dr": dla * rate * rho * (1 - rho), "di": G * m * x * gi * (1 - gi)}
    if s["z"] is not None:
        grads["dz"] = dy * h * sz * (1 + z * (1 - sz))
    if live is not None:
        grads = {k: torch.where(live, v, 0.0) for k, v in grads.items()}
        dla = torch.where(live, dla, 0.0)
    grads = {k: v.to(act) for k, v in grads.items()}
    grads["dA"] = torch.where(s["A"] < 0, (dla * rho).sum((0, 1)), 0.0)
    grads["dstate0"] = a[:, 0] * G[:, 0]
    s["grads"].update(grads)
    return _outputs(s, "state")


def _plain_residual(s):
    act, w, scale, post = _act(s["case"]), s["w"], s["scale"], s["w_post"]
    delta = s["delta"].float()
    n = delta
    if post is not None:
        p = 1 / torch.sqrt((delta * delta).mean(-1, keepdim=True) + EPS)
        n = delta * p * post
    out = s["residual"].float() + (n if scale is None else scale * n)
    s["out"] = out.to(s["residual"].dtype)
    v = s["out"].float()
    q = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    s["y"] = (v * q * w).to(act)
    if "grads" not in s:
        return s["y"], s["out"]
    dy = s["dy"].float()
    dyw = dy * w
    ds = s["ds"].float() + q * (dyw - v * (q * q * (dyw * v).mean(-1, keepdim=True)))
    grads = {"dresidual": ds.to(s["residual"].dtype), "dw": (dy * v * q).sum(0)}
    t = ds
    if scale is not None:
        grads["dscale"] = (ds * n).sum(0)
        t = ds * scale
    if post is not None:
        grads["dw_post"] = (t * delta * p).sum(0)
        tw = t * post
        t = p * (tw - delta * (p * p * (tw * delta).mean(-1, keepdim=True)))
    grads["ddelta"] = t.to(act)
    s["grads"].update(grads)
    return _outputs(s, "out")


def _plain_gated(s):
    c, act, w = s["case"], _act(s["case"]), s["w"]
    o, z = s["o"].float(), s["z"].float()
    sz = _sigmoid(z)
    gate = z * sz
    u = o * gate if c["first"] else o
    q = 1 / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS)
    n = u * q
    y = n * w if c["first"] else n * w * gate
    s["y"] = y.to(act)
    if "grads" not in s:
        return s["y"]
    dy = s["dy"].float()
    dn = dy if c["first"] else dy * gate
    dw = dn * n
    dn = dn * w
    du = q * (dn - n * (dn * n).mean(-1, keepdim=True))
    if c["first"]:
        do, dgate = du * gate, du * o
    else:
        do, dgate = du, dy * n * w
    grads = {"do": do.to(s["o"].dtype), "dz": (dgate * sz * (1 + z * (1 - sz))).to(act),
             "dw": dw.sum(0) if c["per_head"] else dw.sum((0, 1))}
    s["grads"].update(grads)
    return _outputs(s)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "lru_token":
        return _plain_token(state)
    if op.startswith("lru"):
        return _plain_lru(state)
    if op.startswith("residual"):
        return _plain_residual(state)
    return _plain_gated(state)


# ------------------------------------------------------------------ the definition in 64 bits

def _rms(v):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _silu(v):
    return v * torch.sigmoid(v)


def _leaf(s, *names):
    return {k: s[k].double().requires_grad_(True) for k in names if s.get(k) is not None}


def _exact_lru(s, c):
    """Token by token; the gradients by automatic differentiation of the loop over single tokens."""
    B, T, train = c["B"], c["T"], c["op"] == "lru_train"
    until = s["lengths"].tolist() if s["lengths"] is not None else [T] * B
    y, state = s["y"].double(), s["state"].double().clone()
    grads = {k: torch.zeros_like(v, dtype=torch.float64).contiguous() for k, v in s.get("grads", {}).items()
             if v is not None}
    for b in range(B):
        n = until[b]
        if n == 0:
            if train:
                grads["dstate0"][b] = s["dstate"][b].double()
            continue
        with torch.set_grad_enabled(train):
            row = {k: s[k][b, :n].double().requires_grad_(train) for k in ("x", "r", "i", "z") if s[k] is not None}
            A, h0 = s["A"].double().requires_grad_(train), s["state"][b].double().requires_grad_(train)
            log_a = torch.clamp(A, max=0) * torch.sigmoid(row["r"])
            keep = torch.exp(log_a).unbind(0)
            put = (torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(row["i"]) * row["x"]).unbind(0)
            h, path = h0, []
            for t in range(n):
                h = torch.addcmul(put[t], keep[t], h)
                path.append(h)
            out = torch.stack(path)
            if "z" in row:
                out = out * _silu(row["z"])
            y[b, :n], state[b] = out.detach(), h.detach()
            if train:
                loss = (out * s["dy"][b, :n].double()).sum() + (h * s["dstate"][b].double()).sum()
                loss.backward()
                for k, v in row.items():
                    grads["d" + k][b, :n] = v.grad
                grads["dA"] += A.grad
                grads["dstate0"][b] = h0.grad
    if not train:
        return y, state
    return {"y": y, "state": state, **grads}


def _exact_norms(s, c):
    train = "grads" in s
    if c["op"].startswith("residual"):
        v = _leaf(s, "residual", "delta", "w", "scale", "w_post")
        n = _rms(v["delta"]) * v["w_post"] if c["post"] else v["delta"]
        stream = v["residual"] + n * v["scale"] if c["scale"] else v["residual"] + n
        kept = stream.detach().to(s["residual"].dtype).double()       # the stream is rounded where it is stored
        y = _rms(stream + (kept - stream.detach())) * v["w"]
        if not train:
            return y.detach(), kept
        loss = (y * s["dy"].double()).sum() + (stream * s["ds"].double()).sum()
        loss.backward()
        return {"y": y.detach(), "out": kept, **{"d" + k: x.grad for k, x in v.items()}}
    v = _leaf(s, "o", "z", "w")
    gate = _silu(v["z"])
    y = _rms(v["o"] * gate) * v["w"] if c["first"] else _rms(v["o"]) * v["w"] * gate
    if not train:
        return y.detach()
    (y * s["dy"].double()).sum().backward()
    return {"y": y.detach(), **{"d" + k: x.grad for k, x in v.items()}}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"].startswith("lru") and c["op"] != "lru_token":
        # a token of one sequence is one step of the loop
        return None if c["B"] * c["T"] > 2 ** 17 else _exact_lru(s, c)
    if c["op"] != "lru_token":
        return _exact_norms(s, c)
    v = {k: s[k].double() for k in ("state", "x", "r", "i", "A")}
    log_a = torch.clamp(v["A"], max=0) * torch.sigmoid(v["r"])
    h = v["state"] * torch.exp(log_a) + torch.sqrt(-torch.expm1(2 * log_a)) * (torch.sigmoid(v["i"]) * v["x"])
    return (h if s["z"] is None else h * _silu(s["z"].double())), h
