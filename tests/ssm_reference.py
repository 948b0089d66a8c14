"""Plain 64-bit forms of the selective state space layer and of beam search's
selection and reordering, for the tests (NumPy, token by token)."""
import numpy as np


def bf16_round(a):
    """float array -> the nearest bf16 values, as float32 (ties to even)."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return u.astype(np.uint32).view(np.float32)


def make(seed, B, T, H, G, P, N, bf16, scale=1.0, gate=True, state_scale=0.3):
    """Inputs of a layer as float32 arrays (activation values already representable)."""
    r = np.random.default_rng(seed)
    C = H * P + 2 * G * N
    act = bf16_round if bf16 else (lambda a: np.ascontiguousarray(a, dtype=np.float32))
    f32 = lambda a: np.ascontiguousarray(a, dtype=np.float32)
    dt0 = np.exp(r.uniform(np.log(1e-3), np.log(0.1), H))
    return dict(B=B, T=T, H=H, G=G, P=P, N=N, C=C, bf16=bf16,
                state=f32(r.standard_normal((B, H, P, N)) * state_scale), tail=act(r.standard_normal((B, C, 4)) * scale),
                w=act(r.standard_normal((C, 4)) * 0.5), conv_bias=act(r.standard_normal(C) * 0.1),
                x=act(r.standard_normal((B, T, C)) * scale), dt=f32(r.standard_normal((B, T, H))),
                dt_bias=f32(dt0 + np.log(-np.expm1(-dt0))), A=f32(-r.uniform(1, 16, H)),
                D=f32(1 + 0.2 * r.standard_normal(H)), z=act(r.standard_normal((B, T, H, P))) if gate else None)


def run(i, lengths=None):
    """The layer over every token: (y [B][T][H][P] with NaN behind a sequence's end, state, tail)."""
    B, T, H, G, P, N = (i[k] for k in ("B", "T", "H", "G", "P", "N"))
    state, tail = i["state"].astype(np.float64), i["tail"].astype(np.float64).copy()
    y = np.full((B, T, H, P), np.nan)
    opt = lambda name, n: np.zeros(n) if i.get(name) is None else i[name].astype(np.float64)
    bias, dtb, D = opt("conv_bias", i["C"]), opt("dt_bias", H), opt("D", H)
    grp = np.arange(H) // (H // G)
    A = np.minimum(i["A"].astype(np.float64), 0)
    silu = lambda v: v / (1 + np.exp(-v))
    for b in range(B):
        for t in range(T if lengths is None else int(lengths[b])):
            tail[b] = np.concatenate([tail[b][:, 1:], i["x"][b, t][:, None]], 1)
            u = silu((tail[b] * i["w"]).sum(1) + bias)
            x, Bm, Cm = u[:H * P].reshape(H, P), u[H * P:H * P + G * N].reshape(G, N), u[H * P + G * N:].reshape(G, N)
            d = np.logaddexp(0, i["dt"][b, t].astype(np.float64) + dtb)
            state[b] = np.exp(d * A)[:, None, None] * state[b] + (d[:, None] * x)[:, :, None] * Bm[grp][:, None, :]
            yt = (state[b] * Cm[grp][:, None, :]).sum(-1) + D[:, None] * x
            y[b, t] = yt if i["z"] is None else yt * silu(i["z"][b, t].astype(np.float64))
    return y, state, tail


def select(logits, scores, S, finished=None, eos=0):
    """(values, parent, token) of each sequence's S best, by the definition."""
    B, K, V = logits.shape
    lg = logits.astype(np.float64)
    lg = np.where(np.isnan(lg), -np.inf, np.minimum(lg, np.finfo(np.float32).max))
    sc = scores.astype(np.float64)
    sc = np.where(np.isnan(sc), -np.inf, np.minimum(sc, np.finfo(np.float32).max))
    cand = np.full((B, K, V), -np.inf)
    for b in range(B):
        for k in range(K):
            if sc[b, k] == -np.inf:
                continue
            if finished is not None and finished[b, k]:
                cand[b, k, eos] = sc[b, k]
                continue
            m = lg[b, k].max()
            if m == -np.inf:
                continue
            cand[b, k] = sc[b, k] + ((lg[b, k] - m) - np.log(np.exp(lg[b, k] - m).sum()))
    flat = cand.reshape(B, K * V)
    order = np.argsort(-flat, axis=1, kind="stable")[:, :S]
    return np.take_along_axis(flat, order, 1), (order // V).astype(np.int32), (order % V).astype(np.int32)
