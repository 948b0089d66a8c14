"""Plain 64-bit forms of the gated linear recurrent layer, of the norms around a
block, and of their gradients, for the tests (NumPy, token by token), with bounds
on how far an fp32 computation may be from them.

u = 2^-24 is half a step of fp32, relative; an instruction that rounds once costs
one u, the hardware's exp2, reciprocal and square roots two.  Bounds are carried
along beside the values: every term is counted by its magnitude, so that a sum
that cancels is held to its terms and not to what is left of them.

fp32 has no normal number below TINY = 2^-126, and the hardware's exp2, reciprocal
and roots give or take 0 there.  A gate, its derivative, or a square 1 - a^2, that
is smaller may count as 0: its own term is then lost whole (error 1, relative), and a value may be
off by TINY.  sigmoid(r) = 8e-40 at r = -90 and A = -60 say 1 - a^2 = 1e-37, so that
m = 3e-19 of x is such a term.
"""
import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -126
# e^v = 2^(v log2 e): the product rounds (half a step of v log2 e, u relative) and the fp32 constant
# 1.44269502163 is off by 1.34e-8 = 0.224 u, so the result is off by |v| (1 + 0.224) u
EXP = 1.25


def bf16_round(a):
    """float array -> the nearest bf16 values, as float32 (ties to even)."""
    v = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32).astype(np.uint64)
    v = ((v + 0x7FFF + ((v >> 16) & 1)) >> 16) << 16
    return v.astype(np.uint32).view(np.float32)


def half_step(bf16):
    """Half a step of an output's type, relative."""
    return 2.0 ** -8 if bf16 else U


def stored(value, bound, bf16):
    """The bound of a value once it is rounded to its type: half a step of what was computed, which
    may be larger than the true value by the bound."""
    return bound + half_step(bf16) * (np.abs(value) + bound) + TINY


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1, e) / (1 + e)


def slope_of(v):
    """The sigmoid's derivative s (1 - s), without the difference (1 - s loses every digit at v = 40)."""
    e = np.exp(-np.abs(v))
    return e / (1 + e) ** 2


def make(seed, B, T, W, bf16, gate=True, scale=1.0, open_=(0.9, 0.999)):
    """Inputs of a layer as float32 arrays (activation values already representable)."""
    r = np.random.default_rng(seed)
    act = bf16_round if bf16 else (lambda a: np.ascontiguousarray(a, dtype=np.float32))
    n = lambda *s: r.standard_normal(s)
    return dict(B=B, T=T, W=W, bf16=bf16, state=n(B, W).astype(np.float32),
                A=(8 * np.log(r.uniform(*open_, W))).astype(np.float32), x=act(n(B, T, W) * scale), r=act(n(B, T, W)),
                i=act(n(B, T, W)), z=act(n(B, T, W)) if gate else None, dy=act(n(B, T, W)),
                dstate=n(B, W).astype(np.float32))


def _gates(i, b, t):
    """Values of one token and, relative, how far the fp32 ones may be off."""
    rate = np.minimum(i["A"].astype(np.float64), 0)
    r, gi, x = (i[k][b, t].astype(np.float64) for k in ("r", "i", "x"))
    rho, g = sigmoid(r), sigmoid(gi)
    la = rate * rho
    a, m = np.exp(la), np.sqrt(-np.expm1(2 * la))
    e_rho = (EXP * np.abs(r) + 6) * U           # exponent, exp2, add, reciprocal
    e_g = (EXP * np.abs(gi) + 6) * U
    e_la = e_rho + 3 * U                        # the rate in log2 units, the product
    e_a = np.abs(la) * e_la + 3 * U
    # 1 - a to 2e-7 by the polynomial and the error of its argument (of a and one rounding beyond 1/2); m keeps half
    e_m = 0.5 * (e_la + 6 * U + 2 * e_a) + 3 * U
    e_m = np.where((rho < TINY) | (m * m < TINY), 1.0, e_m)
    e_g = np.where(g < TINY, 1.0, e_g)
    e_rho = np.where(rho < TINY, 1.0, e_rho)
    return rate, rho, g, x, a, m, e_rho, e_g, e_a, e_m


def run(i, lengths=None):
    """(y, state) of the layer over every token, y NaN behind a sequence's end, and bounds for both."""
    B, T, W = i["B"], i["T"], i["W"]
    y, ey = np.full((B, T, W), np.nan), np.full((B, T, W), np.nan)
    state, es = i["state"].astype(np.float64).copy(), np.zeros((B, W))
    hs = np.zeros((B, T + 1, W))                # h before each token, its magnitude and its bound
    mag, bound = np.zeros((B, T + 1, W)), np.zeros((B, T + 1, W))
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        h, M, E = state[b].copy(), np.abs(state[b]), np.zeros(W)
        hs[b, 0], mag[b, 0] = h, M
        for t in range(n):
            _, _, g, x, a, m, _, e_g, e_a, e_m = _gates(i, b, t)
            v = m * g * x
            h = a * h + v
            E = a * E + (e_a + 2 * U) * a * M + (e_g + e_m + 2 * U) * np.abs(v)
            M = a * M + np.abs(v)
            E = E + 2 * U * M
            hs[b, t + 1], mag[b, t + 1], bound[b, t + 1] = h, M, E
            s, e_s = 1.0, 0.0
            if i.get("z") is not None:
                z = i["z"][b, t].astype(np.float64)
                s, e_s = z * sigmoid(z), np.where(sigmoid(z) < TINY, 1.0, (EXP * np.abs(z) + 8) * U)
            y[b, t] = h * s
            ey[b, t] = stored(y[b, t], E * np.abs(s) + (e_s + 2 * U) * M * np.abs(s), i["bf16"])
        state[b], es[b] = h, E + TINY
    return dict(y=y, state=state, ey=ey, es=es, hs=hs, mag=mag, bound=bound)


def grad(i, lengths=None, f=None):
    """Gradients of sum(y dy) + sum(state dstate), and {name: bound}."""
    B, T, W = i["B"], i["T"], i["W"]
    f = run(i, lengths) if f is None else f
    out = {k: np.zeros((B, T, W)) for k in ("dx", "dr", "di", "dz")}
    tol = {k: np.zeros((B, T, W)) for k in out}
    out["dA"], tol["dA"], mA = np.zeros(W), np.zeros(W), np.zeros(W)
    out["dstate0"] = np.zeros((B, W)) if i.get("dstate") is None else i["dstate"].astype(np.float64).copy()
    tol["dstate0"] = np.zeros((B, W))
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        K, M, E = out["dstate0"][b].copy(), np.abs(out["dstate0"][b]), np.zeros(W)
        for t in reversed(range(n)):
            rate, rho, g, x, a, m, e_rho, e_g, e_a, e_m = _gates(i, b, t)
            dy = i["dy"][b, t].astype(np.float64)
            s, e_s = 1.0, 0.0
            if i.get("z") is not None:
                z = i["z"][b, t].astype(np.float64)
                sz = sigmoid(z)
                s, e_s = z * sz, np.where(sz < TINY, 1.0, (EXP * np.abs(z) + 8) * U)
                slope = sz + z * slope_of(z)
                d = dy * f["hs"][b, t + 1]
                out["dz"][b, t] = d * slope
                tol["dz"][b, t] = (np.abs(dy) * f["bound"][b, t + 1] * np.abs(slope)
                                   + np.abs(dy) * f["mag"][b, t + 1] * (sz + np.abs(z) * slope_of(z))
                                   * np.where(sz < TINY, 1.0, (EXP * np.abs(z) + 12) * U))
            G = dy * s + K
            EG = E + np.abs(dy * s) * (e_s + 2 * U)
            MG = np.abs(dy * s) + M
            EG = EG + U * MG
            inv = np.where(m > 0, 1 / np.where(m > 0, m, 1), 0)
            before, mb, eb = f["hs"][b, t], f["mag"][b, t], f["bound"][b, t]
            dla = G * (a * before - a * a * inv * g * x)
            t1, t2 = a * mb, a * a * inv * np.abs(g * x)
            e_dla = EG * (t1 + t2) + MG * (a * eb + (e_a + 3 * U) * t1 + (2 * e_a + e_m + e_g + 6 * U) * t2)
            dslope_r, dslope_i = (slope_of(i[k][b, t].astype(np.float64)) for k in ("r", "i"))
            out["dx"][b, t] = G * m * g
            tol["dx"][b, t] = EG * m * g + MG * m * g * (e_m + e_g + 3 * U)
            w = m * x * dslope_i
            out["di"][b, t] = G * w
            tol["di"][b, t] = EG * np.abs(w) + MG * np.abs(w) * (e_m + np.where(dslope_i < TINY, 1.0, 2 * e_g) + 5 * U)
            w = rate * dslope_r
            out["dr"][b, t] = dla * w
            tol["dr"][b, t] = (e_dla + np.abs(MG * (t1 + t2)) * (np.where(dslope_r < TINY, 1.0, 2 * e_rho) + 6 * U)) * np.abs(w)
            out["dA"] += dla * rho
            tol["dA"] += (e_dla + MG * (t1 + t2) * (e_rho + 2 * U)) * rho
            mA += np.abs(MG * (t1 + t2) * rho)
            K = a * G
            E = a * EG + a * MG * (e_a + 2 * U)
            M = a * MG
        out["dstate0"][b], tol["dstate0"][b] = K, E + 2 * U * M
    out["dA"] = np.where(i["A"] < 0, out["dA"], 0)
    tol["dA"] = tol["dA"] + 64 * U * mA         # a tile's sums, its waves', and a quarter of the tiles' in a row
    tol = {k: v + TINY if k in ("dA", "dstate0") else stored(out[k], v, i["bf16"]) for k, v in tol.items()}
    if i.get("z") is None:
        del out["dz"]
    return out, tol


# ------------------------------------------------ norms

def rms(v, eps):
    return 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def norm_error(n):
    """How far 1 / rms may be off, relative: half of a sum's depth over n values, and the reciprocal root."""
    return (0.5 * (32 + 6 + 16 + 4) + 4) * U


def residual_norm(residual, delta, w, scale=None, post=None, eps=1e-6):
    """(out, bound) before any rounding to the stream's type."""
    res = residual.astype(np.float64)
    if delta is None:
        return res, np.zeros_like(res)
    n = delta.astype(np.float64)
    if post is not None:
        n = n * rms(n, eps) * post
    n = n if scale is None else n * scale
    return res + n, (norm_error(0) + 4 * U) * np.abs(n) + U * (np.abs(res) + np.abs(n))


def norm_of(out, w, eps=1e-6):
    v = out.astype(np.float64)
    y = v * rms(v, eps) * w
    return y, (norm_error(0) + 3 * U) * np.abs(y)


def residual_norm_grad(out, delta, w, dy, ds=None, scale=None, post=None, eps=1e-6):
    """Gradients and {name: bound}; bf16 rounding of the outputs is the caller's."""
    v, g = out.astype(np.float64), dy.astype(np.float64)
    rows, W = v.shape
    e = norm_error(0) * 3
    q = rms(v, eps)
    gw = g * w
    back = q * q * (gw * v).mean(-1, keepdims=True)
    back_m = q * q * np.abs(gw * v).mean(-1, keepdims=True)
    d = np.zeros_like(v) if ds is None else ds.astype(np.float64)
    res, tol = {}, {}
    t = d + q * (gw - v * back)
    mt = np.abs(d) + q * (np.abs(gw) + np.abs(v) * back_m)
    et = U * np.abs(d) + q * ((np.abs(gw) + np.abs(v) * back_m) * (e + 6 * U) + np.abs(v) * back_m * 60 * U)
    res["dresidual"], tol["dresidual"] = t, et + U * mt
    depth = (rows + 64) * U
    res["dw"], tol["dw"] = (g * v * q).sum(0), (np.abs(g * v * q) * (e + depth)).sum(0)
    if delta is None:
        return res, tol
    x = delta.astype(np.float64)
    p = rms(x, eps) if post is not None else 1.0
    n = x * p * (1 if post is None else post)
    if scale is not None:
        res["dscale"], tol["dscale"] = (t * n).sum(0), (et * np.abs(n) + mt * np.abs(n) * (e + depth)).sum(0)
        t, et, mt = t * scale, et * np.abs(scale), mt * np.abs(scale)
    if post is not None:
        res["dw_post"], tol["dw_post"] = (t * x * p).sum(0), (np.abs(x * p) * (et + mt * (e + depth))).sum(0)
        t, et, mt = t * post, et * np.abs(post), mt * np.abs(post)
        b2, b2m = p * p * (t * x).mean(-1, keepdims=True), p * p * (mt * np.abs(x)).mean(-1, keepdims=True)
        eb = p * p * (et * np.abs(x)).mean(-1, keepdims=True)
        t = p * (t - x * b2)
        et = p * (et + np.abs(x) * eb) + p * (mt + np.abs(x) * b2m) * (e + 66 * U)
        mt = p * (mt + np.abs(x) * b2m)
    res["ddelta"], tol["ddelta"] = t, et + 2 * U * mt
    return res, tol


def gated_norm(o, z, w, first=False, eps=1e-6):
    """(y, bound) over the last dimension; w broadcasts."""
    v, z = o.astype(np.float64), z.astype(np.float64)
    gate = z * sigmoid(z)
    e = norm_error(0) + (2 * EXP * np.abs(z).max(-1, keepdims=True) + 24) * U
    y = (v * gate) * rms(v * gate, eps) * w if first else v * rms(v, eps) * w * gate
    return y, e * np.abs(y)


def gated_norm_grad(o, z, w, dy, first=False, eps=1e-6, shared=True):
    v, z, g = o.astype(np.float64), z.astype(np.float64), dy.astype(np.float64)
    sz = sigmoid(z)
    gate, slope, mslope = z * sz, sz + z * slope_of(z), sz + np.abs(z) * slope_of(z)
    u = v * gate if first else v
    q = rms(u, eps)
    n = u * q
    dn = g if first else g * gate
    back, back_m = (dn * w * n).mean(-1, keepdims=True), np.abs(dn * w * n).mean(-1, keepdims=True)
    du, mu = q * (dn * w - n * back), q * (np.abs(dn * w) + np.abs(n) * back_m)
    e = 3 * norm_error(0) + (6 * EXP * np.abs(z).max(-1, keepdims=True) + 80) * U
    dgate, mgate = (du * v, mu * np.abs(v)) if first else (g * n * w, np.abs(g * n * w))
    res = {"do": du * gate if first else du, "dz": dgate * slope}
    tol = {"do": e * (mu * np.abs(gate) if first else mu), "dz": e * mgate * mslope}
    rows = v.shape[0]
    axes = (0, 1) if shared else 0
    depth = ((v.shape[0] * (v.shape[1] if shared else 1)) + 64) * U
    res["dw"], tol["dw"] = (dn * n).sum(axes), ((e + depth) * np.abs(dn * n)).sum(axes)
    return res, tol
