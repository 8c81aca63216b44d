"""Plain fp64 implementations of the layer operators, token after token and row after row, for the tests, and the
magnitudes from which their tolerances follow.  Shares no code with the library or with perf/more_operators.py.

A tolerance is |got - ref| <= h |ref| + 2^-24 m: h is half a step of the output's type, m the sum of the
magnitudes that enter an output, each times the number of fp32 roundings that reach it."""
from __future__ import annotations

import numpy as np

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
U = 2.0 ** -24


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def silu(v):
    return v * sigmoid(v)


def silu_slope(v):
    s = sigmoid(v)
    return s * (1 + v * (1 - s))


def close(got, ref, mag, io):
    """The largest excess over the tolerance, as a multiple of it (at most 1 where all is well)."""
    got, ref, mag = (np.asarray(v, np.float64) for v in (got, ref, mag))
    assert got.shape == ref.shape, (got.shape, ref.shape)
    if got.size == 0:
        return 0.0
    tol = HALF[io] * (1 + 1e-3) * np.abs(ref) + U * np.broadcast_to(mag, ref.shape)
    bad = ~np.isfinite(got)
    off = np.where(bad, np.inf, np.abs(got - ref))
    return float(np.max(off / np.maximum(tol, 1e-300)))


# ------------------------------------------------------------------------------------------ convolution


def conv_full(x, window, W):
    batch, _, D = x.shape
    before = np.zeros((batch, W - 1, D)) if window is None else window
    return np.concatenate([before, x], 1)


def conv_reach(reset, batch, L, W):
    """reach[b, t, o]: whether token t sees the input o tokens back."""
    reach = np.ones((batch, L, W), bool)
    if reset is not None:
        for b in range(batch):
            for t in range(L):
                for o in range(1, W):
                    reach[b, t, o] = not any(reset[b, s] for s in range(max(0, t - o + 1), t + 1))
    return reach


def conv_fwd(x, w, bias=None, window=None, reset=None, lengths=None, act=True):
    """out, last_window, c, and the magnitude of out's error."""
    batch, L, D = x.shape
    W = w.shape[1]
    full, reach = conv_full(x, window, W), conv_reach(reset, batch, L, W)
    c = np.zeros((batch, L, D)) + (0 if bias is None else bias)
    mag = np.abs(c)
    for b in range(batch):
        for t in range(L):
            for o in range(W):
                if reach[b, t, o]:
                    c[b, t] += w[:, W - 1 - o] * full[b, t + W - 1 - o]
                    mag[b, t] += np.abs(w[:, W - 1 - o] * full[b, t + W - 1 - o])
    n = [L if lengths is None else min(max(int(lengths[b]), 0), L) for b in range(batch)]
    out = silu(c) if act else c.copy()
    # W + 1 roundings of the sum through a slope of at most 1.1, then SiLU itself: the exponent's rounding
    # is |c| units, exp2, the sum, the reciprocal and the product seven
    m = 1.1 * (W + 1) * mag + (np.abs(out) * (np.abs(c) + 8) if act else 0)
    last = np.zeros((batch, W - 1, D))
    for b in range(batch):
        out[b, n[b]:] = 0
        m[b, n[b]:] = 0
        for j in range(W - 1):
            pos = n[b] - (W - 1) + j
            if reset is None or not any(reset[b, s] for s in range(max(0, pos + 1), n[b])):
                last[b, j] = full[b, pos + W - 1]
    return out, last, c, m


def conv_bwd(x, w, dout, bias=None, window=None, reset=None, act=True, dlast=None):
    """Gradients and the magnitudes of their errors."""
    batch, L, D = x.shape
    W = w.shape[1]
    full, reach = conv_full(x, window, W), conv_reach(reset, batch, L, W)
    _, _, c, m = conv_fwd(x, w, bias, window, reset, None, act)
    _, _, _, s = conv_fwd(np.abs(x), np.abs(w), None if bias is None else np.abs(bias),
                          None if window is None else np.abs(window), reset, None, False)
    g = dout * (silu_slope(c) if act else 1)
    # SiLU' has a slope of at most 0.5 at c's error; its own evaluation is off by 12 + 2 |c| units at most
    gm = np.abs(dout) * (0.5 * s + 12 + 2 * np.abs(c)) if act else np.zeros_like(g)
    gm = gm + 2 * np.abs(g)
    dfull, dm = np.zeros_like(full), np.zeros_like(full)
    dw, dwm = np.zeros((D, W)), np.zeros((D, W))
    # part sums of up to 128 tokens, every 32nd part, 32 sums
    depth = 128 + 32 + batch * L / 8 / 32 + 4
    for b in range(batch):
        for t in range(L):
            for o in range(W):
                if reach[b, t, o]:
                    j, at = W - 1 - o, t + W - 1 - o
                    dfull[b, at] += w[:, j] * g[b, t]
                    dm[b, at] += np.abs(w[:, j]) * (gm[b, t] + (W + 2) * np.abs(g[b, t]))
                    dw[:, j] += g[b, t] * full[b, at]
                    dwm[:, j] += np.abs(full[b, at]) * (gm[b, t] + depth * np.abs(g[b, t]))
    if dlast is not None:
        for b in range(batch):
            for j in range(W - 1):
                pos = L - (W - 1) + j
                if reset is None or not any(reset[b, s] for s in range(max(0, pos + 1), L)):
                    dfull[b, pos + W - 1] += dlast[b, j]
                    dm[b, pos + W - 1] += (W + 2) * np.abs(dlast[b, j])
    res = {"dx": (dfull[:, W - 1:], dm[:, W - 1:]), "dwindow": (dfull[:, :W - 1], dm[:, :W - 1]), "dweight": (dw, dwm),
           "dbias": (g.sum((0, 1)), (gm + depth * np.abs(g)).sum((0, 1)))}
    return res


# ------------------------------------------------------------------------------------------ one token


def softplus(v):
    return np.logaddexp(0.0, v)


def conv_ssm_step(state, window, x, cw, cb, Wx, Wdt, A, z=None, dt_bias=None, Dskip=None, slots=None, out=None):
    """state, window and out behind the token; idle rows leave theirs."""
    batch, D = x.shape
    N, R, W = A.shape[1], Wdt.shape[1], cw.shape[1]
    state, window = state.copy(), window.copy()
    out = np.zeros((batch, D)) if out is None else out.copy()
    for b in range(batch):
        s = b if slots is None else int(slots[b])
        if s < 0 or s >= state.shape[0]:
            continue
        full = np.concatenate([window[s], x[b:b + 1]])
        xc = silu((full * cw.T).sum(0) + (0 if cb is None else cb))
        p = Wx @ xc
        dt = softplus(Wdt @ p[:R] + (0 if dt_bias is None else dt_bias))[:, None]
        safe = np.where(A == 0, 1.0, A)
        weight = np.where(A == 0, dt, np.expm1(dt * A) / safe)
        state[s] = np.exp(dt * A) * state[s] + weight * p[None, R:R + N] * xc[:, None]
        y = (state[s] * p[None, R + N:]).sum(1) + (0 if Dskip is None else Dskip * xc)
        out[b] = y if z is None else y * silu(z[b])
        window[s] = full[1:]
    return state, window, out


# ------------------------------------------------------------------------------------------ norms


def norm_parts(x, pre=None, gate=None, post=None, scale=None, residual=None, alpha=1.0, eps=1e-5, gate_first=True):
    D = x.shape[1]
    s = np.ones_like(x) if gate is None else silu(gate)
    v = x * s if gate_first else x
    k = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps) if post is not None else np.ones((x.shape[0], 1))
    f = (1 if post is None else post) * (1 if gate_first else s) * np.ones(D)
    n = v * k
    p = n * f
    q = alpha * (1 if scale is None else scale) * p
    r = q + (0 if residual is None else residual)
    K = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    return s, v, k, f, n, p, q, r, K


def norm_fwd(x, pre=None, **kw):
    """out (None without pre), residual_out, and the magnitudes of their errors."""
    s, v, k, f, n, p, q, r, K = norm_parts(x, pre, **kw)
    gate = kw.get("gate")
    # a square sum is at most 64 terms a lane and 15 sums over lanes, so 1 / rms is within half of 80 units
    # and two of its own; SiLU 8 + |gate|, products and the sum ten
    e = 60 + 8 + 10 + (0 if gate is None else np.abs(gate))
    rm = np.abs(q) * e + np.abs(r)
    if pre is None:
        return None, r, None, rm
    out = pre * r * K
    # K's error: that of r in the norm, and its own 45 units
    rel = np.sqrt((rm * rm).sum(1, keepdims=True) / np.maximum((r * r).sum(1, keepdims=True), 1e-300))
    return out, r, np.abs(pre) * K * rm + np.abs(out) * (50 + rel), rm


def norm_bwd(x, pre=None, dout=None, dres=None, gate=None, post=None, scale=None, residual=None, alpha=1.0, eps=1e-5,
             gate_first=True):
    """Gradients and the magnitudes of their errors."""
    s, v, k, f, n, p, q, r, K = norm_parts(x, pre, gate, post, scale, residual, alpha, eps, gate_first)
    a = alpha * (1 if scale is None else scale) * np.ones(x.shape[1])
    dr, M = (np.zeros_like(x), np.zeros_like(x)) if dres is None else (dres.copy(), np.abs(dres))
    g = {}
    # r's own relative error matters where the residual cancels the block's output: in units of |q| + |r|
    big = np.abs(q) + np.abs(r)
    if pre is not None:
        dn = dout * pre
        dr = dr + K * (dn - r * K * K * (dn * r).mean(1, keepdims=True))
        M = M + K * (np.abs(dn) + big * K * K * (np.abs(dn) * big).mean(1, keepdims=True)) * \
            (1 + K * np.sqrt((big * big).mean(1, keepdims=True)))
        g["dpre_weight"] = ((dout * r * K).sum(0), (np.abs(dout) * K * big *
                            (1 + K * np.sqrt((big * big).mean(1, keepdims=True)))).sum(0))
    if residual is not None:
        g["dresidual"] = dr, M
    if scale is not None:
        g["dscale"] = alpha * (dr * p).sum(0), abs(alpha) * (M * np.abs(p)).sum(0)
    dp, Mp = dr * a, M * np.abs(a)
    e, Me = dp * f, Mp * np.abs(f)
    if post is not None:
        w = 1 if gate_first else s
        g["dpost_weight"] = (dp * w * n).sum(0), (Mp * np.abs(w) * np.abs(n)).sum(0)
        dv = k * (e - n * (e * n).mean(1, keepdims=True))
        Mv = k * (Me + np.abs(n) * (Me * np.abs(n)).mean(1, keepdims=True))
    else:
        dv, Mv = e, Me
    if gate is not None and gate_first:
        g["dx"] = dv * s, Mv * np.abs(s)
        g["dgate"] = dv * x * silu_slope(gate), Mv * np.abs(x) * (1 + np.abs(gate) / 50)
    else:
        g["dx"] = dv, Mv
        if gate is not None:
            pp = 1 if post is None else post
            g["dgate"] = dp * pp * n * silu_slope(gate), Mp * np.abs(pp) * np.abs(n) * (1 + np.abs(gate) / 50)
    # every factor is within 80 units (norms: 45; SiLU: 8 + |gate|; sums: 80), and no gradient has more than
    # five of them; the sums over rows add as many as a workgroup has rows, and 32 twice
    rows = x.shape[0]
    return {key: (val, mag * (400 + (rows / 768 + 64 + 8 if val.ndim == 1 else 0))) for key, (val, mag) in g.items()}


# ------------------------------------------------------------------------------------------ verification


def verify_row(p, q, drafted, uniform, noise, count):
    """tokens and the number kept of one row, in the fp32 steps that the interface names; p (K + 1, V), q (K, V)."""
    K, V = q.shape
    count = min(max(int(count), 0), K)
    f32 = np.float32
    kept, tokens = 0, np.full(K + 1, -1, np.int64)
    while kept < count and 0 <= drafted[kept] < V and \
            f32(uniform[kept]) * f32(q[kept, drafted[kept]]) < f32(p[kept, drafted[kept]]):
        tokens[kept] = drafted[kept]
        kept += 1
    w = p[kept].astype(f32)
    if kept < count:
        with np.errstate(invalid="ignore"):
            rest = w - q[kept].astype(f32)
        if (rest > 0).any():
            w = rest
    best, at = None, -1
    with np.errstate(divide="ignore", invalid="ignore"):
        score = np.where(noise >= 0, w / np.abs(noise.astype(f32)), f32(-np.inf))
        score = np.where(np.isnan(score), f32(-np.inf), score)
    for i in np.flatnonzero(w > 0):
        if best is None or score[i] > best:
            best, at = score[i], i
    tokens[kept] = at
    return tokens, kept
