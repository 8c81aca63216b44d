"""Plain fp64 implementations of the token-model operators, token after token and row after row,
for the tests.  Shares no code with the library or with perf/operators.py."""
from __future__ import annotations

import math

import numpy as np


def _sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def _softplus(v):
    return np.logaddexp(0.0, v)


def _coefficients(u, ra, rx, lam, c, reset):
    l = -c * _softplus(lam) * _sigmoid(ra)
    a, s = np.exp(l), np.sqrt(-np.expm1(2 * l))
    if reset is not None:
        cut = np.asarray(reset, bool)[..., None]
        a, s = np.where(cut, 0.0, a), np.where(cut, 1.0, s)
    return l, a, s


def gated_fwd(u, ra, rx, lam, c, z=None, reset=None, h0=None):
    """out, last_state, and every state (batch, L + 1, D) with the initial one first."""
    batch, L, D = u.shape
    _, a, s = _coefficients(u, ra, rx, lam, c, reset)
    h = np.zeros((batch, D)) if h0 is None else h0.astype(np.float64)
    states = [h]
    for t in range(L):
        b = s[:, t] * _sigmoid(rx[:, t]) * u[:, t]
        h = np.where(a[:, t] == 0, 0.0, a[:, t] * h) + b
        states.append(h)
    states = np.stack(states, 1)
    out = states[:, 1:]
    if z is not None:
        out = out * z * _sigmoid(z)
    return out, states[:, -1], states


def gated_bwd(u, ra, rx, lam, c, dout, dlast=None, z=None, reset=None, h0=None):
    """The chain rule, last token first."""
    batch, L, D = u.shape
    l, a, s = _coefficients(u, ra, rx, lam, c, reset)
    _, _, states = gated_fwd(u, ra, rx, lam, c, z, reset, h0)
    live = np.ones((batch, L, 1), bool) if reset is None else ~np.asarray(reset, bool)[..., None]
    g = {k: np.zeros((batch, L, D)) for k in ("du", "dgate_a", "dgate_x", "dz")}
    dlam = np.zeros(D)
    dh = np.zeros((batch, D)) if dlast is None else dlast.astype(np.float64)
    kappa = c * _softplus(lam)
    for t in range(L - 1, -1, -1):
        dy = dout[:, t]
        if z is not None:
            sz = _sigmoid(z[:, t])
            g["dz"][:, t] = dy * states[:, t + 1] * (sz + z[:, t] * sz * (1 - sz))
            dy = dy * z[:, t] * sz
        dh = dh + dy
        sx, sa = _sigmoid(rx[:, t]), _sigmoid(ra[:, t])
        g["du"][:, t] = dh * s[:, t] * sx
        g["dgate_x"][:, t] = dh * s[:, t] * u[:, t] * sx * (1 - sx)
        with np.errstate(divide="ignore", invalid="ignore"):
            ds = np.where(s[:, t] > 0, -a[:, t] ** 2 / s[:, t], 0.0)  # ds/dl
        dl = np.where(live[:, t], dh * (a[:, t] * states[:, t] + ds * sx * u[:, t]), 0.0)
        g["dgate_a"][:, t] = dl * -kappa * sa * (1 - sa)
        dlam += (dl * -c * _sigmoid(lam) * sa).sum(0)
        dh = np.where(live[:, t], a[:, t] * dh, 0.0)
    if z is None:
        del g["dz"]
    return {**g, "dlam": dlam, "dh0": dh}


def embed_fwd(ids, weight, scale):
    out = np.zeros((ids.size, weight.shape[1]))
    for i, v in enumerate(ids.ravel()):
        if v >= weight.shape[0]:
            out[i] = np.nan
        elif v >= 0:
            out[i] = scale * weight[v].astype(np.float64)
    return out.reshape(*ids.shape, weight.shape[1])


def embed_bwd(ids, dout, vocab, scale):
    g = np.zeros((vocab, dout.shape[-1]))
    flat = dout.reshape(-1, dout.shape[-1]).astype(np.float64)
    for i, v in enumerate(ids.ravel()):
        if 0 <= v < vocab:
            g[v] += flat[i]
    return g * scale


def sample_row(x, noise, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, kept indices) of one row, by sorting it."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    m = x.max()
    if m == -np.inf:
        return -1, -np.inf, []
    if not temperature > 0 or top_p <= 0:
        top_k = 1
    t = temperature if temperature > 0 else 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == m, 1.0, np.exp((x - m) / t))
    w[x == -np.inf] = 0.0
    order = [i for i in sorted(range(x.size), key=lambda i: (-x[i], i)) if x[i] > -np.inf]
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        total, before, keep = math.fsum(w[i] for i in order), 0.0, []
        for i in order:
            if keep and not before < top_p * total:
                break
            keep.append(i)
            before += w[i]
        order = keep
    if min_p > 0:
        order = [i for i in order if w[i] >= min(min_p, 1.0)]
    order = sorted(i for i in order if w[i] > 0)
    best, token = None, -1
    for i in order:
        with np.errstate(divide="ignore"):
            sc = np.float64(w[i]) / np.float64(noise[i])
        sc = -np.inf if np.isnan(sc) else sc
        if best is None or sc > best:
            best, token = sc, i
    return token, math.log(w[token]) - math.log(math.fsum(w[i] for i in order)), order
