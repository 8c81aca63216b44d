"""Thin ctypes binding of the layer operators (include/mamba_mi355x_layer.h): the short causal
convolution, one token of a layer, the norms around a block, verification of drafted tokens.

As in binding.py the functions keep the C names and only marshal torch tensors
(device memory, the current HIP stream) into the C ABI; there is no fallback.
"""
from __future__ import annotations

import ctypes

from .binding import MambaError, _io_dtype, load_library
from .lm import _arg, _reset_bytes, _stream, _workspace

_typed = None


def _lib():
    """The library with the argument types of mamba_mi355x_layer.h set."""
    global _typed
    if _typed is not None:
        return _typed
    lib = load_library()
    P, I64, I, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    for name, sizes in (("mamba_conv_bwd_workspace_size", 4), ("mamba_conv_ssm_update_workspace_size", 4),
                        ("mamba_residual_norm_bwd_workspace_size", 2), ("mamba_draft_verify_workspace_size", 3)):
        getattr(lib, name).argtypes = [I64] * sizes + [I]
        getattr(lib, name).restype = SZ
    lib.mamba_conv_fwd.argtypes = [I64] * 4 + [I] + [P] * 6 + [I, P, P, P]
    lib.mamba_conv_bwd.argtypes = [I64] * 4 + [I] + [P] * 5 + [I] + [P] * 6 + [P, SZ, P]
    lib.mamba_conv_update.argtypes = [I64] * 3 + [I, I64] + [P] * 5 + [I, P, P]
    lib.mamba_conv_ssm_update.argtypes = [I64] * 5 + [I, I64] + [P] * 13 + [P, SZ, P]
    lib.mamba_residual_norm_fwd.argtypes = [I64, I64, I, I, P, P, I, P, P, P, P, F, F, P, P, P]
    lib.mamba_residual_norm_bwd.argtypes = [I64, I64, I, I, P, P, I, P, P, P, P, F, F] + [P] * 8 + [P, SZ, P]
    lib.mamba_draft_verify.argtypes = [I64] * 3 + [I] + [P] * 8 + [P, SZ, P]
    for name in ("mamba_conv_fwd", "mamba_conv_bwd", "mamba_conv_update", "mamba_conv_ssm_update",
                 "mamba_residual_norm_fwd", "mamba_residual_norm_bwd", "mamba_draft_verify"):
        getattr(lib, name).restype = I
    _typed = lib
    return lib


def mamba_conv_fwd(x, weight, bias=None, window=None, reset=None, lengths=None, silu=True, out=None, last_window=None,
                   return_last_window=True):
    """Short causal convolution: c_t = bias + sum_j weight[:, j] x_{t-(W-1)+j}, out = SiLU(c) (c without silu).

    x: (batch, L, D) float32 or bfloat16; weight: (D, W) float32, W 2 to 4; bias: (D,) float32; window:
    (batch, W - 1, D), the inputs before the first; reset: (batch, L) bool or uint8, a row's first token of
    each document; lengths: (batch,) int32, rows padded behind them (out is zero there).
    Returns (out, last_window): the window with which the rows go on."""
    import torch

    lib = _lib()
    batch, L, D = x.shape
    W = weight.shape[1]
    io, dev, f32, t = _io_dtype(x), x.device, torch.float32, x.dtype
    shape, wshape = (batch, L, D), (batch, W - 1, D)
    out = torch.empty_like(x) if out is None else out
    if last_window is None and return_last_window:
        last_window = torch.empty(wshape, dtype=t, device=dev)
    st = lib.mamba_conv_fwd(
        batch, L, D, W, io, _arg(x, "x", t, shape, dev), _arg(weight, "weight", f32, (D, W), dev),
        _arg(bias, "bias", f32, (D,), dev), _arg(window, "window", t, wshape, dev),
        _reset_bytes(reset, (batch, L), dev), _arg(lengths, "lengths", torch.int32, (batch,), dev), int(bool(silu)),
        _arg(out, "out", t, shape, dev), _arg(last_window, "last_window", t, wshape, dev), _stream(dev))
    if st != 0:
        raise MambaError("mamba_conv_fwd", st)
    return out, last_window


def mamba_conv_bwd_workspace_size(batch: int, seqlen: int, dim: int, width: int, io_dtype: int) -> int:
    return int(_lib().mamba_conv_bwd_workspace_size(batch, seqlen, dim, width, io_dtype))


def mamba_conv_bwd(x, weight, dout, bias=None, window=None, reset=None, silu=True, dlast_window=None, grads=None,
                   workspace=None, want=("dbias", "dwindow")):
    """Gradients of sum(dout * out) + sum(dlast_window * last_window) of mamba_conv_fwd (without lengths).

    Returns a dict with dx, dweight and those of dbias and dwindow named in ``want``.  Preallocated
    outputs may be passed in ``grads`` (same keys)."""
    import torch

    lib = _lib()
    batch, L, D = x.shape
    W = weight.shape[1]
    io, dev, f32, t = _io_dtype(x), x.device, torch.float32, x.dtype
    shape, wshape = (batch, L, D), (batch, W - 1, D)
    like = {"dx": (shape, t), "dweight": ((D, W), f32), "dbias": ((D,), f32), "dwindow": (wshape, t)}
    need = ["dx", "dweight"] + list(want)
    g = dict(grads or {})
    for k in need:
        if k not in g:
            g[k] = torch.empty(like[k][0], dtype=like[k][1], device=dev)
    workspace, ws, ws_bytes = _workspace(workspace, lib.mamba_conv_bwd_workspace_size(batch, L, D, W, io), dev)

    def gp(k):
        return _arg(g[k], k, like[k][1], like[k][0], dev) if k in g else None

    st = lib.mamba_conv_bwd(
        batch, L, D, W, io, _arg(x, "x", t, shape, dev), _arg(weight, "weight", f32, (D, W), dev),
        _arg(bias, "bias", f32, (D,), dev), _arg(window, "window", t, wshape, dev),
        _reset_bytes(reset, (batch, L), dev), int(bool(silu)), _arg(dout, "dout", t, shape, dev),
        _arg(dlast_window, "dlast_window", t, wshape, dev), gp("dx"), gp("dweight"), gp("dbias"), gp("dwindow"), ws,
        ws_bytes, _stream(dev))
    if st != 0:
        raise MambaError("mamba_conv_bwd", st)
    return {k: g[k] for k in need}


def mamba_conv_update(window, x, weight, bias=None, slots=None, silu=True, out=None):
    """One token of mamba_conv_fwd in place on window (nslots, W - 1, D); x: (batch, D).  slots: (batch,) int32,
    the window of each row (None: row b has window b), negative for an idle row, whose out is left as it was."""
    import torch

    lib = _lib()
    batch, D = x.shape
    nslots, W = window.shape[0], weight.shape[1]
    io, dev, f32, t = _io_dtype(x), x.device, torch.float32, x.dtype
    out = torch.empty_like(x) if out is None else out
    st = lib.mamba_conv_update(
        batch, D, W, io, nslots, _arg(window, "window", t, (nslots, W - 1, D), dev), _arg(x, "x", t, (batch, D), dev),
        _arg(weight, "weight", f32, (D, W), dev), _arg(bias, "bias", f32, (D,), dev),
        _arg(slots, "slots", torch.int32, (batch,), dev), int(bool(silu)), _arg(out, "out", t, (batch, D), dev),
        _stream(dev))
    if st != 0:
        raise MambaError("mamba_conv_update", st)
    return out


def mamba_conv_ssm_update_workspace_size(batch: int, dim: int, dstate: int, dt_rank: int, io_dtype: int) -> int:
    return int(_lib().mamba_conv_ssm_update_workspace_size(batch, dim, dstate, dt_rank, io_dtype))


def mamba_conv_ssm_update(state, window, x, conv_weight, W_x, W_dt, A, conv_bias=None, z=None, dt_bias=None,
                          Dskip=None, slots=None, out=None, workspace=None):
    """One token of a layer from its input projection on, in place on state (nslots, D, N) float32 and window
    (nslots, W - 1, D): the convolution with SiLU, the selection projections (W_x (R + 2N, D), W_dt (D, R)) and
    the state update, with fp32 values between them.  x, z: (batch, D); slots as for mamba_conv_update."""
    import torch

    lib = _lib()
    batch, D = x.shape
    nslots, W, N, R = state.shape[0], conv_weight.shape[1], A.shape[1], W_dt.shape[1]
    io, dev, f32, t = _io_dtype(x), x.device, torch.float32, x.dtype
    out = torch.empty_like(x) if out is None else out
    workspace, ws, ws_bytes = _workspace(workspace, lib.mamba_conv_ssm_update_workspace_size(batch, D, N, R, io), dev)
    st = lib.mamba_conv_ssm_update(
        batch, D, N, R, W, io, nslots, _arg(state, "state", f32, (nslots, D, N), dev),
        _arg(window, "window", t, (nslots, W - 1, D), dev), _arg(x, "x", t, (batch, D), dev),
        _arg(conv_weight, "conv_weight", f32, (D, W), dev), _arg(conv_bias, "conv_bias", f32, (D,), dev),
        _arg(W_x, "W_x", t, (R + 2 * N, D), dev), _arg(W_dt, "W_dt", t, (D, R), dev),
        _arg(dt_bias, "dt_bias", f32, (D,), dev), _arg(A, "A", f32, (D, N), dev), _arg(Dskip, "Dskip", f32, (D,), dev),
        _arg(z, "z", t, (batch, D), dev), _arg(slots, "slots", torch.int32, (batch,), dev),
        _arg(out, "out", t, (batch, D), dev), ws, ws_bytes, _stream(dev))
    if st != 0:
        raise MambaError("mamba_conv_ssm_update", st)
    return out


def mamba_residual_norm_fwd(x, pre_weight=None, gate=None, post_weight=None, scale=None, residual=None, alpha=1.0,
                            eps=1e-5, gate_first=True, out=None, residual_out=None, res_dtype=None,
                            return_residual=True):
    """The norm behind a block with its gate, the residual sum, and the norm before the next block:
    p = post_weight v / rms(v) with v = x SiLU(gate) (gate_first=False: v = x and p times SiLU(gate)),
    residual_out = residual + alpha scale p, out = pre_weight residual_out / rms(residual_out).

    x, gate: (..., D) float32 or bfloat16; residual: the same shape, x's type or float32; the weights and scale:
    (D,) float32.  None leaves that part out.  Returns (out, residual_out); out is None without pre_weight.
    res_dtype: residual_out's type where neither residual nor residual_out gives it (default: x's)."""
    import torch

    lib = _lib()
    shape, D = x.shape, x.shape[-1]
    rows = x.numel() // D if D else 0
    io, dev, f32, t = _io_dtype(x), x.device, torch.float32, x.dtype
    rt = residual.dtype if residual is not None else residual_out.dtype if residual_out is not None else res_dtype or t
    if residual_out is None and return_residual:
        residual_out = torch.empty(shape, dtype=rt, device=dev)
    if pre_weight is None:
        out = None
    elif out is None:
        out = torch.empty_like(x)
    st = lib.mamba_residual_norm_fwd(
        rows, D, io, _res_dtype(rt, t), _arg(x, "x", t, shape, dev), _arg(gate, "gate", t, shape, dev),
        int(bool(gate_first)), _arg(post_weight, "post_weight", f32, (D,), dev), _arg(scale, "scale", f32, (D,), dev),
        _arg(residual, "residual", rt, shape, dev), _arg(pre_weight, "pre_weight", f32, (D,), dev), alpha, eps,
        _arg(residual_out, "residual_out", rt, shape, dev), _arg(out, "out", t, shape, dev), _stream(dev))
    if st != 0:
        raise MambaError("mamba_residual_norm_fwd", st)
    return out, residual_out


def _res_dtype(rt, t):
    import torch

    if rt not in (t, torch.float32):
        raise TypeError(f"residual must be {t} or {torch.float32}, got {rt}")
    return 0 if rt == torch.float32 else 1


def mamba_residual_norm_bwd_workspace_size(rows: int, dim: int, io_dtype: int) -> int:
    return int(_lib().mamba_residual_norm_bwd_workspace_size(rows, dim, io_dtype))


def mamba_residual_norm_bwd(x, pre_weight=None, dout=None, dresidual_out=None, gate=None, post_weight=None, scale=None,
                            residual=None, alpha=1.0, eps=1e-5, gate_first=True, grads=None, workspace=None,
                            res_dtype=None, want=("dgate", "dresidual", "dpost_weight", "dscale", "dpre_weight")):
    """Gradients of sum(dout * out) + sum(dresidual_out * residual_out) of mamba_residual_norm_fwd from its inputs.

    dout is given exactly with pre_weight.  Returns a dict with dx and, of those named in ``want``, the
    gradients of the inputs that are given.  Preallocated outputs may be passed in ``grads`` (same keys)."""
    import torch

    lib = _lib()
    shape, D = x.shape, x.shape[-1]
    rows = x.numel() // D if D else 0
    io, dev, f32, t = _io_dtype(x), x.device, torch.float32, x.dtype
    if (dout is None) != (pre_weight is None):
        raise ValueError("dout and pre_weight go together")
    rt = residual.dtype if residual is not None else dresidual_out.dtype if dresidual_out is not None \
        else res_dtype or t
    like = {"dx": (shape, t), "dgate": (shape, t), "dresidual": (shape, rt), "dpost_weight": ((D,), f32),
            "dscale": ((D,), f32), "dpre_weight": ((D,), f32)}
    given = {"dgate": gate, "dresidual": residual, "dpost_weight": post_weight, "dscale": scale,
             "dpre_weight": pre_weight}
    need = ["dx"] + [k for k in want if given[k] is not None]
    g = dict(grads or {})
    for k in need:
        if k not in g:
            g[k] = torch.empty(like[k][0], dtype=like[k][1], device=dev)
    workspace, ws, ws_bytes = _workspace(workspace, lib.mamba_residual_norm_bwd_workspace_size(rows, D, io), dev)

    def gp(k):
        return _arg(g[k], k, like[k][1], like[k][0], dev) if k in need else None

    st = lib.mamba_residual_norm_bwd(
        rows, D, io, _res_dtype(rt, t), _arg(x, "x", t, shape, dev), _arg(gate, "gate", t, shape, dev),
        int(bool(gate_first)), _arg(post_weight, "post_weight", f32, (D,), dev), _arg(scale, "scale", f32, (D,), dev),
        _arg(residual, "residual", rt, shape, dev), _arg(pre_weight, "pre_weight", f32, (D,), dev), alpha, eps,
        _arg(dout, "dout", t, shape, dev), _arg(dresidual_out, "dresidual_out", rt, shape, dev), gp("dx"), gp("dgate"),
        gp("dresidual"), gp("dpost_weight"), gp("dscale"), gp("dpre_weight"), ws, ws_bytes, _stream(dev))
    if st != 0:
        raise MambaError("mamba_residual_norm_bwd", st)
    return {k: g[k] for k in need}


def mamba_draft_verify_workspace_size(rows: int, drafts: int, vocab: int, io_dtype: int) -> int:
    return int(_lib().mamba_draft_verify_workspace_size(rows, drafts, vocab, io_dtype))


def mamba_draft_verify(target, draft, drafted, uniform, noise, counts=None, tokens=None, accepted=None,
                       workspace=None):
    """Drafted tokens against the target's probabilities: draft k stays while uniform q(d) < p(d); behind the kept
    ones a token drawn from max(p - q, 0) (or from p behind the last draft) with Exp(1) noise.

    target: (rows, K + 1, vocab), draft: (rows, K, vocab) float32 or bfloat16; drafted: (rows, K) int64; uniform:
    (rows, K) and noise: (rows, vocab) float32; counts: (rows,) int32, drafts of each row (None: K).
    Returns (tokens int64 (rows, K + 1), -1 behind the drawn one, accepted int32 (rows,))."""
    import torch

    lib = _lib()
    rows, K, V = draft.shape
    io, dev, f32, t = _io_dtype(target), target.device, torch.float32, target.dtype
    tokens = torch.empty((rows, K + 1), dtype=torch.int64, device=dev) if tokens is None else tokens
    accepted = torch.empty((rows,), dtype=torch.int32, device=dev) if accepted is None else accepted
    workspace, ws, ws_bytes = _workspace(workspace, lib.mamba_draft_verify_workspace_size(rows, K, V, io), dev)
    st = lib.mamba_draft_verify(
        rows, K, V, io, _arg(target, "target", t, (rows, K + 1, V), dev), _arg(draft, "draft", t, (rows, K, V), dev),
        _arg(drafted, "drafted", torch.int64, (rows, K), dev), _arg(uniform, "uniform", f32, (rows, K), dev),
        _arg(noise, "noise", f32, (rows, V), dev), _arg(counts, "counts", torch.int32, (rows,), dev),
        _arg(tokens, "tokens", torch.int64, (rows, K + 1), dev),
        _arg(accepted, "accepted", torch.int32, (rows,), dev), ws, ws_bytes, _stream(dev))
    if st != 0:
        raise MambaError("mamba_draft_verify", st)
    return tokens, accepted
