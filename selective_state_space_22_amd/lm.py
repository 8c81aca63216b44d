"""Thin ctypes binding of the token-model operators (include/mamba_mi355x_lm.h):
embedding lookup and gradient, the gated linear recurrence, sampling.

As in binding.py the functions keep the C names and only marshal torch tensors
(device memory, the current HIP stream) into the C ABI; there is no fallback.
"""
from __future__ import annotations

import ctypes

from .binding import MambaError, _check_status, _io_dtype, _ptr, load_library

MAMBA_GATED_STATE_CHUNK = 8

_typed = None


def _lib():
    """The library with the argument types of mamba_mi355x_lm.h set."""
    global _typed
    if _typed is not None:
        return _typed
    lib = load_library()
    P, I64, I, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    for name in ("mamba_gated_scan_fwd_workspace_size", "mamba_gated_scan_bwd_workspace_size",
                 "mamba_embed_bwd_workspace_size"):
        getattr(lib, name).argtypes = [I64, I64, I64, I]
        getattr(lib, name).restype = SZ
    lib.mamba_gated_scan_fwd.argtypes = [I64, I64, I64, I, P, P, P, P, F, P, P, P, P, P, P, P, SZ, P]
    lib.mamba_gated_scan_bwd.argtypes = [I64, I64, I64, I, P, P, P, P, F] + [P] * 13 + [SZ, P]
    lib.mamba_gated_state_update.argtypes = [I64, I64, I, P, P, P, P, P, F, P, P, P, P]
    lib.mamba_embed_fwd.argtypes = [I64, I64, I64, I, P, P, F, P, P]
    lib.mamba_embed_bwd.argtypes = [I64, I64, I64, I, P, P, F, P, P, SZ, P]
    lib.mamba_sample.argtypes = [I64, I64, I, P, P, P, P, P, P, P, P, P]
    for name in ("mamba_gated_scan_fwd", "mamba_gated_scan_bwd", "mamba_gated_state_update", "mamba_embed_fwd",
                 "mamba_embed_bwd", "mamba_sample"):
        getattr(lib, name).restype = I
    _typed = lib
    return lib


# A call on one token is as long as its checks: a tensor that is as expected costs one condition here,
# _ptr names what is wrong with any other (decode of 1 x 2560: 10.1 us a call with _ptr alone, 7.5 so).
def _arg(t, name, dtype, shape, device):
    """Device pointer of a contiguous tensor of that type, shape and device (None -> NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda and t.is_contiguous() and t.numel():
        return t.data_ptr()
    return _ptr(t, name, dtype, shape, device)


def _stream(device):
    import torch

    return torch._C._cuda_getCurrentRawStream(device.index)


def _workspace(workspace, need, device):
    """(tensor, pointer, bytes) of the caller's workspace, or of a new one where need > 0."""
    import torch

    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, _ptr(workspace, "workspace", device=device), workspace.numel() * workspace.element_size()


def _reset_bytes(reset, shape, device):
    """Pointer of a bool or uint8 tensor."""
    import torch

    if reset is None:
        return None
    if reset.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"reset must be bool or uint8, got {reset.dtype}")
    return _ptr(reset, "reset", None, shape, device)


def mamba_gated_scan_fwd_workspace_size(batch: int, seqlen: int, dim: int, io_dtype: int) -> int:
    return int(_lib().mamba_gated_scan_fwd_workspace_size(batch, seqlen, dim, io_dtype))


def mamba_gated_scan_fwd(u, gate_a, gate_x, lam, z=None, h0=None, reset=None, c=8.0, out=None, last_state=None,
                         states=None, workspace=None, return_last_state=True, return_states=False, check=False):
    """Gated linear recurrence over whole sequences: with a = exp(-c softplus(lam) sigmoid(gate_a)),
    h = a h + sqrt(1 - a^2) sigmoid(gate_x) u and out = h SiLU(z) (h without z); reset tokens start anew.

    u, gate_a, gate_x, z: (batch, L, D) float32 or bfloat16; lam: (D,) float32; h0: (batch, D) float32;
    reset: (batch, L) bool or uint8.  Returns (out, last_state), and with return_states=True also the
    states that mamba_gated_scan_bwd takes, (batch, ceil(L / 8), D) float32.
    check=True synchronises the stream and raises MambaError if a wait between sequence chunks gave up."""
    import torch

    lib = _lib()
    batch, L, D = u.shape
    io, dev, f32, t = _io_dtype(u), u.device, torch.float32, u.dtype
    shape = (batch, L, D)
    out = torch.empty_like(u) if out is None else out
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, D), dtype=f32, device=dev)
    chunks = -(-L // MAMBA_GATED_STATE_CHUNK)
    if states is None and return_states:
        states = torch.empty((batch, chunks, D), dtype=f32, device=dev)
    workspace, ws, ws_bytes = _workspace(workspace, lib.mamba_gated_scan_fwd_workspace_size(batch, L, D, io), dev)
    st = lib.mamba_gated_scan_fwd(
        batch, L, D, io, _arg(u, "u", t, shape, dev), _arg(gate_a, "gate_a", t, shape, dev),
        _arg(gate_x, "gate_x", t, shape, dev), _arg(lam, "lam", f32, (D,), dev), c, _arg(z, "z", t, shape, dev),
        _reset_bytes(reset, (batch, L), dev), _arg(h0, "h0", f32, (batch, D), dev), _arg(out, "out", t, shape, dev),
        _arg(last_state, "last_state", f32, (batch, D), dev), _arg(states, "states", f32, (batch, chunks, D), dev),
        ws, ws_bytes, _stream(dev))
    if st != 0:
        raise MambaError("mamba_gated_scan_fwd", st)
    if check:
        _check_status("mamba_gated_scan_fwd", dev)
    return (out, last_state, states) if return_states else (out, last_state)


def mamba_gated_scan_bwd_workspace_size(batch: int, seqlen: int, dim: int, io_dtype: int) -> int:
    return int(_lib().mamba_gated_scan_bwd_workspace_size(batch, seqlen, dim, io_dtype))


def mamba_gated_scan_bwd(u, gate_a, gate_x, lam, dout, z=None, h0=None, reset=None, c=8.0, states=None,
                         dlast_state=None, grads=None, workspace=None, want=("dz", "dh0"), check=False):
    """Gradients of sum(dout * out) + sum(dlast_state * last_state) of mamba_gated_scan_fwd.

    states: what the forward returned with return_states=True from the same inputs (None: computed again).
    Returns a dict with du, dgate_a, dgate_x, dlam and those of dz (only with z) and dh0 named in ``want``.
    Preallocated outputs may be passed in ``grads`` (same keys)."""
    import torch

    lib = _lib()
    batch, L, D = u.shape
    io, dev, f32, t = _io_dtype(u), u.device, torch.float32, u.dtype
    shape = (batch, L, D)
    like = {"du": (shape, t), "dgate_a": (shape, t), "dgate_x": (shape, t), "dlam": ((D,), f32), "dz": (shape, t),
            "dh0": ((batch, D), f32)}
    need = ["du", "dgate_a", "dgate_x", "dlam"] + [k for k in want if k != "dz" or z is not None]
    g = dict(grads or {})
    for k in need:
        if k not in g:
            g[k] = torch.empty(like[k][0], dtype=like[k][1], device=dev)
    chunks = -(-L // MAMBA_GATED_STATE_CHUNK)
    workspace, ws, ws_bytes = _workspace(workspace, lib.mamba_gated_scan_bwd_workspace_size(batch, L, D, io), dev)

    def gp(k):
        return _arg(g[k], k, like[k][1], like[k][0], dev) if k in g else None

    st = lib.mamba_gated_scan_bwd(
        batch, L, D, io, _arg(u, "u", t, shape, dev), _arg(gate_a, "gate_a", t, shape, dev),
        _arg(gate_x, "gate_x", t, shape, dev), _arg(lam, "lam", f32, (D,), dev), c, _arg(z, "z", t, shape, dev),
        _reset_bytes(reset, (batch, L), dev), _arg(h0, "h0", f32, (batch, D), dev),
        _arg(states, "states", f32, (batch, chunks, D), dev), _arg(dout, "dout", t, shape, dev),
        _arg(dlast_state, "dlast_state", f32, (batch, D), dev), gp("du"), gp("dgate_a"), gp("dgate_x"), gp("dlam"),
        gp("dz"), gp("dh0"), ws, ws_bytes, _stream(dev))
    if st != 0:
        raise MambaError("mamba_gated_scan_bwd", st)
    if check:
        _check_status("mamba_gated_scan_bwd", dev)
    return {k: g[k] for k in need}


def mamba_gated_state_update(state, u, gate_a, gate_x, lam, z=None, reset=None, c=8.0, out=None):
    """One token of mamba_gated_scan_fwd in place on state (batch, D) float32.
    u, gate_a, gate_x, z: (batch, D); reset: (batch,) bool or uint8."""
    import torch

    lib = _lib()
    batch, D = u.shape
    io, dev, f32, t = _io_dtype(u), u.device, torch.float32, u.dtype
    shape = (batch, D)
    out = torch.empty_like(u) if out is None else out
    st = lib.mamba_gated_state_update(
        batch, D, io, _arg(state, "state", f32, shape, dev), _arg(u, "u", t, shape, dev),
        _arg(gate_a, "gate_a", t, shape, dev), _arg(gate_x, "gate_x", t, shape, dev),
        _arg(lam, "lam", f32, (D,), dev), c, _arg(z, "z", t, shape, dev),
        _reset_bytes(reset, (batch,), dev), _arg(out, "out", t, shape, dev), _stream(dev))
    if st != 0:
        raise MambaError("mamba_gated_state_update", st)
    return out


def mamba_embed_fwd(ids, weight, scale=1.0, out=None):
    """out = scale * weight[ids]: ids int64 of any shape, weight (vocab, D) float32 or bfloat16.
    A negative id (padding) gives a row of zeros, one of vocab or more a row of NaN."""
    import torch

    lib = _lib()
    V, D = weight.shape
    io, dev, t = _io_dtype(weight), weight.device, weight.dtype
    shape = (*ids.shape, D)
    out = torch.empty(shape, dtype=t, device=dev) if out is None else out
    st = lib.mamba_embed_fwd(ids.numel(), V, D, io, _arg(ids, "ids", torch.int64, ids.shape, dev),
                             _arg(weight, "weight", t, (V, D), dev), scale,
                             _arg(out, "out", t, shape, dev), _stream(dev))
    if st != 0:
        raise MambaError("mamba_embed_fwd", st)
    return out


def mamba_embed_bwd_workspace_size(count: int, vocab: int, dim: int, io_dtype: int) -> int:
    return int(_lib().mamba_embed_bwd_workspace_size(count, vocab, dim, io_dtype))


def mamba_embed_bwd(ids, dout, vocab, scale=1.0, dweight=None, workspace=None):
    """Gradient of mamba_embed_fwd at weight, (vocab, D) in dout's type: dout (*ids.shape, D)."""
    import torch

    lib = _lib()
    D = dout.shape[-1]
    io, dev, t = _io_dtype(dout), dout.device, dout.dtype
    n, V = ids.numel(), int(vocab)
    dweight = torch.empty((V, D), dtype=t, device=dev) if dweight is None else dweight
    workspace, ws, ws_bytes = _workspace(workspace, lib.mamba_embed_bwd_workspace_size(n, V, D, io), dev)
    st = lib.mamba_embed_bwd(n, V, D, io, _arg(ids, "ids", torch.int64, ids.shape, dev),
                             _arg(dout, "dout", t, (*ids.shape, D), dev), scale,
                             _arg(dweight, "dweight", t, (V, D), dev), ws, ws_bytes, _stream(dev))
    if st != 0:
        raise MambaError("mamba_embed_bwd", st)
    return dweight


def mamba_sample(logits, noise, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, logprob=None,
                 return_logprob=True):
    """Draws a token per row of logits (rows, vocab) with Exp(1) noise (rows, vocab) float32, after
    temperature, top_k, top_p and min_p: (rows,) tensors (float32, top_k int32) or None (off).

    Returns (tokens int64 (rows,), logprob float32 (rows,) or None); token -1 where every logit is masked."""
    import torch

    lib = _lib()
    rows, V = logits.shape
    io, dev, f32 = _io_dtype(logits), logits.device, torch.float32
    tokens = torch.empty((rows,), dtype=torch.int64, device=dev) if tokens is None else tokens
    if logprob is None and return_logprob:
        logprob = torch.empty((rows,), dtype=f32, device=dev)
    st = lib.mamba_sample(rows, V, io, _arg(logits, "logits", logits.dtype, (rows, V), dev),
                          _arg(noise, "noise", f32, (rows, V), dev),
                          _arg(temperature, "temperature", f32, (rows,), dev),
                          _arg(top_k, "top_k", torch.int32, (rows,), dev), _arg(top_p, "top_p", f32, (rows,), dev),
                          _arg(min_p, "min_p", f32, (rows,), dev), _arg(tokens, "tokens", torch.int64, (rows,), dev),
                          _arg(logprob, "logprob", f32, (rows,), dev), _stream(dev))
    if st != 0:
        raise MambaError("mamba_sample", st)
    return tokens, logprob
