"""Thin binding of the layer operators (include/mamba_mi355x_layer.h): the short causal
convolution, one token of a layer, the norms around a block, verification of drafted tokens.

As in binding.py the functions keep the C names and only marshal torch tensors (device
memory, the current HIP stream) into the C ABI; there is no fallback.  The marshalling
itself is the module _layer (csrc/bind_layer.cpp), which calls the library that ctypes loads.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

from .binding import MambaError, load_library

_HERE = os.path.dirname(os.path.abspath(__file__))
BIND_PATH = os.path.join(_HERE, "_layer.so")

_typed = None
_module = None


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


def _native():
    """The marshalling module, loaded once.  Raises if it has not been built."""
    global _module
    if _module is not None:
        return _module
    import torch

    if not os.path.exists(BIND_PATH):
        raise ImportError(f"{BIND_PATH} is missing: build it with `python -m selective_state_space_22_amd.build`")
    spec = importlib.util.spec_from_file_location("selective_state_space_22_amd._layer", BIND_PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
    module.use(_lib()._handle, MambaError, stream)
    _module = module
    return module


def mamba_conv_fwd(x, weight, bias=None, window=None, reset=None, lengths=None, silu=True, out=None, last_window=None,
                   return_last_window=True):
    """Short causal convolution: c_t = bias + sum_j weight[:, j] x_{t-(W-1)+j}, out = SiLU(c) (c without silu).

    x: (batch, L, D) float32 or bfloat16; weight: (D, W) float32, W 2 to 4; bias: (D,) float32; window:
    (batch, W - 1, D), the inputs before the first; reset: (batch, L) bool or uint8, a row's first token of
    each document; lengths: (batch,) int32, rows padded behind them (out is zero there).
    Returns (out, last_window): the window with which the rows go on."""
    return _native().conv_fwd(x, weight, bias, window, reset, lengths, silu, out, last_window, return_last_window)


def mamba_conv_bwd_workspace_size(batch: int, seqlen: int, dim: int, width: int, io_dtype: int) -> int:
    return int(_lib().mamba_conv_bwd_workspace_size(batch, seqlen, dim, width, io_dtype))


def mamba_conv_bwd(x, weight, dout, bias=None, window=None, reset=None, silu=True, dlast_window=None, grads=None,
                   workspace=None, want=("dbias", "dwindow")):
    """Gradients of sum(dout * out) + sum(dlast_window * last_window) of mamba_conv_fwd (without lengths).

    Returns a dict with dx, dweight and those of dbias and dwindow named in ``want``.  Preallocated
    outputs may be passed in ``grads`` (same keys)."""
    g = grads or {}
    dx, dweight, dbias, dwindow = _native().conv_bwd(
        x, weight, dout, bias, window, reset, silu, dlast_window, g.get("dx"), g.get("dweight"), g.get("dbias"),
        g.get("dwindow"), "dbias" in want, "dwindow" in want, workspace)
    res = {"dx": dx, "dweight": dweight, "dbias": dbias, "dwindow": dwindow}
    return {k: res[k] for k in ("dx", "dweight", *want)}


def mamba_conv_update(window, x, weight, bias=None, slots=None, silu=True, out=None):
    """One token of mamba_conv_fwd in place on window (nslots, W - 1, D); x: (batch, D).  slots: (batch,) int32,
    the window of each row (None: row b has window b), negative for an idle row, whose out is left as it was (without
    ``out``: as the new tensor's memory was)."""
    return _native().conv_update(window, x, weight, bias, slots, silu, out)


def mamba_conv_ssm_update_workspace_size(batch: int, dim: int, dstate: int, dt_rank: int, io_dtype: int) -> int:
    return int(_lib().mamba_conv_ssm_update_workspace_size(batch, dim, dstate, dt_rank, io_dtype))


def mamba_conv_ssm_update(state, window, x, conv_weight, W_x, W_dt, A, conv_bias=None, z=None, dt_bias=None,
                          Dskip=None, slots=None, out=None, workspace=None):
    """One token of a layer from its input projection on, in place on state (nslots, D, N) float32 and window
    (nslots, W - 1, D): the convolution with SiLU, the selection projections (W_x (R + 2N, D), W_dt (D, R)) and
    the state update, with fp32 values between them.  x, z: (batch, D); slots and out as for mamba_conv_update."""
    return _native().conv_ssm_update(state, window, x, conv_weight, W_x, W_dt, A, conv_bias, z, dt_bias, Dskip, slots, out,
                                     workspace)


def _res_code(res_dtype):
    """The residual stream's type as the module takes it."""
    if res_dtype is None:
        return -1
    import torch

    if res_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"residual must be float32 or bfloat16, got {res_dtype}")
    return 0 if res_dtype == torch.float32 else 1


def mamba_residual_norm_fwd(x, pre_weight=None, gate=None, post_weight=None, scale=None, residual=None, alpha=1.0,
                            eps=1e-5, gate_first=True, out=None, residual_out=None, res_dtype=None,
                            return_residual=True):
    """The norm behind a block with its gate, the residual sum, and the norm before the next block:
    p = post_weight v / rms(v) with v = x SiLU(gate) (gate_first=False: v = x and p times SiLU(gate)),
    residual_out = residual + alpha scale p, out = pre_weight residual_out / rms(residual_out).

    x, gate: (..., D) float32 or bfloat16; residual: the same shape, x's type or float32; the weights and scale:
    (D,) float32.  None leaves that part out.  Returns (out, residual_out); out is None without pre_weight.
    res_dtype: residual_out's type where neither residual nor residual_out gives it (default: x's)."""
    return _native().norm_fwd(x, pre_weight, gate, post_weight, scale, residual, alpha, eps, gate_first, out, residual_out,
                              _res_code(res_dtype), return_residual)


def mamba_residual_norm_bwd_workspace_size(rows: int, dim: int, io_dtype: int) -> int:
    return int(_lib().mamba_residual_norm_bwd_workspace_size(rows, dim, io_dtype))


def mamba_residual_norm_bwd(x, pre_weight=None, dout=None, dresidual_out=None, gate=None, post_weight=None, scale=None,
                            residual=None, alpha=1.0, eps=1e-5, gate_first=True, grads=None, workspace=None,
                            res_dtype=None, want=("dgate", "dresidual", "dpost_weight", "dscale", "dpre_weight")):
    """Gradients of sum(dout * out) + sum(dresidual_out * residual_out) of mamba_residual_norm_fwd from its inputs.

    dout is given exactly with pre_weight.  Returns a dict with dx and, of those named in ``want``, the
    gradients of the inputs that are given.  Preallocated outputs may be passed in ``grads`` (same keys)."""
    g = grads or {}
    wanted = [("dgate" in want and gate is not None), ("dresidual" in want and residual is not None),
              ("dpost_weight" in want and post_weight is not None), ("dscale" in want and scale is not None),
              ("dpre_weight" in want and pre_weight is not None)]
    given = [g.get(k) if w else None for k, w in zip(_NORM_GRADS, wanted)]
    made = _native().norm_bwd(x, pre_weight, dout, dresidual_out, gate, post_weight, scale, residual, alpha, eps, gate_first,
                              _res_code(res_dtype), g.get("dx"), *given, *wanted, workspace)
    return {"dx": made[0], **{k: t for k, t in zip(_NORM_GRADS, made[1:]) if t is not None}}


_NORM_GRADS = ("dgate", "dresidual", "dpost_weight", "dscale", "dpre_weight")


def mamba_draft_verify_workspace_size(rows: int, drafts: int, vocab: int, io_dtype: int) -> int:
    return int(_lib().mamba_draft_verify_workspace_size(rows, drafts, vocab, io_dtype))


def mamba_draft_verify(target, draft, drafted, uniform, noise, counts=None, tokens=None, accepted=None,
                       workspace=None):
    """Drafted tokens against the target's probabilities: draft k stays while uniform q(d) < p(d); behind the kept
    ones a token drawn from max(p - q, 0) (or from p behind the last draft) with Exp(1) noise.

    target: (rows, K + 1, vocab), draft: (rows, K, vocab) float32 or bfloat16; drafted: (rows, K) int64; uniform:
    (rows, K) and noise: (rows, vocab) float32; counts: (rows,) int32, drafts of each row (None: K).
    Returns (tokens int64 (rows, K + 1), -1 behind the drawn one, accepted int32 (rows,))."""
    return _native().draft_verify(target, draft, drafted, uniform, noise, counts, tokens, accepted, workspace)
