"""The C ABI of the layer operators on the host: symbols, workspace sizes and refusals.  Every call is decided by
the host-side checks (the fake device pointers are never dereferenced)."""
import ctypes
import os
import re

import pytest

from selective_state_space_22_amd import binding, layer
from selective_state_space_22_amd import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mamba_mi355x_layer.h")
OK, ERR_NULL, ERR_DIM, ERR_UNSUPPORTED, ERR_DTYPE, ERR_WORKSPACE, ERR_ALIGN, ERR_HIP, _, ERR_OPTION = range(10)
FAKE = 0x10000
BIG = 1 << 40  # more workspace than any of these shapes needs


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        lib_build.build()
    return layer._lib()


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mamba_\w+)\s*\(", text)))
    assert names == sorted([
        "mamba_conv_fwd", "mamba_conv_bwd", "mamba_conv_bwd_workspace_size", "mamba_conv_update",
        "mamba_conv_ssm_update", "mamba_conv_ssm_update_workspace_size", "mamba_residual_norm_fwd",
        "mamba_residual_norm_bwd", "mamba_residual_norm_bwd_workspace_size", "mamba_draft_verify",
        "mamba_draft_verify_workspace_size"])
    raw = ctypes.CDLL(binding.LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n


# name: (function, sizes, {size: position}, arguments in order)
HOST = {"silu": 1, "gate_first": 1, "alpha": 1.0, "eps": 1e-5, "ws_bytes": BIG, "stream": None}
ENTRY = {
    "conv_fwd": ((2, 8, 64, 4, 0), ["x", "weight", "bias?", "window?", "reset?", "lengths?", "silu", "out", "last?",
                                    "stream"]),
    "conv_bwd": ((2, 8, 64, 4, 0), ["x", "weight", "bias?", "window?", "reset?", "silu", "dout", "dlast?", "dx", "dweight",
                                    "dbias?", "dwindow?", "ws", "ws_bytes", "stream"]),
    "conv_update": ((2, 64, 4, 0, 2), ["window", "x", "weight", "bias?", "slots?", "silu", "out", "stream"]),
    "conv_ssm_update": ((2, 64, 16, 4, 4, 0, 2), ["state", "window", "x", "cw", "cb?", "Wx", "Wdt", "dtb?", "A", "Dskip?",
                                                  "z?", "slots?", "out", "ws", "ws_bytes", "stream"]),
    "residual_norm_fwd": ((2, 64, 0, 0), ["x", "gate?", "gate_first", "post?", "scale?", "residual?", "pre?", "alpha",
                                          "eps", "residual_out?", "out", "stream"]),
    "residual_norm_bwd": ((2, 64, 0, 0), ["x", "gate?", "gate_first", "post?", "scale?", "residual?", "pre?", "alpha",
                                          "eps", "dout", "dres?", "dx", "dgate?", "dresidual?", "dpost?", "dscale?",
                                          "dpre?", "ws", "ws_bytes", "stream"]),
    "draft_verify": ((2, 3, 500, 0), ["target", "draft", "drafted", "uniform", "noise", "counts?", "tokens", "accepted",
                                      "ws", "ws_bytes", "stream"]),
}
TYPE_AT = {"conv_fwd": 4, "conv_bwd": 4, "conv_update": 3, "conv_ssm_update": 5, "residual_norm_fwd": 2,
           "residual_norm_bwd": 2, "draft_verify": 3}
SIZES = {"conv_fwd": (0, 1, 2), "conv_bwd": (0, 1, 2), "conv_update": (0, 1, 4), "conv_ssm_update": (0, 1, 3, 6),
         "residual_norm_fwd": (0, 1), "residual_norm_bwd": (0, 1), "draft_verify": (0, 1, 2)}


def _call(lib, name, head=None, **kw):
    sizes, order = ENTRY[name]
    args = []
    for a in order:
        k = a.rstrip("?")
        args.append(kw[k] if k in kw else HOST[k] if k in HOST else None if a.endswith("?") else FAKE)
    return getattr(lib, "mamba_" + name)(*(head or sizes), *args)


def _with(t, i, v):
    return (*t[:i], v, *t[i + 1:])


@pytest.mark.parametrize("name", ENTRY)
def test_refusals_of_pointers(lib, name):
    for a in ENTRY[name][1]:
        k = a.rstrip("?")
        if k in HOST:
            continue
        assert _call(lib, name, **{k: FAKE + 4}) == ERR_ALIGN, k
        if not a.endswith("?") and k != "ws":
            more = {"pre": FAKE} if name.startswith("residual") else {}  # out and dout go with the weight
            assert _call(lib, name, **{k: None}, **more) == ERR_NULL, k


@pytest.mark.parametrize("name", ENTRY)
def test_refusals_of_sizes_and_types(lib, name):
    head = ENTRY[name][0]
    for io in (2, -1):
        assert _call(lib, name, _with(head, TYPE_AT[name], io)) == ERR_DTYPE
    for i in SIZES[name]:
        for bad in (-1, 1 << 41):
            assert _call(lib, name, _with(head, i, bad)) == ERR_DIM, (i, bad)


def test_refusals_of_widths_states_and_ranks(lib):
    for width in (-1, 0, 1, 5, 1 << 40):
        for name, i in (("conv_fwd", 3), ("conv_bwd", 3), ("conv_update", 2), ("conv_ssm_update", 4)):
            assert _call(lib, name, _with(ENTRY[name][0], i, width)) == ERR_UNSUPPORTED
    for n in (0, 3, 32):
        assert _call(lib, "conv_ssm_update", (2, 64, n, 4, 4, 0, 2)) == ERR_UNSUPPORTED
    for r in (0, 513):
        assert _call(lib, "conv_ssm_update", (2, 64, 16, r, 4, 0, 2)) == ERR_DIM


def test_refusals_of_a_convolution_over_its_inputs(lib):
    a, b, c, d, e, f = (FAKE + 4096 * i for i in range(6))
    apart = {"x": a, "window": b, "out": c, "last": d}
    for out, of in (("out", "x"), ("out", "window"), ("last", "window"), ("last", "x")):
        assert _call(lib, "conv_fwd", **{**apart, out: apart[of]}) == ERR_OPTION, (out, of)
    apart = {"x": a, "window": b, "dout": c, "dlast": d, "dx": e, "dwindow": f}
    for out, of in (("dx", "x"), ("dx", "dout"), ("dwindow", "window"), ("dwindow", "dlast")):
        assert _call(lib, "conv_bwd", **{**apart, out: apart[of]}) == ERR_OPTION, (out, of)


def test_refusals_of_too_few_slots(lib):
    assert _call(lib, "conv_update", (2, 64, 4, 0, 1)) == ERR_DIM
    assert _call(lib, "conv_ssm_update", (2, 64, 16, 4, 4, 0, 1)) == ERR_DIM


def test_refusals_of_norm_options(lib):
    nan, inf = float("nan"), float("inf")
    for name in ("residual_norm_fwd", "residual_norm_bwd"):
        for kw in ({"alpha": nan}, {"alpha": inf}, {"eps": 0.0}, {"eps": -1.0}, {"eps": nan}, {"eps": inf}):
            assert _call(lib, name, **kw) == ERR_OPTION, kw
        assert _call(lib, name, (2, 64, 0, 1)) == ERR_DTYPE  # a narrower residual than the I/O type
        assert _call(lib, name, (2, 64, 1, 2)) == ERR_DTYPE
        assert _call(lib, name, (2, 0, 0, 0)) == ERR_DIM
        assert _call(lib, name, (2, 16385, 0, 0)) == ERR_DIM


def test_refusals_of_what_a_launch_cannot_count(lib):
    assert _call(lib, "conv_fwd", (65535, 1 << 30, 4096, 4, 0)) == ERR_DIM
    assert _call(lib, "conv_bwd", (65535, 1 << 30, 4096, 4, 0)) == ERR_DIM
    assert _call(lib, "conv_update", (65535, 4194304, 4, 0, 65535)) == ERR_DIM
    assert _call(lib, "conv_ssm_update", (65535, 4194304, 16, 4, 4, 0, 65535)) == ERR_DIM
    assert _call(lib, "residual_norm_fwd", ((1 << 31) - 1, 8192, 0, 0)) == ERR_DIM
    assert _call(lib, "draft_verify", ((1 << 20) + 1, 1, 9, 0)) == ERR_DIM
    assert _call(lib, "draft_verify", (1, 4097, 9, 0)) == ERR_DIM
    assert _call(lib, "draft_verify", (1, 1, 0, 0)) == ERR_DIM


@pytest.mark.parametrize("name,size,args", [
    ("conv_bwd", "mamba_conv_bwd_workspace_size", (2, 8, 64, 4, 0)),
    ("conv_ssm_update", "mamba_conv_ssm_update_workspace_size", (2, 64, 16, 4, 0)),
    ("residual_norm_bwd", "mamba_residual_norm_bwd_workspace_size", (2, 64, 0)),
    ("draft_verify", "mamba_draft_verify_workspace_size", (2, 3, 50000, 0))])
def test_workspace_sizes_and_their_refusal(lib, name, size, args):
    f = getattr(layer, size)
    need = f(*args)
    assert need > 0 and need == f(*args)
    assert f(-1, *args[1:]) == 0 and f(*args[:-1], 7) == 0
    head = (2, 3, 50000, 0) if name == "draft_verify" else None
    assert _call(lib, name, head, ws=None) == ERR_WORKSPACE
    assert _call(lib, name, head, ws_bytes=need - 1) == ERR_WORKSPACE


def test_empty_problems_need_no_pointers(lib):
    for name, heads in (("conv_fwd", [(0, 8, 64, 4, 0), (2, 8, 0, 4, 0), (2, 0, 64, 4, 0)]),
                        ("conv_bwd", [(2, 8, 0, 4, 0)]), ("conv_update", [(0, 64, 4, 0, 0), (2, 0, 4, 0, 2)]),
                        ("conv_ssm_update", [(0, 64, 16, 4, 4, 0, 0), (2, 0, 16, 4, 4, 0, 2)]),
                        ("residual_norm_fwd", [(0, 64, 0, 0), (0, 0, 0, 0)]), ("residual_norm_bwd", [(0, 0, 0, 0)]),
                        ("draft_verify", [(0, 3, 50, 0)])):
        none = {a.rstrip("?"): None for a in ENTRY[name][1] if a.rstrip("?") not in HOST}
        for head in heads:
            assert _call(lib, name, head, ws_bytes=0, **none) == OK, (name, head)


def test_binding_refuses_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    z = torch.zeros
    for call in (lambda: layer.mamba_conv_fwd(z(1, 4, 8), z(8, 4)), lambda: layer.mamba_conv_bwd(z(1, 4, 8), z(8, 4), z(1, 4, 8)),
                 lambda: layer.mamba_conv_update(z(1, 3, 8), z(1, 8), z(8, 4)),
                 lambda: layer.mamba_conv_ssm_update(z(1, 8, 16), z(1, 3, 8), z(1, 8), z(8, 4), z(34, 8), z(8, 2), z(8, 16)),
                 lambda: layer.mamba_residual_norm_fwd(z(2, 8), z(8)),
                 lambda: layer.mamba_residual_norm_bwd(z(2, 8), z(8), z(2, 8)),
                 lambda: layer.mamba_draft_verify(z(1, 2, 9), z(1, 1, 9), z(1, 1, dtype=torch.int64), z(1, 1), z(1, 9))):
        with pytest.raises(ValueError):
            call()


def test_the_limits_that_the_header_states_are_those_of_the_library(lib):
    text = " ".join(open(HEADER).read().replace("\n *", " ").split())
    assert "batch * ceil(dim / 2) * (ceil(seqlen / 32) + 1) < 2^31" in text
    for seqlen, fits in ((32 * ((1 << 20) - 2), True), (32 * ((1 << 20) - 2) + 1, False)):  # 2^10 x 2 x 2^20
        assert (layer.mamba_conv_bwd_workspace_size(1024, seqlen, 4, 4, 0) > 0) == fits
        if not fits:
            assert _call(lib, "conv_fwd", (1024, seqlen, 4, 4, 0)) == ERR_DIM
    assert "batch * ceil(dim / 2) < 2^30" in text
    assert _call(lib, "conv_update", (1 << 15, 1 << 16, 4, 0, 1 << 15)) == ERR_DIM
    assert "ceil(batch / 16) * dim < 2^28" in text
    for dim, fits in (((1 << 16) - 1, True), (1 << 16, False)):
        assert (layer.mamba_conv_ssm_update_workspace_size(65535, dim, 16, 8, 0) > 0) == fits
    assert "64 (up to 768 elements), 192 (up to 1536), 512 (up to 4096) or 1024 (beyond) below 2^31" in text
    for dim, threads in ((768, 64), (769, 192), (1536, 192), (1537, 512), (4096, 512), (4097, 1024), (16384, 1024)):
        most = -(-(1 << 31) // threads)
        assert layer.mamba_residual_norm_bwd_workspace_size(most - 1, dim, 0) > 0
        assert layer.mamba_residual_norm_bwd_workspace_size(most, dim, 0) == 0
