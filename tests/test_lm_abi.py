"""The C ABI of the token-model operators on the host: symbols, workspace sizes and refusals.  Every
call is decided by the host-side checks (the fake device pointers are never dereferenced)."""
import ctypes
import os
import re

import pytest

from selective_state_space_22_amd import binding, lm
from selective_state_space_22_amd import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mamba_mi355x_lm.h")
OK, ERR_NULL, ERR_DIM, ERR_UNSUPPORTED, ERR_DTYPE, ERR_WORKSPACE, ERR_ALIGN, ERR_HIP, _, ERR_OPTION = range(10)
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        lib_build.build()
    return lm._lib()


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mamba_\w+)\s*\(", text)))
    assert names == sorted([
        "mamba_embed_bwd", "mamba_embed_bwd_workspace_size", "mamba_embed_fwd", "mamba_gated_scan_bwd",
        "mamba_gated_scan_bwd_workspace_size", "mamba_gated_scan_fwd", "mamba_gated_scan_fwd_workspace_size",
        "mamba_gated_state_update", "mamba_sample"])
    raw = ctypes.CDLL(binding.LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n


BIG = 1 << 40  # more workspace than any of these shapes needs


def _call(fn, order, head, values, **kw):
    return fn(*head, *[kw.get(k, values[k]) for k in order])


FWD = ["u", "gate_a", "gate_x", "lam", "c", "z", "reset", "h0", "out", "last", "states", "ws", "ws_bytes", "stream"]
BWD = ["u", "gate_a", "gate_x", "lam", "c", "z", "reset", "h0", "states", "dout", "dlast", "du", "dgate_a", "dgate_x",
       "dlam", "dz", "dh0", "ws", "ws_bytes", "stream"]
STEP = ["state", "u", "gate_a", "gate_x", "lam", "c", "z", "reset", "out", "stream"]
OPTIONAL = {"z", "reset", "h0", "last", "states", "dlast", "dz", "dh0", "stream", "temperature", "top_k", "top_p",
            "min_p", "logprob"}


def _values(order):
    v = {k: None if k in OPTIONAL else FAKE for k in order}
    v.update({k: x for k, x in (("c", 8.0), ("ws_bytes", BIG), ("scale", 1.0)) if k in v})
    return v


def _entry(lib, name):
    order = {"fwd": FWD, "bwd": BWD, "step": STEP,
             "embed_fwd": ["ids", "weight", "scale", "out", "stream"],
             "embed_bwd": ["ids", "dout", "scale", "dweight", "ws", "ws_bytes", "stream"],
             "sample": ["logits", "noise", "temperature", "top_k", "top_p", "min_p", "tokens", "logprob", "stream"]}[name]
    fn = {"fwd": lib.mamba_gated_scan_fwd, "bwd": lib.mamba_gated_scan_bwd, "step": lib.mamba_gated_state_update,
          "embed_fwd": lib.mamba_embed_fwd, "embed_bwd": lib.mamba_embed_bwd, "sample": lib.mamba_sample}[name]
    head = {"step": (2, 64, 0), "sample": (2, 64, 0)}.get(name, (2, 8, 64, 0))
    return fn, order, head


ENTRIES = ["fwd", "bwd", "step", "embed_fwd", "embed_bwd", "sample"]


@pytest.mark.parametrize("name", ENTRIES)
def test_refusals_of_pointers(lib, name):
    fn, order, head = _entry(lib, name)
    v = _values(order)
    for k in order:
        if k in ("c", "scale", "ws_bytes", "stream"):
            continue
        assert _call(fn, order, head, v, **{k: FAKE + 4}) == ERR_ALIGN, k
        if k not in OPTIONAL and k != "ws":
            assert _call(fn, order, head, v, **{k: None}) == ERR_NULL, k


@pytest.mark.parametrize("name", ENTRIES)
def test_refusals_of_sizes_and_types(lib, name):
    fn, order, head = _entry(lib, name)
    v = _values(order)
    assert _call(fn, order, (*head[:-1], 2), v) == ERR_DTYPE
    assert _call(fn, order, (*head[:-1], -1), v) == ERR_DTYPE
    for i in range(len(head) - 1):
        for bad in (-1, 1 << 41):
            assert _call(fn, order, (*head[:i], bad, *head[i + 1:]), v) == ERR_DIM, (i, bad)
    if "c" in order:
        for c in (0.0, -1.0, float("inf"), float("nan")):
            assert _call(fn, order, head, v, c=c) == ERR_OPTION
    if "scale" in order:
        for s in (float("inf"), float("nan")):
            assert _call(fn, order, head, v, scale=s) == ERR_OPTION


def test_refusal_of_a_vocabulary_of_none(lib):
    fn, order, _ = _entry(lib, "sample")
    assert _call(fn, order, (2, 0, 0), _values(order)) == ERR_DIM
    assert _call(fn, order, (2, (1 << 20) + 1, 0), _values(order)) == ERR_DIM


@pytest.mark.parametrize("name,size,head", [
    ("fwd", "mamba_gated_scan_fwd_workspace_size", (1, 1 << 20, 256, 0)),
    ("bwd", "mamba_gated_scan_bwd_workspace_size", (2, 4096, 256, 1)),
    ("embed_bwd", "mamba_embed_bwd_workspace_size", (4096, 1000, 64, 0))])
def test_workspace_sizes_and_their_refusal(lib, name, size, head):
    fn, order, _ = _entry(lib, name)
    need = getattr(lm, size)(*head)
    assert need == getattr(lm, size)(*head)
    assert getattr(lm, size)(-1, *head[1:]) == 0 and getattr(lm, size)(*head[:-1], 7) == 0
    if need:
        v = _values(order)
        assert _call(fn, order, head, v, ws=None) == ERR_WORKSPACE
        assert _call(fn, order, head, v, ws_bytes=need - 1) == ERR_WORKSPACE


def test_empty_problems_need_no_pointers(lib):
    for name, heads in (("fwd", [(0, 8, 64, 0), (2, 8, 0, 0)]), ("bwd", [(2, 8, 0, 0)]),
                        ("step", [(0, 64, 0), (2, 0, 0)]), ("embed_fwd", [(0, 8, 64, 0), (2, 8, 0, 0)]),
                        ("embed_bwd", [(2, 0, 64, 0), (2, 8, 0, 0)]), ("sample", [(0, 64, 0)])):
        fn, order, _ = _entry(lib, name)
        none = {k: x if k in ("c", "scale") else (0 if k == "ws_bytes" else None) for k, x in _values(order).items()}
        for head in heads:
            assert _call(fn, order, head, none) == OK, (name, head)


def test_binding_refuses_cpu_tensors_and_wrong_types(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 4, 64)
    for call in (lambda: lm.mamba_gated_scan_fwd(x, x, x, torch.zeros(64)),
                 lambda: lm.mamba_gated_scan_bwd(x, x, x, torch.zeros(64), x),
                 lambda: lm.mamba_gated_state_update(x[0], x[0], x[0], x[0], torch.zeros(64)),
                 lambda: lm.mamba_embed_fwd(torch.zeros(3, dtype=torch.int64), x[0]),
                 lambda: lm.mamba_embed_bwd(torch.zeros(4, dtype=torch.int64), x[0], 9),
                 lambda: lm.mamba_sample(x[0], x[0])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lm.mamba_sample(x[0].half(), x[0]), lambda: lm.mamba_embed_fwd(x, x[0].half())):
        with pytest.raises(TypeError):
            call()
