"""The token-model operators on the GPU, through the binding, against the fp64 reference (lm_ref.py).

Tolerances: elementwise results get the framework's bounds (max relative error with the tensor's rms
as floor, 1e-4 fp32 I/O, 2e-2 bf16 I/O: fp32 arithmetic carries some 2^-24 times the root of a state's
memory, about 1e-5 at the longest memory used here, and bf16 output rounds by 2^-9).  dlam adds
batch * L fp32 terms of both signs: 5e-4, as for the sums of mamba_scan_bwd.  A table's gradient adds at
most count fp32 terms: 1e-4.  Sampled tokens are whole numbers and have to be equal; logprob is a
difference of two fp32 logarithms of numbers that carry 2^-22: 1e-5 absolute."""
import math

import lm_ref as R
import numpy as np
import pytest

from gpu_util import TOL, library_option, parity_error
from selective_state_space_22_amd import binding

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _lib():
    import selective_state_space_22_amd as lib

    return lib


def _dev(x, io=None):
    """Host array to the GPU; io rounds to the I/O type."""
    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x)).to("cuda")
    return t.to(DT[io]) if io else t


def _host(t):
    return t.detach().double().cpu().numpy()


def _f32(rng, *shape):
    return rng.standard_normal(shape).astype(np.float32)


def _gated_inputs(batch, L, D, io, seed, z=True, reset=0.1, h0=True, lam=None):
    rng = np.random.default_rng(seed)
    r = lambda *s: _host(_dev(_f32(rng, *s), io))  # noqa: E731  values the I/O type holds
    kappa = -np.log(rng.uniform(0.9, 0.999, D))
    p = {"u": r(batch, L, D), "ra": r(batch, L, D), "rx": r(batch, L, D),
         "lam": (np.log(np.expm1(kappa / 8.0)) if lam is None else lam).astype(np.float32)}
    opt = {"z": r(batch, L, D) if z else None, "h0": _f32(rng, batch, D) if h0 else None,
           "reset": (rng.random((batch, L)) < reset) if reset else None}
    return p, opt, r(batch, L, D), _f32(rng, batch, D)


def _gated_dev(p, opt, io):
    args = (_dev(p["u"], io), _dev(p["ra"], io), _dev(p["rx"], io), _dev(p["lam"]))
    return args, dict(z=_dev(opt["z"], io), h0=_dev(opt["h0"]), reset=_dev(opt["reset"]))


def _check_gated(p, opt, dout, dlast, io, c=8.0, label="", states_too=True):
    lib = _lib()
    args, kw = _gated_dev(p, opt, io)
    tol = TOL[io]
    p64 = {k: v.astype(np.float64) for k, v in p.items()}
    with np.errstate(over="ignore"):
        want, wlast, wstates = R.gated_fwd(**p64, c=c, **opt)
        wg = R.gated_bwd(**p64, c=c, dout=dout, dlast=dlast, **opt)
    out, last, states = lib.mamba_gated_scan_fwd(*args, c=c, **kw, return_states=True, check=True)
    errs = {"out": parity_error(_host(out), want), "last": parity_error(_host(last), wlast),
            "states": parity_error(_host(states), wstates[:, :-1][:, ::lib.MAMBA_GATED_STATE_CHUNK])}
    assert errs["out"] <= tol and errs["last"] <= 1e-4 and errs["states"] <= 1e-4, (label, errs)
    for given in (states, None) if states_too else (states,):
        g = lib.mamba_gated_scan_bwd(*args, _dev(dout, io), c=c, **kw, states=given, dlast_state=_dev(dlast),
                                     check=True)
        assert set(g) == set(wg)
        e = {k: parity_error(_host(g[k]), wg[k]) for k in g}
        for k, v in e.items():
            assert v <= (5e-4 if k == "dlam" else 1e-4 if k == "dh0" else tol), (label, k, e)
    return out, last, g


# lengths around the saved states and the tiles, widths that are and are not multiples of the vector
GATED = [(1, 1, 1), (2, 2, 3), (1, 63, 64), (3, 64, 65), (2, 65, 130), (1, 127, 8), (2, 129, 256), (1, 1000, 48),
         (5, 257, 1), (1, 4100, 72), (2, 700, 520), (1, 20011, 16)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", GATED, ids=str)
def test_gated_scan_and_gradients(shape, io):
    for k, (z, reset, h0) in enumerate([(True, 0.05, True), (False, 0, False)]):
        p, opt, dout, dlast = _gated_inputs(*shape, io, 11 + k, z, reset, h0)
        _check_gated(p, opt, dout, dlast if h0 else None, io, label=(shape, io, z))


@pytest.mark.parametrize("flags", [(True, 0, False), (False, 0.02, False), (False, 0, True), (True, 0.02, False)])
def test_gated_scan_with_each_option_alone(flags):
    z, reset, h0 = flags
    p, opt, dout, dlast = _gated_inputs(2, 300, 96, "f32", 5, z, reset, h0)
    _check_gated(p, opt, dout, None, "f32", label=flags)


def test_gated_scan_where_every_token_or_none_of_a_row_resets():
    p, opt, dout, dlast = _gated_inputs(3, 200, 40, "f32", 6)
    opt["reset"] = np.zeros((3, 200), bool)
    opt["reset"][0] = True          # nothing of the past anywhere
    opt["reset"][1, [0, 64, 128, 199]] = True  # at the edges of the saved states
    _check_gated(p, opt, dout, dlast, "f32")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_scan_at_extreme_gates_and_rates(io):
    lam = np.array([-60.0, -20.0, -8.0, -1.0, 0.0, 3.0, 20.0, 60.0], np.float32)
    p, opt, dout, dlast = _gated_inputs(2, 150, 8, io, 7, lam=lam)
    p["ra"][:, ::3] *= 16
    p["rx"][:, 1::3] *= 16
    _check_gated(p, opt, dout, dlast, io, label="extreme")


def test_gated_scan_of_long_memory_carries_no_bias():
    """kappa near 1e-5: 1e5 tokens of memory, through every chunk hand-over."""
    D = 16
    lam = np.log(np.expm1(np.full(D, 1e-5 / 8))).astype(np.float32)
    p, opt, dout, _ = _gated_inputs(1, 30000, D, "f32", 8, False, 0, True, lam)
    p["u"] = np.abs(p["u"])  # a bias would not average out
    _check_gated(p, opt, dout, None, "f32")


def test_gated_scan_keeps_a_fault_inside_its_sequence():
    """An infinity or NaN in one row and channel stays there, and ends at a reset."""
    lib = _lib()
    p, opt, dout, _ = _gated_inputs(2, 300, 64, "f32", 9, True, 0, False)
    opt["reset"] = np.zeros((2, 300), bool)
    opt["reset"][:, 200] = True
    clean, _ = lib.mamba_gated_scan_fwd(*_gated_dev(p, opt, "f32")[0], **_gated_dev(p, opt, "f32")[1])
    p["u"][0, 70, 5], p["u"][1, 130, 9] = np.nan, np.inf
    args, kw = _gated_dev(p, opt, "f32")
    out, last, states = lib.mamba_gated_scan_fwd(*args, **kw, return_states=True)
    g = lib.mamba_gated_scan_bwd(*args, _dev(dout, "f32"), **kw, states=states)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 70:200, 5] = True
    want[1, 130:200, 9] = True
    assert torch.equal(bad, want)
    assert torch.equal(out[~want], clean[~want]) and torch.isfinite(last).all()
    finite = torch.isfinite(g["du"])  # du does not read u or h
    assert finite.all()
    badg = ~torch.isfinite(g["dgate_a"])
    assert not badg[:, 200:].any() and not badg[0, :, :5].any() and not badg[1, :, :9].any()
    # a NaN gradient after the reset does not flow before it
    dy = dout.copy()
    dy[0, 250, 3] = np.nan
    g = lib.mamba_gated_scan_bwd(*args, _dev(dy, "f32"), **kw, states=states)
    assert torch.isnan(g["du"][0, 200:251, 3]).all() and not torch.isnan(g["du"][0, :200, 3]).any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_steps_equal_the_scan(io):
    lib = _lib()
    p, opt, _, _ = _gated_inputs(3, 20, 77, io, 10)
    args, kw = _gated_dev(p, opt, io)
    out, last = lib.mamba_gated_scan_fwd(*args, **kw)
    state = kw["h0"].clone()
    got = [lib.mamba_gated_state_update(state, *(a[:, t].contiguous() for a in args[:3]), args[3],
                                        z=kw["z"][:, t].contiguous(), reset=kw["reset"][:, t].contiguous())
           for t in range(20)]
    assert parity_error(_host(torch.stack(got, 1)), _host(out)) <= TOL[io]
    assert parity_error(_host(state), _host(last)) <= 1e-5


def test_gated_scan_continues_from_its_last_state():
    lib = _lib()
    p, opt, _, _ = _gated_inputs(2, 500, 130, "f32", 12)
    args, kw = _gated_dev(p, opt, "f32")
    out, last = lib.mamba_gated_scan_fwd(*args, **kw)
    cut = 193
    first = lambda t: t[:, :cut].contiguous()  # noqa: E731
    rest = lambda t: t[:, cut:].contiguous()  # noqa: E731
    o1, s1 = lib.mamba_gated_scan_fwd(*map(first, args[:3]), args[3], z=first(kw["z"]), reset=first(kw["reset"]),
                                      h0=kw["h0"])
    o2, s2 = lib.mamba_gated_scan_fwd(*map(rest, args[:3]), args[3], z=rest(kw["z"]), reset=rest(kw["reset"]), h0=s1)
    assert parity_error(_host(torch.cat([o1, o2], 1)), _host(out)) <= 1e-5
    assert parity_error(_host(s2), _host(last)) <= 1e-5


def test_gated_scan_empty_sequences():
    lib = _lib()
    lam = torch.zeros(5, device="cuda")
    e = torch.empty((2, 0, 5), device="cuda")
    h0 = torch.randn((2, 5), device="cuda")
    out, last, states = lib.mamba_gated_scan_fwd(e, e, e, lam, h0=h0, return_states=True)
    assert out.numel() == 0 and states.numel() == 0 and torch.equal(last, h0)
    g = lib.mamba_gated_scan_bwd(e, e, e, lam, e, dlast_state=h0)
    assert torch.equal(g["dh0"], h0) and not g["dlam"].any()
    n = torch.empty((0, 7, 5), device="cuda")
    g = lib.mamba_gated_scan_bwd(n, n, n, lam, n)
    assert not g["dlam"].any()


@pytest.mark.parametrize("shape", [(2, 3000, 264, "bf16"), (1, 60000, 64, "f32"), (3, 5000, 1500, "bf16")])
def test_gated_scan_repeats_bit_for_bit_on_another_stream(shape):
    """Few and many sequence chunks in flight: what a chunk finds published differs from run to run."""
    lib = _lib()
    io = shape[3]
    p, opt, dout, dlast = _gated_inputs(*shape, 13, reset=0.001)
    args, kw = _gated_dev(p, opt, io)
    dev = _dev(dout, io)

    def both():
        out, last, states = lib.mamba_gated_scan_fwd(*args, **kw, return_states=True)
        return {"out": out, "last": last, **lib.mamba_gated_scan_bwd(*args, dev, **kw, states=states)}

    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [both() for _ in range(12)]
    torch.cuda.current_stream().wait_stream(side)
    for a in again:
        for k in first:
            assert torch.equal(first[k], a[k]), k


def test_gated_scan_reports_a_wait_that_gives_up():
    """With no polls allowed a chunk gives up at once where its predecessor is not ready: then the call
    reports it, and without a report the results are right."""
    lib = _lib()
    p, opt, _, _ = _gated_inputs(1, 20000, 64, "f32", 14, False, 0, False)
    args, kw = _gated_dev(p, opt, "f32")
    want, wlast = lib.mamba_gated_scan_fwd(*args, **kw, check=True)
    with library_option(binding.MAMBA_OPT_SPIN_LIMIT, 0):
        out, last = lib.mamba_gated_scan_fwd(*args, **kw)
        status = binding.mamba_stream_status()
    assert status in (0, binding.MAMBA_ERR_TIMEOUT)
    same = torch.isnan(out) | (out == want)
    assert same.all()
    assert torch.isfinite(out).all() or status == binding.MAMBA_ERR_TIMEOUT
    out, last = lib.mamba_gated_scan_fwd(*args, **kw, check=True)
    assert torch.equal(out, want) and torch.equal(last, wlast)


# ------------------------------------------------------------------------------------------ embedding

EMBED = [(20000, 300, 24), (17000, 40000, 8), (40000, 1000000, 3), (1, 7, 8), (5, 3, 1), (64, 1, 16), (777, 300, 96), (1000, 70000, 33), (2500, 11, 520), (4097, 1023, 8),
         (9000, 5000, 64), (3, 1024, 2560)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", EMBED, ids=str)
def test_embedding_and_its_gradient(shape, io):
    lib = _lib()
    n, V, D = shape
    rng = np.random.default_rng(n + V)
    ids = np.minimum((V * rng.random(n) ** 3).astype(np.int64), V - 1)  # a few ids often
    ids[rng.random(n) < 0.1] = -1
    W, dout = _host(_dev(_f32(rng, V, D), io)), _host(_dev(_f32(rng, n, D), io))
    out = lib.mamba_embed_fwd(_dev(ids), _dev(W, io), scale=1.7)
    want = R.embed_fwd(ids, W, np.float64(np.float32(1.7)))
    assert parity_error(_host(out), want) <= (1e-6 if io == "f32" else TOL[io])
    assert not _host(out)[ids < 0].any()
    g = lib.mamba_embed_bwd(_dev(ids), _dev(dout, io), V, scale=1.7)
    wg = R.embed_bwd(ids, dout, V, np.float64(np.float32(1.7)))
    assert parity_error(_host(g), wg) <= TOL[io]
    untouched = np.setdiff1d(np.arange(V), ids)
    assert not _host(g)[untouched].any()
    assert torch.equal(g, lib.mamba_embed_bwd(_dev(ids), _dev(dout, io), V, scale=1.7))


@pytest.mark.parametrize("n", [1, 7, 8, 9, 31, 32, 33, 64, 65, 1000, 5000, 30000])
def test_embedding_gradient_of_one_repeated_id(n):
    lib = _lib()
    rng = np.random.default_rng(n)
    dout = _f32(rng, n, 20)
    for v in (0, 4, 9):
        g = _host(lib.mamba_embed_bwd(torch.full((n,), v, device="cuda"), _dev(dout), 10))
        want = np.zeros((10, 20))
        want[v] = dout.astype(np.float64).sum(0)
        assert parity_error(g, want) <= 1e-4
        assert not np.delete(g, v, 0).any()


def test_embedding_ids_outside_the_table():
    lib = _lib()
    ids = torch.tensor([[-1, 0, 4], [5, 2 ** 40, -2 ** 62]], device="cuda")
    W = torch.randn((5, 24), device="cuda")
    out = lib.mamba_embed_fwd(ids, W)
    assert out.shape == (2, 3, 24)
    assert torch.equal(out[0, 1], W[0]) and torch.equal(out[0, 2], W[4])
    assert not out[0, 0].any() and not out[1, 2].any()
    assert torch.isnan(out[1, 0]).all() and torch.isnan(out[1, 1]).all()
    dout = torch.randn((2, 3, 24), device="cuda")
    dout[1] = float("nan")  # of ids that are not in the table: not read into any sum
    g = lib.mamba_embed_bwd(ids, dout, 5)
    assert torch.equal(g[0], dout[0, 1]) and torch.equal(g[4], dout[0, 2]) and not g[1:4].any()
    none = lib.mamba_embed_bwd(torch.full((40,), -1, device="cuda"), torch.randn((40, 8), device="cuda"), 6)
    assert not none.any()
    empty = lib.mamba_embed_bwd(torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty((0, 8), device="cuda"), 6)
    assert empty.shape == (6, 8) and not empty.any()
    assert lib.mamba_embed_fwd(torch.empty(0, dtype=torch.int64, device="cuda"), W).shape == (0, 24)


# ------------------------------------------------------------------------------------------- sampling


def _sample(x, noise, io="f32", **kw):
    lib = _lib()
    dev = {k: torch.as_tensor(np.asarray(v)).to("cuda", torch.int32 if k == "top_k" else torch.float32)
           for k, v in kw.items()}
    tok, lp = lib.mamba_sample(_dev(x, io), _dev(noise.astype(np.float32)), **dev)
    return tok.cpu().numpy(), _host(lp)


def _check_sample(x, noise, io="f32", **kw):
    """x holds values of the I/O type; kw: per-row lists."""
    tok, lp = _sample(x, noise, io, **kw)
    for r in range(x.shape[0]):
        row = {k: float(np.float32(v[r])) if k != "top_k" else int(v[r]) for k, v in kw.items()}
        wt, wl, _ = R.sample_row(x[r].astype(np.float64), noise[r].astype(np.float32), **row)
        assert tok[r] == wt, (r, row, tok[r], wt, lp[r], wl)
        assert lp[r] == wl or abs(lp[r] - wl) <= 1e-5 * max(1, abs(wl)), (r, row, lp[r], wl)


def _logits(rows, V, io, seed, scale=3.0):
    rng = np.random.default_rng(seed)
    return _host(_dev(scale * _f32(rng, rows, V), io)).astype(np.float32), rng.exponential(size=(rows, V)), rng


FILTERS = {"none": {}, "top_k": {"top_k": [1, 2, 5, 40, 300]}, "top_p": {"top_p": [0.1, 0.5, 0.9, 0.99, 1.0]},
           "min_p": {"min_p": [0.5, 0.1, 0.01, 1.0, 0.0]}, "t": {"temperature": [0.0, 0.5, 1.0, 2.0, 0.05]},
           "all": {"temperature": [0.7, 0.9, 1.0, 1.3, 0.0], "top_k": [50, 3, 0, 1000, 7],
                   "top_p": [0.95, 0.6, 0.8, 0.99, 0.9], "min_p": [0.0, 0.05, 0.02, 0.001, 0.1]}}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 63, 1000, 1025, 5003, 40000])
@pytest.mark.parametrize("name", FILTERS)
def test_sampling(name, V, io):
    x, noise, _ = _logits(5, V, io, V + len(name))
    _check_sample(x, noise, io, **FILTERS[name])


@pytest.mark.parametrize("name", FILTERS)
def test_sampling_with_equal_logits(name):
    """Few distinct values: every cut falls between equal logits."""
    rng = np.random.default_rng(3)
    for V, kinds in ((400, 3), (3000, 8), (9000, 1)):
        x = rng.integers(0, kinds, (5, V)).astype(np.float32)
        _check_sample(x, rng.exponential(size=(5, V)), "bf16", **FILTERS[name])


@pytest.mark.parametrize("name", FILTERS)
def test_sampling_with_masked_logits(name):
    x, noise, rng = _logits(5, 3000, "f32", 4)
    x[rng.random(x.shape) < 0.9] = -np.inf
    x[1, ::7] = np.nan
    x[2] = -np.inf
    x[2, 1234] = 5.0        # one left
    x[3] = np.nan           # none left
    x[4, ::2] = np.finfo(np.float32).min
    _check_sample(x, noise, "f32", **FILTERS[name])


def test_sampling_with_infinite_and_lowest_logits():
    noise = np.random.default_rng(6).exponential(size=(4, 300))
    x = np.zeros((4, 300), np.float32)
    x[0, [17, 200, 250]] = np.inf
    x[1] = np.finfo(np.float32).min
    x[2] = -np.inf
    x[3, 5], x[3, 6:] = np.finfo(np.float32).max, np.finfo(np.float32).min
    for kw in ({}, {"top_k": [2, 2, 2, 2]}, {"top_p": [0.5] * 4}):
        _check_sample(x, noise, **kw)


def test_sampling_zero_infinite_and_invalid_noise():
    x = np.zeros((3, 200), np.float32)
    noise = np.ones((3, 200), np.float32)
    noise[0, 50] = 0.0
    noise[1, :100] = np.nan
    noise[2] = np.inf
    assert _sample(x, noise)[0].tolist() == [50, 100, 0]


@pytest.mark.parametrize("kw", [{}, {"top_p": [0.5] * 5}, {"top_k": [40] * 5}, {"min_p": [0.01] * 5}], ids=str)
def test_sampling_where_no_noise_is_a_number(kw):
    """Every score counts as -inf: the first element that stays is drawn."""
    x, noise, _ = _logits(5, 9001, "f32", 31)
    noise[:, :] = np.nan
    noise[1, 5000:] = np.inf  # a score of 0 beats the others, wherever it is
    x[1, 5000:] -= 1.0
    noise[2] = -1.0           # negative scores: the smallest weight is the best
    for r in range(5):
        row = {k: float(np.float32(v[r])) if k != "top_k" else v[r] for k, v in kw.items()}
        want = R.sample_row(x[r].astype(np.float64), noise[r].astype(np.float32), **row)[0]
        assert _sample(x, noise, **kw)[0][r] == want, (r, kw)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("k", [256, 257, 300, 600, 2000, 5000])
def test_sampling_of_long_lists(k, io):
    """Lists that are ranked, searched by digits, by counts and then by masses, and that do not fit."""
    x, noise, _ = _logits(3, 20000, io, k)
    for p in ([1.0, 1.0, 1.0], [0.9, 0.5, 0.999]):
        _check_sample(x, noise, io, top_k=[k, k + 1, k], top_p=p, temperature=[1.0, 3.0, 8.0])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_sampling_where_the_largest_logits_come_late(io):
    """The row's first pieces are no guide to its maximum: far below it, masked, or above all the rest."""
    x, noise, _ = _logits(6, 30011, io, 41)
    x[0, 20000] = 60.0
    x[1, :10000] = -np.inf
    x[2, :10000] -= 7.0
    x[3, :10000] = np.nan
    x[4, 5] = 40.0
    x[5, 25000:] += 9.0
    x = _host(_dev(x, io)).astype(np.float32)
    for p in (0.3, 0.9, 0.999):
        _check_sample(x, noise, io, top_p=[p] * 6, temperature=[1.0, 0.7, 1.0, 1.5, 8.0, 1.0])


def test_sampling_of_a_flat_long_row():
    """More elements within one bin of the end than the list holds, and more pieces than LDS holds."""
    rng = np.random.default_rng(12)
    x = (rng.standard_normal((3, 130001)) * 0.01).astype(np.float32)
    _check_sample(x, rng.exponential(size=x.shape), "f32", top_p=[0.3, 0.9, 0.9999], min_p=[0.0, 0.98, 0.0])
    longest = np.full((1, 1 << 20), 3.0, np.float32)  # of one bin
    longest[0, 77::2] += (rng.standard_normal(longest[0, 77::2].shape) * 1e-3).astype(np.float32)
    _check_sample(longest, rng.exponential(size=longest.shape), "f32", top_p=[0.4])
    y = _host(_dev(x + 2, "bf16")).astype(np.float32)
    _check_sample(y, rng.exponential(size=x.shape), "bf16", top_p=[0.3, 0.9, 0.9999], top_k=[0, 0, 70000])


def test_sampling_of_spread_logits_beyond_the_exponent_range():
    """Differences of hundreds, and a temperature that makes them so: weights that underflow are not drawn."""
    rng = np.random.default_rng(8)
    x = (rng.standard_normal((4, 2000)) * 300).astype(np.float32)
    _check_sample(x, rng.exponential(size=x.shape), temperature=[1.0, 0.01, 30.0, 100.0],
                  top_p=[0.9, 0.9, 0.9, 0.999], top_k=[0, 10, 0, 0])


@pytest.mark.parametrize("name", ["top_p", "top_k", "both", "none"])
def test_sampling_repeats_bit_for_bit(name):
    x, noise, _ = _logits(16, 12345, "bf16", 21)
    kw = dict(temperature=np.linspace(0.5, 1.5, 16))
    if name in ("top_p", "both"):
        kw["top_p"] = np.linspace(0.5, 0.99, 16)
    if name in ("top_k", "both"):
        kw["top_k"] = np.arange(5, 800, 50)
    first = _sample(x, noise, "bf16", **kw)
    for _ in range(10):
        again = _sample(x, noise, "bf16", **kw)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_sampling_frequencies():
    """Many rows of one distribution: the drawn shares are the probabilities after the filters."""
    lib = _lib()
    n, V = 60000, 16
    logits = torch.linspace(0, 3, V, device="cuda").repeat(n, 1)
    noise = torch.empty((n, V), device="cuda").exponential_(generator=torch.Generator("cuda").manual_seed(1))
    tok, lp = lib.mamba_sample(logits, noise, top_k=torch.full((n,), 6, dtype=torch.int32, device="cuda"))
    p = torch.softmax(logits[0].double(), 0)
    p[: V - 6] = 0
    p /= p.sum()
    share = torch.bincount(tok, minlength=V).double() / n
    assert ((share - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all()
    assert (lp.double() - p.log()[tok]).abs().max() < 1e-5
