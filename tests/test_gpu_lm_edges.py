"""Token-model operators where a shortcut of the kernels could end, against the fp64 reference (lm_ref.py):
sums that a small weight decides, temperatures, differences of logits, rates, gates and faults at the edges
of their ranges.

Tolerances are those of test_gpu_lm.py where no other is derived at a test."""
import lm_ref as R
import numpy as np
import pytest

from test_gpu_lm import (DT, _check_gated, _check_sample, _dev, _gated_dev, _gated_inputs, _host, _lib, _logits)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ------------------------------------------------------------------------------------------- sampling


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("small", [100, 400])
def test_sampling_where_small_weights_decide_the_end(small, io):
    """Ten equal weights and many of e^-34, 1.7e-15: half of the mass is a little more than five of the ten,
    so a sixth stays.  The masses' unit is 2^-52 of the largest weight for rows of this length, 2.2e-16."""
    rng = np.random.default_rng(small)
    x = np.full((3, 1003), -np.inf, np.float32)
    for r in range(3):
        at = rng.permutation(1003)
        x[r, at[:10]], x[r, at[10:10 + small]] = 0.0, -34.0
    _check_sample(x, rng.exponential(size=x.shape), io, top_k=[10 + small] * 3, top_p=[0.5] * 3)


HOT = [1e30, 1e31, 1e32, 1e36, 4e36, 1e37, 1e38, 3e38, np.inf]
HOT_FILTERS = {"none": {}, "top_p": {"top_p": [0.3, 0.9, 0.999] * 3}, "min_p": {"min_p": [0.0, 0.5, 0.9] * 3},
               "top_k": {"top_k": [2, 40, 700] * 3},
               "all": {"top_k": [0, 40, 2500] * 3, "top_p": [0.7, 0.9, 0.5] * 3, "min_p": [0.01, 0.5, 0.02] * 3}}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 1003, 8193, 20001])
@pytest.mark.parametrize("name", HOT_FILTERS)
def test_sampling_at_temperatures_that_level_the_row(name, V, io):
    """Up to an infinite temperature, where every logit that is not masked weighs the same: masked ones and
    what lies past the row's end have no part in it.  The type's lowest value is a logit like any other."""
    x, noise, rng = _logits(9, V, io, V)
    kw = {"temperature": HOT, **HOT_FILTERS[name]}
    _check_sample(x, noise, io, **kw)
    x[rng.random(x.shape) < 0.5] = -np.inf
    x[rng.random(x.shape) < 0.1] = np.nan
    x[:, 0] = 1.0
    noise[np.isnan(x) | (x == -np.inf)] = 1e-6  # the best scores by far, if they counted
    _check_sample(x, noise, io, **kw)
    x[:, 1::3] = _host(torch.tensor(torch.finfo(torch.bfloat16).min))
    _check_sample(x, noise, io, **kw)


# (temperature, difference of two logits): the difference in bins of 1/64 of the temperature rounds to
# just below a whole number, while that number of bins rounds to the difference itself
BIN_EDGES = [(0.55, 2.0625), (0.55, 4.125), (0.55, 8.25), (1.1, 1.03125), (1.1, 4.125), (1.35, 1.265625),
             (1.35, 2.53125), (1.35, 5.0625), (1.35, 10.125), (0.72, 10.125), (2.2, 4.125)]


def test_the_differences_lie_at_the_edge_of_a_bin():
    for t, d in BIN_EDGES:
        bins = np.float32(64) / np.float32(t)
        edge = np.floor(np.float32(d) * bins) + np.float32(1)
        assert np.float32(d) * bins < edge and np.float32(edge / bins) == np.float32(d), (t, d)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("ties", [1, 5, 300])
@pytest.mark.parametrize("above", [1, 7, 700])
def test_top_k_that_ends_at_the_edge_of_a_bin(above, ties, io):
    """`above` logits of the largest value, `ties` at the edge and others far below: the k-th largest is one
    of those at the edge.  700 above: the histogram of all elements, else that of the threads' maxima."""
    rng = np.random.default_rng(above + ties)
    n = len(BIN_EDGES)
    x = np.full((n, 6000), -40.0, np.float32)
    x[:, ::2] = -np.inf
    for r, (_, d) in enumerate(BIN_EDGES):
        at = rng.permutation(6000)
        x[r, at[:above]], x[r, at[above:above + ties]] = d, 0.0
    noise = rng.exponential(size=x.shape)
    kw = {"temperature": [t for t, _ in BIN_EDGES], "top_k": [above + (r % ties) + 1 for r in range(n)]}
    _check_sample(x, noise, io, **kw)
    _check_sample(x, noise, io, **kw, top_p=[0.999999] * n)


# ---------------------------------------------------------------------------------- gated recurrence

# relative bound per element of products of up to 60 decays: the exponent's rounding, 2^-24 of a sum of
# logarithms of 85 at most and of its partial sums (some 1e-5), and a few ulp of each factor (60 * 2e-7)
PRODUCT_TOL = 1e-4


def _rate(lam, c):
    return c * np.log1p(np.exp(np.float64(np.float32(lam))))


def _lam_for(l, c):
    """lam of the decay e^l of one token at gate_a = 0."""
    return np.log(np.expm1(-2.0 * l / c)).astype(np.float32)


def _relative(got, want):
    return float(np.max(np.abs(_host(got) / want - 1.0)))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("c", [1.0, 8.0, 30.0])
@pytest.mark.parametrize("l,L", [(-0.01, 60), (-0.3, 60), (-0.4, 60), (-1.0, 60), (-4.0, 20), (-8.0, 1), (-8.0, 9),
                                 (-12.0, 6), (-16.0, 1), (-16.0, 5), (-30.0, 2), (-60.0, 1)])
def test_decays_keep_their_relative_accuracy(l, L, c, io):
    """Without inputs a state is the product of its decays, and so is the gradient that reaches h0: channels
    that forget within a token or two, each rate alone, element by element."""
    lib = _lib()
    batch, D = 2, 72
    rng = np.random.default_rng(int(-l * 100) + L)
    lam = _lam_for(np.full(D, l), c)
    kappa = _rate(lam, c)[None]
    h0, dlast = 1.0 + rng.random((batch, D)).astype(np.float32), 1.0 + rng.random((batch, D)).astype(np.float32)
    zero = torch.zeros((batch, L, D), device="cuda", dtype=DT[io])
    args = (zero, zero, zero, _dev(lam))
    decay = np.exp(-0.5 * kappa * L)
    out, last, states = lib.mamba_gated_scan_fwd(*args, h0=_dev(h0), c=c, return_states=True)
    assert _relative(last, decay * h0) <= PRODUCT_TOL
    state = _dev(h0)
    for _ in range(L):
        lib.mamba_gated_state_update(state, zero[:, 0].contiguous(), zero[:, 0].contiguous(), zero[:, 0].contiguous(),
                                     args[3], c=c)
    assert _relative(state, decay * h0) <= PRODUCT_TOL
    g = lib.mamba_gated_scan_bwd(*args, zero, h0=_dev(h0), c=c, states=states, dlast_state=_dev(dlast))
    assert _relative(g["dh0"], decay * dlast) <= PRODUCT_TOL
    # dL/dl is the same product for every token, and gate_a = 0 halves it times -kappa
    e = decay * h0 * dlast
    assert _relative(g["dgate_a"], (-0.25 * kappa * e)[:, None].repeat(L, 1)) <= (PRODUCT_TOL if io == "f32" else 2e-2)
    dkappa = c / (1.0 + np.exp(-lam.astype(np.float64)))
    assert _relative(g["dlam"], (-0.5 * dkappa * L * e).sum(0)) <= PRODUCT_TOL


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lam", [0.0, 1.0, 2.0, 4.0])
@pytest.mark.parametrize("c", [0.5, 8.0])
def test_layers_of_channels_that_all_forget_fast(c, lam, io):
    p, opt, dout, dlast = _gated_inputs(2, 300, 70, io, 17, lam=np.full(70, lam))
    _check_gated(p, opt, dout, dlast, io, c=c, label=(c, lam))


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("which", ["u", "ra", "rx", "z"])
@pytest.mark.parametrize("shape", [(2, 300, 70), (1, 3000, 64), (2, 700, 4100)], ids=str)
def test_a_fault_ends_at_a_reset(shape, which, value):
    """Inputs that are no numbers show where the definition has them and leave the other sequences of the
    row alone, to the bit: on the same wave, on others of its tile of tokens, and on later tiles."""
    lib = _lib()
    batch, L, D = shape
    for io in ("f32", "bf16"):
        p, opt, _, _ = _gated_inputs(*shape, io, 18, reset=0)
        opt["reset"] = np.zeros((batch, L), bool)
        opt["reset"][:, [L // 3, L // 3 + 5, 2 * L // 3]] = True
        args, kw = _gated_dev(p, opt, io)
        clean, clast = lib.mamba_gated_scan_fwd(*args, **kw)
        holder = p if which in p else opt
        for r, t, d in ((0, L // 3 - 1, 0), (0, L // 3 + 1, 7), (batch - 1, 2 * L // 3 - 40, D - 1)):
            holder[which][r, t, d] = value
        args, kw = _gated_dev(p, opt, io)
        out, last = lib.mamba_gated_scan_fwd(*args, **kw)
        with np.errstate(invalid="ignore", over="ignore"):
            want, wlast, _ = R.gated_fwd(**{k: v.astype(np.float64) for k, v in p.items()}, c=8.0, **opt)
        assert np.array_equal(np.isfinite(_host(out)), np.isfinite(want))
        assert torch.equal(last, clast)
        same = torch.from_numpy(np.isfinite(want)).cuda()
        if value != value or which in ("u", "z"):  # (an infinite gate gives other numbers, not faults)
            assert torch.equal(out[same], clean[same])


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("c", [0.05, 8.0])
def test_a_fault_outlasts_every_decay(c, value):
    """Without a reset a state that is no number stays so, in channels that forget within a token and in
    those of long memory, through every hand-over; a decay that underflows is no reset."""
    lib = _lib()
    p, opt, dout, dlast = _gated_inputs(2, 2500, 70, "f32", 21, z=False, reset=0, lam=np.linspace(-6.0, 2.0, 70))
    at = 100 + 7 * np.arange(70)
    for d in range(70):
        p["u"][1, at[d], d] = value
    args, kw = _gated_dev(p, opt, "f32")
    out, last, states = lib.mamba_gated_scan_fwd(*args, c=c, **kw, return_states=True)
    bad = ~np.isfinite(_host(out))
    assert not bad[0].any()
    assert np.array_equal(bad[1], np.arange(2500)[:, None] >= at[None])
    assert torch.isfinite(last[0]).all() and not torch.isfinite(last[1]).any()
    p["u"][1] = 0.0  # and a gradient that is no number, towards the first token
    dout[1, at, np.arange(70)] = value
    args, kw = _gated_dev(p, opt, "f32")
    g = lib.mamba_gated_scan_bwd(*args, _dev(dout, "f32"), c=c, **kw, dlast_state=_dev(dlast))
    assert torch.isfinite(g["dh0"][0]).all() and not torch.isfinite(g["dh0"][1]).any()
    bad = ~np.isfinite(_host(g["du"]))
    assert not bad[0].any()
    assert np.array_equal(bad[1], np.arange(2500)[:, None] <= at[None])


@pytest.mark.parametrize("shape", [(2, 520, 70), (1, 130, 64), (9, 60, 1024), (3, 2, 5)], ids=str)
@pytest.mark.parametrize("where", ["h0", "u"])
def test_values_that_a_reset_cuts_off_stay_out_of_the_sums(where, shape):
    """h0 before a first token that starts anew, or the input of a last token whose state nothing reads:
    infinities and NaN there do not reach dlam, whatever is left of the last tile of tokens."""
    lib = _lib()
    batch, L, D = shape
    p, opt, dout, dlast = _gated_inputs(*shape, "f32", 20, z=False, reset=0)
    opt["reset"] = np.zeros((batch, L), bool)
    opt["reset"][:, 0 if where == "h0" else -1] = True
    args, kw = _gated_dev(p, opt, "f32")
    clean = lib.mamba_gated_scan_bwd(*args, _dev(dout, "f32"), **kw, dlast_state=_dev(dlast))
    bad = {k: v.copy() for k, v in (("h0", opt["h0"]), ("u", p["u"]))}
    bad["h0"][:, ::2], bad["h0"][:, 1::2] = np.nan, np.inf
    bad["u"][:, -1, ::2], bad["u"][:, -1, 1::2] = np.nan, np.inf
    args, kw = _gated_dev({**p, "u": bad["u"]} if where == "u" else p, {**opt, "h0": bad["h0"]} if where == "h0" else opt,
                          "f32")
    g = lib.mamba_gated_scan_bwd(*args, _dev(dout, "f32"), **kw, dlast_state=_dev(dlast))
    assert torch.isfinite(g["dlam"]).all()
    for k in ("dlam", "dh0", "du", "dgate_a"):
        assert torch.equal(g[k], clean[k]), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["ra", "rx", "z"])
def test_gates_that_are_no_numbers_show_in_the_gradients(which, io):
    """A NaN gate makes NaN what depends on it, in the backward as in the forward, and nothing else."""
    lib = _lib()
    p, opt, dout, dlast = _gated_inputs(2, 300, 70, io, 18, reset=0, lam=np.linspace(-6.0, 2.0, 70))
    opt["reset"] = np.zeros((2, 300), bool)
    opt["reset"][:, 180] = True
    (p if which in p else opt)[which][0, 100, 7] = np.nan
    (p if which in p else opt)[which][1, 233, 69] = np.nan
    args, kw = _gated_dev(p, opt, io)
    p64 = {k: v.astype(np.float64) for k, v in p.items()}
    want = R.gated_bwd(**p64, c=8.0, dout=dout, dlast=dlast, **opt)
    out, last, states = lib.mamba_gated_scan_fwd(*args, **kw, return_states=True)
    for given in (states, None):
        g = lib.mamba_gated_scan_bwd(*args, _dev(dout, io), **kw, states=given, dlast_state=_dev(dlast))
        for k in want:
            assert np.array_equal(np.isnan(_host(g[k])), np.isnan(want[k])), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_gate_that_a_reset_leaves_out_has_no_gradient(io):
    """l does not enter at a reset token: whatever gate_a holds there, its gradient is 0 and no other sees it."""
    lib = _lib()
    p, opt, dout, dlast = _gated_inputs(2, 100, 70, io, 19, reset=0)
    opt["reset"] = np.zeros((2, 100), bool)
    opt["reset"][:, [0, 37, 99]] = True
    args, kw = _gated_dev(p, opt, io)
    clean = lib.mamba_gated_scan_bwd(*args, _dev(dout, io), **kw, dlast_state=_dev(dlast))
    for value in (np.nan, np.inf, -np.inf):
        p["ra"][:, [0, 37, 99]] = value
        g = lib.mamba_gated_scan_bwd(*_gated_dev(p, opt, io)[0], _dev(dout, io), **kw, dlast_state=_dev(dlast))
        assert not _host(g["dgate_a"])[:, [0, 37, 99]].any()
        for k in clean:
            assert torch.equal(g[k], clean[k]), (value, k)
