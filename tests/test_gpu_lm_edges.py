"""Token-model operators where a shortcut of the kernels could end, against the fp64 reference (lm_ref.py):
sums that a small weight decides, temperatures, differences of logits, rates, gates and faults at the edges
of their ranges.

Tolerances are those of test_gpu_lm.py where no other is derived at a test."""
import numpy as np
import pytest

from test_gpu_lm import _check_sample, _host, _logits

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
