"""The fp64 reference of the token-model operators against finite differences, closed forms and
distributions, on the CPU."""
import math

import lm_ref as R
import numpy as np
import pytest


def _inputs(batch, L, D, seed, z, reset, h0):
    rng = np.random.default_rng(seed)
    p = {"u": rng.standard_normal((batch, L, D)), "ra": rng.standard_normal((batch, L, D)),
         "rx": rng.standard_normal((batch, L, D)), "lam": rng.standard_normal(D) - 2.0}
    opt = {"z": rng.standard_normal((batch, L, D)) if z else None,
           "h0": rng.standard_normal((batch, D)) if h0 else None,
           "reset": rng.random((batch, L)) < 0.3 if reset else None}
    return p, opt, rng.standard_normal((batch, L, D)), rng.standard_normal((batch, D))


@pytest.mark.parametrize("z,reset,h0", [(False, False, False), (True, False, True), (True, True, True)])
def test_gradients_against_central_differences(z, reset, h0):
    p, opt, dout, dlast = _inputs(2, 5, 3, 7, z, reset, h0)
    grads = R.gated_bwd(**p, c=8.0, dout=dout, dlast=dlast, **opt)

    def value(p, opt):
        out, last, _ = R.gated_fwd(**p, c=8.0, **opt)
        return (out * dout).sum() + (last * dlast).sum()

    names = {"u": "du", "ra": "dgate_a", "rx": "dgate_x", "lam": "dlam", "z": "dz", "h0": "dh0"}
    for k, gk in names.items():
        where = p if k in p else opt
        if where[k] is None:
            continue
        for i in np.ndindex(where[k].shape):
            e = 1e-5
            side = []
            for sgn in (1, -1):
                moved = {**where, k: where[k].copy()}
                moved[k][i] += sgn * e
                side.append(value(moved if k in p else p, opt if k in p else moved))
            assert abs((side[0] - side[1]) / (2 * e) - grads[gk][i]) < 1e-7 * (1 + abs(grads[gk][i])), (k, i)


def test_constant_gates_have_the_geometric_closed_form():
    L, c = 40, 8.0
    lam = np.array([-3.0, 0.5])
    u, zero = np.ones((1, L, 2)), np.zeros((1, L, 2))
    a = np.exp(-c * np.log1p(np.exp(lam)) * 0.5)
    want = 0.5 * np.sqrt(1 - a ** 2) * (1 - a ** np.arange(1, L + 1)[:, None]) / (1 - a)
    out, last, _ = R.gated_fwd(u, zero, zero, lam, c)
    assert np.allclose(out[0], want, rtol=1e-12) and np.allclose(last[0], want[-1], rtol=1e-12)


def test_reset_equals_starting_anew():
    p, opt, _, _ = _inputs(1, 9, 2, 3, True, False, True)
    reset = np.zeros((1, 9), bool)
    reset[0, 4] = True
    out, last, _ = R.gated_fwd(**p, c=8.0, z=opt["z"], reset=reset, h0=opt["h0"])
    tail = {k: v[:, 4:] if k != "lam" else v for k, v in p.items()}
    first = np.zeros((1, 5), bool)
    first[0, 0] = True
    out2, last2, _ = R.gated_fwd(**tail, c=8.0, z=opt["z"][:, 4:], reset=first)
    assert np.array_equal(out[:, 4:], out2) and np.array_equal(last, last2)


def test_sampling_draws_each_kept_token_with_its_probability():
    rng = np.random.default_rng(5)
    x = np.log(np.array([0.4, 0.3, 0.2, 0.06, 0.04]))
    n = 20000
    for kw, keep in (({}, [0, 1, 2, 3, 4]), ({"top_k": 3}, [0, 1, 2]), ({"top_p": 0.69}, [0, 1]),
                     ({"min_p": 0.14}, [0, 1, 2, 3])):
        count = np.zeros(5)
        for _ in range(n):
            count[R.sample_row(x, rng.exponential(size=5), **kw)[0]] += 1
        p = np.exp(x) * np.isin(np.arange(5), keep)
        p /= p.sum()
        assert np.all(np.abs(count / n - p) < 5 * np.sqrt(p * (1 - p) / n) + 1e-12), kw


def test_sampling_logprob_and_ties():
    ones = np.ones(4)
    tok, lp, kept = R.sample_row(np.array([1.0, 2.0, 2.0, 2.0]), ones, top_k=2)
    assert (tok, kept) == (1, [1, 2]) and math.isclose(lp, -math.log(2))
    assert R.sample_row(np.full(4, -np.inf), ones)[:2] == (-1, -np.inf)
    assert R.sample_row(np.array([0.0, 3.0, 3.0, 1.0]), ones, temperature=0.0)[:2] == (1, 0.0)
