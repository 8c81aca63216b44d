"""The fp64 reference of the layer operators against differences, brute force and each other, on the CPU."""
import numpy as np
import pytest

import layer_ref as ref

RNG = np.random.default_rng


def _difference(f, arrays, grads, h=1e-6, picks=6, seed=0):
    rng = RNG(seed)
    for name, a in arrays.items():
        flat = a.reshape(-1)
        for i in rng.choice(flat.size, min(picks, flat.size), replace=False):
            keep = flat[i]
            flat[i] = keep + h
            up = f()
            flat[i] = keep - h
            down = f()
            flat[i] = keep
            want = (up - down) / (2 * h)
            got = grads[name].reshape(-1)[i]
            assert abs(got - want) <= 1e-6 * (1 + abs(want)), (name, i, got, want)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("L", [1, 2, 9])
@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("act", [False, True])
def test_convolution_gradients_against_differences(W, L, cut, act):
    rng = RNG(W + 10 * L)
    a = {"x": rng.normal(size=(2, L, 3)), "weight": rng.normal(size=(3, W)), "bias": rng.normal(size=3),
         "window": rng.normal(size=(2, W - 1, 3))}
    reset = rng.random((2, L)) < 0.4 if cut else None
    dout, dlast = rng.normal(size=(2, L, 3)), rng.normal(size=(2, W - 1, 3))

    def total():
        out, last, _, _ = ref.conv_fwd(a["x"], a["weight"], a["bias"], a["window"], reset, None, act)
        return (out * dout).sum() + (last * dlast).sum()

    g = ref.conv_bwd(a["x"], a["weight"], dout, a["bias"], a["window"], reset, act, dlast)
    _difference(total, a, {k: g["d" + k][0] for k in a})


def test_convolution_is_causal_and_goes_on_from_its_window():
    rng = RNG(1)
    x, w, b = rng.normal(size=(2, 11, 3)), rng.normal(size=(3, 4)), rng.normal(size=3)
    reset = rng.random((2, 11)) < 0.3
    out, last, _, _ = ref.conv_fwd(x, w, b, None, reset)
    o1, l1, _, _ = ref.conv_fwd(x[:, :2], w, b, None, reset[:, :2])
    o2, l2, _, _ = ref.conv_fwd(x[:, 2:], w, b, l1, reset[:, 2:])
    assert np.allclose(out, np.concatenate([o1, o2], 1)) and np.allclose(last, l2)
    padded, l3, _, _ = ref.conv_fwd(x, w, b, None, reset, [2, 0])
    assert np.allclose(padded[0, :2], o1[0]) and not padded[0, 2:].any() and np.allclose(l3[0], l1[0])
    assert not l3[1].any()


@pytest.mark.parametrize("gate", [None, True, False])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("rest", [False, True])
def test_norm_gradients_against_differences(gate, post, pre, rest):
    rng = RNG(7)
    a = {"x": rng.normal(size=(3, 5))}
    if gate is not None:
        a["gate"] = rng.normal(size=(3, 5))
    if post:
        a["post"] = rng.normal(size=5)
    if rest:
        a["scale"], a["residual"] = rng.normal(size=5), rng.normal(size=(3, 5))
    if pre:
        a["pre"] = rng.normal(size=5)
    dout, dres = rng.normal(size=(3, 5)) if pre else None, rng.normal(size=(3, 5))

    def total():
        out, r, _, _ = ref.norm_fwd(alpha=0.7, gate_first=gate is not False, **a)
        return (r * dres).sum() + ((out * dout).sum() if pre else 0.0)

    g = ref.norm_bwd(dout=dout, dres=dres, alpha=0.7, gate_first=gate is not False, **a)
    names = {"post": "post_weight", "pre": "pre_weight"}
    _difference(total, a, {k: g["d" + names.get(k, k)][0] for k in a})


def test_a_token_is_the_convolution_the_projections_and_the_state_in_turn():
    rng = RNG(3)
    D, N, R, W = 6, 4, 2, 3
    cw, cb, Wx, Wdt = (rng.normal(size=s) for s in ((D, W), D, (R + 2 * N, D), (D, R)))
    A, xs = -rng.random((D, N)) - 0.1, rng.normal(size=(1, 7, D))
    state, window = np.zeros((1, D, N)), np.zeros((1, W - 1, D))
    conv, _, _, _ = ref.conv_fwd(xs, cw, cb)
    h = np.zeros((D, N))
    for t in range(7):
        state, window, out = ref.conv_ssm_step(state, window, xs[:, t], cw, cb, Wx, Wdt, A)
        p = Wx @ conv[0, t]
        dt = np.log1p(np.exp(Wdt @ p[:R]))[:, None]
        h = np.exp(dt * A) * h + (np.exp(dt * A) - 1) / A * p[R:R + N] * conv[0, t][:, None]
        assert np.allclose(state[0], h) and np.allclose(out[0], h @ p[R + N:])
    assert np.array_equal(window[0], xs[0, -2:])


def test_verification_keeps_the_target_distribution():
    # every token of a two-step draft, counted over a grid of uniforms and many noises
    rng = RNG(5)
    V, n = 4, 40000
    p, q = rng.dirichlet(np.ones(V), 2).astype(np.float32), rng.dirichlet(np.ones(V), 1).astype(np.float32)
    first = np.zeros(V)
    for _ in range(n):
        d = rng.choice(V, p=q[0].astype(float) / q[0].astype(float).sum())
        tokens, kept = ref.verify_row(p, q, [d], rng.random(1), rng.exponential(size=V), 1)
        first[tokens[0]] += 1
        assert kept == (tokens[1] >= 0)
    # four standard deviations of a count
    assert (np.abs(first / n - p[0]) < 4 * np.sqrt(p[0] * (1 - p[0]) / n) + 1e-9).all()
