"""The layer operators on the GPU against their fp64 definitions (tests/layer_ref.py, which derives the tolerances)."""
import numpy as np
import pytest

import layer_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def io_values(rng, shape, io, scale=1.0):
    """Normal values that the I/O type holds exactly, in fp64."""
    t = torch.from_numpy(np.asarray(rng.normal(size=shape) * scale, np.float32)).to(DT[io])
    return t.double().numpy()


def f32_values(rng, shape, scale=1.0):
    return np.asarray(rng.normal(size=shape) * scale, np.float32).astype(np.float64)


def dev(a, io="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda", DT[io])


def host(t):
    return None if t is None else t.double().cpu().numpy()


def u8(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return None if a is None else torch.tensor(np.asarray(a, np.int32)).cuda()


# ------------------------------------------------------------------------------------------ convolution

# rows of one element, of a group and a bit, odd ones; sequences shorter than the taps, of a chunk and a bit
CONV_SHAPES = [(1, 1, 1), (2, 3, 5), (3, 17, 64), (2, 70, 130), (1, 203, 259), (2, 1, 8), (4, 129, 12), (5, 8, 3),
               (1, 600, 36), (2, 40, 700), (2, 4500, 9)]


def _conv_case(shape, W, io, flags, seed=0):
    rng = np.random.default_rng(seed + sum(shape) + 7 * W)
    b, L, D = shape
    c = {"x": io_values(rng, shape, io), "w": f32_values(rng, (D, W), 0.6),
         "bias": f32_values(rng, D, 0.2) if "b" in flags else None,
         "window": io_values(rng, (b, W - 1, D), io) if "w" in flags else None,
         "reset": rng.random((b, L)) < (0.5 if L < 20 else 0.1) if "r" in flags else None,
         "lengths": rng.integers(-1, L + 2, b) if "l" in flags else None, "act": "n" not in flags}
    return rng, c


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("flags", ["", "bw", "br", "bwrl", "l", "bn", "wr"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("shape", CONV_SHAPES, ids=str)
def test_convolution(shape, W, flags, io):
    import selective_state_space_22_amd as lib

    _, c = _conv_case(shape, W, io, flags)
    out, last, _, m = ref.conv_fwd(c["x"], c["w"], c["bias"], c["window"], c["reset"], c["lengths"], c["act"])
    got, glast = lib.mamba_conv_fwd(dev(c["x"], io), dev(c["w"]), bias=dev(c["bias"]), window=dev(c["window"], io),
                                    reset=u8(c["reset"]), lengths=i32(c["lengths"]), silu=c["act"])
    assert got.dtype == DT[io] and glast.dtype == DT[io]
    assert ref.close(host(got), out, m, io) <= 1
    assert np.array_equal(host(glast), last)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("flags", ["", "bw", "br", "bwr", "bn", "wrn"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("shape", CONV_SHAPES, ids=str)
def test_convolution_gradients(shape, W, flags, io):
    import selective_state_space_22_amd as lib

    rng, c = _conv_case(shape, W, io, flags, seed=100)
    b, L, D = shape
    dout, dlast = io_values(rng, shape, io), io_values(rng, (b, W - 1, D), io) if "w" in flags else None
    want = ref.conv_bwd(c["x"], c["w"], dout, c["bias"], c["window"], c["reset"], c["act"], dlast)
    got = lib.mamba_conv_bwd(dev(c["x"], io), dev(c["w"]), dev(dout, io), bias=dev(c["bias"]),
                             window=dev(c["window"], io), reset=u8(c["reset"]), silu=c["act"],
                             dlast_window=dev(dlast, io))
    assert sorted(got) == sorted(want)
    for k, (v, m) in want.items():
        assert ref.close(host(got[k]), v, m, io if got[k].dtype == torch.bfloat16 else "f32") <= 1, k


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W,D", [(2, 1), (3, 10), (4, 64), (4, 259)])
def test_convolution_token_by_token(W, D, io):
    import selective_state_space_22_amd as lib

    rng, c = _conv_case((3, 9, D), W, io, "bw")
    x, w, bias = dev(c["x"], io), dev(c["w"]), dev(c["bias"])
    out, last = lib.mamba_conv_fwd(x, w, bias=bias, window=dev(c["window"], io))
    window = dev(c["window"], io)
    steps = torch.stack([lib.mamba_conv_update(window, x[:, t].contiguous(), w, bias=bias) for t in range(9)], 1)
    assert torch.equal(steps, out) and torch.equal(window, last)


@pytest.mark.parametrize("cut", [False, True])
def test_convolution_in_pieces_gives_the_same_bits(cut):
    import selective_state_space_22_amd as lib

    rng, c = _conv_case((2, 150, 72), 4, "bf16", "br" if cut else "b")
    x, w, bias, reset = dev(c["x"], "bf16"), dev(c["w"]), dev(c["bias"]), u8(c["reset"])
    out, last = lib.mamba_conv_fwd(x, w, bias=bias, reset=reset)
    window, at, parts = None, 0, []
    for n in (1, 2, 40, 0, 107):
        piece = slice(at, at + n)
        o, window = lib.mamba_conv_fwd(x[:, piece].contiguous(), w, bias=bias, window=window,
                                       reset=None if reset is None else reset[:, piece].contiguous())
        parts.append(o)
        at += n
    assert torch.equal(torch.cat(parts, 1), out) and torch.equal(window, last)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_reset_or_a_length_cuts_off_does_not_leak(bad):
    import selective_state_space_22_amd as lib

    _, c = _conv_case((2, 40, 24), 4, "bf16", "b")
    x, w, bias = dev(c["x"], "bf16"), dev(c["w"]), dev(c["bias"])
    reset = torch.zeros((2, 40), dtype=torch.bool, device="cuda")
    reset[:, 20] = True
    clean, last = lib.mamba_conv_fwd(x, w, bias=bias, reset=reset)
    dirty = x.clone()
    dirty[:, 17:20] = bad
    out, _ = lib.mamba_conv_fwd(dirty, w, bias=bias, reset=reset)
    assert torch.equal(out[:, 20:], clean[:, 20:]) and torch.equal(out[:, :17], clean[:, :17])
    dout = torch.ones_like(x)
    dout[:, 17:20] = 0
    g = lib.mamba_conv_bwd(dirty, w, dout, bias=bias, reset=reset)
    assert torch.equal(g["dx"][:, 20:], lib.mamba_conv_bwd(x, w, dout, bias=bias, reset=reset)["dx"][:, 20:])
    # behind a length nothing is read: the row as if it were that short
    n = torch.tensor([17, 0], dtype=torch.int32, device="cuda")
    short, slast = lib.mamba_conv_fwd(dirty, w, bias=bias, lengths=n)
    assert torch.equal(short[0, :17], clean[0, :17]) and not short[0, 17:].any() and not short[1].any()
    assert torch.equal(slast[0], x[0, 14:17]) and not slast[1].any()


def test_convolution_of_no_tokens_hands_the_window_on():
    import selective_state_space_22_amd as lib

    rng = np.random.default_rng(0)
    window, w = dev(io_values(rng, (2, 3, 9), "bf16"), "bf16"), dev(f32_values(rng, (9, 4)))
    x = torch.empty((2, 0, 9), dtype=torch.bfloat16, device="cuda")
    out, last = lib.mamba_conv_fwd(x, w, window=window)
    assert out.shape == x.shape and torch.equal(last, window)
    assert not lib.mamba_conv_fwd(x, w)[1].any()
    g = lib.mamba_conv_bwd(x, w, x, window=window, dlast_window=window)
    assert torch.equal(g["dwindow"], window) and not g["dweight"].any() and not g["dbias"].any()
    g = lib.mamba_conv_bwd(x[:0], w, x[:0])
    assert not g["dweight"].any() and not g["dbias"].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_convolution_update_with_slots(io):
    import selective_state_space_22_amd as lib

    rng = np.random.default_rng(3)
    pool, x, w = dev(io_values(rng, (7, 3, 33), io), io), dev(io_values(rng, (5, 33), io), io), dev(f32_values(rng, (33, 4)))
    slots = i32([6, -1, 0, 7, 3])  # 7 is no window of the pool
    out = torch.full((5, 33), 9.0, dtype=DT[io], device="cuda")
    before = pool.clone()
    lib.mamba_conv_update(pool, x, w, slots=slots, out=out)
    live = [0, 2, 4]
    place = slots.long()[live]
    own = before[place].contiguous()
    assert torch.equal(lib.mamba_conv_update(own, x[live].contiguous(), w), out[live]) and torch.equal(own, pool[place])
    assert (out[[1, 3]] == 9).all()
    rest = [i for i in range(7) if i not in place.tolist()]
    assert torch.equal(pool[rest], before[rest])


# ------------------------------------------------------------------------------------------ one token

# relative to max(|ref|, rms): 1.4e-5 of the input weight's bracket form, and fp32 sums of at most dim terms
# whose errors add like independent ones: 2 sqrt(dim) 2^-24 for dim up to 768 is 3.3e-6, thrice (r, dt, B C)
STEP_TOL = 3e-5
STEP_SHAPES = [(1, 1, 1, 1), (3, 8, 2, 3), (2, 60, 4, 24), (5, 130, 8, 33), (4, 259, 16, 8), (17, 64, 16, 32),
               (33, 300, 16, 17), (1, 768, 16, 24), (16, 128, 4, 160), (18, 520, 2, 512),
               # tiles of eight rows
               (131, 1030, 16, 33), (517, 130, 4, 24), (1030, 8, 8, 3), (1029, 60, 2, 5), (1027, 5, 1, 2)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 33), (5, 1101)], ids=str)
def test_convolution_update_over_its_input(shape, io):
    import selective_state_space_22_amd as lib

    batch, D = shape
    rng = np.random.default_rng(batch + D)
    window, x, w = dev(io_values(rng, (batch, 2, D), io), io), dev(io_values(rng, (batch, D), io), io), dev(f32_values(rng, (D, 3)))
    apart = window.clone()
    want = lib.mamba_conv_update(apart, x, w)
    assert lib.mamba_conv_update(window, x, w, out=x) is x
    assert torch.equal(x, want) and torch.equal(window, apart)


def test_refusals_of_a_convolution_over_its_inputs():
    import selective_state_space_22_amd as lib

    x, w, window = torch.ones(1, 8, 16, device="cuda"), torch.ones(16, 4, device="cuda"), torch.ones(1, 3, 16, device="cuda")
    for kw in ({"out": x}, {"window": window, "last_window": window}):
        with pytest.raises(lib.MambaError):
            lib.mamba_conv_fwd(x, w, **kw)
    assert (x == 1).all() and (window == 1).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 130, 16, 5), (5, 261, 4, 9), (9, 512, 16, 32)], ids=str)
def test_one_token_over_its_input_and_its_gate(shape, io):
    import selective_state_space_22_amd as lib

    batch, D, N, R = shape
    rng, c = _step_case(shape, 4, io, seed=2)
    state, window = dev(f32_values(rng, (batch, D, N))), dev(io_values(rng, (batch, 3, D), io), io)
    rest = [dev(c["cw"]), dev(c["Wx"], io), dev(c["Wdt"], io), dev(c["A"])]
    want = None
    for over in (None, "x", "z"):
        s, v, t = state.clone(), window.clone(), {k: dev(c[k], io) for k in "xz"}
        got = lib.mamba_conv_ssm_update(s, v, t["x"], *rest, z=t["z"], out=t.get(over))
        want = (got, s, v) if want is None else want
        assert all(torch.equal(a, b) for a, b in zip((got, s, v), want)), over


def _step_case(shape, W, io, seed=0):
    batch, D, N, R = shape
    rng = np.random.default_rng(seed + sum(shape))
    return rng, {
        "x": io_values(rng, (batch, D), io), "z": io_values(rng, (batch, D), io), "cw": f32_values(rng, (D, W), 0.5),
        "cb": f32_values(rng, D, 0.1), "Wx": io_values(rng, (R + 2 * N, D), io, D ** -0.5),
        "Wdt": io_values(rng, (D, R), io, R ** -0.5), "A": -np.asarray(rng.random((D, N)) * N + 0.1, np.float32).astype(float),
        "dt_bias": f32_values(rng, D) - 3, "Dskip": f32_values(rng, D)}


def _step(c, state, window, io, slots=None, out=None, drop=()):
    import selective_state_space_22_amd as lib

    v = {k: None if k in drop else a for k, a in c.items()}
    return lib.mamba_conv_ssm_update(
        state, window, dev(v["x"], io), dev(v["cw"]), dev(v["Wx"], io), dev(v["Wdt"], io), dev(v["A"]),
        conv_bias=dev(v["cb"]), z=dev(v["z"], io), dt_bias=dev(v["dt_bias"]), Dskip=dev(v["Dskip"]), slots=slots, out=out)


def _far(got, want):
    rms = np.sqrt(np.mean(want * want)) if want.size else 0.0
    assert np.isfinite(got).all()
    return np.max(np.abs(got - want) / np.maximum(np.maximum(np.abs(want), rms), 1e-300)) if want.size else 0.0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("shape", STEP_SHAPES, ids=str)
def test_one_token(shape, W, io):
    batch, D, N, R = shape
    rng, c = _step_case(shape, W, io)
    drop = () if W == 4 else ("cb", "z", "dt_bias", "Dskip")
    state, window = f32_values(rng, (batch, D, N)), io_values(rng, (batch, W - 1, D), io)
    v = {k: None if k in drop else a for k, a in c.items()}
    h, win, out = ref.conv_ssm_step(state, window, v["x"], v["cw"], v["cb"], v["Wx"], v["Wdt"], v["A"], v["z"],
                                    v["dt_bias"], v["Dskip"])
    gs, gw = dev(state), dev(window, io)
    got = _step(c, gs, gw, io, drop=drop)
    assert _far(host(gs), h) <= STEP_TOL
    assert np.array_equal(host(gw), win)
    assert _far(host(got), out) <= 3 * STEP_TOL + ref.HALF[io]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 40, 16, 5), (21, 200, 16, 24), (6, 70, 2, 8), (517, 130, 16, 40)], ids=str)
def test_one_token_with_slots(shape, io):
    batch, D, N, R = shape
    rng, c = _step_case(shape, 4, io, seed=1)
    places = 2 * batch + 1
    state, window = f32_values(rng, (places, D, N)), io_values(rng, (places, 3, D), io)
    slots = rng.permutation(places)[:batch].astype(np.int32)
    if batch > 1:
        slots[1], slots[-1] = -5, places
    before = np.full((batch, D), 7.0)
    h, win, out = ref.conv_ssm_step(state, window, c["x"], c["cw"], c["cb"], c["Wx"], c["Wdt"], c["A"], c["z"],
                                    c["dt_bias"], c["Dskip"], slots, before)
    gs, gw, go = dev(state), dev(window, io), dev(before, io)
    _step(c, gs, gw, io, slots=i32(slots), out=go)
    idle = [i for i in range(places) if i not in slots.tolist()]
    assert np.array_equal(host(gs)[idle], state[idle]) and np.array_equal(host(gw), win)
    assert (host(go)[(slots < 0) | (slots >= places)] == 7).all()
    live = (slots >= 0) & (slots < places)
    assert _far(host(gs)[slots[live]], h[slots[live]]) <= STEP_TOL
    assert _far(host(go)[live], out[live]) <= 3 * STEP_TOL + ref.HALF[io]


def test_a_row_does_not_depend_on_the_batch_around_it():
    # the same bits for rows of batches that take the join launch, and of those that do not too
    for shape in ((40, 136, 16, 24), (4, 136, 16, 24)):
        rng, c = _step_case(shape, 4, "bf16")
        state, window = f32_values(rng, (shape[0], 136, 16)), io_values(rng, (shape[0], 3, 136), "bf16")
        gs, gw = dev(state), dev(window, "bf16")
        out = _step(c, gs, gw, "bf16")
        for r in (0, shape[0] - 1):
            one = {k: v[r:r + 1] if k in ("x", "z") else v for k, v in c.items()}
            s1, w1 = dev(state[r:r + 1]), dev(window[r:r + 1], "bf16")
            assert torch.equal(_step(one, s1, w1, "bf16"), out[r:r + 1]) and torch.equal(s1, gs[r:r + 1])


def test_one_token_with_a_zero_state_matrix_and_a_held_state():
    # A = 0 takes the limit dt of the input weight; a dt that underflows leaves the state bit for bit
    rng, c = _step_case((2, 70, 16, 9), 4, "f32")
    c["A"][::3] = 0
    state, window = f32_values(rng, (2, 70, 16)), io_values(rng, (2, 3, 70), "f32")
    h, _, _ = ref.conv_ssm_step(state, window, c["x"], c["cw"], c["cb"], c["Wx"], c["Wdt"], c["A"], c["z"], c["dt_bias"],
                                c["Dskip"])
    gs = dev(state)
    _step(c, gs, dev(window), "f32")
    assert _far(host(gs), h) <= STEP_TOL
    c["dt_bias"] = np.full(70, -1e4)
    gs = dev(state)
    _step(c, gs, dev(window), "f32")
    assert np.array_equal(host(gs), state)


# ------------------------------------------------------------------------------------------ norms

NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (2, 511), (4, 512), (3, 513), (9, 776), (2, 1101), (3, 2050), (2, 2560),
               (1, 4095), (2, 4097), (2, 5000), (3, 5121), (2, 6144), (2, 6145), (1, 8192), (2, 12001), (1, 16384)]
NORM_FLAGS = ["", "p", "gPsrp", "aPsrp", "gr", "aPp", "sr", "gsrp"]


def _norm_case(shape, flags, io, res, seed=0):
    """flags: g gate first, a gate after, P post weight, s scale, r residual, p pre weight."""
    rng = np.random.default_rng(seed + sum(shape))
    M, D = shape
    x = io_values(rng, shape, io)
    kw = {"pre": 1 + f32_values(rng, D, 0.3) if "p" in flags else None,
          "gate": io_values(rng, shape, io) if "g" in flags or "a" in flags else None,
          "post": 1 + f32_values(rng, D, 0.3) if "P" in flags else None,
          "scale": f32_values(rng, D) if "s" in flags else None,
          "residual": io_values(rng, shape, res, 3.0) if "r" in flags else None, "gate_first": "a" not in flags}
    for k in ("pre", "post"):
        if kw[k] is not None:
            kw[k] = kw[k].astype(np.float32).astype(float)
    return rng, x, kw


def _norm_args(kw, io, res):
    return {"gate": dev(kw["gate"], io), "post_weight": dev(kw["post"]), "scale": dev(kw["scale"]),
            "residual": dev(kw["residual"], res), "gate_first": kw["gate_first"]}


TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("flags", NORM_FLAGS)
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_norm(shape, flags, io, res):
    import selective_state_space_22_amd as lib

    _, x, kw = _norm_case(shape, flags, io, res)
    alpha, eps = float(np.float32(0.7)), float(np.float32(1e-5))
    out, r, om, rm = ref.norm_fwd(x, alpha=alpha, eps=eps, **kw)
    got, gr = lib.mamba_residual_norm_fwd(dev(x, io), dev(kw["pre"]), alpha=alpha, eps=eps, res_dtype=DT[res],
                                          **_norm_args(kw, io, res))
    assert gr.dtype == DT[res] and ref.close(host(gr), r, rm, res) <= 1
    assert (got is None) == (out is None)
    if out is not None:
        assert got.dtype == DT[io] and ref.close(host(got), out, om, io) <= 1


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("flags", NORM_FLAGS)
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_norm_gradients(shape, flags, io, res):
    import selective_state_space_22_amd as lib

    rng, x, kw = _norm_case(shape, flags, io, res, seed=50)
    alpha, eps = float(np.float32(-1.3)), float(np.float32(1e-5))
    dout = io_values(rng, shape, io) if "p" in flags else None
    dres = io_values(rng, shape, res) if len(flags) % 2 == 0 else None
    want = ref.norm_bwd(x, dout=dout, dres=dres, alpha=alpha, eps=eps, **kw)
    got = lib.mamba_residual_norm_bwd(dev(x, io), dev(kw["pre"]), dev(dout, io), dresidual_out=dev(dres, res), alpha=alpha,
                                      eps=eps, res_dtype=DT[res], **_norm_args(kw, io, res))
    assert sorted(got) == sorted(want)
    for k, (v, m) in want.items():
        assert ref.close(host(got[k]), v, m, "bf16" if got[k].dtype == torch.bfloat16 else "f32") <= 1, k


@pytest.mark.parametrize("rows,D", [(2049, 40), (2500, 520), (4097, 1101), (2100, 2560), (2048, 4096), (300, 4609), (70, 5124), (40, 6147)])
def test_norm_of_many_rows_is_that_of_few(rows, D):
    import selective_state_space_22_amd as lib

    _, x, kw = _norm_case((16, D), "gPsrp", "bf16", "f32")
    pick = np.random.default_rng(0).integers(0, 16, rows)
    x, kw = x[pick], {k: v[pick] if k in ("gate", "residual") else v for k, v in kw.items()}
    alpha, eps = 0.5, float(np.float32(1e-5))
    out, r, om, rm = ref.norm_fwd(x, alpha=alpha, eps=eps, **kw)
    got, gr = lib.mamba_residual_norm_fwd(dev(x, "bf16"), dev(kw["pre"]), alpha=alpha, eps=eps, **_norm_args(kw, "bf16", "f32"))
    assert ref.close(host(got), out, om, "bf16") <= 1 and ref.close(host(gr), r, rm, "f32") <= 1
    rng = np.random.default_rng(1)
    dout, dres = io_values(rng, (rows, D), "bf16"), f32_values(rng, (rows, D))
    want = ref.norm_bwd(x, dout=dout, dres=dres, alpha=alpha, eps=eps, **kw)
    got = lib.mamba_residual_norm_bwd(dev(x, "bf16"), dev(kw["pre"]), dev(dout, "bf16"), dresidual_out=dev(dres), alpha=alpha,
                                      eps=eps, **_norm_args(kw, "bf16", "f32"))
    for k, (v, m) in want.items():
        assert ref.close(host(got[k]), v, m, "bf16" if got[k].dtype == torch.bfloat16 else "f32") <= 1, k


@pytest.mark.parametrize("D", [96, 1101, 4096])
def test_norm_in_place(D):
    import selective_state_space_22_amd as lib

    rng, x, kw = _norm_case((7, D), "gPsrp", "bf16", "bf16")
    args = _norm_args(kw, "bf16", "bf16")
    x, pre = dev(x, "bf16"), dev(kw["pre"])
    out, r = lib.mamba_residual_norm_fwd(x, pre, **args)
    x2, args2 = x.clone(), {**args, "residual": args["residual"].clone()}
    lib.mamba_residual_norm_fwd(x2, pre, out=x2, residual_out=args2["residual"], **args2)
    assert torch.equal(x2, out) and torch.equal(args2["residual"], r)
    dout, dres = dev(io_values(rng, (7, D), "bf16"), "bf16"), dev(io_values(rng, (7, D), "bf16"), "bf16")
    g = lib.mamba_residual_norm_bwd(x, pre, dout, dresidual_out=dres, **args)
    x3, args3, dres3 = x.clone(), {**args, "gate": args["gate"].clone()}, dres.clone()
    lib.mamba_residual_norm_bwd(x3, pre, dout, dresidual_out=dres3, grads={"dx": x3, "dgate": args3["gate"], "dresidual": dres3},
                                **args3)
    assert torch.equal(x3, g["dx"]) and torch.equal(args3["gate"], g["dgate"]) and torch.equal(dres3, g["dresidual"])


def test_norm_of_rows_of_zeros_and_of_what_is_no_number():
    import selective_state_space_22_amd as lib

    x = torch.zeros((4, 520), device="cuda")
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    x[3] = 1
    pre = torch.ones(520, device="cuda")
    out, r = lib.mamba_residual_norm_fwd(x, pre, post_weight=pre, eps=1e-6)
    assert not out[0].any() and out[1].isnan().all() and out[2].isnan().any() and torch.isfinite(out[3]).all()
    g = lib.mamba_residual_norm_bwd(x, pre, torch.ones_like(x), post_weight=pre, eps=1e-6)
    assert torch.isfinite(g["dx"][[0, 3]]).all() and g["dx"][1].isnan().all()


def test_norm_of_no_rows():
    import selective_state_space_22_amd as lib

    x, w = torch.empty((0, 33), device="cuda"), torch.ones(33, device="cuda")
    out, r = lib.mamba_residual_norm_fwd(x, w)
    assert out.shape == r.shape == (0, 33)
    g = lib.mamba_residual_norm_bwd(x, w, x, post_weight=w, scale=w)
    assert all(not g[k].any() for k in ("dpost_weight", "dscale", "dpre_weight"))


# ------------------------------------------------------------------------------------------ verification


def _verify_case(rows, K, V, io, seed=0, near=0.3):
    rng = np.random.default_rng(seed + rows + K + V)
    logits = 2 * rng.normal(size=(rows, K + 1, V))
    soft = lambda v: np.exp(v - v.max(-1, keepdims=True)) / np.exp(v - v.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
    p, q = soft(logits), soft(logits[:, :K] + near * rng.normal(size=(rows, K, V)))
    rounded = [torch.from_numpy(v.astype(np.float32)).to(DT[io]) for v in (p, q)]
    drafted = np.array([[rng.choice(V, p=q[r, k]) for k in range(K)] for r in range(rows)], np.int64).reshape(rows, K)
    return {"p": rounded[0], "q": rounded[1], "drafted": drafted, "uniform": rng.random((rows, K)).astype(np.float32),
            "noise": rng.exponential(size=(rows, V)).astype(np.float32)}


def _verify(c, counts=None):
    import selective_state_space_22_amd as lib

    tokens, kept = lib.mamba_draft_verify(c["p"].cuda(), c["q"].cuda(), torch.from_numpy(c["drafted"]).cuda(),
                                          torch.from_numpy(c["uniform"]).cuda(), torch.from_numpy(c["noise"]).cuda(),
                                          counts=i32(counts) if counts is not None else None)
    return tokens.cpu().numpy(), kept.cpu().numpy()


def _verify_check(c, counts=None):
    rows, K = c["drafted"].shape
    tokens, kept = _verify(c, counts)
    p, q = c["p"].float().numpy(), c["q"].float().numpy()
    for r in range(rows):
        want, n = ref.verify_row(p[r], q[r], c["drafted"][r], c["uniform"][r], c["noise"][r],
                                 K if counts is None else counts[r])
        assert kept[r] == n and np.array_equal(tokens[r], want), (r, kept[r], n, tokens[r], want)
    return kept


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,K,V", [(1, 1, 1), (1, 0, 5), (3, 2, 7), (2, 5, 1000), (65, 3, 4099), (1, 4, 50000),
                                      (2, 70, 33), (1, 130, 9), (4, 3, 2048), (1500, 1, 40), (300, 2, 4099),
                                      (1, 2, 16384), (2, 2, 16385), (256, 1, 2049)])
def test_verification(rows, K, V, io):
    _verify_check(_verify_case(rows, K, V, io))


def test_verification_of_drafts_that_all_stay_and_that_never_do():
    c = _verify_case(4, 6, 300, "f32", near=0.0)
    c["uniform"][:] = 0.999
    c["q"] = c["p"][:, :6] * 0.5
    assert (_verify_check(c) == 6).all()
    c["uniform"][:] = 1.0
    c["q"] = c["p"][:, :6] * 2
    assert (_verify_check(c) == 0).all()


def test_verification_with_counts():
    c = _verify_case(7, 5, 500, "bf16", near=0.05)
    _verify_check(c, [-3, 0, 1, 2, 5, 9, 4])


def test_verification_where_the_distributions_are_equal():
    # a refusal of equal distributions leaves no weight above 0: the target's own decides
    c = _verify_case(5, 3, 5000, "f32", near=0.0)
    c["q"] = c["p"][:, :3].clone()
    c["uniform"][:] = 1.0
    assert (_verify_check(c) == 0).all()


def test_verification_of_bad_values():
    c = _verify_case(6, 3, 700, "f32")
    c["drafted"][0, 0], c["drafted"][1, 1] = -1, 700
    c["drafted"][2, 0] = 1 << 40
    c["noise"][3, ::2] = -1.0
    c["noise"][3, 1::4] = np.nan
    c["noise"][4, 11] = 0.0
    c["noise"][4, 13] = -0.0
    p = c["p"]
    p[5, :, ::3] = float("nan")
    _verify_check(c)
    c["p"] = torch.zeros_like(p)
    tokens, kept = _verify(c)
    assert (kept == 0).all() and (tokens == -1).all()
    c["noise"][:] = -1.0  # nothing can win: the lowest index of what has weight
    c["p"][:, :, 20:30] = 0.1
    _verify_check(c)


def test_verification_where_the_drafts_probabilities_are_nan():
    c = _verify_case(4, 3, 600, "f32")
    c["q"][0, 0] = float("nan")        # refused; nothing of p - q is above 0: the target's own decides
    c["q"][1, 0, ::2] = float("nan")
    c["uniform"][1, 0] = 1.0
    c["q"][2, 1, c["drafted"][2, 1]] = float("nan")
    assert _verify_check(c)[0] == 0


def test_verification_prefers_the_lowest_index_of_equal_scores():
    c = _verify_case(3, 2, 9000, "f32")
    c["p"][:] = 0.25
    c["q"][:] = 0.5
    c["uniform"][:] = 1.0
    c["noise"][:] = 2.0
    c["noise"][1, [8000, 4000, 6000]] = 1.0
    tokens, kept = _verify(c)
    assert kept.tolist() == [0, 0, 0] and tokens[:, 0].tolist() == [0, 4000, 0]


# ------------------------------------------------------------------------------------------ calls


def test_refusals_of_the_binding():
    import selective_state_space_22_amd as lib

    f = lambda *s, **k: torch.zeros(s, device="cuda", **k)  # noqa: E731
    x, w = f(2, 8, 16), f(16, 4)
    for bad in (lambda: lib.mamba_conv_fwd(x, f(16, 5)), lambda: lib.mamba_conv_fwd(x, f(16, 1)),
                lambda: lib.mamba_residual_norm_fwd(x, w[:, 0].contiguous(), eps=0.0),
                lambda: lib.mamba_residual_norm_fwd(x, w[:, 0].contiguous(), alpha=float("inf")),
                lambda: lib.mamba_residual_norm_fwd(f(1, 16392), f(16392)),
                lambda: lib.mamba_conv_update(f(1, 3, 16), x[:, 0].contiguous(), w),
                lambda: lib.mamba_conv_ssm_update(f(2, 16, 3), f(2, 3, 16), x[:, 0].contiguous(), w, f(8, 16), f(16, 2),
                                                  f(16, 3))):
        with pytest.raises(lib.MambaError):
            bad()
    for bad in (lambda: lib.mamba_conv_fwd(x[:, :, ::2], w), lambda: lib.mamba_conv_fwd(x, w, window=f(2, 2, 16)),
                lambda: lib.mamba_conv_fwd(x.cpu(), w), lambda: lib.mamba_conv_bwd(x, w, x[:, :4]),
                lambda: lib.mamba_residual_norm_bwd(x, w[:, 0].contiguous()),
                lambda: lib.mamba_draft_verify(f(2, 2, 9), f(2, 2, 9), f(2, 2, dtype=torch.int64), f(2, 2), f(2, 9)),
                lambda: lib.mamba_conv_fwd(x.transpose(0, 1), w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.mamba_conv_fwd(x.half(), w), lambda: lib.mamba_conv_fwd(x, w.bfloat16()),
                lambda: lib.mamba_conv_fwd(x, w, reset=f(2, 8)), lambda: lib.mamba_conv_fwd(x, w, lengths=f(2)),
                lambda: lib.mamba_residual_norm_fwd(x, residual=x.bfloat16()),
                lambda: lib.mamba_conv_update(f(2, 3, 16), x[:, 0].contiguous(), w, slots=f(2, dtype=torch.int64))):
        with pytest.raises(TypeError):
            bad()


def test_calls_on_another_stream_and_twice():
    import selective_state_space_22_amd as lib

    _, c = _conv_case((2, 300, 100), 4, "bf16", "b")
    x, w, bias = dev(c["x"], "bf16"), dev(c["w"]), dev(c["bias"])
    pre, noise = torch.ones(100, device="cuda"), torch.rand((2, 30000), device="cuda")
    p, d, u = torch.rand((2, 3, 30000), device="cuda"), torch.zeros((2, 2), dtype=torch.int64, device="cuda"), torch.rand((2, 2), device="cuda")

    def work():
        g = lib.mamba_conv_bwd(x, w, x, bias=bias)
        n = lib.mamba_residual_norm_bwd(x, pre, x, residual=x, post_weight=pre)
        t = lib.mamba_draft_verify(p, p[:, :2].contiguous(), d, u, noise)
        return [*lib.mamba_conv_fwd(x, w, bias=bias), *g.values(), *n.values(), *t]

    want = work()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(work())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("D", [513, 1101, 4099, 5001])
def test_an_infinity_in_a_row_that_chunks_share(D):
    # rms is infinite: what is finite becomes 0, the infinity itself no number
    import selective_state_space_22_amd as lib

    x = torch.ones((3, D), device="cuda")
    x[0, D - 1], x[1, D - 3], x[2, 0] = float("inf"), -float("inf"), float("inf")
    w = torch.ones(D, device="cuda")
    out, _ = lib.mamba_residual_norm_fwd(x, w, post_weight=None)
    assert out.isnan().sum(1).tolist() == [1, 1, 1] and not torch.nan_to_num(out).any()
