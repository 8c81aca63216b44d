"""The layer operators at the sizes that real calls have, where the small cases of test_gpu_layer.py do not reach: the
convolution with more than the fewest tokens to a thread, one token's products of more matrix steps than are loaded ahead in
every tile, gradients of many long rows.  References are fp64 with the tolerances of layer_ref.py; those of the convolution are
formed for all tokens at once, on the GPU."""
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
    yield
    torch.cuda.empty_cache()


def _excess(got, want, mag, io):
    """layer_ref.close for tensors on the GPU."""
    assert got.shape == want.shape
    tol = ref.HALF[io] * (1 + 1e-3) * want.abs() + ref.U * mag
    off = torch.where(torch.isfinite(got), (got.double() - want).abs(), float("inf"))
    return float((off / tol.clamp(min=1e-300)).max())


def _silu_slope(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


class Conv:
    """x, weight, ... of a shape, and the definition over all tokens."""

    def __init__(self, shape, W, io, flags):
        g = torch.Generator("cuda").manual_seed(sum(shape) + W)

        def randn(*s, scale=1.0):
            return torch.randn(s, generator=g, device="cuda") * scale

        b, L, D = shape
        self.W, self.io, self.act = W, io, "n" not in flags
        self.x, self.dout = randn(*shape).to(DT[io]), randn(*shape).to(DT[io])
        self.w, self.bias = randn(D, W, scale=0.6), randn(D, scale=0.2)
        self.window = randn(b, W - 1, D).to(DT[io]) if "w" in flags else None
        self.dlast = randn(b, W - 1, D).to(DT[io]) if "w" in flags else None
        self.reset = torch.rand((b, L), generator=g, device="cuda") < 0.02 if "r" in flags else None
        if self.reset is not None:  # a long stretch without any, and some one after the other
            self.reset[:, L // 3: L // 3 + 300] = False
            self.reset[:, 37:43] = True
        before = self.x.new_zeros((b, W - 1, D)) if self.window is None else self.window
        self.full = torch.cat([before, self.x], 1).double()
        document = torch.zeros((b, L), device="cuda", dtype=torch.int64) if self.reset is None else self.reset.long().cumsum(1)
        self.of = torch.cat([document.new_zeros((b, W - 1)), document], 1)
        self.L = L

    def sees(self, j):
        """Whether token t sees its tap j, the input W - 1 - j tokens back."""
        return (self.of[:, j:j + self.L] == self.of[:, self.W - 1:]).unsqueeze(-1)

    def sums(self):
        """c, and the sum of the magnitudes in it."""
        c = self.bias.double().expand(self.x.shape).clone()
        mag = c.abs()
        for j in range(self.W):
            v = torch.where(self.sees(j), self.full[:, j:j + self.L] * self.w[:, j].double(), 0.0)
            c += v
            mag += v.abs()
        return c, mag

    def forward(self, n):
        """out, last_window and out's magnitude where row b has n[b] tokens."""
        W, (b, L, D) = self.W, self.x.shape
        c, mag = self.sums()
        out = c * torch.sigmoid(c) if self.act else c
        m = 1.1 * (W + 1) * mag + (out.abs() * (c.abs() + 8) if self.act else 0)
        alive = (torch.arange(L, device="cuda") < n.unsqueeze(1)).unsqueeze(-1)
        at, row = n.unsqueeze(1) + torch.arange(W - 1, device="cuda"), torch.arange(b, device="cuda").unsqueeze(1)
        same = self.of[row, at] == self.of[row, n.unsqueeze(1) + W - 2]
        last = torch.where(same.unsqueeze(-1), self.full[row, at], 0.0)
        return torch.where(alive, out, 0.0), last, torch.where(alive, m, 0.0)

    def backward(self):
        W, L, (b, _, D) = self.W, self.L, self.x.shape
        c, mag = self.sums()
        dout = self.dout.double()
        g = dout * _silu_slope(c) if self.act else dout
        gm = 2 * g.abs() + (dout.abs() * (0.5 * mag + 12 + 2 * c.abs()) if self.act else 0)
        depth = 128 + 32 + b * L / 8 / 32 + 4
        dfull, dm = torch.zeros_like(self.full), torch.zeros_like(self.full)
        dw, dwm = torch.zeros_like(self.w, dtype=torch.float64), torch.zeros_like(self.w, dtype=torch.float64)
        for j in range(W):
            w, tap, see = self.w[:, j].double(), self.full[:, j:j + L], self.sees(j)
            dfull[:, j:j + L] += torch.where(see, g * w, 0.0)
            dm[:, j:j + L] += torch.where(see, w.abs() * (gm + (W + 2) * g.abs()), 0.0)
            dw[:, j] = torch.where(see, g * tap, 0.0).sum((0, 1))
            dwm[:, j] = torch.where(see, tap.abs() * (gm + depth * g.abs()), 0.0).sum((0, 1))
        if self.dlast is not None:
            same = (self.of[:, L:] == self.of[:, L + W - 2:L + W - 1]).unsqueeze(-1)
            dfull[:, L:] += torch.where(same, self.dlast.double(), 0.0)
            dm[:, L:] += torch.where(same, (W + 2) * self.dlast.double().abs(), 0.0)
        return {"dx": (dfull[:, W - 1:], dm[:, W - 1:]), "dwindow": (dfull[:, :W - 1], dm[:, :W - 1]), "dweight": (dw, dwm),
                "dbias": (g.sum((0, 1)), (gm + depth * g.abs()).sum((0, 1)))}


# Tokens to a thread, forward and gradients: 16 and 16, 32 and 44, 32 and 64, 32 and 128, 12 and 12
LONG = [(3, 1537, 1101), (1, 4099, 4100), (8, 2048, 1536), (2, 16411, 1601), (5, 250, 3500)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W,flags", [(4, "r"), (4, "wr"), (3, "w"), (2, "rn")])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_convolution_of_long_chunks(shape, W, flags, io):
    import selective_state_space_22_amd as lib

    b, L, D = shape
    c = Conv(shape, W, io, flags)
    short = torch.tensor([L - 1, L // 2 + 5, 0, 13, L // 3 + 100, 36, 1, L][:b], device="cuda")
    for n in (torch.full((b,), L, device="cuda"), short):
        want, last, m = c.forward(n)
        lengths = None if n is not short else n.to(torch.int32)
        out, glast = lib.mamba_conv_fwd(c.x, c.w, bias=c.bias, window=c.window, reset=c.reset, lengths=lengths, silu=c.act)
        assert _excess(out, want, m, io) <= 1
        assert torch.equal(glast.double(), last)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W,flags", [(4, "r"), (4, "wr"), (3, "w"), (2, "rn")])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_convolution_gradients_of_long_chunks(shape, W, flags, io):
    import selective_state_space_22_amd as lib

    c = Conv(shape, W, io, flags)
    got = lib.mamba_conv_bwd(c.x, c.w, c.dout, bias=c.bias, window=c.window, reset=c.reset, silu=c.act, dlast_window=c.dlast)
    want = c.backward()
    assert sorted(got) == sorted(want)
    for k, (v, m) in want.items():
        assert _excess(got[k], v, m, io if got[k].dtype == torch.bfloat16 else "f32") <= 1, k


def _host(t):
    return t.double().cpu().numpy()


# relative to max(|ref|, rms) as in test_gpu_layer.py: 1.4e-5 of the input weight, three sums of at most 1030 terms
STEP_TOL = 3e-5


def _far(got, want):
    assert np.isfinite(got).all()
    return np.max(np.abs(got - want) / np.maximum(np.abs(want), np.sqrt(np.mean(want * want))))


# tiles of eight rows, then of four; ranks of one to sixteen matrix steps, a part of a step behind them
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("pool", [False, True])
@pytest.mark.parametrize("shape", [(131, 1030, 16, 160), (131, 1030, 16, 512), (517, 130, 4, 97), (1030, 8, 1, 200),
                                   (1029, 60, 2, 65), (520, 129, 8, 161), (7, 1030, 16, 161), (3, 1030, 8, 449),
                                   (1, 1030, 16, 193)], ids=str)
def test_one_token_of_larger_ranks(shape, pool, io):
    import selective_state_space_22_amd as lib

    batch, D, N, R = shape
    rng = np.random.default_rng(sum(shape))

    def values(*s, scale=1.0, dtype=torch.float32):
        return torch.from_numpy(np.asarray(rng.normal(size=s) * scale, np.float32)).to("cuda", dtype)

    t = DT[io]
    places = 2 * batch + 1 if pool else batch
    x, z, cw, cb = values(batch, D, dtype=t), values(batch, D, dtype=t), values(D, 4, scale=0.5), values(D, scale=0.1)
    Wx, Wdt = values(R + 2 * N, D, scale=D ** -0.5, dtype=t), values(D, R, scale=R ** -0.5, dtype=t)
    A = torch.from_numpy(-np.asarray(rng.random((D, N)) * N + 0.1, np.float32)).cuda()
    dtb, ds = values(D) - 3, values(D)
    state, window = values(places, D, N), values(places, 3, D, dtype=t)
    slots = None
    if pool:
        slots = torch.from_numpy(rng.permutation(places)[:batch].astype(np.int32)).cuda()
        if batch > 1:
            slots[batch // 2] = -1
    out = torch.full((batch, D), 7.0, device="cuda", dtype=t)
    want = ref.conv_ssm_step(*(_host(v) for v in (state, window, x, cw, cb, Wx, Wdt, A, z, dtb, ds)),
                             None if slots is None else slots.cpu().numpy(), _host(out))
    lib.mamba_conv_ssm_update(state, window, x, cw, Wx, Wdt, A, conv_bias=cb, z=z, dt_bias=dtb, Dskip=ds, slots=slots, out=out)
    assert _far(_host(state), want[0]) <= STEP_TOL
    assert np.array_equal(_host(window), want[1])
    assert _far(_host(out), want[2]) <= 3 * STEP_TOL + ref.HALF[io]


@pytest.mark.parametrize("io,res", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,D", [(1300, 776), (700, 2052), (515, 3001), (130, 8191), (90, 8192), (70, 8193), (50, 12003),
                                    (40, 16384)])
def test_norm_of_many_long_rows(rows, D, io, res):
    import selective_state_space_22_amd as lib

    rng = np.random.default_rng(rows + D)

    def values(*s, scale=1.0, dtype=torch.float32):
        return torch.from_numpy(np.asarray(rng.normal(size=s) * scale, np.float32)).to("cuda", dtype)

    t, r = DT[io], DT[res]
    x, gate, dout, residual, dres = (values(rows, D, dtype=d) for d in (t, t, t, r, r))
    pre, post, scale = (1 + values(D, scale=0.3) for _ in range(3))
    alpha, eps = 0.5, float(np.float32(1e-5))
    for first in (True, False):
        kw = {"gate": _host(gate), "post": _host(post), "scale": _host(scale), "residual": _host(residual),
              "gate_first": first, "alpha": alpha, "eps": eps}
        args = {"gate": gate, "post_weight": post, "scale": scale, "residual": residual, "gate_first": first, "alpha": alpha,
                "eps": eps}
        want, rsum, om, rm = ref.norm_fwd(_host(x), _host(pre), **kw)
        out, rout = lib.mamba_residual_norm_fwd(x, pre, **args)
        assert ref.close(_host(out), want, om, io) <= 1 and ref.close(_host(rout), rsum, rm, res) <= 1
        grads = ref.norm_bwd(_host(x), _host(pre), _host(dout), _host(dres), **kw)
        got = lib.mamba_residual_norm_bwd(x, pre, dout, dresidual_out=dres, **args)
        assert sorted(got) == sorted(grads)
        for k, (v, m) in grads.items():
            assert ref.close(_host(got[k]), v, m, "bf16" if got[k].dtype == torch.bfloat16 else "f32") <= 1, k
