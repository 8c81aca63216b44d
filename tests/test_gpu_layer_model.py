"""The layer operators as a model uses them: the token model with its convolution and norms against plain float64
torch, its steps against its sequences, drafted generation; and a selective layer's tokens against its prompt.

Tolerances: float32 throughout, so the framework's 1e-4 (max relative error, rms floor) for logits and
5e-4 for gradients, sums over all tokens of both signs."""
import pytest

from gpu_util import parity_error

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _err(a, b):
    return parity_error(a.detach().double().cpu().numpy(), b.detach().double().cpu().numpy())


def _norm(v, w):
    return w * v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-5)


def _plain_logits(p, scale, ids, reset, taps, norms):
    """The model in CPU float64: p its parameters by name."""
    x = scale * p["table"][ids]
    n = _norm(x, p["norm_in"]) if norms else x
    u, a, g, z = (n @ p["w_in"]).chunk(4, -1)
    if taps:
        document, full = reset.long().cumsum(1), torch.nn.functional.pad(u, (0, 0, taps - 1, 0))
        of = torch.nn.functional.pad(document, (taps - 1, 0), value=-1)
        c = p["conv_bias"]
        for j in range(taps):
            same = (of[:, j:j + ids.shape[1]] == document).unsqueeze(-1)
            c = c + torch.where(same, full[:, j:j + ids.shape[1]] * p["conv_weight"][:, j], 0.0)
        u = torch.nn.functional.silu(c)
    log_a = -8.0 * torch.nn.functional.softplus(p["lam"]) * torch.sigmoid(a)
    h, ys = torch.zeros_like(u[:, 0]), []
    for t in range(ids.shape[1]):
        keep = ~reset[:, t, None]
        decay = torch.where(keep, torch.exp(log_a[:, t]), 0.0)
        weight = torch.where(keep, torch.sqrt(-torch.expm1(2 * log_a[:, t])), 1.0)
        h = decay * h + weight * torch.sigmoid(g[:, t]) * u[:, t]
        ys.append(h * torch.nn.functional.silu(z[:, t]))
    y = torch.stack(ys, 1) @ p["w_out"]
    x = _norm(x + p["norm_scale"] * _norm(y, p["norm_block"]), p["norm_out"]) if norms else x + y
    return x @ p["table"].t()


@pytest.mark.parametrize("taps,norms", [(4, True), (2, False), (0, True)])
def test_logits_and_gradients_against_float64(taps, norms):
    from selective_state_space_22_amd import token_model as M

    model = M.TokenModel(vocab=41, dim=24, seed=3, conv=taps, norms=norms)
    ids, target, reset = M.batch_of(torch.Generator().manual_seed(5), 3, 77, 41, 3)
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in model.named_parameters()}
    want = _plain_logits(p, model.scale, ids, reset, taps, norms)
    torch.nn.functional.cross_entropy(want.reshape(-1, 41), target.reshape(-1)).backward()
    got = model(ids.cuda(), reset.cuda())
    assert _err(got, want) <= 1e-4
    torch.nn.functional.cross_entropy(got.reshape(-1, 41), target.reshape(-1).cuda()).backward()
    for k, v in model.named_parameters():
        assert _err(v.grad, p[k].grad) <= 5e-4, k


def test_the_plain_model_is_what_it_was():
    from selective_state_space_22_amd import token_model as M

    a, b = M.TokenModel(vocab=9, dim=16, seed=1), M.TokenModel(vocab=9, dim=16, seed=1, conv=3, norms=True)
    for k, v in a.named_parameters():
        assert torch.equal(v, dict(b.named_parameters())[k])


@pytest.mark.parametrize("taps,norms", [(4, True), (3, False)])
def test_steps_continue_the_prompt(taps, norms):
    from selective_state_space_22_amd import token_model as M

    model = M.TokenModel(vocab=41, dim=24, seed=4, conv=taps, norms=norms)
    ids = torch.randint(0, 41, (5, 60), generator=torch.Generator().manual_seed(1)).cuda()
    with torch.no_grad():
        whole = model(ids)
    logits, state = model.prefill(ids[:, :50].contiguous())
    assert _err(logits, whole[:, 49]) <= 1e-4
    for t in range(50, 60):
        assert _err(model.step(ids[:, t].contiguous(), state), whole[:, t]) <= 1e-4
    assert model.generate(ids, 3, top_k=1).shape == (5, 3)


def test_a_model_that_drafts_for_itself_keeps_every_draft():
    from selective_state_space_22_amd import token_model as M

    model = M.TokenModel(vocab=30, dim=32, seed=2, conv=4, norms=True)
    ids = torch.randint(0, 30, (6, 12), generator=torch.Generator().manual_seed(2)).cuda()
    said = model.speculate(ids, 3, model, drafts=4, generator=torch.Generator("cuda").manual_seed(0))
    assert [len(r) for r in said] == [15] * 6
    assert all(0 <= t < 30 for r in said for t in r)


def test_drafted_tokens_are_the_models_own_where_it_has_one_choice():
    """At a temperature that leaves one token its whole probability, drafted generation says what greedy
    generation says, whatever the drafting model proposes."""
    from selective_state_space_22_amd import token_model as M

    model, draft = M.TokenModel(vocab=30, dim=32, seed=2, conv=3), M.TokenModel(vocab=30, dim=16, seed=9)
    ids = torch.randint(0, 30, (4, 9), generator=torch.Generator().manual_seed(3)).cuda()
    said = model.speculate(ids, 4, draft, drafts=3, temperature=1e-4, generator=torch.Generator("cuda").manual_seed(1))
    want = model.generate(ids, max(len(r) for r in said), top_k=1).tolist()
    for got, line in zip(said, want):
        assert 4 <= len(got) <= 16 and got == line[:len(got)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_selective_layers_tokens_go_on_from_its_prompt(io):
    """Norm, convolution, selective scan, norm over a prompt, then token by token with slots: the outputs of the
    whole sequence.  f32: the framework's 1e-4.  bf16: the sequence rounds the convolution, r, B, C and dt to bf16
    where the token keeps fp32, so they differ by those roundings: the framework's 2e-2."""
    import selective_state_space_22_amd as lib

    t = {"f32": torch.float32, "bf16": torch.bfloat16}[io]
    g = torch.Generator().manual_seed(7)
    batch, L, more, D, N, R = 3, 40, 6, 96, 16, 6

    def randn(*s, scale=1.0, dtype=torch.float32):
        return (torch.randn(s, generator=g) * scale).to("cuda", dtype)

    res, block, z = (randn(batch, L + more, D, dtype=t) for _ in range(3))
    cw, cb, pre, post, scale = randn(D, 4, scale=0.5), randn(D, scale=0.1), randn(D), randn(D), randn(D)
    Wx, Wdt = randn(R + 2 * N, D, scale=D ** -0.5, dtype=t), randn(D, R, scale=R ** -0.5, dtype=t)
    A, dtb, ds = -torch.rand(D, N, generator=g).cuda() * 8 - 0.1, randn(D) - 3, randn(D)
    x, _ = lib.mamba_residual_norm_fwd(block, pre, post_weight=post, scale=scale, residual=res, gate=z, gate_first=False)

    def prompt(n):
        xc, window = lib.mamba_conv_fwd(x[:, :n].contiguous(), cw, bias=cb)
        y, state = lib.mamba_ssm_fwd(xc, Wx, Wdt, A, z=z[:, :n].contiguous(), dt_bias=dtb, Dskip=ds)
        return y, window, state

    whole, _, _ = prompt(L + more)
    _, window, state = prompt(L)
    pool, windows = torch.zeros((7, D, N), device="cuda"), torch.zeros((7, 3, D), device="cuda", dtype=t)
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()], windows[slots.long()] = state, window
    for k in range(L, L + more):
        out = lib.mamba_conv_ssm_update(pool, windows, x[:, k].contiguous(), cw, Wx, Wdt, A, conv_bias=cb,
                                        z=z[:, k].contiguous(), dt_bias=dtb, Dskip=ds, slots=slots)
        assert _err(out, whole[:, k]) <= {"f32": 1e-4, "bf16": 2e-2}[io], k
