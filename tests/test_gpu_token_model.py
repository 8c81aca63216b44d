"""The example model on the token-model operators: its logits and gradients against plain float64
torch, its steps against its scan, and that it learns and says what it learned.

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


def _plain_logits(p, scale, ids, reset):
    """The model in CPU float64: p its parameters by name."""
    x = scale * p["table"][ids]
    u, a, g, z = (x @ p["w_in"]).chunk(4, -1)
    log_a = -8.0 * torch.nn.functional.softplus(p["lam"]) * torch.sigmoid(a)
    h, ys = torch.zeros_like(u[:, 0]), []
    for t in range(ids.shape[1]):
        keep = ~reset[:, t, None]
        decay = torch.where(keep, torch.exp(log_a[:, t]), 0.0)
        weight = torch.where(keep, torch.sqrt(-torch.expm1(2 * log_a[:, t])), 1.0)
        h = decay * h + weight * torch.sigmoid(g[:, t]) * u[:, t]
        ys.append(h * torch.nn.functional.silu(z[:, t]))
    return (x + torch.stack(ys, 1) @ p["w_out"]) @ p["table"].t()


def _err(a, b):
    return parity_error(a.detach().double().cpu().numpy(), b.detach().double().cpu().numpy())


def test_logits_and_gradients_against_float64():
    from selective_state_space_22_amd import token_model as M

    model = M.TokenModel(vocab=41, dim=24, seed=3)
    ids, target, reset = M.batch_of(torch.Generator().manual_seed(5), 3, 77, 41, 3)
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in model.named_parameters()}
    want = _plain_logits(p, model.scale, ids, reset)
    torch.nn.functional.cross_entropy(want.reshape(-1, 41), target.reshape(-1)).backward()
    got = model(ids.cuda(), reset.cuda())
    assert _err(got, want) <= 1e-4
    torch.nn.functional.cross_entropy(got.reshape(-1, 41), target.reshape(-1).cuda()).backward()
    for k, v in model.named_parameters():
        assert _err(v.grad, p[k].grad) <= 5e-4, k


def test_steps_continue_the_prompt():
    from selective_state_space_22_amd import token_model as M

    model = M.TokenModel(vocab=41, dim=24, seed=4)
    ids = torch.randint(0, 41, (5, 60), generator=torch.Generator().manual_seed(1)).cuda()
    with torch.no_grad():
        whole = model(ids)
    logits, state = model.prefill(ids[:, :50].contiguous())
    assert _err(logits, whole[:, 49]) <= 1e-4
    for t in range(50, 60):
        assert _err(model.step(ids[:, t].contiguous(), state), whole[:, t]) <= 1e-4


def test_learns_to_repeat_a_word():
    from selective_state_space_22_amd import token_model as M

    model = M.TokenModel(vocab=16, dim=64)
    losses = M.train(model, 150, rows=8, length=128, period=1)
    assert losses[-1] < 0.5 * losses[0]
    prompt = torch.tensor([[3] * 8, [9] * 8], device="cuda")
    said = model.generate(prompt, 6, top_k=1)
    assert said.tolist() == [[3] * 6, [9] * 6]
