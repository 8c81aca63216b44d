"""The example model reads a prompt as training reads a document: its first token starts anew."""
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


def test_a_prompt_is_read_as_a_document_of_training():
    """Tolerance: float32 throughout, the framework's 1e-4."""
    from selective_state_space_22_amd import token_model as M

    model = M.TokenModel(vocab=41, dim=24, seed=6)
    ids = torch.randint(0, 41, (3, 30), generator=torch.Generator().manual_seed(2)).cuda()
    reset = torch.zeros((3, 30), dtype=torch.bool)
    reset[:, 0] = True  # as batch_of marks a document
    with torch.no_grad():
        whole = model(ids, reset.cuda())
        # and the same document behind another one, in a packed row
        packed = torch.cat([torch.randint(0, 41, (3, 17)).cuda(), ids], 1)
        marks = torch.zeros((3, 47), dtype=torch.bool)
        marks[:, [0, 17]] = True
        behind = model(packed, marks.cuda())[:, 17:]
    assert _err(behind, whole) <= 1e-4
    assert _err(model(ids), whole) <= 1e-4
    logits, state = model.prefill(ids[:, :10].contiguous())
    assert _err(logits, whole[:, 9]) <= 1e-4
    for t in range(10, 30):
        assert _err(model.step(ids[:, t].contiguous(), state), whole[:, t]) <= 1e-4
    first, _ = model.prefill(ids[:, :1].contiguous())
    assert _err(first, whole[:, 0]) <= 1e-4
