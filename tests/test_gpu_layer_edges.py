"""The layer operators where lengths, pointers and values are out of the ordinary."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def _randn(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


@pytest.mark.parametrize("length", [5, 2 ** 31 - 1])
@pytest.mark.parametrize("cut", [False, True])
def test_a_length_in_a_row_of_more_than_2_31_tokens(cut, length):
    import selective_state_space_22_amd as lib

    L = 2 ** 31 + 4096
    x, w, bias = torch.ones((1, L, 1), device="cuda", dtype=BF), _randn(1, 4), _randn(1)
    ends = [slice(0, 64), slice(length - 64, length)] if length > 64 else [slice(0, length)]
    for at in ends:
        x[:, at] = _randn(1, at.stop - at.start, 1, dtype=BF, seed=at.stop)
    x[:, length:] = float("nan")  # not to be read
    reset = None
    if cut:
        reset = torch.zeros((1, L), device="cuda", dtype=torch.bool)
        reset[:, [2, max(2, length - 20)]] = True
        reset[:, length:length + 8] = True
    lengths = torch.tensor([length], dtype=torch.int32, device="cuda")
    out, last = lib.mamba_conv_fwd(x, w, bias=bias, reset=reset, lengths=lengths)
    for at in ends:
        window = x[:, at.start - 3:at.start].clone() if at.start else None
        part, plast = lib.mamba_conv_fwd(x[:, at].clone(), w, bias=bias, window=window,
                                         reset=None if reset is None else reset[:, at].clone())
        assert torch.equal(out[:, at], part)
    assert torch.equal(last, plast)
    assert torch.count_nonzero(out[:, length:]) == 0
