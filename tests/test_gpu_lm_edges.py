"""Token-model operators where a shortcut of the kernels could end, against the fp64 reference (lm_ref.py):
sums that a small weight decides, temperatures, differences of logits, rates, gates and faults at the edges
of their ranges.

Tolerances are those of test_gpu_lm.py where no other is derived at a test."""
import numpy as np
import pytest

from test_gpu_lm import _check_sample

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
