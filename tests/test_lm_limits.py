"""The limits on sizes that the header of the token-model operators states are those that the library has
(host only: sizes of workspaces, and refusals before anything is enqueued)."""
import os
import re

import pytest

from selective_state_space_22_amd import binding, lm
from selective_state_space_22_amd import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mamba_mi355x_lm.h")
ERR_DIM = 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(binding.LIB_PATH):
        lib_build.build()
    return lm._lib()


def _documented():
    """(channels, tokens) of the stated bound batch * ceil(dim / channels) * ceil(seqlen / tokens) < 2^31, and
    the longest sequence."""
    text = " ".join(open(HEADER).read().replace("*/", " ").replace("\n *", " ").split())
    c, t = re.search(r"batch \* ceil\(dim / (\d+)\) \* ceil\(seqlen / (\d+)\) < 2\^31", text).groups()
    longest = re.search(r"0 <= seqlen <= 2\^(\d+)", text)
    return int(c), int(t), 1 << int(longest.group(1)) if longest else None


@pytest.mark.parametrize("batch,blocks", [(1, 1), (1, 3), (7, 5), (65535, 1)])
def test_scan_sizes_up_to_the_stated_product(batch, blocks):
    channels, tokens, _ = _documented()
    dim = blocks * channels - channels // 2 if blocks > 1 else channels
    levels = (2 ** 31 - 1) // (batch * blocks)
    for size in (lm.mamba_gated_scan_fwd_workspace_size, lm.mamba_gated_scan_bwd_workspace_size):
        for io in (0, 1):
            assert size(batch, levels * tokens, dim, io) > 0, (batch, blocks, io)
            assert size(batch, levels * tokens + tokens * batch * blocks, dim, io) == 0


def test_scan_length_up_to_the_stated_one(lib):
    _, _, longest = _documented()
    assert longest is not None
    none = [None] * 4
    for L, status in ((longest, 0), (longest + 1, ERR_DIM)):  # no channels: nothing else is in the way
        assert lib.mamba_gated_scan_fwd(1, L, 0, 0, *none, 8.0, *[None] * 7, 0, None) == status
