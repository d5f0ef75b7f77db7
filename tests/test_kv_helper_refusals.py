"""Calls that the rotation and tree helpers refuse with AttnError before anything else
happens."""
import pytest
import torch

import block_skipping_softmax_b200 as bss
from block_skipping_softmax_b200 import build as bss_build


@pytest.fixture(scope="module", autouse=True)
def built():
    bss_build.build()


def test_a_rotation_needs_positions():
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(bss.AttnError, match="positions"):
        bss.qk_norm_rope(x, x, None, torch.ones(32))
