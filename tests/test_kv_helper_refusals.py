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


@pytest.mark.parametrize("max_q,max_seq_len", [(5, (1 << 32) + 100), ((1 << 32) + 5, 100), (5, 1 << 31), (5, -1), (-(1 << 32) + 5, 100)])
def test_sizes_that_wrap_around_are_refused(max_q, max_seq_len):
    """2^32 + 100 keys were taken for 100."""
    q = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, 2, 64, 64, dtype=torch.bfloat16)
    codes, scales = pages.to(torch.uint8), torch.ones(3, 2, 64)
    table, lens, cu = (torch.tensor(x, dtype=torch.int32) for x in ([[0, 1, 2]], [100], [0, 5]))
    with pytest.raises(bss.AttnError, match="31 bits"):
        bss.tree_paged(q, pages, pages, table, lens, cu, max_q, max_seq_len)
    with pytest.raises(bss.AttnError, match="31 bits"):
        bss.tree_paged_e4m3(q, codes, codes, scales, scales, table, lens, cu, max_q, max_seq_len)
