"""How the work of tree_paged and tree_paged_e4m3 is divided: a long sequence is shared
out whatever stands beside it, and a limit above the lengths changes nothing."""
import random

import pytest
import torch

import block_skipping_softmax_b200 as bss
from block_skipping_softmax_b200 import build as bss_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    bss_build.build()


@pytest.mark.parametrize("max_q", [1, 4, 16, 64])
@pytest.mark.parametrize("Hkv", [1, 2, 8])
@pytest.mark.parametrize("L", [4096, 32768, 131072])
def test_a_long_sequence_can_be_shared_out_at_any_batch_size(max_q, Hkv, L):
    """One CTA a KV head needs no workspace; its time would be that of the longest sequence."""
    for B in [1, 2, 3, 18, 37, 55, 56, 73, 74, 75, 110, 111, 112, 148, 185, 221, 222, 223, 296, 444, 512, 888]:
        assert bss.attn_tree_workspace_bytes(B, max_q, B * max_q, 4 * Hkv, Hkv, L, 128) > 0, B


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,T,g", [(111, 1, 1), (74, 4, 5), (74, 3, 4)])  # multiples of the CTAs that run at once
@pytest.mark.parametrize("limit", [20000, 131072])
def test_one_long_sequence_among_short_ones(cache, B, T, g, limit):
    from test_tree_batches_gpu import check
    from test_tree_gpu import Case

    rng = random.Random(B)
    lens = [rng.randrange(T, 300) for _ in range(B)]
    lens[B // 2] = 20000
    c = Case(cache, lens, [T] * B, 8 * g, 8, 64, seed=B)
    wide = torch.full((B, -(-limit // 64)), -1, dtype=torch.int32, device="cuda")
    wide[:, : c.max_pages] = c.table
    c.table = wide
    check(c, c.run(max_len=limit))
