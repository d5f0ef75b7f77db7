"""A value that is not finite makes the tokens that see it NaN, however small its
weight, and no others."""
import math

import pytest
import torch

import block_skipping_softmax_b200 as bss
import kv_reference as ref
from block_skipping_softmax_b200 import build as bss_build
from test_tree_batches_gpu import chain
from test_tree_gpu import CACHES, PAGE, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    bss_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,g", [(1, 4), (4, 2), (4, 4), (40, 4)])
@pytest.mark.parametrize("drafted", [False, True])
def test_a_value_that_is_not_finite_counts_at_any_weight(cache, d, T, g, drafted):
    """One key a thousand log2 units below the others: its probability is 0 in 32 bits."""
    lens = [300, 73 + T]
    keys = [n - T + T // 2 if drafted else n - T - 7 for n in lens]

    def spoil(c, K, V):
        K[..., 0] = torch.where(K[..., 0].isnan(), K[..., 0], torch.zeros((), dtype=K.dtype, device="cuda"))
        for b, key in enumerate(keys):
            p = int(c.table_cpu[b, key // PAGE])
            K[p, :, key % PAGE, 0] = -1000.0
            V[p, :, key % PAGE, 3] = math.inf

    c = Case(cache, lens, [T, T], 2 * g, 2, d, seed=d + T, v_hook=spoil)
    c.q.zero_()
    c.q[..., 0] = 8.0
    o = c.run()
    for b, (n, key) in enumerate(zip(lens, keys)):
        K, V = c.kv(b)
        for i in range(T):
            row = o[c.starts[b] + i]
            if n - T + i >= key:
                # e4m3: the whole value is NaN; bf16: its one element at least
                assert row.isnan().all() if cache == "e4m3" else row[:, 3].isnan().all()
            else:
                seen = n - T + i + 1
                want, tol = chain(c.q[c.starts[b] + i][None], K[:, :seen], V[:, :seen])
                ref.close(row[None], want, tol, f"sequence {b} token {i}")
    assert bss.attn_sync_status() == 0
