"""Keys with the same score weigh the same, however large the score is and wherever
the work of a sequence is divided."""
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
@pytest.mark.parametrize("T,g", [(1, 1), (4, 4), (9, 8), (40, 8)])
@pytest.mark.parametrize("q_exp", [0, 16, 40])
def test_equal_scores_of_any_size_weigh_equally(cache, T, g, q_exp):
    """All keys the same: the mean of the values, wherever the keys are divided."""
    lens = [20000, 7001, 1300]

    def same(c, K, V):
        for x in (K, V):
            x[:] = torch.where(x.isnan(), x, torch.ones((), dtype=x.dtype, device="cuda"))
        for b, n in enumerate(lens):  # values that rise along the sequence
            for i in range(-(-n // PAGE)):
                V[int(c.table_cpu[b, i]), :, : min(PAGE, n - i * PAGE)] = (i % 100) / 8.0

    c = Case(cache, lens, [T] * 3, g, 1, 128, seed=T, v_hook=same)
    c.q = torch.full_like(c.q, 2.0 ** q_exp)
    o = c.run()
    for b in range(3):
        rows = slice(c.starts[b], c.starts[b + 1])
        want, tol = chain(c.q[rows], *c.kv(b))
        ref.close(o[rows], want, tol, f"sequence {b}")
    assert bss.attn_sync_status() == 0
