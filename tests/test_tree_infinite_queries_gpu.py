"""Rows whose visible scores are all -inf: softmax has no value there, so they are
NaN, while a row that sees no key at all is 0."""
import math

import pytest
import torch

import block_skipping_softmax_b200 as bss
from block_skipping_softmax_b200 import build as bss_build
from test_tree_batches_gpu import chain
from test_tree_gpu import CACHES, Case, as_int64
import kv_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    bss_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,g", [(1, 4), (2, 4), (4, 4), (40, 8)])
@pytest.mark.parametrize("lens", [[1, 65, 300], [9000, 7000], [900] * 30])  # one CTA a head; few and many shares
def test_scores_of_minus_infinity_alone_give_nan(cache, d, T, g, lens):
    lens = [max(n, T) for n in lens]

    def negative(c, K, V):
        K[..., 5] = -K[..., 5].abs() - 0.5

    c = Case(cache, lens, [T] * len(lens), 2 * g, 2, d, seed=T + d, v_hook=negative)
    c.q[..., 5] = c.q[..., 5].abs()
    bits = [(2 << i) - 1 for i in range(T)] * len(lens) + [0] * 3
    spoiled = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    blind = spoiled.clone()
    for b, n in enumerate(lens):
        s = c.starts[b]
        spoiled[s, 0] = spoiled[s + T - 1, 2 * g - 1] = True
        if T > 1:  # a token that sees no drafted key: nothing where there is no prefix
            bits[s + 1] = 0
            spoiled[s + 1] = n > T
            blind[s + 1] = n == T
    c.q[..., 5][spoiled | blind] = math.inf
    o = c.run(as_int64(bits))
    assert o[spoiled].isnan().all()
    assert (o[blind] == 0).all()
    assert not o[~spoiled].isnan().any()
    for b, n in enumerate(lens):  # the rows beside them are what they are
        s = c.starts[b]
        rows = [i for i in range(T) if not (T > 1 and i == 1)]
        K, V = c.kv(b)
        q = torch.where(spoiled[s: s + T, :, None], torch.zeros((), dtype=c.q.dtype, device="cuda"), c.q[s: s + T])
        if not q.isfinite().all():
            q = q.nan_to_num(0, 0, 0)
        want, tol = chain(q, K, V)
        keep = ~spoiled[s: s + T]
        for i in rows:
            ref.close(o[s + i][keep[i]], want[i][keep[i]], tol[i][keep[i]], f"sequence {b} token {i}")
    assert bss.attn_sync_status() == 0
