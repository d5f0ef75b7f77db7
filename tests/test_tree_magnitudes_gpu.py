"""tree_paged and tree_paged_e4m3 up to the largest keys and values that they are for.

Values: a term of the sums is a value times up to 2^8 (bf16) or 2^15 (e4m3), so a
sequence's keys times its largest value have to stay below 2^120 or 2^113.
Keys: over e4m3 a score is held at 2^14 to 2^15 of the query's largest element, so
that keys up to 2^104 stay in fp32 whatever the query; over bf16 q k has to."""
import math

import pytest
import torch

import block_skipping_softmax_b200 as bss
from block_skipping_softmax_b200 import build as bss_build
from test_tree_batches_gpu import check
from test_tree_gpu import CACHES, PAGE, Case

pytestmark = pytest.mark.gpu
ROWS = [(1, 4), (4, 4), (9, 8)]  # 4, 16 and 72 rows a KV head
TERMS = {"bf16": 120, "e4m3": 113}


@pytest.fixture(scope="module", autouse=True)
def lib():
    bss_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def scaled(side, exps, seed):
    """A hook that multiplies each key (0) or value (1) by one of 2^exps; every third page by the first."""
    def hook(case, K, V):
        x = (K, V)[side]
        e = torch.tensor(exps, dtype=torch.float64)[torch.randint(len(exps), x.shape[:3], generator=torch.Generator().manual_seed(seed))]
        e[::3] = exps[0]
        x *= torch.exp2(e).to(x)[..., None]
    return hook


def largest(cache, n):
    """The exponent for values of N(0, 1), none beyond 5."""
    return math.floor(TERMS[cache] - math.log2(5 * n))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,g", ROWS)
@pytest.mark.parametrize("others", [(), (0,), (-40, 0)])
@pytest.mark.parametrize("lens", [[1], [64, 700, 130], [9000, 3000]])  # one CTA a head; shares
def test_values_up_to_the_largest(cache, d, T, g, others, lens):
    lens = [max(n, T) for n in lens]
    exps = (largest(cache, max(lens)), *others)
    c = Case(cache, lens, [T] * len(lens), 2 * g, 2, d, seed=d + T, v_hook=scaled(1, exps, T))
    o = c.run()
    assert o[: c.starts[-1]].isfinite().all()
    check(c, o)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("T,g", ROWS)
def test_the_largest_values_meet_a_rising_score(cache, T, g):
    """They come under probabilities of nearly 2^8 of the running reference."""
    n = 640

    def rising(c, K, V):
        for i in range(n // PAGE):
            p = int(c.table_cpu[0, i])
            K[p] = 0
            K[p, :, :, 0] = float(i)
            V[p] *= 2.0 ** largest(cache, n) if i >= 5 else 1.0

    c = Case(cache, [n], [T], 2 * g, 2, 128, seed=T, v_hook=rising)
    c.q.zero_()
    c.q[..., 0] = 30.0  # 3.8 log2 units a page, and from one page to the next but one 7.6
    check(c, c.run())


@pytest.mark.parametrize("cache,k_exp,q_exp", [("bf16", 116, -116), ("bf16", -110, 110), ("bf16", 118, 0), ("bf16", 60, -120),
                                               ("e4m3", 101, -101), ("e4m3", -110, 110), ("e4m3", 101, 0), ("e4m3", 60, -120)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,g", ROWS)
def test_keys_up_to_the_largest(cache, d, T, g, k_exp, q_exp):
    lens = [1, 64, 700, 3000]
    lens = [max(n, T) for n in lens]
    c = Case(cache, lens, [T] * 4, 2 * g, 2, d, seed=d + T, v_hook=scaled(0, (k_exp, min(k_exp, 0)), T))
    c.q = (c.q.double() * 2.0 ** q_exp).to(torch.bfloat16)
    check(c, c.run())
