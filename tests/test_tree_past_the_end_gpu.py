"""What lies in a page behind a sequence's last key changes no bit of the result."""
import math

import pytest
import torch

import block_skipping_softmax_b200 as bss
from block_skipping_softmax_b200 import build as bss_build
from test_tree_batches_gpu import check
from test_tree_gpu import NAN, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    bss_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def same_bits(c, fills):
    """c.run() with each fill of the slots that no sequence owns."""
    unowned = ~c.owned(c.pool[0].shape[0]).cuda()[:, None].expand(c.pool[0].shape[:3])
    first = None
    for fill in fills:
        for x, value in zip(c.pool, fill):
            x[unowned] = value
        o = c.run()
        check(c, o)
        if first is None:
            first = o
        assert torch.equal(o.view(torch.int16), first.view(torch.int16)), f"other bits with {fill}"


ROWS = [(1, 4), (4, 4), (3, 8), (17, 8), (40, 8)]  # 4, 16, 24, 136 and 320 rows a KV head


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,g", ROWS)
@pytest.mark.parametrize("lens", [[41, 70, 127, 500], [3001, 4100]])
def test_codes_and_scales_past_the_end(d, T, g, lens):
    c = Case("e4m3", lens, [T] * len(lens), 2 * g, 2, d, seed=d + T)
    same_bits(c, [(0x7F, 0x7F, 1.0, 0.5), (0, 0, 0.0, 0.0), (0x7F, 0xFF, NAN, NAN), (0x7E, 0x7E, 2.0 ** 100, 2.0 ** 100),
                  (1, 1, 2.0 ** -126, 2.0 ** -126), (0x7F, 0x7F, math.inf, -math.inf)])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,g", ROWS)
def test_values_past_the_end(d, T, g):
    c = Case("bf16", [41, 70, 127, 500], [T] * 4, 2 * g, 2, d, seed=d + T)
    same_bits(c, [(NAN, NAN), (0.0, 0.0), (math.inf, -math.inf), (3e38, 3e38)])
