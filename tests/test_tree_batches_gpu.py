"""tree_paged and tree_paged_e4m3 over batches whose work is divided in every
way: many sequences, more heads than CTAs run at once, empty ones between long
ones, pages that sequences share; and over keys, values and queries of any
magnitude."""
import math
import random

import pytest
import torch

import block_skipping_softmax_b200 as bss
import kv_reference as ref
from block_skipping_softmax_b200 import build as bss_build
from test_tree_gpu import CACHES, NAN, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    bss_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def chain(q, K, V):
    """ref.tree of a chain of finite values, by whole matrices."""
    T, Hq, d = q.shape
    Hkv, n, _ = K.shape
    K, V = (x.repeat_interleave(Hq // Hkv, 0) for x in (K, V))
    x = q.double().transpose(0, 1) @ K.transpose(1, 2) / math.sqrt(d)
    prefix = max(0, n - T)
    key, token = torch.arange(n, device=q.device), torch.arange(T, device=q.device)
    x = x.masked_fill((key >= prefix) & (key - prefix > token[:, None]), -math.inf)
    p = torch.softmax(x, -1)
    o, size = (p @ V).transpose(0, 1), (p @ V.abs()).transpose(0, 1)
    return o, (ref.BF16 + 2.0 ** -11) * (size + o.abs()) + ref.BF16 * o.abs() + 1e-30


def check(c, o):
    for b, (n, T) in enumerate(zip(c.lens, c.drafted)):
        if T == 0:
            continue
        rows = slice(c.starts[b], c.starts[b] + T)
        if n == 0:
            assert (o[rows] == 0).all()
            continue
        want, tol = chain(c.q[rows], *c.kv(b))
        ref.close(o[rows], want, tol, f"sequence {b}: {n} keys, {T} tokens")
    assert (o[c.starts[-1]:] == 55.0).all(), "rows of no sequence were written"
    assert bss.attn_sync_status() == 0


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("B,Hkv,g,T,most,d", [
    (40, 2, 4, 1, 2500, 64),     # equal pieces, segments of several sequences
    (70, 2, 4, 20, 1500, 128),
    (33, 1, 4, 4, 5000, 128),    # 16 rows
    (200, 4, 1, 1, 900, 64),     # more heads than CTAs
    (90, 4, 4, 33, 700, 64),     # the same, in two planes of rows
    (300, 2, 2, 2, 400, 128),    # few tiles: a CTA a head
    (600, 1, 2, 9, 100, 64),     # the same, of many rows
    (130, 1, 2, 3, 3000, 64),    # pieces over several times 32 sequences
])
def test_many_ragged_sequences(cache, B, Hkv, g, T, most, d):
    rng = random.Random(B)
    lens = [rng.choice([0, 1, 63, 64, 65, rng.randrange(most), rng.randrange(most), most]) for _ in range(B)]
    drafted = [rng.choice([0, 1, T, T, rng.randrange(T + 1)]) for _ in range(B)]
    lens = [max(n, t) if n else 0 for n, t in zip(lens, drafted)]
    c = Case(cache, lens, drafted, g * Hkv, Hkv, d, seed=B)
    check(c, c.run(max_q=T))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("T", [1, 4, 24])
@pytest.mark.parametrize("lens", [[0] * 40 + [9000], [9000] + [0] * 40, [1] * 35 + [6000, 0, 6001] + [2] * 5])
def test_one_long_sequence_among_empty_ones(cache, T, lens):
    drafted = [T if n >= T else min(n, T) for n in lens]
    c = Case(cache, lens, drafted, 4, 1, 128, seed=T)
    check(c, c.run(max_q=T))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("T", [2, 12])
def test_a_limit_far_above_the_lengths(cache, T):
    """max_seq_len sizes the division of the work; the lengths on the device decide it."""
    lens = [T, 700, 65, 3000]
    c = Case(cache, lens, [T] * 4, 8, 2, 64, seed=T)
    wide = torch.full((4, 2000), -1, dtype=torch.int32, device="cuda")
    wide[:, : c.max_pages] = c.table
    c.table = wide
    check(c, c.run(max_q=64, max_len=128000))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("T", [1, 16])
def test_sequences_share_pages(cache, T):
    c = Case(cache, [2000, 2000, 1300], [T, T, T], 8, 2, 128, seed=T)
    c.table[1] = c.table[0]
    c.table[2, : c.max_pages] = c.table[0]
    check(c, c.run())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,g", [(1, 4), (4, 4), (9, 8)])
@pytest.mark.parametrize("k_exp,v_exp", [((0, -40), (0, -30, -100)), ((20, -20), (0, 12, 20)), ((0,), (100, 60))])
def test_scales_of_any_size(d, T, g, k_exp, v_exp):
    """Scales beyond what an fp16 operand holds, in some keys of a page or in all.
    The products are exact, so the bound is that of ordinary values."""
    rng = torch.Generator().manual_seed(d + T)
    lens = [700, 130, 64 + T, 2000]

    def scale(case, K, V):
        for x, exps in ((K, k_exp), (V, v_exp)):
            e = torch.tensor(exps, dtype=torch.float64)[torch.randint(len(exps), x.shape[:3], generator=rng)]
            e[::3] = exps[0]  # some pages are ordinary
            x *= torch.exp2(e).to(x)[..., None]

    c = Case("e4m3", lens, [T] * 4, 2 * g, 2, d, seed=T, v_hook=scale)
    c.q = (c.q.float() * 2.0 ** -max(k_exp)).to(torch.bfloat16)
    check(c, c.run())


@pytest.mark.parametrize("T", [1, 4, 40])
@pytest.mark.parametrize("side", [0, 1])
def test_a_scale_that_is_nan_reaches_its_sequence_alone(T, side):
    def poison(case, K, V):
        page = int(case.table_cpu[1, 2])
        (K, V)[side][page, 0, 7, 3] = math.inf

    lens = [500, 600, 400]
    c = Case("e4m3", lens, [T] * 3, 8, 2, 64, seed=T, v_hook=poison)
    o = c.run()
    rows = slice(c.starts[1], c.starts[2])
    assert o[rows, :4].isnan().all(), "a NaN key or value before the drafted ones reaches every row of its head"
    rest = [b for b in range(3) if b != 1]
    for b in rest:
        want, tol = chain(c.q[c.starts[b]: c.starts[b + 1]], *c.kv(b))
        ref.close(o[c.starts[b]: c.starts[b + 1]], want, tol)
    want, tol = chain(c.q[rows, 4:], *(x[1:] for x in c.kv(1)))
    ref.close(o[rows, 4:], want, tol)
    assert bss.attn_sync_status() == 0


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,g", [(4, 2), (4, 4), (17, 8)])
def test_queries_of_any_size(cache, d, T, g):
    """Rows of zeros (a plain mean), tiny ones (nearly so) and huge ones (one key)."""
    c = Case(cache, [900, 70 + T, 1500], [T] * 3, 2 * g, 2, d, seed=d + g)
    rows = torch.arange(c.q.shape[0] * c.q.shape[1], device="cuda").view(*c.q.shape[:2], 1)
    e = torch.tensor([0.0, 2.0 ** -100, 2.0 ** -30, 1.0, 2.0 ** 60], device="cuda")[rows % 5]
    c.q = (c.q.float() * e).to(torch.bfloat16)
    check(c, c.run())


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("T,g", [(1, 4), (4, 4), (40, 4)])
def test_the_same_call_gives_the_same_bits(cache, T, g):
    """No atomics: the division of the work, and so every rounding, follows from the lengths."""
    c = Case(cache, [3000, T, 900, 5000], [T] * 4, 2 * g, 2, 128, seed=T)
    first = c.run()
    for _ in range(20):
        assert torch.equal(c.run().view(torch.int16), first.view(torch.int16))
    check(c, first)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("T,g", [(1, 4), (9, 8)])
def test_what_follows_in_the_stream_sees_the_result(cache, T, g):
    """Heads that one CTA finishes leave the merge nothing to do; a copy behind it still waits for them."""
    c = Case(cache, [800] * 37, [T] * 37, 8 * g, 8, 128, seed=T)
    first = c.run()
    out = torch.empty_like(first)
    copies = []
    for _ in range(30):
        out.fill_(NAN)
        c.run(out=out)
        copies.append(out.clone())
    rows = slice(0, c.starts[-1])
    assert all(torch.equal(x[rows], first[rows]) for x in copies)
    check(c, first)
