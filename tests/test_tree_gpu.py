"""tree_paged and tree_paged_e4m3 against softmax attention in 64 bits.

Slots that no sequence owns hold NaN (bf16 pools) or NaN scales and codes of
all ones (e4m3 pools), table entries past a sequence's end are invalid, and
rows of no sequence hold a mark: a kernel that reads or writes there fails."""
import random

import pytest
import torch

import block_skipping_softmax_b200 as bss
import kv_reference as ref
from block_skipping_softmax_b200 import build as bss_build

pytestmark = pytest.mark.gpu
PAGE = 64
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    bss_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def tree_masks(T, rng, empty=()):
    bits = [1]
    for i in range(1, T):
        bits.append(bits[rng.randrange(i)] | 1 << i)
    return [0 if i in empty else b for i, b in enumerate(bits)][:T]


def as_int64(bits):
    return torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device="cuda")


class Case:
    """A batch over a shuffled pool; K, V of sequence b as float64 [Hkv, len, d]."""

    def __init__(self, cache, lens, drafted, Hq, Hkv, d, seed=0, extra_rows=3, q_sigma=2.0, v_hook=None):
        self.cache, self.lens, self.drafted, self.Hq, self.Hkv, self.d = cache, lens, drafted, Hq, Hkv, d
        g = torch.Generator(device="cuda").manual_seed(seed)
        B = len(lens)
        n_pages = [-(-n // PAGE) for n in lens]
        self.max_pages = max(max(n_pages), 1)
        pool = sum(n_pages) + 3
        order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed))
        table = torch.full((B, self.max_pages), -1, dtype=torch.int32)
        K = torch.full((pool, Hkv, PAGE, d), NAN, dtype=torch.bfloat16, device="cuda")
        V = K.clone()
        at = 0
        for b, n in enumerate(lens):
            pages = order[at: at + n_pages[b]]
            at += n_pages[b]
            table[b, : n_pages[b]] = pages
            for i, p in enumerate(pages.tolist()):
                m = min(PAGE, n - i * PAGE)
                K[p, :, :m] = torch.randn(Hkv, m, d, generator=g, device="cuda").to(torch.bfloat16)
                V[p, :, :m] = torch.randn(Hkv, m, d, generator=g, device="cuda").to(torch.bfloat16)
        self.table_cpu = table
        if v_hook:
            v_hook(self, K, V)
        total = sum(drafted) + extra_rows
        self.q = (q_sigma * torch.randn(total, Hq, d, generator=g, device="cuda")).to(torch.bfloat16)
        self.table, self.lens_t = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = [0]
        for t in drafted:
            starts.append(starts[-1] + t)
        self.starts = starts
        self.cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
        if cache == "bf16":
            self.pool = (K, V)
            self.values = (K.double(), V.double())
        else:
            owned = ~K[:, 0, :, 0].isnan() if v_hook is None else self.owned(pool)
            codes, scales, values = [], [], []
            for x in (K, V):
                c, s = ref.quantised(torch.where(owned.cpu()[:, None, :, None], x.cpu(), torch.zeros((), dtype=x.dtype)))
                c[~owned.cpu()[:, None].expand(s.shape)] = 0x7F
                s[~owned.cpu()[:, None].expand(s.shape)] = NAN
                codes.append(c.cuda())
                scales.append(s.cuda())
                values.append(ref.dequantised(c, s).cuda())
            self.pool = (*codes, *scales)
            self.values = tuple(values)

    def owned(self, pool):
        o = torch.zeros(pool, PAGE, dtype=torch.bool)
        for b, n in enumerate(self.lens):
            for i in range(-(-n // PAGE)):
                o[int(self.table_cpu[b, i]), : min(PAGE, n - i * PAGE)] = True
        return o

    def run(self, mask=None, max_q=None, max_len=None, **kw):
        fn = bss.tree_paged if self.cache == "bf16" else bss.tree_paged_e4m3
        kw.setdefault("out", torch.full_like(self.q, 55.0))
        return fn(self.q, *self.pool, self.table, self.lens_t, self.cu, max_q or max(max(self.drafted), 1),
                  max_len or max(max(self.lens), 1), mask, **kw)

    def kv(self, b):
        n = self.lens[b]
        pages = self.table[b, : -(-n // PAGE)].long()
        return [x[pages].transpose(0, 1).reshape(self.Hkv, -1, self.d)[:, :n] for x in self.values]

    def check(self, o, bits=None):
        for b, (n, T) in enumerate(zip(self.lens, self.drafted)):
            if T == 0:
                continue
            s = self.starts[b]
            K, V = self.kv(b)
            want, tol = ref.tree(self.q[s: s + T], K, V, None if bits is None else bits[s: s + T], T)
            ref.close(o[s: s + T], want, tol, f"sequence {b}: {n} keys, {T} tokens")
        assert (o[self.starts[-1]:] == 55.0).all(), "rows of no sequence were written"
        assert bss.attn_sync_status() == 0


CACHES = ["bf16", "e4m3"]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 3, 4, 8])
def test_single_tokens(cache, d, g):
    lens = [1, 2, 63, 64, 65, 129, 700, 4096]
    c = Case(cache, lens, [1] * len(lens), 2 * g, 2, d, seed=g)
    c.check(c.run())


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,T", [(1, 2), (1, 64), (2, 17), (4, 5), (4, 8), (4, 33), (5, 7), (8, 16), (8, 64)])
def test_trees_and_chains_in_a_ragged_batch(cache, d, g, T):
    rng = random.Random(T * g)
    lens = [T, T + 1, 64, 64 + T // 2, 130, 1000, 128 + T, 3001]
    drafted = [T, T, max(1, T // 2), T, 1, T, T, max(1, T - 1)]
    c = Case(cache, lens, drafted, 2 * g, 2, d, seed=T + d)
    c.check(c.run())
    bits = sum((tree_masks(t, rng) for t in drafted), []) + [0] * 3
    c.check(c.run(as_int64(bits)), bits)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("g", [1, 4])
def test_empty_rows_empty_sequences_and_fewer_keys_than_tokens(cache, g):
    T = 6
    rng = random.Random(5)
    lens, drafted = [0, 6, 3, 70, 500, 0, 64], [T, T, T, T, T, 0, 0]
    c = Case(cache, lens, drafted, 2 * g, 2, 128, seed=3)
    bits = sum((tree_masks(t, rng, empty=(0, 3)) for t in drafted), []) + [0] * 3
    o = c.run(as_int64(bits))
    c.check(o, bits)
    assert (o[:T] == 0).all(), "a sequence without keys gives zeros"
    assert (o[T] == 0).all() and (o[T + 3] == 0).all(), "a row that sees nothing gives zeros"
    c.check(c.run())
    c = Case(cache, [0, 0], [2, 1], 2, 1, 64)
    o = c.run()
    assert (o[:3] == 0).all()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("T,g", [(8, 1), (8, 8), (40, 4)])
def test_values_that_are_not_finite_reach_only_the_tokens_that_see_them(cache, T, g):
    """Drafted key 3 is inf or NaN; only its descendants and itself see it."""
    lens = [200, 64 + T]

    def spoil(c, K, V):
        for b, n in enumerate(lens):
            key = n - T + 3
            p = int(c.table_cpu[b, key // PAGE])
            (K if b == 0 else V)[p, :, key % PAGE, 5] = float("inf") if b else NAN

    c = Case(cache, lens, [T, T], g, 1, 128, seed=8, v_hook=spoil)
    bits = []
    for _ in lens:  # tokens 0..3 a chain; even later tokens hang off 3, odd ones off 2
        chain = [1, 3, 7, 15]
        bits += chain + [(15 if i % 2 == 0 else 7) | 1 << i for i in range(4, T)]
    bits += [0] * 3
    o = c.run(as_int64(bits))
    for b in range(2):
        for i in range(T):
            row = o[b * T + i]
            if (bits[b * T + i] >> 3) & 1:
                assert row.isnan().any(-1).all()
            else:
                K, V = c.kv(b)
                want, tol = ref.tree(c.q[b * T + i: b * T + i + 1], K, V.nan_to_num(0, 0, 0), None, 1)
                s = [j for j in range(lens[b]) if j < lens[b] - T or (bits[b * T + i] >> (j - lens[b] + T)) & 1]
                want, tol = ref.tree(c.q[b * T + i: b * T + i + 1], K[:, s], V[:, s], [1], 1)
                ref.close(row[None], want, tol, f"sequence {b} token {i}")
    assert bss.attn_sync_status() == 0


@pytest.mark.parametrize("cache", CACHES)
def test_queries_that_are_not_finite_stay_in_their_rows(cache):
    c = Case(cache, [300, 90], [4, 4], 4, 2, 64)
    c.q[1, 2, 5] = NAN
    c.q[6, 0] = float("inf")
    o = c.run()
    assert o[1, 2].isnan().all()
    keep = [(t, h) for t in range(8) for h in range(4) if (t, h) not in ((1, 2), (6, 0))]
    q = c.q.clone()
    c.q[1, 2] = 0
    c.q[6, 0] = 0
    ok = c.run()
    c.q = q
    for t, h in keep:
        assert torch.equal(o[t, h], ok[t, h])


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("B,T,L", [(1, 1, 100000), (1, 40, 50001), (3, 9, 20000)])
def test_long_caches_are_split_and_merged(cache, B, T, L):
    rng = random.Random(L)
    c = Case(cache, [L - 77 * b for b in range(B)], [T] * B, 4, 1, 128, seed=1)
    assert bss.attn_tree_workspace_bytes(B, T, B * T + 3, 4, 1, L, 128) > 0
    bits = sum((tree_masks(T, rng) for _ in range(B)), []) + [0] * 3
    o = c.run(as_int64(bits))
    c.check(o, bits)
    # a caller's workspace full of NaN gives the same bits, and so does a second call
    need = bss.attn_tree_workspace_bytes(B, T, c.q.shape[0], 4, 1, L, 128)
    ws = torch.full((need // 4,), NAN, device="cuda").view(torch.uint8)
    assert torch.equal(c.run(as_int64(bits), workspace=ws), o)
    assert torch.equal(c.run(as_int64(bits), workspace=ws), o)


@pytest.mark.parametrize("cache", CACHES)
def test_a_chain_is_each_token_over_its_own_prefix(cache):
    """A chain of T tokens equals T decodes over growing caches."""
    T, n = 5, 333
    c = Case(cache, [n], [T], 8, 2, 128)
    o = c.run()
    for i in range(T):
        one = Case(cache, [n], [1], 8, 2, 128, extra_rows=0)
        one.pool, one.table = c.pool, c.table
        one.lens_t = torch.tensor([n - T + 1 + i], dtype=torch.int32, device="cuda")
        one.q = c.q[i: i + 1].clone()
        K, V = c.kv(0)
        want, tol = ref.tree(one.q, K[:, : n - T + 1 + i], V[:, : n - T + 1 + i], None, 1)
        ref.close(one.run(), want, tol)
        ref.close(o[i: i + 1], want, tol)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("T", [1, 30])
def test_page_ids_outside_the_pool_read_zeros(cache, T):
    c = Case(cache, [64 * 6], [T], 4, 1, 128)
    c.table[0, 1], c.table[0, 2], c.table[0, 3] = -7, c.pool[0].shape[0], (1 << 31) - 1
    o = c.run()
    c.table[0, 1:4] = 0
    K, V = c.kv(0)
    K[:, 64:256] = 0
    V[:, 64:256] = 0
    want, tol = ref.tree(c.q[:T], K, V, None, T)
    ref.close(o[:T], want, tol)
    assert bss.attn_sync_status() == 0


@pytest.mark.parametrize("cache", CACHES)
def test_malformed_offsets_and_lengths_stay_inside(cache):
    """cu_q outside the batch, lengths past the table and more tokens than max_q are cut."""
    c = Case(cache, [200, 128], [6, 4], 4, 2, 64)
    full = c.run()
    c.lens_t = torch.tensor([200, 1 << 30], dtype=torch.int32, device="cuda")  # cut to max_seq_len
    o = c.run(max_len=128)
    K, V = c.kv(1)
    ref.close(o[6:10], *ref.tree(c.q[6:10], K[:, :128], V[:, :128], None, 4))
    c.lens_t = torch.tensor([200, 128], dtype=torch.int32, device="cuda")
    c.cu = torch.tensor([-5, 6, 1 << 30], dtype=torch.int32, device="cuda")  # rows 6..12 are sequence 1's now
    o = c.run(max_q=7)
    assert torch.equal(o[:6], full[:6])
    K, V = c.kv(1)
    ref.close(o[6:13], *ref.tree(c.q[6:13], K, V, None, 7))
    c.cu = torch.tensor([0, 6, 10], dtype=torch.int32, device="cuda")
    o = c.run(max_q=3)  # the first three tokens of each
    assert (o[3:6] == 55).all() and (o[9:] == 55).all()
    K, V = c.kv(0)
    ref.close(o[:3], *ref.tree(c.q[:3], K, V, None, 3))
    assert bss.attn_sync_status() == 0


@pytest.mark.parametrize("cache", CACHES)
def test_a_pool_beyond_32_bit_offsets(cache):
    Hkv, d, T = 8, 128, 12
    row = PAGE * d * (2 if cache == "bf16" else 1)
    pages = (1 << 32) // (Hkv * row) + 40
    small = Case(cache, [1000], [T], 16, Hkv, d)
    want = small.run()
    n = small.pool[0].shape[0]
    big = []
    for p in small.pool:
        x = torch.empty((pages, *p.shape[1:]), dtype=p.dtype, device="cuda")
        x[pages - n:] = p
        big.append(x)
    small.pool = tuple(big)
    small.table = torch.where(small.table >= 0, small.table + (pages - n), small.table)
    assert torch.equal(small.run(), want)


@pytest.mark.parametrize("cache", CACHES)
def test_two_streams_at_once_and_captured_graphs(cache):
    a = Case(cache, [5000, 4000], [7, 7], 8, 2, 128, seed=1)
    b = Case(cache, [6000, 300], [20, 3], 8, 2, 128, seed=2)
    wa, wb = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got.append((a.run(stream=s1), wa))
        got.append((b.run(stream=s2), wb))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)
    # two graphs, replayed at once, inputs changed in place
    graphs, outs = [], []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run(out=torch.empty_like(c.q)))
        graphs.append(g)
    a.q.neg_()
    b.q.mul_(0.5)
    for s, g in ((s1, graphs[0]), (s2, graphs[1])):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(10):
                g.replay()
    torch.cuda.synchronize()
    for c, o in ((a, outs[0]), (b, outs[1])):
        assert torch.equal(c.run()[: c.starts[-1]], o[: c.starts[-1]])
    assert bss.attn_sync_status() == 0


def test_agrees_with_the_decode_of_single_tokens():
    """T = 1 over a bf16 pool is decode_paged at tau = inf."""
    c = Case("bf16", [1, 64, 700, 5000], [1] * 4, 8, 2, 128, extra_rows=0)
    o = c.run()
    p = bss.decode_paged(c.q, *c.pool, c.table, c.lens_t, 5000)
    for b in range(4):
        want, tol = ref.tree(c.q[b: b + 1], *c.kv(b), None, 1)
        ref.close(o[b: b + 1], want, tol)
        ref.close(p[b: b + 1], want, tol)


def test_refusals_of_the_helper():
    c = Case("bf16", [100], [4], 4, 2, 64, extra_rows=0)
    e = Case("e4m3", [100], [4], 4, 2, 64, extra_rows=0)
    q, (K, V), t, n, cu = c.q, c.pool, c.table, c.lens_t, c.cu
    for call in (lambda: bss.tree_paged(q, K, V, t, n, cu, 65, 100),
                 lambda: bss.tree_paged(q, K, V, t, n, cu, 0, 100),
                 lambda: bss.tree_paged(q, K, V, t, n, cu, 4, 129),
                 lambda: bss.tree_paged(q, K, V, t, n, cu, 4, 0),
                 lambda: bss.tree_paged(q[:, :3], K, V, t, n, cu, 4, 100),
                 lambda: bss.tree_paged(q[:, :3].contiguous(), K, V, t, n, cu, 4, 100),
                 lambda: bss.tree_paged(q, K[..., :32], V[..., :32], t, n, cu, 4, 100),
                 lambda: bss.tree_paged(q, K, V, t.long(), n, cu, 4, 100),
                 lambda: bss.tree_paged(q, K, V, t, n, cu.cpu(), 4, 100),
                 lambda: bss.tree_paged(q, K, V, t, n, cu, 4, 100, torch.zeros(3, dtype=torch.int64, device="cuda")),
                 lambda: bss.tree_paged(q, K, V, t, n, cu, 4, 100, out=torch.empty(4, 4, 64, device="cuda")),
                 lambda: bss.tree_paged_e4m3(q, K, V, *e.pool[2:], t, n, cu, 4, 100),
                 lambda: bss.tree_paged_e4m3(q, *e.pool[:3], e.pool[3][:1], t, n, cu, 4, 100)):
        with pytest.raises(bss.AttnError):
            call()
