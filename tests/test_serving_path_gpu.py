"""The operators of a serving step together: rotation, cache, tree attention,
and the accepted branch moved to its place in the cache."""
import pytest
import torch

import block_skipping_softmax_b200 as bss
import kv_reference as ref
from block_skipping_softmax_b200 import build as bss_build

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def lib():
    bss_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("d,Hq,Hkv,rot,norm", [(128, 8, 2, 128, True), (64, 4, 4, 32, False)])
def test_prompt_drafts_and_acceptance(d, Hq, Hkv, rot, norm):
    g = torch.Generator(device="cuda").manual_seed(d)
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    w = (1 + 0.1 * torch.randn(2, d, generator=g, device="cuda")).to(torch.bfloat16)
    wq, wk = (w[0], w[1]) if norm else (None, None)
    lens, T = [130, 61, 1], 6
    pages_per = 4
    order = torch.randperm(3 * pages_per).view(3, pages_per)
    table = order.to(torch.int32).cuda()
    pool = [torch.full((14, Hkv, PAGE, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pool += [torch.full((14, Hkv, PAGE), float("nan"), device="cuda") for _ in range(2)]
    slot = lambda b, pos: int(order[b, pos // PAGE]) * PAGE + pos % PAGE  # noqa: E731
    kept = [[], [], []]  # what each cached position means, in 64 bits: (k, v) [Hkv, d]

    def step(positions, slots):
        """Projection output -> rotated q, cached k and v; returns q and the cached values."""
        n = len(positions)
        fused = torch.randn(n, Hq + 2 * Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
        q0, k0, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
        q, k = bss.qk_norm_rope(q0, k0, pos, f, wq, wk)
        for got, x, weight in ((q, q0, wq), (k, k0, wk)):
            want, tol = ref.norm_rope(x.transpose(0, 1), weight, pos, f, False)
            ref.close(got.transpose(0, 1), want, tol)
        bss.cache_write_e4m3(k, v, torch.tensor(slots, device="cuda"), *pool)
        return q, ref.dequantised(*ref.quantised(k)), ref.dequantised(*ref.quantised(v))

    # prompts
    where = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    _, k, v = step([p for _, p in where], [slot(b, p) for b, p in where])
    for i, (b, _) in enumerate(where):
        kept[b].append((k[i], v[i]))

    # drafts: two branches from the root (0-1-2 and 0-3-4-5), by depth in position
    parent = [-1, 0, 1, 0, 3, 4]
    depth, bits = [], []
    for i, p in enumerate(parent):
        depth.append(0 if p < 0 else depth[p] + 1)
        bits.append((0 if p < 0 else bits[p]) | 1 << i)
    where = [(b, i) for b in range(3) for i in range(T)]
    q, k, v = step([lens[b] + depth[i] for b, i in where], [slot(b, lens[b] + i) for b, i in where])
    cu = torch.tensor([0, T, 2 * T, 3 * T], dtype=torch.int32, device="cuda")
    now = torch.tensor([n + T for n in lens], dtype=torch.int32, device="cuda")
    mask = torch.tensor(bits * 3, dtype=torch.int64, device="cuda")
    o = bss.tree_paged_e4m3(q, *pool, table, now, cu, T, pages_per * PAGE, mask)
    for b in range(3):
        K, V = (torch.stack([x[j] for x in kept[b]] + [y[b * T + i] for i in range(T)], 1).cuda()
                for j, y in ((0, k), (1, v)))
        want, tol = ref.tree(q[b * T: b * T + T], K, V, bits, T)
        ref.close(o[b * T: b * T + T], want, tol, f"drafts of sequence {b}")

    # tokens 0, 3, 4 are accepted: their slots move up behind the prefix
    accepted = [0, 3, 4]
    src = torch.tensor([slot(b, lens[b] + i) for b in range(3) for i in accepted], device="cuda")
    dst = torch.tensor([slot(b, lens[b] + j) for b in range(3) for j in range(3)], device="cuda")
    bss.cache_write_e4m3(*bss.cache_read_e4m3(*pool, src), dst, *pool)
    for b in range(3):
        kept[b] += [(k[b * T + i], v[b * T + i]) for i in accepted]
        lens[b] += 3

    # the next single token of each sequence
    q, k, v = step(lens, [slot(b, lens[b]) for b in range(3)])
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    now = torch.tensor([n + 1 for n in lens], dtype=torch.int32, device="cuda")
    o = bss.tree_paged_e4m3(q, *pool, table, now, cu, 1, pages_per * PAGE)
    for b in range(3):
        K, V = (torch.stack([x[j] for x in kept[b]] + [y[b]], 1).cuda() for j, y in ((0, k), (1, v)))
        want, tol = ref.tree(q[b: b + 1], K, V, None, 1)
        ref.close(o[b: b + 1], want, tol, f"next token of sequence {b}")
    # the cached prefix, read back into the contiguous decode's layout
    n = max(lens) + 1
    slots = torch.tensor([[slot(b, p) if p <= lens[b] else -1 for p in range(n)] for b in range(3)], device="cuda")
    Kc, Vc = bss.cache_read_e4m3(*pool, slots)
    longest = lens.index(max(lens))
    contiguous = bss.decode(q, Kc, Vc)
    K, V = Kc[longest].double(), Vc[longest].double()
    want, tol = ref.tree(q[longest: longest + 1], K, V, None, 1)
    ref.close(contiguous[longest: longest + 1], want, tol)
    assert bss.attn_sync_status() == 0
