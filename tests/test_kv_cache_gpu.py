"""cache_write_e4m3 and cache_read_e4m3: exact against the C oracle's quantiser."""
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


def pool(pages, Hkv, d, fill=0xAB):
    codes = [torch.full((pages, Hkv, PAGE, d), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, Hkv, PAGE), 77.0, device="cuda") for _ in range(2)]
    return (*codes, *scales)


def vectors(N, Hkv, d, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, 2 * Hkv, d, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-20, 20, (N, 2 * Hkv, 1), generator=g, device="cuda").float())
    return x.to(torch.bfloat16)


def at(p, slots):
    """Rows [tokens, Hkv, ...] of a pool tensor [pages, Hkv, 64, ...]."""
    return p.transpose(1, 2).flatten(0, 1)[slots]


@pytest.mark.parametrize("N,Hkv,d", [(1, 1, 64), (1, 8, 128), (7, 3, 128), (63, 2, 64), (1000, 8, 128), (20011, 1, 64),
                                     (6000, 8, 64), (9001, 4, 128)])
def test_codes_scales_and_values_are_exact(N, Hkv, d):
    fused = vectors(N, Hkv, d, seed=N)
    k, v = fused[:, :Hkv], fused[:, Hkv:]  # strided slices
    pages = N // PAGE + 3
    Kc, Vc, Ks, Vs = pool(pages, Hkv, d)
    slots = torch.randperm(pages * PAGE, generator=torch.Generator().manual_seed(N))[:N].cuda()
    bss.cache_write_e4m3(k, v, slots, Kc, Vc, Ks, Vs)
    back = bss.cache_read_e4m3(Kc, Vc, Ks, Vs, slots)
    untouched = torch.ones(pages * PAGE, dtype=torch.bool, device="cuda")
    untouched[slots] = False
    for x, codes, scales, r in ((k, Kc, Ks, back[0]), (v, Vc, Vs, back[1])):
        wc, ws = ref.quantised(x)
        assert torch.equal(at(codes, slots).cpu(), wc) and torch.equal(at(scales, slots).cpu(), ws)
        assert torch.equal(r.cpu().double(), ref.dequantised(wc, ws))  # exact in bf16
        rest = codes.transpose(1, 2).flatten(0, 1)[untouched]
        assert (rest == 0xAB).all() and (scales.transpose(1, 2).flatten(0, 1)[untouched] == 77).all()
    # written back, the values do not change
    K2 = pool(pages, Hkv, d)
    bss.cache_write_e4m3(*back, slots, *K2)
    again = bss.cache_read_e4m3(*K2, slots)
    assert torch.equal(again[0], back[0]) and torch.equal(again[1], back[1])


def test_prefill_layout_padded_tokens_and_slots_outside_the_pool():
    B, N, Hkv, d, pages = 3, 65, 2, 128, 4
    fused = vectors(B * N, Hkv, d)
    k, v = (x.unflatten(0, (B, N)).transpose(1, 2).contiguous() for x in (fused[:, :Hkv], fused[:, Hkv:]))
    slots = torch.randperm(pages * PAGE)[:B * N].view(B, N).cuda()
    slots[0, 60:] = -1
    slots[1, 3], slots[1, 4] = pages * PAGE, 1 << 40
    slots[2, 0] = -(1 << 62)
    Kc, Vc, Ks, Vs = pool(pages, Hkv, d)
    bss.cache_write_e4m3(k, v, slots, Kc, Vc, Ks, Vs)
    good = (slots >= 0) & (slots < pages * PAGE)
    for x, codes, scales in ((k, Kc, Ks), (v, Vc, Vs)):
        wc, ws = ref.quantised(x.transpose(1, 2)[good])
        assert torch.equal(at(codes, slots[good]).cpu(), wc) and torch.equal(at(scales, slots[good]).cpu(), ws)
        assert int((scales != 77).sum()) <= int(good.sum()) * Hkv
    out = tuple(torch.full_like(k, 5.0) for _ in range(2))
    r = bss.cache_read_e4m3(Kc, Vc, Ks, Vs, slots, out=out)
    assert r[0] is out[0]
    for x, got in ((k, r[0]), (v, r[1])):
        want = ref.dequantised(*ref.quantised(x))
        want[~good[:, None].expand(B, Hkv, N).cpu()] = 0  # a slot outside the pool reads zeros
        assert torch.equal(got.cpu().double(), want)
    # one slot read many times
    one = slots[0, 0].repeat(100)
    a, _ = bss.cache_read_e4m3(Kc, Vc, Ks, Vs, one)
    assert torch.equal(a, r[0][0, :, 0].expand(100, Hkv, d))


def test_edges_of_the_format():
    d = 64
    rows = torch.zeros(10, d)
    rows[0] = 0.0
    rows[1, 0] = 448.0
    rows[2, 0] = 449.0
    rows[2, 1] = 2.0 ** -9
    rows[3] = 2.0 ** -133  # the least bf16 subnormal
    rows[4, 5] = 3.3895e38
    rows[5, 0], rows[5, 1:] = 1.0, torch.linspace(-1, 1, d - 1)
    rows[6, 3] = float("inf")
    rows[7, 4] = float("nan")
    rows[8, 0], rows[8, 1:4] = -256.0, torch.tensor([17.0, 18.0, 19.0])  # ties go to even codes
    rows[9, 0] = -(2.0 ** -126)
    x = rows.to(torch.bfloat16).cuda()[:, None]
    slots = torch.arange(10).cuda()
    p = pool(1, 1, d)
    bss.cache_write_e4m3(x, x, slots, *p)
    wc, ws = ref.quantised(x)
    assert torch.equal(at(p[2], slots).cpu().nan_to_num(-1), ws.nan_to_num(-1))
    finite = torch.tensor([0, 1, 2, 3, 4, 5, 8, 9])
    assert torch.equal(at(p[0], slots).cpu()[finite], wc[finite])
    k, _ = bss.cache_read_e4m3(*p, slots)
    # row 4: 255 * 2^120 rounds to the code of 256, and 256 * 2^120 = 2^128 lies
    # beyond bf16: rounded to bf16 it is inf.  The other values are exact.
    want = ref.dequantised(wc, ws)
    assert torch.equal(k.cpu()[finite], want.to(torch.bfloat16)[finite])
    rest = torch.tensor([0, 1, 2, 3, 5, 8, 9])
    assert torch.equal(k.cpu().double()[rest], want[rest]) and k[4, 0, 5] == float("inf")
    assert k[6].isnan().all() and k[7].isnan().all()
    # every code, under a scale of 1
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 1, 4, d)
    full = torch.zeros(1, 1, PAGE, d, dtype=torch.uint8, device="cuda")
    full[:, :, :4] = codes
    one = torch.ones(1, 1, PAGE, device="cuda")
    k, _ = bss.cache_read_e4m3(full, full, one, one, slots[:4])
    want = ref.dequantised(codes.cpu()[0, 0], torch.ones(4))
    assert torch.equal(k.cpu().double()[:, 0].nan_to_num(1e9), want.nan_to_num(1e9))


def test_offsets_beyond_32_bits():
    """Codes past 2^32 bytes of a pool (its last pages)."""
    Hkv, d = 8, 128
    pages = (1 << 32) // (Hkv * PAGE * d) + 3
    Kc = torch.empty(pages, Hkv, PAGE, d, dtype=torch.uint8, device="cuda")
    Vc = torch.empty_like(Kc)
    Ks, Vs = (torch.empty(pages, Hkv, PAGE, device="cuda") for _ in range(2))
    fused = vectors(130, Hkv, d, seed=9)
    slots = torch.cat([torch.arange(pages * PAGE - 100, pages * PAGE), torch.arange(30)]).cuda()
    Kc[0] = 1
    bss.cache_write_e4m3(fused[:, :Hkv], fused[:, Hkv:], slots, Kc, Vc, Ks, Vs)
    k, v = bss.cache_read_e4m3(Kc, Vc, Ks, Vs, slots)
    assert (Kc[0, :, 30:] == 1).all()
    for x, r in ((fused[:, :Hkv], k), (fused[:, Hkv:], v)):
        assert torch.equal(r.cpu().double(), ref.dequantised(*ref.quantised(x)))


def test_another_stream_and_a_captured_graph():
    N, Hkv, d = 200, 4, 128
    fused = vectors(N, Hkv, d)
    k, v = fused[:, :Hkv], fused[:, Hkv:]
    slots = torch.arange(N).cuda()
    p, p2 = pool(4, Hkv, d), pool(4, Hkv, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bss.cache_write_e4m3(k, v, slots, *p, stream=s)
    got = bss.cache_read_e4m3(*p, slots, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    want = ref.dequantised(*ref.quantised(k))
    assert torch.equal(got[0].cpu().double(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bss.cache_write_e4m3(k, v, slots, *p2)
        out = bss.cache_read_e4m3(*p2, slots)
    fused.copy_(vectors(N, Hkv, d, seed=4))
    slots.copy_(torch.arange(N).flip(0))
    graph.replay()
    assert torch.equal(out[1].cpu().double(), ref.dequantised(*ref.quantised(v)))


def test_refusals_of_the_helpers():
    fused = vectors(4, 2, 64)
    k, v = fused[:, :2], fused[:, 2:]
    slots = torch.arange(4).cuda()
    Kc, Vc, Ks, Vs = pool(2, 2, 64)
    for call in (lambda: bss.cache_write_e4m3(k, v, slots.int(), Kc, Vc, Ks, Vs),
                 lambda: bss.cache_write_e4m3(k, v, slots[:3], Kc, Vc, Ks, Vs),
                 lambda: bss.cache_write_e4m3(k[:, :1], v[:, :1], slots, Kc, Vc, Ks, Vs),
                 lambda: bss.cache_write_e4m3(k[..., :32], v[..., :32], slots, Kc, Vc, Ks, Vs),
                 lambda: bss.cache_write_e4m3(k, v, slots, Kc.transpose(0, 1), Vc, Ks, Vs),
                 lambda: bss.cache_write_e4m3(k, v, slots.cpu(), Kc, Vc, Ks, Vs),
                 lambda: bss.cache_write_e4m3(k[:0], v[:0], slots[:0], Kc, Vc, Ks, Vs),
                 lambda: bss.cache_read_e4m3(Kc, Vc, Ks, Vs[:1], slots),
                 lambda: bss.cache_read_e4m3(Kc, Vc, Ks, Vs, slots, out=(k.float(), v))):
        with pytest.raises(bss.AttnError):
            call()
