"""qk_norm_rope against the formula in 64 bits."""
import pytest
import torch

import block_skipping_softmax_b200 as bss
import kv_reference as ref
from block_skipping_softmax_b200 import build as bss_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    bss_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def inputs(N, Hq, Hkv, d, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    fused = (torch.randn(N, Hq + 2 * Hkv, d, generator=g, device="cuda") * 3).to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(2, d, generator=g, device="cuda")).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (N,), generator=g, device="cuda", dtype=torch.int32)
    return fused, w, pos


def check(got, x, w, pos, f, interleaved, eps=1e-6):
    """got and x [tokens, H, d]."""
    want, tol = ref.norm_rope(x.transpose(0, 1), w, pos, f, interleaved, eps)
    ref.close(got.transpose(0, 1), want, tol, "norm_rope")


@pytest.mark.parametrize("N", [1, 3, 1000])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (32, 8), (5, 3), (64, 8)])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48)])
def test_slices_of_a_fused_projection(N, Hq, Hkv, d, rot):
    fused, w, pos = inputs(N, Hq, Hkv, d, seed=N + Hq + d)
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hkv]
    before = fused.clone()
    for interleaved in (False, True):
        for wq, wk in ((w[0], w[1]), (None, w[1]), (None, None)):
            qo, ko = bss.qk_norm_rope(q, k, pos, freqs(rot), wq, wk, interleaved=interleaved)
            assert qo.is_contiguous() and ko.shape == k.shape
            check(qo, q, wq, pos, freqs(rot), interleaved)
            check(ko, k, wk, pos, freqs(rot), interleaved)
    assert torch.equal(fused, before)


@pytest.mark.parametrize("per_sequence", [False, True])
def test_prefill_layout_and_in_place(per_sequence):
    B, N, Hq, Hkv, d = 3, 257, 8, 2, 128
    fused, w, _ = inputs(B * N, Hq, Hkv, d)
    q, k = (x.unflatten(0, (B, N)).transpose(1, 2) for x in (fused[:, :Hq], fused[:, Hq:Hq + Hkv]))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    if per_sequence:
        pos = (pos + torch.tensor([[0], [70000], [5]], device="cuda")).to(torch.int32)
    f = freqs(d)
    qo, ko = bss.qk_norm_rope(q, k, pos, f, w[0], w[1])
    assert qo.shape == (B, Hq, N, d) and qo.is_contiguous()
    for b in range(B):
        p = pos[b] if per_sequence else pos
        for got, x, weight in ((qo, q, w[0]), (ko, k, w[1])):
            want, tol = ref.norm_rope(x[b], weight, p, f, False)
            ref.close(got[b], want, tol)
    # in place: the strided slices themselves; the values between them stay
    v = fused[:, Hq + Hkv:].clone()
    r = bss.qk_norm_rope(q, k, pos, f, w[0], w[1], out=(q, k))
    assert r[0] is q and torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(fused[:, Hq + Hkv:], v)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    d = 128
    pos = torch.tensor([0, 1, -1, 1 << 17, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32, device="cuda")
    fused, _, _ = inputs(len(pos), 2, 1, d)
    f = freqs(d, 500000.0)
    qo, ko = bss.qk_norm_rope(fused[:, :2], fused[:, 2:3], pos, f, interleaved=interleaved)
    check(qo, fused[:, :2], None, pos, f, interleaved)
    check(ko, fused[:, 2:3], None, pos, f, interleaved)


def test_no_rotation_zeros_eps_and_nonfinite_rows():
    N, Hq, Hkv, d = 9, 4, 2, 64
    fused, w, pos = inputs(N, Hq, Hkv, d)
    fused[3] = 0
    fused[5, 1, 7] = float("nan")
    fused[6, 0, 63] = float("inf")  # outside the rotated part
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hkv]
    qo, ko = bss.qk_norm_rope(q, k, None, None, w[0], w[1], eps=1e-2)
    ok = torch.ones(N, Hq, dtype=torch.bool)
    ok[5, 1] = ok[6, 0] = False
    want, tol = ref.norm_rope(q.transpose(0, 1), w[0], pos, torch.empty(0, device="cuda"), False, 1e-2)
    ref.close(qo.cpu()[ok], want.transpose(0, 1).cpu()[ok], tol.transpose(0, 1).cpu()[ok])
    assert (qo[3] == 0).all() and (ko[3] == 0).all()
    assert qo[5, 1].isnan().all()
    # without a norm a value outside the rotated part is copied, whatever it is
    qo, _ = bss.qk_norm_rope(q, k, pos, freqs(32))
    assert torch.equal(qo[..., 32:].nan_to_num(7), q[..., 32:].nan_to_num(7))


def test_another_stream_and_a_captured_graph():
    fused, w, pos = inputs(64, 8, 2, 128)
    q, k, f = fused[:, :8], fused[:, 8:10], freqs(128)
    want = bss.qk_norm_rope(q, k, pos, f, w[0], w[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bss.qk_norm_rope(q, k, pos, f, w[0], w[1], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bss.qk_norm_rope(q, k, pos, f, w[0], w[1])
    fused.mul_(-2)
    pos.add_(3)
    graph.replay()
    want = bss.qk_norm_rope(q, k, pos, f, w[0], w[1])
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_refusals_of_the_helper():
    fused, w, pos = inputs(4, 4, 2, 64)
    q, k, f = fused[:, :4], fused[:, 4:6], freqs(64)
    buf = torch.zeros(4 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    odd = torch.as_strided(fused, (4, 4, 64), (260, 64, 1))  # a token stride that is no multiple of 8
    for call in (lambda: bss.qk_norm_rope(buf[1:].view(4, 4, 64), k, pos, f),  # 2-byte aligned
                 lambda: bss.qk_norm_rope(odd, k, pos, f),
                 lambda: bss.qk_norm_rope(q, k, pos, freqs(8)),
                 lambda: bss.qk_norm_rope(q, k, pos, f, w[0, :32]),
                 lambda: bss.qk_norm_rope(q, k, pos, f, eps=-1.0),
                 lambda: bss.qk_norm_rope(q, k, pos.cpu(), f),
                 lambda: bss.qk_norm_rope(q[:0], k[:0], pos[:0], f),
                 lambda: bss.qk_norm_rope(q, k, pos, f, out=(q[:2], k))):
        with pytest.raises(bss.AttnError):
            call()
