"""Refusals of the rotation, cache and tree entry points, checked without a GPU:
the C ABI rejects bad arguments before it touches the device, and the Python
helpers reject tensors of the wrong kind."""
import pytest
import torch

import block_skipping_softmax_b200 as bss
from block_skipping_softmax_b200 import build as bss_build

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses are passed only without a GPU")
P = 1 << 20  # aligned fake address: validation fails before it is ever used


@pytest.fixture(scope="module", autouse=True)
def built():
    bss_build.build()


ROPE = dict(q=P, k=P, q_out=P, k_out=P, positions=P, inv_freq=P, q_weight=P, k_weight=P, B=1, N=5, Hq=4, Hkv=2, d=64,
            rot_dim=64, interleaved=False, eps=1e-6, strides=(0, 384, 64) * 4, pos_stride_b=0)


@no_gpu
@pytest.mark.parametrize("args", [
    dict(q=0), dict(k_out=0), dict(q=P + 8), dict(k_weight=P + 2), dict(B=0), dict(N=0), dict(Hq=-1), dict(Hkv=0),
    dict(d=96), dict(rot_dim=8), dict(rot_dim=80), dict(rot_dim=-16), dict(positions=0), dict(inv_freq=0),
    dict(positions=P + 2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(strides=(0, 384, 60) + (0, 384, 64) * 3), dict(strides=(0, 384, 64) * 3 + (0, 4, 64)),
])
def test_norm_rope_rejects_bad_arguments(args):
    assert bss.attn_qk_norm_rope(**{**ROPE, **args}) == 1


@no_gpu
@pytest.mark.parametrize("args", [dict(B=1 << 16, N=1 << 15), dict(Hq=65535, Hkv=1)])
def test_norm_rope_refuses_what_it_does_not_support(args):
    assert bss.attn_qk_norm_rope(**{**ROPE, **args}) == 2


@no_gpu
def test_valid_arguments_reach_the_device_check():
    """What the refusals above leave is accepted: the first thing missing is the GPU."""
    assert bss.attn_qk_norm_rope(**ROPE) == 2
    assert bss.attn_qk_norm_rope(**{**ROPE, "rot_dim": 0, "positions": 0, "inv_freq": 0}) == 2
    assert bss.attn_cache_write_e4m3(**CACHE) == 2
    assert bss.attn_cache_read_e4m3(**CACHE) == 2
    assert bss.attn_tree_paged(**TREE) == 2
    assert bss.attn_tree_paged(**{**TREE, "tree_mask": 0}) == 2
    assert bss.attn_tree_paged_e4m3(**{**E4M3}) == 2


CACHE = dict(k=P, v=P, slots=P, K_codes=P, V_codes=P, K_scales=P, V_scales=P, B=1, N=5, Hkv=2, num_pages=3, d=64,
             strides=(0, 128, 64) * 2)


@no_gpu
@pytest.mark.parametrize("fn", ["attn_cache_write_e4m3", "attn_cache_read_e4m3"])
@pytest.mark.parametrize("args", [
    dict(k=0), dict(slots=0), dict(V_codes=0), dict(K_scales=0), dict(k=P + 8), dict(slots=P + 4), dict(K_codes=P + 8),
    dict(V_scales=P + 4), dict(B=0), dict(N=-1), dict(Hkv=0), dict(num_pages=0), dict(d=32),
    dict(strides=(0, 128, 4, 0, 128, 64)),
])
def test_cache_rejects_bad_arguments(fn, args):
    assert getattr(bss, fn)(**{**CACHE, **args}) == 1


TREE = dict(q=P, K_pages=P, V_pages=P, block_table=P, seq_lens=P, cu_q=P, tree_mask=P, o=P, B=2, max_q=8, total_q=16,
            Hq=8, Hkv=2, num_pages=10, max_pages_per_seq=4, max_seq_len=256, d=128, ws=P, ws_bytes=1 << 30)
E4M3 = {("K_codes" if k == "K_pages" else "V_codes" if k == "V_pages" else k): v for k, v in TREE.items()}
E4M3 |= dict(K_scales=P, V_scales=P)


@no_gpu
@pytest.mark.parametrize("args", [
    dict(q=0), dict(o=0), dict(block_table=0), dict(seq_lens=0), dict(cu_q=0), dict(q=P + 8), dict(o=P + 2),
    dict(block_table=P + 2), dict(cu_q=P + 1), dict(tree_mask=P + 4), dict(B=0), dict(max_q=0), dict(max_q=65),
    dict(total_q=0), dict(Hq=7), dict(Hkv=0), dict(num_pages=0), dict(max_pages_per_seq=0), dict(max_seq_len=0),
    dict(max_seq_len=257), dict(d=96),
])
def test_tree_rejects_bad_arguments(args):
    assert bss.attn_tree_paged(**{**TREE, **args}) == 1
    assert bss.attn_tree_paged_e4m3(**{**E4M3, **args}) == 1


@no_gpu
def test_tree_rejects_missing_scales_and_unsupported_sizes():
    assert bss.attn_tree_paged_e4m3(**{**E4M3, "K_scales": 0}) == 1
    assert bss.attn_tree_paged_e4m3(**{**E4M3, "V_scales": P + 4}) == 1
    assert bss.attn_tree_paged(**{**TREE, "B": 65536}) == 2
    assert bss.attn_tree_paged(**{**TREE, "num_pages": (1 << 30) - 1}) == 2


@no_gpu
def test_tree_rejects_bad_workspace():
    big = {**TREE, "max_pages_per_seq": 1000, "max_seq_len": 64000}
    need = bss.attn_tree_workspace_bytes(2, 8, 16, 8, 2, 64000, 128)
    assert need > 0
    assert bss.attn_tree_paged(**{**big, "ws": 0, "ws_bytes": 0}) == 1
    assert bss.attn_tree_paged(**{**big, "ws_bytes": need - 1}) == 1
    assert bss.attn_tree_paged(**{**big, "ws": P + 16}) == 1
    assert bss.attn_tree_paged(**{**big, "ws_bytes": need}) == 2  # only the GPU is missing


def test_tree_workspace_follows_the_sizes():
    ws = bss.attn_tree_workspace_bytes
    assert ws(1, 1, 1, 8, 8, 64, 128) == 0  # one page: one split
    assert ws(1, 65, 1, 8, 8, 64, 128) == 0 and ws(1, 1, 1, 8, 3, 64, 128) == 0  # refused sizes
    for (B, T, Hq, Hkv, L) in [(1, 1, 8, 8, 100000), (16, 8, 32, 8, 32768), (4, 64, 64, 8, 16384), (64, 1, 8, 1, 999)]:
        for d in (64, 128):
            n = ws(B, T, B * T, Hq, Hkv, L, d)
            assert n == ws(B, T, B * T, Hq, Hkv, L, d) and n % 256 == 0
            if n:  # at least two splits of fp32 partial results
                assert n >= B * T * Hq * 2 * (d + 1) * 4
            assert n < 4 << 30


def test_helpers_reject_host_tensors_and_wrong_kinds():
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    pos, freq = torch.zeros(5, dtype=torch.int32), torch.ones(32)
    codes, scales = torch.zeros(3, 2, 64, 64, dtype=torch.uint8), torch.ones(3, 2, 64)
    slots = torch.arange(5)
    table, lens, cu = torch.zeros(1, 3, dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.tensor([0, 5], dtype=torch.int32)
    pages = torch.zeros(3, 2, 64, 64, dtype=torch.bfloat16)
    calls = [
        lambda: bss.qk_norm_rope(x, x, pos, freq),
        lambda: bss.cache_write_e4m3(x, x, slots, codes, codes, scales, scales),
        lambda: bss.cache_read_e4m3(codes, codes, scales, scales, slots),
        lambda: bss.tree_paged(x, pages, pages, table, lens, cu, 5, 100),
        lambda: bss.tree_paged_e4m3(x, codes, codes, scales, scales, table, lens, cu, 5, 100),
        lambda: bss.qk_norm_rope(x.float(), x, pos, freq),
        lambda: bss.qk_norm_rope(x, x[:4], pos, freq),
        lambda: bss.qk_norm_rope(x, x, pos.long(), freq),
        lambda: bss.qk_norm_rope(x, x, pos[:3], freq),
        lambda: bss.qk_norm_rope(x.transpose(1, 2), x.transpose(1, 2), pos, freq),
        lambda: bss.cache_write_e4m3(x, x[:, :1], slots, codes, codes, scales, scales),
        lambda: bss.cache_write_e4m3(x, x, slots.int(), codes, codes, scales, scales),
        lambda: bss.cache_write_e4m3(x, x, slots, codes, codes, scales[:2], scales),
        lambda: bss.cache_read_e4m3(codes, codes[:, :, :32], scales, scales, slots),
        lambda: bss.tree_paged(x, pages, pages[:2], table, lens, cu, 5, 100),
        lambda: bss.tree_paged(x, pages, pages, table, lens, cu[:1], 5, 100),
        lambda: bss.tree_paged(x, pages, pages, table.long(), lens, cu, 5, 100),
        lambda: bss.tree_paged(x, pages, pages, table, lens, cu, 5, 100, tree_mask=torch.zeros(4, dtype=torch.int64)),
    ]
    for call in calls:
        with pytest.raises(bss.AttnError):
            call()
