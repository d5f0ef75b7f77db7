"""Skip Softmax attention for NVIDIA B200 (sm_100a): Python binding of libattn.so.

The functions named like the C ABI (``attn_prefill``, ``attn_decode`` ...)
take raw device pointers and sizes and only marshal arguments; the torch
helpers ``prefill`` and ``decode`` take tensors and pass their pointers.
Every step of the computation runs in the library's CUDA kernels.  There is
no CPU fallback: if the library cannot be loaded, or no sm_100 device is
present, calls raise ``AttnError``.

Method: "Accelerating Long-Context Inference with Skip Softmax in NVIDIA
TensorRT-LLM" (Key Points; Detailed Analysis) -- a key tile is skipped when
every query row's tile maximum is below its running maximum minus tau.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

__all__ = [
    "AttnError", "lib", "attn_prefill", "attn_prefill_ex", "attn_prefill_host", "prefill_host",
    "attn_prefill_varlen", "prefill_varlen", "attn_quantize_e4m3", "quantize_e4m3",
    "attn_prefill_qk8", "prefill_qk8", "attn_quantize_i8", "quantize_i8", "attn_prefill_qki8",
    "prefill_qki8", "attn_prefill_poly", "prefill_poly", "attn_decode", "attn_decode_ex",
    "attn_decode_noalloc", "attn_decode_rule", "attn_decode_paged", "decode_paged", "RULE_GROUP", "RULE_PER_HEAD", "RULE_SINK_SEED",
    "attn_qk_norm_rope", "qk_norm_rope", "attn_cache_write_e4m3", "cache_write_e4m3",
    "attn_cache_read_e4m3", "cache_read_e4m3", "attn_tree_paged", "tree_paged", "attn_tree_paged_e4m3",
    "tree_paged_e4m3", "attn_tree_workspace_bytes",
    "attn_decode_split_len", "attn_decode_tile", "attn_decode_workspace_bytes",
    "attn_set_stream", "attn_sync_status", "attn_last_timeout_site", "attn_set_wait_limit_ms",
    "attn_test_withhold_copy", "attn_status_string", "attn_shutdown", "prefill", "decode", "STATUS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn.so")
STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_CUDA",
          4: "ATTN_ERR_TIMEOUT"}


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {STATUS.get(status, status)}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libattn.so (built in-tree by ``block_skipping_softmax_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise AttnError(-1, f"loading {LIB_PATH} (not built; run python -m block_skipping_softmax_b200.build)")
    L = ctypes.CDLL(LIB_PATH)
    vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    ll = ctypes.c_longlong
    sig = {
        "attn_prefill": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, ci]),
        "attn_prefill_ex": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, ci, vp, vp]),
        "attn_prefill_host": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, ci, ci, vp]),
        "attn_prefill_poly": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, ci, ci, vp, vp]),
        "attn_prefill_varlen": (ci, [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf, ci, ci, vp, vp]),
        "attn_quantize_e4m3": (ci, [vp, vp, vp, ctypes.c_longlong, ctypes.c_longlong, vp]),
        "attn_prefill_qk8": (ci, [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, ci, vp, vp]),
        "attn_quantize_i8": (ci, [vp, vp, vp, ctypes.c_longlong, ctypes.c_longlong, vp]),
        "attn_prefill_qki8": (ci, [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, ci, vp, vp]),
        "attn_decode": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf]),
        "attn_decode_ex": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, vp, vp, vp, sz]),
        "attn_decode_noalloc": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, vp, vp]),
        "attn_decode_rule": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, vp, vp, vp, sz]),
        "attn_decode_paged": (ci, [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf, ci, vp, vp,
                                   vp, sz]),
        "attn_qk_norm_rope": (ci, [vp] * 8 + [ci] * 7 + [cf, vp, ll, vp]),
        "attn_cache_write_e4m3": (ci, [vp] * 7 + [ci] * 5 + [vp, vp]),
        "attn_cache_read_e4m3": (ci, [vp] * 7 + [ci] * 5 + [vp, vp]),
        "attn_tree_paged": (ci, [vp] * 8 + [ci] * 9 + [vp, vp, sz]),
        "attn_tree_paged_e4m3": (ci, [vp] * 10 + [ci] * 9 + [vp, vp, sz]),
        "attn_tree_workspace_bytes": (sz, [ci] * 7),
        "attn_decode_split_len": (ci, [ci, ci, ci]),
        "attn_decode_tile": (ci, []),
        "attn_decode_workspace_bytes": (sz, [ci, ci, ci, ci, ci]),
        "attn_set_stream": (ci, [vp]),
        "attn_sync_status": (ci, []),
        "attn_last_timeout_site": (ci, []),
        "attn_set_wait_limit_ms": (ci, [ci]),
        "attn_test_withhold_copy": (ci, [ci]),
        "attn_status_string": (ctypes.c_char_p, [ci]),
        "attn_shutdown": (None, []),
    }
    for name, (res, args) in sig.items():
        try:
            f = getattr(L, name)
        except AttributeError:  # an older build: the entry point raises when called
            continue
        f.restype, f.argtypes = res, args
    _lib = L
    return L


# ---- C-ABI names: argument marshalling only ---------------------------------

def attn_prefill(Q, K, V, O, B, Hq, Hkv, N, d, causal, tau, Br, Bc) -> int:
    return lib().attn_prefill(Q, K, V, O, B, Hq, Hkv, N, d, int(causal), float(tau), Br, Bc)


def attn_prefill_ex(Q, K, V, O, B, Hq, Hkv, N, d, causal, tau, Br, Bc, stream=None, skip_mask=None) -> int:
    return lib().attn_prefill_ex(Q, K, V, O, B, Hq, Hkv, N, d, int(causal), float(tau), Br, Bc,
                                 stream, skip_mask)


def attn_prefill_poly(Q, K, V, O, B, Hq, Hkv, N, d, causal, tau, Br, Bc, poly_pairs, stream=None,
                      skip_mask=None) -> int:
    return lib().attn_prefill_poly(Q, K, V, O, B, Hq, Hkv, N, d, int(causal), float(tau), Br, Bc,
                                   int(poly_pairs), stream, skip_mask)


def attn_prefill_host(Qh, Kh, Vh, Oh, B, Hq, Hkv, N, d, causal, tau, Br, Bc, chunk=0, stream=None) -> int:
    return lib().attn_prefill_host(Qh, Kh, Vh, Oh, B, Hq, Hkv, N, d, int(causal), float(tau), Br, Bc,
                                   int(chunk), stream)


def attn_prefill_varlen(Q, K, V, O, cu_seqlens, B, max_seqlen, total_tokens, Hq, Hkv, d, causal, tau,
                        Br, Bc, stream=None, skip_mask=None) -> int:
    return lib().attn_prefill_varlen(Q, K, V, O, cu_seqlens, B, max_seqlen, total_tokens, Hq, Hkv, d,
                                     int(causal), float(tau), Br, Bc, stream, skip_mask)


def attn_quantize_e4m3(x, q, scales, groups, group_elems, stream=None) -> int:
    return lib().attn_quantize_e4m3(x, q, scales, int(groups), int(group_elems), stream)


def attn_prefill_qk8(Q8, K8, q_scales, k_scales, V, O, B, Hq, Hkv, N, d, causal, tau, Br, Bc, stream=None,
                     skip_mask=None) -> int:
    return lib().attn_prefill_qk8(Q8, K8, q_scales, k_scales, V, O, B, Hq, Hkv, N, d, int(causal),
                                  float(tau), Br, Bc, stream, skip_mask)


def attn_quantize_i8(x, q, scales, groups, group_elems, stream=None) -> int:
    return lib().attn_quantize_i8(x, q, scales, int(groups), int(group_elems), stream)


def attn_prefill_qki8(Q8, K8, q_scales, k_scales, V, O, B, Hq, Hkv, N, d, causal, tau, Br, Bc, stream=None,
                      skip_mask=None) -> int:
    return lib().attn_prefill_qki8(Q8, K8, q_scales, k_scales, V, O, B, Hq, Hkv, N, d, int(causal),
                                   float(tau), Br, Bc, stream, skip_mask)


def attn_decode(q, K, V, o, B, Hq, Hkv, L, d, tau) -> int:
    return lib().attn_decode(q, K, V, o, B, Hq, Hkv, L, d, float(tau))


def attn_decode_ex(q, K, V, o, B, Hq, Hkv, L, d, tau, stream=None, skip_mask=None, ws=None, ws_bytes=0) -> int:
    return lib().attn_decode_ex(q, K, V, o, B, Hq, Hkv, L, d, float(tau), stream, skip_mask, ws, ws_bytes)


RULE_GROUP, RULE_PER_HEAD, RULE_SINK_SEED = 0, 1, 2


def attn_decode_rule(q, K, V, o, B, Hq, Hkv, L, d, tau, rule, stream=None, skip_mask=None, ws=None,
                     ws_bytes=0) -> int:
    return lib().attn_decode_rule(q, K, V, o, B, Hq, Hkv, L, d, float(tau), int(rule), stream,
                                  skip_mask, ws, ws_bytes)


def attn_decode_paged(q, K_pages, V_pages, block_table, seq_lens, o, B, Hq, Hkv, num_pages,
                      max_pages_per_seq, max_seq_len, d, tau, rule=0, stream=None, skip_mask=None,
                      ws=None, ws_bytes=0) -> int:
    return lib().attn_decode_paged(q, K_pages, V_pages, block_table, seq_lens, o, B, Hq, Hkv,
                                   num_pages, max_pages_per_seq, max_seq_len, d, float(tau),
                                   int(rule), stream, skip_mask, ws, ws_bytes)


def attn_decode_noalloc(q, K, V, o, B, Hq, Hkv, L, d, tau, stream=None, skip_mask=None) -> int:
    """Decode with the library's fixed scratch array: no device allocation."""
    return lib().attn_decode_noalloc(q, K, V, o, B, Hq, Hkv, L, d, float(tau), stream, skip_mask)


@functools.lru_cache(maxsize=256)
def _strides(values):
    """The C array of a tuple of strides (the library only reads it)."""
    return (ctypes.c_longlong * len(values))(*values)


def attn_qk_norm_rope(q, k, q_out, k_out, positions, inv_freq, q_weight, k_weight, B, N, Hq, Hkv, d, rot_dim,
                      interleaved, eps, strides, pos_stride_b, stream=None) -> int:
    """``strides``: 12 ints (batch, token and head stride of q, k, q_out, k_out, in elements)."""
    return lib().attn_qk_norm_rope(q, k, q_out, k_out, positions, inv_freq, q_weight, k_weight, B, N, Hq, Hkv, d,
                                   rot_dim, int(interleaved), eps, _strides(tuple(strides)), pos_stride_b, stream)


def attn_cache_write_e4m3(k, v, slots, K_codes, V_codes, K_scales, V_scales, B, N, Hkv, num_pages, d, strides,
                          stream=None) -> int:
    """``strides``: 6 ints (batch, token and head stride of k and v, in elements)."""
    return lib().attn_cache_write_e4m3(k, v, slots, K_codes, V_codes, K_scales, V_scales, B, N, Hkv, num_pages,
                                       d, _strides(tuple(strides)), stream)


def attn_cache_read_e4m3(K_codes, V_codes, K_scales, V_scales, slots, k, v, B, N, Hkv, num_pages, d, strides,
                         stream=None) -> int:
    """``strides``: 6 ints (batch, token and head stride of k and v, in elements)."""
    return lib().attn_cache_read_e4m3(K_codes, V_codes, K_scales, V_scales, slots, k, v, B, N, Hkv, num_pages,
                                      d, _strides(tuple(strides)), stream)


def attn_tree_paged(q, K_pages, V_pages, block_table, seq_lens, cu_q, tree_mask, o, B, max_q, total_q, Hq, Hkv,
                    num_pages, max_pages_per_seq, max_seq_len, d, stream=None, ws=None, ws_bytes=0) -> int:
    return lib().attn_tree_paged(q, K_pages, V_pages, block_table, seq_lens, cu_q, tree_mask, o, B, max_q,
                                 total_q, Hq, Hkv, num_pages, max_pages_per_seq, max_seq_len, d, stream, ws,
                                 ws_bytes)


def attn_tree_paged_e4m3(q, K_codes, V_codes, K_scales, V_scales, block_table, seq_lens, cu_q, tree_mask, o, B,
                         max_q, total_q, Hq, Hkv, num_pages, max_pages_per_seq, max_seq_len, d, stream=None,
                         ws=None, ws_bytes=0) -> int:
    return lib().attn_tree_paged_e4m3(q, K_codes, V_codes, K_scales, V_scales, block_table, seq_lens, cu_q,
                                      tree_mask, o, B, max_q, total_q, Hq, Hkv, num_pages, max_pages_per_seq,
                                      max_seq_len, d, stream, ws, ws_bytes)


def attn_tree_workspace_bytes(B, max_q, total_q, Hq, Hkv, max_seq_len, d) -> int:
    return lib().attn_tree_workspace_bytes(B, max_q, total_q, Hq, Hkv, max_seq_len, d)


def attn_decode_split_len(B, Hkv, L) -> int:
    return lib().attn_decode_split_len(B, Hkv, L)


def attn_decode_tile() -> int:
    return lib().attn_decode_tile()


def attn_decode_workspace_bytes(B, Hq, Hkv, L, d) -> int:
    return lib().attn_decode_workspace_bytes(B, Hq, Hkv, L, d)


def attn_set_stream(stream) -> int:
    return lib().attn_set_stream(stream)


def attn_sync_status() -> int:
    return lib().attn_sync_status()


def attn_last_timeout_site() -> int:
    return lib().attn_last_timeout_site()


def attn_set_wait_limit_ms(ms) -> int:
    return lib().attn_set_wait_limit_ms(int(ms))


def attn_test_withhold_copy(which) -> int:
    """Test support: 1 = decode CTAs withhold their first V copy (the waits run out)."""
    return lib().attn_test_withhold_copy(int(which))


def attn_status_string(status) -> str:
    return lib().attn_status_string(int(status)).decode()


def attn_shutdown() -> None:
    lib().attn_shutdown()


# ---- torch helpers: pass tensor pointers, no compute -------------------------

def _check(st: int, what: str):
    if st != 0:
        raise AttnError(st, what)


def _stream_ptr(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def prefill(Q, K, V, causal: bool, tau: float = math.inf, Br: int = 128, Bc: int = 128,
            out=None, skip_mask: bool = False, stream=None):
    """O = Skip Softmax attention of bf16 CUDA tensors Q [B,Hq,N,d], K/V [B,Hkv,N,d].

    Returns O (and the uint8 skip mask [B,Hq,ceil(N/Br),ceil(N/Bc)] when asked).
    """
    import torch

    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    for t in (Q, K, V):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise AttnError(1, "prefill (tensors must be contiguous bf16 CUDA tensors)")
    O = out if out is not None else torch.empty_like(Q)
    mask = None
    if skip_mask:
        mask = torch.empty(B, Hq, -(-N // Br), -(-N // Bc), dtype=torch.uint8, device=Q.device)
    st = attn_prefill_ex(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), B, Hq, Hkv, N, d,
                         causal, tau, Br, Bc, _stream_ptr(stream),
                         mask.data_ptr() if mask is not None else None)
    _check(st, "attn_prefill_ex")
    return (O, mask) if skip_mask else O


def prefill_poly(Q, K, V, causal: bool, tau: float = math.inf, poly_pairs: int = 4, out=None,
                 skip_mask: bool = False, stream=None):
    """attn_prefill_poly on bf16 CUDA tensors (d = 128, Br = Bc = 128):
    poly_pairs of every 16 exponential pairs on the FMA-pipe polynomial."""
    import torch

    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    for t in (Q, K, V):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise AttnError(1, "prefill_poly (tensors must be contiguous bf16 CUDA tensors)")
    O = out if out is not None else torch.empty_like(Q)
    mask = None
    if skip_mask:
        mask = torch.empty(B, Hq, -(-N // 128), -(-N // 128), dtype=torch.uint8, device=Q.device)
    st = attn_prefill_poly(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), B, Hq, Hkv, N, d,
                           causal, tau, 128, 128, poly_pairs, _stream_ptr(stream),
                           mask.data_ptr() if mask is not None else None)
    _check(st, "attn_prefill_poly")
    return (O, mask) if skip_mask else O


def prefill_varlen(Q, K, V, cu_seqlens, max_seqlen: int, causal: bool, tau: float = math.inf,
                   Br: int = 128, Bc: int = 128, out=None, skip_mask: bool = False, stream=None):
    """Packed variable-length prefill: Q [total, Hq, d], K/V [total, Hkv, d]
    bf16 CUDA tensors; cu_seqlens int32 CUDA tensor [B + 1]."""
    import torch

    total, Hq, d = Q.shape
    Hkv = K.shape[1]
    B = cu_seqlens.numel() - 1
    for t in (Q, K, V):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise AttnError(1, "prefill_varlen (tensors must be contiguous bf16 CUDA tensors)")
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
        raise AttnError(1, "prefill_varlen (cu_seqlens must be an int32 CUDA tensor)")
    O = out if out is not None else torch.empty_like(Q)
    mask = None
    if skip_mask:
        mask = torch.empty(B, Hq, -(-max_seqlen // Br), -(-max_seqlen // Bc), dtype=torch.uint8,
                           device=Q.device)
    st = attn_prefill_varlen(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), cu_seqlens.data_ptr(),
                             B, max_seqlen, total, Hq, Hkv, d, causal, tau, Br, Bc, _stream_ptr(stream),
                             mask.data_ptr() if mask is not None else None)
    _check(st, "attn_prefill_varlen")
    return (O, mask) if skip_mask else O


def quantize_e4m3(x, out=None, stream=None):
    """e4m3 codes (uint8, x's shape) and one power-of-two scale per head slab
    (float32 [B, H]) of a contiguous bf16 CUDA tensor x [B, H, N, d].
    ``out`` = (codes, scales) writes into existing tensors."""
    return _quantize(x, out, stream, int8=False)


def quantize_i8(x, out=None, stream=None):
    """int8 codes (int8, x's shape) and one power-of-two scale per head slab
    (float32 [B, H]) of a contiguous bf16 CUDA tensor x [B, H, N, d]."""
    return _quantize(x, out, stream, int8=True)


def _quantize(x, out, stream, int8):
    import torch

    code_dtype = torch.int8 if int8 else torch.uint8
    what = "quantize_i8" if int8 else "quantize_e4m3"

    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous() or x.dim() != 4:
        raise AttnError(1, f"{what} (x must be a contiguous 4-d bf16 CUDA tensor)")
    B, H, N, d = x.shape
    if out is not None:
        q, scales = out
        if (q.dtype != code_dtype or q.shape != x.shape or not q.is_contiguous() or
                scales.dtype != torch.float32 or scales.numel() != B * H or not scales.is_contiguous()):
            raise AttnError(1, f"{what} (out must be {code_dtype} codes of x's shape and float32 [B, H])")
    else:
        q = torch.empty(x.shape, dtype=code_dtype, device=x.device)
        scales = torch.empty(B, H, dtype=torch.float32, device=x.device)
    fn = attn_quantize_i8 if int8 else attn_quantize_e4m3
    _check(fn(x.data_ptr(), q.data_ptr(), scales.data_ptr(), B * H, N * d, _stream_ptr(stream)),
           "attn_" + what)
    return q, scales


def prefill_qk8(Q8, K8, q_scales, k_scales, V, causal: bool, tau: float = math.inf, Br: int = 128,
                Bc: int = 128, out=None, skip_mask: bool = False, stream=None):
    """Prefill with e4m3 Q8 [B,Hq,N,d], K8 [B,Hkv,N,d] (uint8 codes from
    quantize_e4m3), float32 scales [B,Hq] / [B,Hkv], and bf16 V."""
    return _prefill_8bit(Q8, K8, q_scales, k_scales, V, causal, tau, Br, Bc, out, skip_mask, stream, False)


def prefill_qki8(Q8, K8, q_scales, k_scales, V, causal: bool, tau: float = math.inf, Br: int = 128,
                 Bc: int = 128, out=None, skip_mask: bool = False, stream=None):
    """Prefill with int8 Q8 [B,Hq,N,d], K8 [B,Hkv,N,d] (codes from
    quantize_i8), float32 scales [B,Hq] / [B,Hkv], and bf16 V."""
    return _prefill_8bit(Q8, K8, q_scales, k_scales, V, causal, tau, Br, Bc, out, skip_mask, stream, True)


def _prefill_8bit(Q8, K8, q_scales, k_scales, V, causal, tau, Br, Bc, out, skip_mask, stream, int8):
    import torch

    what = "prefill_qki8" if int8 else "prefill_qk8"
    code_dtype = torch.int8 if int8 else torch.uint8
    B, Hq, N, d = Q8.shape
    Hkv = K8.shape[1]
    for t in (Q8, K8):
        if t.dtype != code_dtype or not t.is_cuda or not t.is_contiguous():
            raise AttnError(1, f"{what} (Q8, K8 must be contiguous {code_dtype} CUDA tensors)")
    for t in (q_scales, k_scales):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise AttnError(1, f"{what} (scales must be contiguous float32 CUDA tensors)")
    if V.dtype != torch.bfloat16 or not V.is_cuda or not V.is_contiguous():
        raise AttnError(1, f"{what} (V must be a contiguous bf16 CUDA tensor)")
    O = out if out is not None else torch.empty(Q8.shape, dtype=torch.bfloat16, device=Q8.device)
    mask = None
    if skip_mask:
        mask = torch.empty(B, Hq, -(-N // Br), -(-N // Bc), dtype=torch.uint8, device=Q8.device)
    fn = attn_prefill_qki8 if int8 else attn_prefill_qk8
    st = fn(Q8.data_ptr(), K8.data_ptr(), q_scales.data_ptr(), k_scales.data_ptr(),
            V.data_ptr(), O.data_ptr(), B, Hq, Hkv, N, d, causal, tau, Br, Bc,
            _stream_ptr(stream), mask.data_ptr() if mask is not None else None)
    _check(st, "attn_" + what)
    return (O, mask) if skip_mask else O


def prefill_host(Qh, Kh, Vh, causal: bool, tau: float = math.inf, Br: int = 128, Bc: int = 128,
                 out=None, chunk: int = 0, stream=None):
    """attn_prefill_host on host (CPU) bf16 tensors; pinned memory lets the
    copies overlap.  Asynchronous on ``stream``: synchronise it before reading
    the returned tensor."""
    import torch

    B, Hq, N, d = Qh.shape
    Hkv = Kh.shape[1]
    for t in (Qh, Kh, Vh):
        if t.dtype != torch.bfloat16 or t.is_cuda or not t.is_contiguous():
            raise AttnError(1, "prefill_host (tensors must be contiguous bf16 host tensors)")
    Oh = out if out is not None else torch.empty_like(Qh, pin_memory=Qh.is_pinned())
    st = attn_prefill_host(Qh.data_ptr(), Kh.data_ptr(), Vh.data_ptr(), Oh.data_ptr(), B, Hq, Hkv, N, d,
                           causal, tau, Br, Bc, chunk, _stream_ptr(stream))
    _check(st, "attn_prefill_host")
    return Oh


def decode(q, K, V, tau: float = math.inf, out=None, skip_mask: bool = False, stream=None,
           workspace=None, rule: int = RULE_GROUP):
    """o = Skip Softmax decode attention: q [B,Hq,d], K/V [B,Hkv,L,d] bf16 CUDA tensors.

    ``workspace``: optional uint8 CUDA tensor of at least
    attn_decode_workspace_bytes(...) bytes; otherwise the library's own is used.
    """
    import torch

    B, Hq, d = q.shape
    Hkv, L = K.shape[1], K.shape[2]
    for t in (q, K, V):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise AttnError(1, "decode (tensors must be contiguous bf16 CUDA tensors)")
    o = out if out is not None else torch.empty_like(q)
    mask = None
    if skip_mask:
        rows = Hq if rule & RULE_PER_HEAD else Hkv
        mask = torch.empty(B, rows, -(-L // attn_decode_tile()), dtype=torch.uint8, device=q.device)
    ws, wsb = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    st = attn_decode_rule(q.data_ptr(), K.data_ptr(), V.data_ptr(), o.data_ptr(), B, Hq, Hkv, L, d,
                          tau, rule, _stream_ptr(stream),
                          mask.data_ptr() if mask is not None else None, ws, wsb)
    _check(st, "attn_decode_rule")
    return (o, mask) if skip_mask else o


def decode_paged(q, K_pages, V_pages, block_table, seq_lens, max_seq_len: int, tau: float = math.inf,
                 out=None, skip_mask: bool = False, stream=None, rule: int = RULE_GROUP):
    """o = Skip Softmax decode from a paged KV cache.

    q [B,Hq,d]; K_pages/V_pages [num_pages,Hkv,64,d] bf16; block_table int32
    [B,max_pages]; seq_lens int32 [B]; all CUDA tensors.
    """
    import torch

    B, Hq, d = q.shape
    num_pages, Hkv = K_pages.shape[0], K_pages.shape[1]
    for t in (q, K_pages, V_pages):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise AttnError(1, "decode_paged (tensors must be contiguous bf16 CUDA tensors)")
    for t in (block_table, seq_lens):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise AttnError(1, "decode_paged (block_table/seq_lens must be contiguous int32 CUDA tensors)")
    o = out if out is not None else torch.empty_like(q)
    mask = None
    if skip_mask:
        rows = Hq if rule & RULE_PER_HEAD else Hkv
        mask = torch.empty(B, rows, -(-max_seq_len // attn_decode_tile()), dtype=torch.uint8,
                           device=q.device)
    st = attn_decode_paged(q.data_ptr(), K_pages.data_ptr(), V_pages.data_ptr(), block_table.data_ptr(),
                           seq_lens.data_ptr(), o.data_ptr(), B, Hq, Hkv, num_pages,
                           block_table.shape[1], max_seq_len, d, tau, rule, _stream_ptr(stream),
                           mask.data_ptr() if mask is not None else None)
    _check(st, "attn_decode_paged")
    return (o, mask) if skip_mask else o


# ---- rotation, cache and tree helpers -----------------------------------------
#
# These run once a layer and token, beside kernels of a few microseconds: checks
# are plain comparisons, and messages are made only when one fails.

def _no(what: str, why: str) -> AttnError:
    return AttnError(1, f"{what} ({why})")


def _device(what, tensors, torch) -> int:
    """The index of the tensors' one device, which is the current one (the library launches there)."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise _no(what, "tensors must be on one CUDA device")
    if dev < 0:
        raise _no(what, "tensors must be CUDA tensors")
    try:
        current = torch._C._cuda_getDevice()  # CUDA is up: there are tensors on it
    except AttributeError:
        current = torch.cuda.current_device()
    if dev != current:
        raise _no(what, "tensors must be on the current CUDA device")
    return dev


def _raw_stream(dev: int, torch) -> int:
    """The current stream's cudaStream_t, without making a Stream object."""
    try:
        return torch._C._cuda_getCurrentRawStream(dev)
    except AttributeError:
        return torch.cuda.current_stream(dev).cuda_stream


def _run(dev, stream, tensors, make, call, torch):
    """call(make(), raw stream) on `stream` (None: the current one).  Memory that
    make() allocates belongs to that stream, and tensors that meet it from
    another one are recorded on it, so that the caching allocator keeps them
    until the call's kernels are done."""
    raw = _raw_stream(dev, torch)
    if stream is None or stream.cuda_stream == raw:
        new = make()
        return new, call(new, raw)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    current = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        new = make()
    for t in new:
        if t is not None:
            t.record_stream(current)
            t.record_stream(stream)
    return new, call(new, stream.cuda_stream)


def _token_strides(what, x):
    """(batch, token, head) strides of [tokens, H, d] or [B, H, N, d]; an axis of length 1 counts as 0."""
    strides = x.stride()
    if len(strides) == 3:
        (N, H, _), (sn, sh, sd), sb = x.shape, strides, 0
    else:
        (B, H, N, _), (sb, sh, sn, sd) = x.shape, strides
        if B == 1:
            sb = 0
    if sd != 1:
        raise _no(what, "the d elements of a head must be contiguous")
    return sb, sn if N > 1 else 0, sh if H > 1 else 0


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, out=None, stream=None):
    """Norms of queries and keys for each head, and their rotation by position, in one pass.

    q, k: bf16 CUDA tensors [tokens, H, d] or [B, H, N, d], of any strides that
    are multiples of 8 (d contiguous), for instance slices of a fused
    projection.  positions: int32 [tokens], or [N] or [B, N].  inv_freq:
    float32 [rot_dim / 2], None for no rotation.  q_weight, k_weight: bf16 [d],
    None for no norm.  interleaved: the pairs are (2i, 2i+1) instead of
    (i, i + rot_dim/2).  Returns (q, k), contiguous, or ``out`` = (q, k), which
    may be the inputs themselves.
    """
    import torch

    what = "qk_norm_rope"
    bf16 = torch.bfloat16
    q_shape, k_shape = q.shape, k.shape
    axes = len(q_shape)
    if axes not in (3, 4) or len(k_shape) != axes:
        raise _no(what, "q and k must be [tokens, H, d] or [B, H, N, d]")
    if axes == 3:
        (N, Hq, d), (Nk, Hkv, dk), B, Bk = q_shape, k_shape, 1, 1
    else:
        (B, Hq, N, d), (Bk, Hkv, Nk, dk) = q_shape, k_shape
    if N != Nk or d != dk or B != Bk:
        raise _no(what, "q and k must have the same tokens and head size")
    if q.dtype is not bf16 or k.dtype is not bf16:
        raise _no(what, "q and k must be bf16")
    rot = pos_stride = 0
    pos_ptr = freq_ptr = None
    tensors = [q, k]
    n_freq = 0 if inv_freq is None else inv_freq.numel()
    if n_freq:
        if inv_freq.dtype is not torch.float32 or not inv_freq.is_contiguous():
            raise _no(what, "inv_freq must be contiguous float32")
        if positions is None:
            raise _no(what, "a rotation needs positions")
        shape = positions.shape
        if (positions.dtype is not torch.int32 or (N > 1 and positions.stride(-1) != 1) or
                not (shape == (N,) or (axes == 4 and shape == (B, N)))):
            raise _no(what, "positions must be int32 [N] or [B, N]")
        if len(shape) == 2 and B > 1:
            pos_stride = positions.stride(0)
        rot, pos_ptr, freq_ptr = 2 * n_freq, positions.data_ptr(), inv_freq.data_ptr()
        tensors += (positions, inv_freq)
    for w in (q_weight, k_weight):
        if w is not None:
            if w.dtype is not bf16 or w.shape != (d,) or not w.is_contiguous():
                raise _no(what, "weights must be contiguous bf16 [d]")
            tensors.append(w)
    if out is not None:
        if out[0].shape != q_shape or out[1].shape != k_shape or out[0].dtype is not bf16 or out[1].dtype is not bf16:
            raise _no(what, "out must be bf16 of the inputs' shapes")
        tensors += out
    strides = _token_strides(what, q) + _token_strides(what, k)
    if out is not None:
        strides += _token_strides(what, out[0]) + _token_strides(what, out[1])
    elif axes == 3:  # contiguous ones; a stride of an axis of length 1 is not used
        strides += (0, Hq * d, d, 0, Hkv * d, d)
    else:
        strides += (Hq * N * d, d, N * d, Hkv * N * d, d, N * d)
    dev = _device(what, tensors, torch)

    def call(new, raw):
        qo, ko = new
        return lib().attn_qk_norm_rope(
            q.data_ptr(), k.data_ptr(), qo.data_ptr(), ko.data_ptr(), pos_ptr, freq_ptr,
            None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
            B, N, Hq, Hkv, d, rot, interleaved, eps, _strides(strides), pos_stride, raw)

    def make():
        if out is not None:
            return out
        form = torch.contiguous_format
        return torch.empty_like(q, memory_format=form), torch.empty_like(k, memory_format=form)

    new, st = _run(dev, stream, tensors, make, call, torch)
    if st:
        raise AttnError(st, "attn_qk_norm_rope")
    return new


def _check_codes(what, K_codes, V_codes, K_scales, V_scales, torch):
    shape = K_codes.shape
    if len(shape) != 4 or shape[2] != 64 or V_codes.shape != shape or K_codes.dtype is not torch.uint8 or \
            V_codes.dtype is not torch.uint8 or not K_codes.is_contiguous() or not V_codes.is_contiguous():
        raise _no(what, "codes must be contiguous uint8 [num_pages, Hkv, 64, d]")
    groups = shape[:3]
    if K_scales.shape != groups or V_scales.shape != groups or K_scales.dtype is not torch.float32 or \
            V_scales.dtype is not torch.float32 or not K_scales.is_contiguous() or not V_scales.is_contiguous():
        raise _no(what, "scales must be contiguous float32 [num_pages, Hkv, 64]")
    return shape


def _check_slots(what, slots, torch):
    if slots.dtype is not torch.int64 or slots.dim() not in (1, 2) or not slots.is_contiguous():
        raise _no(what, "slots must be contiguous int64, [tokens] or [B, N]")


def cache_write_e4m3(k, v, slots, K_codes, V_codes, K_scales, V_scales, stream=None) -> None:
    """Quantise keys and values to e4m3 and write them into a paged cache, in place.

    k, v: bf16 CUDA tensors [tokens, Hkv, d] or [B, Hkv, N, d] (strides as in
    qk_norm_rope).  slots: int64 [tokens] or [B, N]: page * 64 + key, no two
    alike; a token whose slot lies outside the pool (-1) is not written.
    K_codes, V_codes: uint8 [num_pages, Hkv, 64, d]; K_scales, V_scales: float32
    [num_pages, Hkv, 64].
    """
    import torch

    what = "cache_write_e4m3"
    shape = k.shape
    if len(shape) not in (3, 4) or v.shape != shape:
        raise _no(what, "k and v must be [tokens, H, d] or [B, H, N, d], of one shape")
    if k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16:
        raise _no(what, "k and v must be bf16")
    pages, pool_heads, _, pool_d = _check_codes(what, K_codes, V_codes, K_scales, V_scales, torch)
    _check_slots(what, slots, torch)
    if len(shape) == 3:
        (N, Hkv, d), B, tokens = shape, 1, shape[:1]
    else:
        B, Hkv, N, d = shape
        tokens = (B, N)
    if pool_heads != Hkv or pool_d != d:
        raise _no(what, "the pool has other heads than k")
    if slots.shape != tokens:
        raise _no(what, "slots must have one entry a token")
    tensors = (k, v, slots, K_codes, V_codes, K_scales, V_scales)
    dev = _device(what, tensors, torch)
    strides = _strides(_token_strides(what, k) + _token_strides(what, v))
    _, st = _run(dev, stream, tensors, tuple, lambda _, raw: lib().attn_cache_write_e4m3(
        k.data_ptr(), v.data_ptr(), slots.data_ptr(), K_codes.data_ptr(), V_codes.data_ptr(), K_scales.data_ptr(),
        V_scales.data_ptr(), B, N, Hkv, pages, d, strides, raw), torch)
    if st:
        raise AttnError(st, "attn_cache_write_e4m3")


def cache_read_e4m3(K_codes, V_codes, K_scales, V_scales, slots, out=None, stream=None):
    """(k, v) of the given slots of an e4m3 cache, as bf16.

    slots int64 [tokens] gives [tokens, Hkv, d]; [B, N] gives [B, Hkv, N, d].  A
    slot outside the pool reads zeros.  ``out`` = (k, v) writes into existing
    tensors of those shapes (strides as in qk_norm_rope).
    """
    import torch

    what = "cache_read_e4m3"
    bf16 = torch.bfloat16
    pages, Hkv, _, d = _check_codes(what, K_codes, V_codes, K_scales, V_scales, torch)
    _check_slots(what, slots, torch)
    tokens = slots.shape
    if len(tokens) == 1:
        N, B = tokens[0], 1
        shape = (N, Hkv, d)
        strides = (0, Hkv * d, d) * 2  # contiguous; a stride of an axis of length 1 is not used
    else:
        B, N = tokens
        shape = (B, Hkv, N, d)
        strides = (Hkv * N * d, d, N * d) * 2
    tensors = (K_codes, V_codes, K_scales, V_scales, slots)
    if out is not None:
        for t in out:
            if t.shape != shape or t.dtype is not bf16:
                raise _no(what, "out must be bf16, [tokens, Hkv, d] or [B, Hkv, N, d] as slots are")
        tensors += tuple(out)
        strides = _token_strides(what, out[0]) + _token_strides(what, out[1])
    dev = _device(what, tensors, torch)

    def make():
        if out is not None:
            return out
        k = K_scales.new_empty(shape, dtype=bf16)
        return k, torch.empty_like(k)

    new, st = _run(dev, stream, tensors, make, lambda new, raw: lib().attn_cache_read_e4m3(
        K_codes.data_ptr(), V_codes.data_ptr(), K_scales.data_ptr(), V_scales.data_ptr(), slots.data_ptr(),
        new[0].data_ptr(), new[1].data_ptr(), B, N, Hkv, pages, d, _strides(strides), raw), torch)
    if st:
        raise AttnError(st, "attn_cache_read_e4m3")
    return new


def tree_paged(q, K_pages, V_pages, block_table, seq_lens, cu_q, max_q: int, max_seq_len: int, tree_mask=None,
               out=None, stream=None, workspace=None):
    """Attention of each sequence's drafted tokens over its paged bf16 cache.

    q: bf16 [total_q, Hq, d], sequence b's tokens at rows cu_q[b]..cu_q[b+1]
    (cu_q int32 [B + 1], at most max_q <= 64 tokens each).  K_pages, V_pages,
    block_table and seq_lens as in decode_paged; seq_lens count the drafted
    tokens' own keys, which are each sequence's last.  tree_mask: int64
    [total_q], bit j set iff the token sees drafted key j; None: a chain.
    Rows of no sequence stay as they are in ``out``, and are undefined without
    it.  ``workspace``: optional uint8 CUDA tensor of at least
    attn_tree_workspace_bytes(...) bytes.
    """
    import torch

    if K_pages.dtype is not torch.bfloat16 or V_pages.dtype is not torch.bfloat16 or V_pages.shape != K_pages.shape or \
            not K_pages.is_contiguous() or not V_pages.is_contiguous():
        raise _no("tree_paged", "pages must be contiguous bf16 of one shape")
    return _tree("tree_paged", q, K_pages, V_pages, None, None, block_table, seq_lens, cu_q, max_q, max_seq_len,
                 tree_mask, out, stream, workspace)


def tree_paged_e4m3(q, K_codes, V_codes, K_scales, V_scales, block_table, seq_lens, cu_q, max_q: int,
                    max_seq_len: int, tree_mask=None, out=None, stream=None, workspace=None):
    """tree_paged over the e4m3 cache that cache_write_e4m3 writes."""
    import torch

    _check_codes("tree_paged_e4m3", K_codes, V_codes, K_scales, V_scales, torch)
    return _tree("tree_paged_e4m3", q, K_codes, V_codes, K_scales, V_scales, block_table, seq_lens, cu_q, max_q,
                 max_seq_len, tree_mask, out, stream, workspace)


@functools.lru_cache(maxsize=256)
def _tree_workspace(*sizes) -> int:
    return lib().attn_tree_workspace_bytes(*sizes)


def _tree(what, q, K, V, K_scales, V_scales, block_table, seq_lens, cu_q, max_q, max_seq_len, tree_mask, out,
          stream, workspace):
    import torch

    bf16, int32 = torch.bfloat16, torch.int32
    q_shape, pool, table = q.shape, K.shape, block_table.shape
    if len(q_shape) != 3 or q.dtype is not bf16 or not q.is_contiguous():
        raise _no(what, "q must be contiguous bf16 [total_q, Hq, d]")
    total, Hq, d = q_shape
    if len(pool) != 4 or pool[2] != 64 or pool[3] != d:
        raise _no(what, "the cache must be [num_pages, Hkv, 64, d]")
    pages, Hkv, _, _ = pool
    if block_table.dtype is not int32 or seq_lens.dtype is not int32 or cu_q.dtype is not int32 or \
            not block_table.is_contiguous() or not seq_lens.is_contiguous() or not cu_q.is_contiguous():
        raise _no(what, "block_table, seq_lens and cu_q must be contiguous int32")
    B = seq_lens.numel()
    if len(table) != 2 or table[0] != B or cu_q.numel() != B + 1:
        raise _no(what, "block_table must be [B, max_pages] and cu_q [B + 1]")
    if max_q >> 31 or max_seq_len >> 31:  # the C interface would take them for others
        raise _no(what, "max_q and max_seq_len must be ints of 31 bits")
    tensors = [q, K, V, block_table, seq_lens, cu_q]
    if K_scales is not None:
        tensors += (K_scales, V_scales)
    if tree_mask is not None:
        if tree_mask.dtype is not torch.int64 or tree_mask.shape != (total,) or not tree_mask.is_contiguous():
            raise _no(what, "tree_mask must be contiguous int64 [total_q]")
        tensors.append(tree_mask)
    if out is not None:
        if out.shape != q_shape or out.dtype is not bf16 or not out.is_contiguous():
            raise _no(what, "out must be contiguous bf16 of q's shape")
        tensors.append(out)
    need = 0
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
            raise _no(what, "workspace must be contiguous uint8")
        tensors.append(workspace)
    else:
        need = _tree_workspace(B, max_q, total, Hq, Hkv, max_seq_len, d)
    dev = _device(what, tensors, torch)

    def make():
        return (torch.empty_like(q) if out is None else out,
                seq_lens.new_empty((need,), dtype=torch.uint8) if need else workspace)

    def call(new, raw):
        o, ws = new
        mask = None if tree_mask is None else tree_mask.data_ptr()
        ws_ptr, ws_bytes = (None, 0) if ws is None else (ws.data_ptr(), ws.numel())
        if K_scales is None:
            return lib().attn_tree_paged(
                q.data_ptr(), K.data_ptr(), V.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), cu_q.data_ptr(),
                mask, o.data_ptr(), B, max_q, total, Hq, Hkv, pages, table[1], max_seq_len, d, raw, ws_ptr,
                ws_bytes)
        return lib().attn_tree_paged_e4m3(
            q.data_ptr(), K.data_ptr(), V.data_ptr(), K_scales.data_ptr(), V_scales.data_ptr(), block_table.data_ptr(),
            seq_lens.data_ptr(), cu_q.data_ptr(), mask, o.data_ptr(), B, max_q, total, Hq, Hkv, pages,
            table[1], max_seq_len, d, raw, ws_ptr, ws_bytes)

    new, st = _run(dev, stream, tensors, make, call, torch)
    if st:
        raise AttnError(st, "attn_" + what)
    return new[0]
