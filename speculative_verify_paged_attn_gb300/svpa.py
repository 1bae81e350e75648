"""ctypes binding of libsvpa.so -- argument marshalling only.

Every function here forwards to the C entry point of the same name in
``include/svpa.h``: it checks nothing the library does not check itself,
computes nothing, and passes device pointers (``tensor.data_ptr()``) plus the
current CUDA stream.  Device memory is allocated by the caller (PyTorch).

There is no CPU fallback: if the compiled library is missing, importing the
library raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsvpa.so")

SVPA_KV_BF16 = 0
SVPA_KV_FP8_E4M3 = 1
SVPA_LOGITS_FP32 = 0
SVPA_LOGITS_BF16 = 1
STATUS = {0: "SVPA_OK", 1: "SVPA_ERR_INVALID_ARG", 2: "SVPA_ERR_UNSUPPORTED", 3: "SVPA_ERR_CUDA",
          4: "SVPA_ERR_OUT_OF_BLOCKS", 5: "SVPA_ERR_BAD_BLOCK", 6: "SVPA_ERR_WORKSPACE",
          7: "SVPA_ERR_TIMEOUT"}
EXPORTS = ("svpa_attn_workspace_size", "svpa_attn_kernel", "svpa_paged_verify_attn", "svpa_spec_accept_workspace_size",
           "svpa_spec_accept", "svpa_spec_accept_tree", "svpa_block_table_commit", "svpa_check_error",
           "svpa_status_string", "svpa_version", "svpa_paged_verify_attn_noalloc", "svpa_kv_append",
           "svpa_gamma_update", "svpa_attn_launches", "svpa_spec_accept_logits",
           "svpa_spec_accept_logits_workspace_size", "svpa_wait_selftest", "svpa_spec_accept_tree_logits",
           "svpa_paged_prompt_attn_workspace_size", "svpa_paged_prompt_attn",
           "svpa_prefix_verify_attn_workspace_size", "svpa_prefix_verify_attn",
           "svpa_block_table_build_workspace_size", "svpa_block_table_build", "svpa_kv_write", "svpa_logits_process")


class SvpaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class AttnParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("split_pages", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("scale_tile", ctypes.c_int32)]


class PromptParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("total_q", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("q_stride", ctypes.c_int32)]


class LogitsParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("rows", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("max_history", ctypes.c_int32), ("logits_dtype", ctypes.c_int32)]


_BF16, _F32, _I32, _U32 = torch.bfloat16, torch.float32, torch.int32, torch.uint32

_lib = None


def load(path: str = LIB_PATH):
    """Load libsvpa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libsvpa.so not found at {path}; build it with "
                           "`python -m speculative_verify_paged_attn_gb300.build`")
    L = ctypes.CDLL(path)
    P, I, U, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    L.svpa_attn_workspace_size.argtypes = [ctypes.POINTER(AttnParams), ctypes.POINTER(U)]
    L.svpa_attn_kernel.argtypes = [ctypes.POINTER(AttnParams), ctypes.POINTER(I)]
    L.svpa_attn_launches.argtypes = [ctypes.POINTER(AttnParams), ctypes.POINTER(I)]
    L.svpa_paged_verify_attn.argtypes = [ctypes.POINTER(AttnParams)] + [P] * 11 + [U, P, P]
    L.svpa_spec_accept_workspace_size.argtypes = [I, I, ctypes.POINTER(U)]
    L.svpa_spec_accept.argtypes = [I, I, I] + [P] * 9 + [U, P, P]
    L.svpa_spec_accept_tree.argtypes = [I, I, I] + [P] * 11 + [U, P, P]
    L.svpa_spec_accept_logits.argtypes = [I, I, I, ctypes.c_float, ctypes.c_float] + [P] * 9 + [U, P, P]
    L.svpa_spec_accept_logits_workspace_size.argtypes = [I, I, I, ctypes.POINTER(U)]
    L.svpa_spec_accept_tree_logits.argtypes = [I, I, I, P, ctypes.c_float, ctypes.c_float] + [P] * 11
    L.svpa_block_table_commit.argtypes = [I] * 5 + [P] * 7 + [I, P, P, I, I, I, P, P]
    L.svpa_paged_verify_attn_noalloc.argtypes = [ctypes.POINTER(AttnParams)] + [P] * 12
    L.svpa_kv_append.argtypes = [I] * 9 + [P] * 13
    L.svpa_gamma_update.argtypes = [I, I] + [P] * 6 + [ctypes.c_float, ctypes.c_float, P, P]
    L.svpa_paged_prompt_attn_workspace_size.argtypes = [ctypes.POINTER(PromptParams), ctypes.POINTER(U)]
    L.svpa_paged_prompt_attn.argtypes = [ctypes.POINTER(PromptParams)] + [P] * 9 + [U, P, P]
    L.svpa_prefix_verify_attn_workspace_size.argtypes = [ctypes.POINTER(AttnParams), I, ctypes.POINTER(U)]
    L.svpa_prefix_verify_attn.argtypes = [ctypes.POINTER(AttnParams)] + [P] * 4 + [I] + [P] * 6 + [U, P, P]
    L.svpa_block_table_build_workspace_size.argtypes = [I, ctypes.POINTER(U)]
    L.svpa_block_table_build.argtypes = [I] * 5 + [P, P, I] + [P] * 7 + [U, P, P]
    L.svpa_kv_write.argtypes = [I] * 7 + [P, P, ctypes.c_int64, ctypes.c_int64] + [P] * 7
    L.svpa_logits_process.argtypes = [ctypes.POINTER(LogitsParams)] + [P] * 16
    L.svpa_check_error.argtypes = [P, P]
    L.svpa_wait_selftest.argtypes = [ctypes.c_uint64, P, P, P]
    L.svpa_status_string.argtypes = [I]
    L.svpa_status_string.restype = ctypes.c_char_p
    L.svpa_version.argtypes = []
    for name in EXPORTS:
        if name != "svpa_status_string":
            getattr(L, name).restype = I
    _lib = L
    return L


def _p(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _arr(t, dtype, n: int, what: str) -> Optional[int]:
    """The pointer of a contiguous array of at least n values of dtype, or of None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise SvpaError(1, f"{what}: {n} contiguous values of {dtype} expected, not {tuple(t.shape)} of {t.dtype}")
    return t.data_ptr()


try:
    # the current stream's handle without a Stream object around it (0.3 us against 3)
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:  # not part of torch's public interface
    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, what: str):
    if status != 0:
        raise SvpaError(status, what)


VARIANT_AUTO, VARIANT_MMA, VARIANT_TCGEN05 = 0, 1, 2


def attn_params(batch, n_q, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, num_blocks,
                kv_fp8=False, sm_scale=None, split_pages=0, block_size=16, variant=0,
                scale_tile=0) -> AttnParams:
    return AttnParams(batch, n_q, num_q_heads, num_kv_heads, head_dim, block_size,
                      max_blocks_per_seq, num_blocks, SVPA_KV_FP8_E4M3 if kv_fp8 else SVPA_KV_BF16,
                      1.0 / math.sqrt(head_dim) if sm_scale is None else sm_scale, split_pages,
                      variant, scale_tile)


def attn_workspace_size(params: AttnParams) -> int:
    n = ctypes.c_size_t(0)
    _check(load().svpa_attn_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "svpa_attn_workspace_size")
    return n.value


def attn_kernel(params: AttnParams) -> int:
    """The attention kernel the library runs for `params`: 1 warp-level MMA, 2 tcgen05."""
    k = ctypes.c_int32(0)
    _check(load().svpa_attn_kernel(ctypes.byref(params), ctypes.byref(k)), "svpa_attn_kernel")
    return k.value


def attn_launches(params: AttnParams) -> int:
    """Kernel launches of one svpa_paged_verify_attn call for `params` (1, or 2 with the unit ranking)."""
    n = ctypes.c_int32(0)
    _check(load().svpa_attn_launches(ctypes.byref(params), ctypes.byref(n)), "svpa_attn_launches")
    return n.value


def spec_accept_workspace_size(batch: int, vocab: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().svpa_spec_accept_workspace_size(batch, vocab, ctypes.byref(n)),
           "svpa_spec_accept_workspace_size")
    return n.value


def _mask_array(mask: Optional[Sequence[int]]):
    if mask is None:
        return None
    vals = [int(m) & ((1 << 64) - 1) for m in (mask.tolist() if hasattr(mask, "tolist") else mask)]
    return (ctypes.c_uint64 * len(vals))(*vals)


def paged_verify_attn(params: AttnParams, q, k_pool, v_pool, block_table, context_lens, out, *,
                      workspace, error_flag, k_scale=None, v_scale=None, ancestor_mask=None,
                      lse=None, stream=None, check=True) -> int:
    """svpa_paged_verify_attn.  ancestor_mask: host sequence of n_q 64-bit masks or None."""
    m = _mask_array(ancestor_mask)
    st = load().svpa_paged_verify_attn(
        ctypes.byref(params), _p(q), _p(k_pool), _p(v_pool), _p(k_scale), _p(v_scale),
        _p(block_table), _p(context_lens), None if m is None else ctypes.cast(m, ctypes.c_void_p),
        _p(out), _p(lse), _p(workspace), workspace.numel() * workspace.element_size(),
        _p(error_flag), _stream(stream))
    if check:
        _check(st, "svpa_paged_verify_attn")
    return st


def paged_verify_attn_noalloc(params: AttnParams, q, k_pool, v_pool, block_table, context_lens, out,
                              *, error_flag, k_scale=None, v_scale=None, ancestor_mask=None,
                              lse=None, stream=None, check=True) -> int:
    """svpa_paged_verify_attn_noalloc: no workspace argument; the library's own
    fixed scratch array is used (for callers that may not allocate)."""
    m = _mask_array(ancestor_mask)
    st = load().svpa_paged_verify_attn_noalloc(
        ctypes.byref(params), _p(q), _p(k_pool), _p(v_pool), _p(k_scale), _p(v_scale),
        _p(block_table), _p(context_lens), None if m is None else ctypes.cast(m, ctypes.c_void_p),
        _p(out), _p(lse), _p(error_flag), _stream(stream))
    if check:
        _check(st, "svpa_paged_verify_attn_noalloc")
    return st


def _pool_type(params, pool):
    """bf16, or for FP8 pages (which the packed attention calls refuse) the pool's own type."""
    return _BF16 if params.kv_dtype == SVPA_KV_BF16 else pool.dtype


def prompt_params(batch, total_q, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, num_blocks, *,
                  sm_scale=None, q_stride=0, block_size=16, kv_fp8=False) -> PromptParams:
    """q_stride: elements from one token of q to the next (q.stride(0)); 0 = contiguous."""
    return PromptParams(batch, total_q, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                        num_blocks, SVPA_KV_FP8_E4M3 if kv_fp8 else SVPA_KV_BF16,
                        1.0 / math.sqrt(head_dim) if sm_scale is None else sm_scale, q_stride)


def paged_prompt_attn_workspace_size(params: PromptParams) -> int:
    n = ctypes.c_size_t(0)
    _check(load().svpa_paged_prompt_attn_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "svpa_paged_prompt_attn_workspace_size")
    return n.value


def paged_prompt_attn(params: PromptParams, q, k_pool, v_pool, block_table, cu_seqlens, kv_lens, out, *,
                      workspace, error_flag, lse=None, stream=None, check=True) -> int:
    """svpa_paged_prompt_attn: causal attention of packed prompts (or chunks) over
    their pages; q [T, Hq, D], its tokens params.q_stride elements apart."""
    b, rows, d = params.batch, params.total_q * params.num_q_heads, params.head_dim
    if q.dtype is not _BF16 or q.dim() != 3 or q.shape[0] < params.total_q or \
            q.shape[1] != params.num_q_heads or q.shape[2] != d:
        raise SvpaError(1, "q: bf16 [total_q, num_q_heads, head_dim] expected")
    if _row_stride(q, "q") != (params.q_stride or params.num_q_heads * d) and q.shape[0] > 1:
        raise SvpaError(1, "q: its tokens are not q_stride elements apart")
    page, pool = params.num_blocks * params.num_kv_heads * params.block_size * d, _pool_type(params, k_pool)
    st = load().svpa_paged_prompt_attn(
        ctypes.byref(params), _p(q), _arr(k_pool, pool, page, "k_pool"), _arr(v_pool, pool, page, "v_pool"),
        _arr(block_table, _I32, b * params.max_blocks_per_seq, "block_table"),
        _arr(cu_seqlens, _I32, b + 1, "cu_seqlens"), _arr(kv_lens, _I32, b, "kv_lens"),
        _arr(out, _BF16, rows * d, "out"), _arr(lse, _F32, rows, "lse"), _p(workspace),
        workspace.numel() * workspace.element_size(), _arr(error_flag, _I32, 1, "error_flag"), _stream(stream))
    if check:
        _check(st, "svpa_paged_prompt_attn")
    return st


def prefix_verify_attn_workspace_size(params: AttnParams, prefix_len: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().svpa_prefix_verify_attn_workspace_size(ctypes.byref(params), prefix_len, ctypes.byref(n)),
           "svpa_prefix_verify_attn_workspace_size")
    return n.value


def prefix_verify_attn(params: AttnParams, q, k_pool, v_pool, prefix_blocks, block_table, context_lens, out, *,
                       workspace, error_flag, ancestor_mask=None, lse=None, stream=None, check=True) -> int:
    """svpa_prefix_verify_attn: paged_verify_attn with the attention over the
    blocks of prefix_blocks (int32, or None) formed once for all sequences."""
    m = _mask_array(ancestor_mask)
    if m is not None and len(m) < params.n_q:
        raise SvpaError(1, "svpa_prefix_verify_attn: one ancestor mask per query")
    b, d = params.batch, params.head_dim
    rows = b * params.n_q * params.num_q_heads
    page, pool = params.num_blocks * params.num_kv_heads * params.block_size * d, _pool_type(params, k_pool)
    st = load().svpa_prefix_verify_attn(
        ctypes.byref(params), _arr(q, _BF16, rows * d, "q"), _arr(k_pool, pool, page, "k_pool"),
        _arr(v_pool, pool, page, "v_pool"),
        _arr(prefix_blocks, _I32, 0, "prefix_blocks"),
        0 if prefix_blocks is None else prefix_blocks.shape[0] * params.block_size,
        _arr(block_table, _I32, b * params.max_blocks_per_seq, "block_table"),
        _arr(context_lens, _I32, b, "context_lens"),
        None if m is None else ctypes.cast(m, ctypes.c_void_p),
        _arr(out, _BF16, rows * d, "out"), _arr(lse, _F32, rows, "lse"), _p(workspace),
        workspace.numel() * workspace.element_size(), _arr(error_flag, _I32, 1, "error_flag"), _stream(stream))
    if check:
        _check(st, "svpa_prefix_verify_attn")
    return st


def spec_accept(p_probs, q_probs, draft_tokens, u_accept, u_sample, accepted_len, out_tokens, *,
                workspace, error_flag, near_boundary=None, stream=None, check=True) -> int:
    B, g1, V = p_probs.shape
    st = load().svpa_spec_accept(B, g1 - 1, V, _p(p_probs), _p(q_probs), _p(draft_tokens),
                                 _p(u_accept), _p(u_sample), _p(accepted_len), _p(out_tokens),
                                 _p(near_boundary), _p(workspace),
                                 workspace.numel() * workspace.element_size(), _p(error_flag),
                                 _stream(stream))
    if check:
        _check(st, "svpa_spec_accept")
    return st


def spec_accept_logits_workspace_size(batch: int, gamma: int, vocab: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().svpa_spec_accept_logits_workspace_size(batch, gamma, vocab, ctypes.byref(n)),
           "svpa_spec_accept_logits_workspace_size")
    return n.value


def spec_accept_logits(target_logits, draft_logits, draft_tokens, u_accept, u_sample, accepted_len, out_tokens,
                       *, workspace, error_flag, temperature=1.0, draft_temperature=None, near_boundary=None,
                       stream=None, check=True) -> int:
    """The linear sampler on P = softmax(target_logits / T), Q = softmax(draft_logits / T_draft)."""
    B, g1, V = target_logits.shape
    td = temperature if draft_temperature is None else draft_temperature
    st = load().svpa_spec_accept_logits(B, g1 - 1, V, float(temperature), float(td), _p(target_logits),
                                        _p(draft_logits), _p(draft_tokens), _p(u_accept), _p(u_sample),
                                        _p(accepted_len), _p(out_tokens), _p(near_boundary), _p(workspace),
                                        workspace.numel() * workspace.element_size(), _p(error_flag),
                                        _stream(stream))
    if check:
        _check(st, "svpa_spec_accept_logits")
    return st


def spec_accept_tree(parent: Sequence[int], p_probs, q_probs, node_tokens, u_accept, u_sample,
                     accepted_len, path_nodes, out_tokens, *, error_flag, near_boundary=None,
                     workspace=None, stream=None, check=True) -> int:
    """parent: host sequence (parent[0] = -1)."""
    par = [int(x) for x in (parent.tolist() if hasattr(parent, "tolist") else parent)]
    arr = (ctypes.c_int32 * len(par))(*par)
    B, n, V = p_probs.shape
    st = load().svpa_spec_accept_tree(B, n, V, ctypes.cast(arr, ctypes.c_void_p), _p(p_probs),
                                      _p(q_probs), _p(node_tokens), _p(u_accept), _p(u_sample),
                                      _p(accepted_len), _p(path_nodes), _p(out_tokens),
                                      _p(near_boundary), _p(workspace),
                                      0 if workspace is None else workspace.numel() * workspace.element_size(),
                                      _p(error_flag), _stream(stream))
    if check:
        _check(st, "svpa_spec_accept_tree")
    return st


def spec_accept_tree_logits(parent: Sequence[int], target_logits, draft_logits, node_tokens, u_accept, u_sample,
                            accepted_len, path_nodes, out_tokens, *, error_flag, temperature=1.0,
                            draft_temperature=None, near_boundary=None, stream=None, check=True) -> int:
    """The draft-tree sampler on P = softmax(target_logits / T) at every node and
    Q = softmax(draft_logits / T_draft) at every internal node; parent: host
    sequence (parent[0] = -1)."""
    par = [int(x) for x in (parent.tolist() if hasattr(parent, "tolist") else parent)]
    arr = (ctypes.c_int32 * len(par))(*par)
    B, n, V = target_logits.shape
    td = temperature if draft_temperature is None else draft_temperature
    st = load().svpa_spec_accept_tree_logits(B, n, V, ctypes.cast(arr, ctypes.c_void_p), float(temperature),
                                             float(td), _p(target_logits), _p(draft_logits), _p(node_tokens),
                                             _p(u_accept), _p(u_sample), _p(accepted_len), _p(path_nodes),
                                             _p(out_tokens), _p(near_boundary), _p(error_flag), _stream(stream))
    if check:
        _check(st, "svpa_spec_accept_tree_logits")
    return st


def block_table_commit(n_q, block_table, context_lens, accepted_len, refcount, free_stack, free_top,
                       *, error_flag, path_nodes=None, k_pool=None, v_pool=None, num_kv_heads=0,
                       head_dim=0, kv_fp8=False, stream=None, check=True) -> int:
    B, max_blocks = block_table.shape
    st = load().svpa_block_table_commit(
        B, n_q, 16, max_blocks, refcount.shape[0], _p(block_table), _p(context_lens),
        _p(accepted_len), _p(refcount), _p(free_stack), _p(free_top), _p(path_nodes),
        0 if path_nodes is None else path_nodes.shape[1], _p(k_pool), _p(v_pool), num_kv_heads,
        head_dim, SVPA_KV_FP8_E4M3 if kv_fp8 else SVPA_KV_BF16, _p(error_flag), _stream(stream))
    if check:
        _check(st, "svpa_block_table_commit")
    return st


def kv_append(new_k, new_v, block_table, context_lens, refcount, free_stack, free_top, k_pool, v_pool,
              *, error_flag, k_scale=None, v_scale=None, scale_tile=0, stream=None, check=True) -> int:
    """svpa_kv_append: write new_k/new_v [B, n_new, Hkv, D] (bf16) at positions
    context_lens[b] .. + n_new - 1, allocating and cloning pages as needed; the
    pools are bf16 or float8_e4m3fn/uint8 [num_blocks, Hkv, 16, D]."""
    B, n_new, Hkv, D = new_k.shape
    fp8 = k_pool.element_size() == 1
    st = load().svpa_kv_append(
        B, n_new, Hkv, D, 16, block_table.shape[1], k_pool.shape[0],
        SVPA_KV_FP8_E4M3 if fp8 else SVPA_KV_BF16, scale_tile, _p(new_k), _p(new_v), _p(block_table),
        _p(context_lens), _p(refcount), _p(free_stack), _p(free_top), _p(k_pool), _p(v_pool),
        _p(k_scale), _p(v_scale), _p(error_flag), _stream(stream))
    if check:
        _check(st, "svpa_kv_append")
    return st


def block_table_build_workspace_size(batch: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().svpa_block_table_build_workspace_size(batch, ctypes.byref(n)),
           "svpa_block_table_build_workspace_size")
    return n.value


def block_table_build(seq_lens, block_table, cu_seqlens, slot_map, refcount, free_stack, free_top, *, workspace,
                      error_flag, prefix_blocks=None, stream=None, check=True) -> int:
    """svpa_block_table_build: tables [B, max_blocks], packed offsets [B + 1] and
    slots of the new tokens of requests with seq_lens [B] tokens, the first of
    them in the shared blocks of prefix_blocks (int32, or None)."""
    B, max_blocks = block_table.shape
    blocks = refcount.shape[0]
    st = load().svpa_block_table_build(
        B, 16, max_blocks, blocks, slot_map.shape[0], _arr(seq_lens, _I32, B, "seq_lens"),
        _arr(prefix_blocks, _I32, 0, "prefix_blocks"), 0 if prefix_blocks is None else prefix_blocks.shape[0] * 16,
        _arr(block_table, _I32, 0, "block_table"), _arr(cu_seqlens, _I32, B + 1, "cu_seqlens"),
        _arr(slot_map, _I32, 0, "slot_map"), _arr(refcount, _I32, 0, "refcount"),
        _arr(free_stack, _I32, blocks, "free_stack"), _arr(free_top, _I32, 1, "free_top"), _p(workspace),
        workspace.numel() * workspace.element_size(), _arr(error_flag, _I32, 1, "error_flag"), _stream(stream))
    if check:
        _check(st, "svpa_block_table_build")
    return st


def _row_stride(t, what: str) -> int:
    """Elements from one token of t [T, H, D] to the next; the tokens' own values must be contiguous."""
    if t.shape[0] > 0 and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2])):
        raise SvpaError(1, f"{what}: the values of a token are not contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def kv_write(new_k, new_v, slot_map, k_pool, v_pool, *, error_flag, k_scale=None, v_scale=None, scale_tile=0,
             stream=None, check=True) -> int:
    """svpa_kv_write: new_k/new_v [T, Hkv, D] (bf16; slices of a fused projection
    along the heads are taken as they are) to the slots of slot_map [T]; the
    pools are bf16 or float8_e4m3fn/uint8 [num_blocks, Hkv, 16, D]."""
    T, Hkv, D = new_k.shape
    blocks, fp8 = k_pool.shape[0], k_pool.element_size() == 1
    if new_k.dtype is not _BF16 or new_v.dtype is not _BF16 or new_v.shape != new_k.shape:
        raise SvpaError(1, "new_k, new_v: bf16 rows of one shape expected")
    page, scales = blocks * Hkv * 16 * D, blocks * Hkv * 16 * (D // 64) if fp8 else 0
    pool = k_pool.dtype if fp8 else _BF16
    st = load().svpa_kv_write(
        T, Hkv, D, 16, blocks, SVPA_KV_FP8_E4M3 if fp8 else SVPA_KV_BF16, scale_tile, _p(new_k), _p(new_v),
        _row_stride(new_k, "new_k"), _row_stride(new_v, "new_v"), _arr(slot_map, _I32, T, "slot_map"),
        _arr(k_pool, pool, page, "k_pool"), _arr(v_pool, pool, page, "v_pool"),
        _arr(k_scale, _F32, scales, "k_scale"), _arr(v_scale, _F32, scales, "v_scale"),
        _arr(error_flag, _I32, 1, "error_flag"), _stream(stream))
    if check:
        _check(st, "svpa_kv_write")
    return st


def logits_process(logits, out, *, error_flag, history=None, prompt_lens=None, hist_lens=None, draft_tokens=None,
                   parent: Optional[Sequence[int]] = None, repetition=None, presence=None, frequency=None,
                   bias_offsets=None, bias_tokens=None, bias_values=None, mask=None, stream=None, check=True) -> int:
    """svpa_logits_process: penalties, biases and grammar masks on logits [B,
    rows, V] (fp32 or bf16, contiguous) into out (fp32, may be logits); parent:
    host sequence of the draft tree (parent[0] = -1) or None for a chain."""
    B, rows, V = logits.shape
    bf16, hist = logits.dtype is _BF16, 0 if history is None else history.shape[1]
    p = LogitsParams(B, rows, V, hist, SVPA_LOGITS_BF16 if bf16 else SVPA_LOGITS_FP32)
    arr = None
    if parent is not None:
        par = [int(x) for x in (parent.tolist() if hasattr(parent, "tolist") else parent)]
        if len(par) != rows:
            raise SvpaError(1, "svpa_logits_process: one parent per row")
        arr = (ctypes.c_int32 * rows)(*par)
    # (the arrays of one value a sequence are taken as they are)
    st = load().svpa_logits_process(
        ctypes.byref(p), _arr(logits, _BF16 if bf16 else _F32, 0, "logits"),
        _arr(history, _I32, B * hist, "history"), _p(prompt_lens), _p(hist_lens),
        _arr(draft_tokens, _I32, B * (rows - 1 if arr is None else rows), "draft_tokens"),
        None if arr is None else ctypes.cast(arr, ctypes.c_void_p), _p(repetition), _p(presence), _p(frequency),
        _p(bias_offsets), _p(bias_tokens), _p(bias_values),
        None if mask is None else _arr(mask, _U32 if mask.dtype is _U32 else _I32, B * rows * ((V + 31) // 32), "mask"),
        _arr(out, _F32, B * rows * V, "out"), _p(error_flag), _stream(stream))
    if check:
        _check(st, "svpa_logits_process")
    return st


def gamma_update(gamma, accepted_len, batch_state, batch_gamma, telemetry, *, error_flag, seq_state=None,
                 seq_gamma=None, decay=0.9, draft_cost_ratio=0.0, stream=None, check=True) -> int:
    """svpa_gamma_update: acceptance moving averages (per sequence when
    seq_state [B, 2] is given, and for the batch in batch_state [2]) and the
    draft length of the next step (seq_gamma [B], batch_gamma [1])."""
    st = load().svpa_gamma_update(
        accepted_len.shape[0], gamma, _p(accepted_len), _p(seq_state), _p(seq_gamma), _p(batch_state),
        _p(batch_gamma), _p(telemetry), float(decay), float(draft_cost_ratio), _p(error_flag), _stream(stream))
    if check:
        _check(st, "svpa_gamma_update")
    return st


def check_error(error_flag, stream=None) -> int:
    """svpa_check_error: synchronise the stream and map the device error word."""
    return load().svpa_check_error(_p(error_flag), _stream(stream))


def wait_selftest(limit_ns: int, error_flag, reached, stream=None, check=True) -> int:
    """svpa_wait_selftest: one kernel waits, bounded by limit_ns, on an
    mbarrier no thread arrives on (the wait-limit path of every kernel)."""
    st = load().svpa_wait_selftest(int(limit_ns), _p(error_flag), _p(reached), _stream(stream))
    if check:
        _check(st, "svpa_wait_selftest")
    return st

def status_string(status: int) -> str:
    return load().svpa_status_string(status).decode()


def version() -> int:
    return load().svpa_version()
