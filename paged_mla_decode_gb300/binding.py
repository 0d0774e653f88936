"""Thin ctypes binding of libmla.so (argument marshalling only).

Each function has the name of the C entry point it calls and takes PyTorch
tensors, from which it passes device pointers, sizes and the current CUDA
stream. All computation happens in the library's CUDA kernels; there is no
fallback: if ``libmla.so`` is missing the first call raises.
"""

from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB_PATH

MLA_OK = 0
MLA_ERR_INVALID_ARG = 1
MLA_ERR_UNSUPPORTED = 2
MLA_ERR_WORKSPACE = 3
MLA_ERR_CUDA = 4

MLA_KV_E4M3 = 0
MLA_KV_BF16 = 1
MLA_KV_E2M1 = 2

MLA_E2M1_PAGE_BYTES = 19008

MLA_DEVICE_ERR_BAD_PAGE = 0x1
MLA_DEVICE_ERR_BAD_LENGTH = 0x2
MLA_DEVICE_ERR_TIMEOUT = 0x4

MLA_KV_CHECK_TAG_MISMATCH = 0x1
MLA_KV_CHECK_PAGE_RANGE = 0x2
MLA_KV_CHECK_BAD_LENGTH = 0x4

MLA_KV_ALLOC_BAD_LENGTH = 0x1
MLA_KV_ALLOC_TABLE_FULL = 0x2
MLA_KV_ALLOC_SLOTS_FULL = 0x4
MLA_KV_ALLOC_NO_PAGES = 0x8

MLA_PROB_F32 = 0
MLA_PROB_BF16 = 1
MLA_MAX_DRAFTS = 31
MLA_MAX_TREE_NODES = 64
MLA_MAX_PROBS_VOCAB = 393216
MLA_MAX_BIASES = 1024

EXPORTED = ("mla_abi_version", "mla_status_string", "mla_kv_append",
            "mla_decode_workspace_size", "mla_decode", "mla_decode_f16_operands",
            "mla_decode_grouped_workspace_size", "mla_decode_grouped",
            "mla_decode_combine", "mla_kv_check", "mla_decode_static_scratch",
            "mla_kv_gather", "mla_kv_alloc", "mla_verify_drafts",
            "mla_decode_tree_workspace_size", "mla_decode_tree", "mla_logits_to_probs",
            "mla_verify_tree", "mla_kv_compact")

_lib = None


class MlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmla.so once and declare the argument types of every entry point."""
    global _lib
    if _lib is None:
        _lib = open_library(path)
    return _lib


def open_library(path: str) -> ctypes.CDLL:
    """Open a build of the library at ``path`` (not cached) with its argument types."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run paged_mla_decode_gb300.build.build() "
                           "(or __graft_entry__.build()) first")
    lib = ctypes.CDLL(path)
    c = ctypes
    lib.mla_abi_version.restype = c.c_int
    lib.mla_abi_version.argtypes = []
    lib.mla_status_string.restype = c.c_char_p
    lib.mla_status_string.argtypes = [c.c_int]
    lib.mla_kv_append.restype = c.c_int
    lib.mla_kv_append.argtypes = [c.c_void_p, c.c_void_p, c.c_void_p, c.c_int64, c.c_void_p,
                                  c.c_int64, c.c_int, c.c_int, c.c_float, c.c_void_p]
    lib.mla_decode_workspace_size.restype = c.c_size_t
    lib.mla_decode_workspace_size.argtypes = [c.c_int, c.c_int, c.c_int, c.c_int]
    lib.mla_decode.restype = c.c_int
    lib.mla_decode.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_int, c.c_int, c.c_void_p,
                               c.c_int, c.c_void_p, c.c_int, c.c_int, c.c_int, c.c_float,
                               c.c_float, c.c_int, c.c_void_p, c.c_size_t, c.c_void_p,
                               c.c_void_p, c.c_void_p]
    lib.mla_decode_f16_operands.restype = c.c_int
    lib.mla_decode_f16_operands.argtypes = lib.mla_decode.argtypes
    lib.mla_decode_grouped_workspace_size.restype = c.c_size_t
    lib.mla_decode_grouped_workspace_size.argtypes = [c.c_int, c.c_int, c.c_int, c.c_int]
    lib.mla_decode_grouped.restype = c.c_int
    lib.mla_decode_grouped.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_int, c.c_int,
                                       c.c_void_p, c.c_int, c.c_void_p, c.c_int, c.c_int,
                                       c.c_int, c.c_int, c.c_void_p, c.c_float, c.c_float,
                                       c.c_int, c.c_void_p, c.c_size_t, c.c_void_p, c.c_void_p,
                                       c.c_void_p]
    lib.mla_decode_tree_workspace_size.restype = c.c_size_t
    lib.mla_decode_tree_workspace_size.argtypes = [c.c_int, c.c_int, c.c_int, c.c_int]
    lib.mla_decode_tree.restype = c.c_int
    lib.mla_decode_tree.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_int, c.c_int, c.c_void_p,
                                    c.c_int, c.c_void_p, c.c_void_p, c.c_void_p, c.c_int, c.c_int,
                                    c.c_int, c.c_float, c.c_float, c.c_int, c.c_void_p, c.c_size_t,
                                    c.c_void_p, c.c_void_p, c.c_void_p]
    lib.mla_decode_combine.restype = c.c_int
    lib.mla_decode_combine.argtypes = [c.c_void_p, c.c_void_p, c.c_int, c.c_int64, c.c_void_p,
                                       c.c_void_p, c.c_void_p]
    lib.mla_kv_check.restype = c.c_int
    lib.mla_kv_check.argtypes = [c.c_void_p, c.c_int64, c.c_void_p, c.c_void_p, c.c_int,
                                 c.c_void_p, c.c_int, c.c_int, c.c_void_p, c.c_void_p,
                                 c.c_void_p]
    lib.mla_decode_static_scratch.restype = c.c_int
    lib.mla_decode_static_scratch.argtypes = [
        c.c_void_p, c.c_void_p, c.c_int64, c.c_int, c.c_int, c.c_void_p, c.c_int, c.c_void_p,
        c.c_int, c.c_int, c.c_int, c.c_float, c.c_float, c.c_int, c.c_void_p, c.c_void_p,
        c.c_void_p, c.c_void_p]
    lib.mla_kv_gather.restype = c.c_int
    lib.mla_kv_gather.argtypes = [c.c_void_p, c.c_int64, c.c_int, c.c_int, c.c_float, c.c_void_p,
                                  c.c_int, c.c_void_p, c.c_void_p, c.c_int, c.c_int64, c.c_void_p,
                                  c.c_void_p, c.c_void_p]
    lib.mla_kv_alloc.restype = c.c_int
    lib.mla_kv_alloc.argtypes = [c.c_void_p, c.c_void_p, c.c_int, c.c_int, c.c_void_p, c.c_void_p,
                                 c.c_void_p, c.c_int64, c.c_int64, c.c_void_p, c.c_int, c.c_void_p,
                                 c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p,
                                 c.c_void_p, c.c_int64, c.c_void_p, c.c_void_p]
    lib.mla_verify_drafts.restype = c.c_int
    lib.mla_verify_drafts.argtypes = [c.c_void_p, c.c_int64, c.c_void_p, c.c_int64, c.c_int,
                                      c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p, c.c_int,
                                      c.c_int, c.c_int, c.c_void_p, c.c_void_p, c.c_void_p,
                                      c.c_void_p]
    lib.mla_logits_to_probs.restype = c.c_int
    lib.mla_logits_to_probs.argtypes = [
        c.c_void_p, c.c_int64, c.c_int, c.c_void_p, c.c_int64, c.c_int, c.c_int, c.c_int, c.c_int,
        c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p,
        c.c_void_p, c.c_void_p, c.c_void_p, c.c_int, c.c_void_p, c.c_void_p]
    lib.mla_verify_tree.restype = c.c_int
    lib.mla_verify_tree.argtypes = [
        c.c_void_p, c.c_int64, c.c_void_p, c.c_int64, c.c_int, c.c_void_p, c.c_void_p, c.c_void_p,
        c.c_void_p, c.c_void_p, c.c_int, c.c_int, c.c_int, c.c_void_p, c.c_void_p, c.c_void_p,
        c.c_void_p, c.c_void_p, c.c_void_p]
    lib.mla_kv_compact.restype = c.c_int
    lib.mla_kv_compact.argtypes = [
        c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_int, c.c_int, c.c_void_p, c.c_int, c.c_void_p,
        c.c_void_p, c.c_void_p, c.c_int, c.c_int, c.c_void_p]
    return lib


def status_string(status: int) -> str:
    return load_library().mla_status_string(int(status)).decode()


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream, device: int | None = None) -> int:
    """The stream's handle; the current stream of the current device (`device`, if it is known to
    be) by default.

    (Read without a Stream object, which costs as much host time as a kernel launch.)
    """
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device)
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != MLA_OK:
        raise MlaError(status, where)


def _refuse(what: str):
    """An argument that the library cannot check. (Not an assert statement: python -O drops those,
    and the pointer would go to a kernel.)"""
    raise AssertionError(what)


def kv_dtype_code(kv_pages: torch.Tensor) -> int:
    """The cache's element type, from its tensor (and a check of its shape).

    uint8 ``[num_pages, 64, 576]`` holds e4m3 codes, bfloat16 of that shape bf16
    values, uint8 ``[num_pages, 19008]`` e2m1 pages.
    """
    if not kv_pages.is_contiguous():
        _refuse("kv_pages is not contiguous")
    if kv_pages.dtype == torch.uint8 and kv_pages.dim() == 2:
        if kv_pages.shape[1] != MLA_E2M1_PAGE_BYTES:
            _refuse("kv_pages of an e2m1 cache are [num_pages, 19008]")
        return MLA_KV_E2M1
    if kv_pages.dim() != 3 or kv_pages.shape[2] != 576:
        _refuse("kv_pages are [num_pages, 64, 576]")
    if kv_pages.dtype == torch.uint8:
        return MLA_KV_E4M3
    if kv_pages.dtype == torch.bfloat16:
        return MLA_KV_BF16
    raise TypeError("kv_pages must be uint8 (e4m3 codes or e2m1 pages) or bfloat16")


def _page_size(kv_pages: torch.Tensor) -> int:
    """Tokens per page: the second dimension, 64 by definition of an e2m1 page."""
    return 64 if kv_pages.dim() == 2 else int(kv_pages.shape[1])


_I32, _U32 = torch.int32, torch.uint32


def _int32(device: int, *tensors) -> None:
    """Each tensor is a contiguous int32 (for tags and status words also uint32) one on `device`."""
    for t in tensors:
        if t.dtype is not _I32 and t.dtype is not _U32:
            _refuse("an index tensor is not int32")
        if not t.is_contiguous() or t.get_device() != device:
            _refuse("an index tensor is not contiguous, or on another device")


def _device_of(t: torch.Tensor) -> int:
    """The tensor's CUDA device, which must be the current one (the library launches there)."""
    device = t.get_device()
    if not t.is_cuda or device != torch.cuda.current_device():
        _refuse("a tensor is not on the current CUDA device")
    return device


def _same_device(device: int, *tensors) -> None:
    """Each tensor is contiguous and on `device`: its pointer is all the library gets."""
    for t in tensors:
        if not t.is_contiguous() or t.get_device() != device:
            _refuse("a tensor is not contiguous, or on another device")


def _entries(latent: torch.Tensor, rope: torch.Tensor, rows: int) -> None:
    if latent.dtype != torch.bfloat16 or latent.shape != (rows, 512):
        _refuse("latent is bfloat16 [tokens, 512]")
    if rope.dtype != torch.bfloat16 or rope.shape != (rows, 64):
        _refuse("rope is bfloat16 [tokens, 64]")


def _decode_shape(q, block_table, seq_lens, out, lse):
    """Batch, queries and heads of a decode, whose types and shapes fit."""
    if q.dtype != torch.bfloat16 or q.dim() != 4 or q.shape[3] != 576:
        _refuse("q is bfloat16 [batch, queries, heads, 576]")
    batch, nq, heads, _ = q.shape
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != batch:
        _refuse("block_table is int32 [batch, max_pages]")
    if seq_lens.dtype != torch.int32 or seq_lens.numel() != batch:
        _refuse("seq_lens is int32 [batch]")
    if out.dtype != torch.bfloat16 or out.shape != (batch, nq, heads, 512):
        _refuse("out is bfloat16 [batch, queries, heads, 512]")
    if lse.dtype != torch.float32 or lse.shape != (batch, nq, heads):
        _refuse("lse is float32 [batch, queries, heads]")
    return batch, nq, heads


def mla_kv_append(latent: torch.Tensor, rope: torch.Tensor, slot_mapping: torch.Tensor,
                  kv_pages: torch.Tensor, kv_scale: float, stream=None) -> None:
    """Write tokens' 512 latent + 64 rope elements into their cache slots."""
    num_tokens = int(slot_mapping.numel())
    if slot_mapping.dtype != torch.int32:
        _refuse("slot_mapping is int32")
    _entries(latent, rope, num_tokens)
    dtype = kv_dtype_code(kv_pages)
    _same_device(_device_of(kv_pages), latent, rope, slot_mapping)
    st = load_library().mla_kv_append(_ptr(latent), _ptr(rope), _ptr(slot_mapping), num_tokens,
                                      _ptr(kv_pages), int(kv_pages.shape[0]),
                                      _page_size(kv_pages), dtype,
                                      float(kv_scale), _stream(stream))
    _check(st, "mla_kv_append")


def mla_decode_workspace_size(batch: int, num_queries: int, num_heads: int,
                              num_ctas: int = 0) -> int:
    return int(load_library().mla_decode_workspace_size(batch, num_queries, num_heads, num_ctas))


def mla_decode(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
               seq_lens: torch.Tensor, sm_scale: float, kv_scale: float, out: torch.Tensor,
               lse: torch.Tensor, workspace: torch.Tensor, num_ctas: int = 0,
               stream=None, f16_operands: bool = False) -> None:
    """Split-KV paged MLA decode (combine included) into ``out`` and ``lse``.

    ``kv_pages`` as in :func:`kv_dtype_code` (e4m3, bf16 or e2m1 pages).
    ``f16_operands`` calls mla_decode_f16_operands (the e4m3 cache widened to f16
    operands) instead of mla_decode."""
    batch, nq, heads = _decode_shape(q, block_table, seq_lens, out, lse)
    dtype = kv_dtype_code(kv_pages)
    _same_device(_device_of(kv_pages), q, block_table, seq_lens, out, lse, workspace)
    lib = load_library()
    fn = lib.mla_decode_f16_operands if f16_operands else lib.mla_decode
    st = fn(
        _ptr(q), _ptr(kv_pages), int(kv_pages.shape[0]), _page_size(kv_pages),
        dtype, _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
        batch, nq, heads, float(sm_scale), float(kv_scale), int(num_ctas), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _ptr(out), _ptr(lse),
        _stream(stream))
    _check(st, "mla_decode_f16_operands" if f16_operands else "mla_decode")


def mla_decode_grouped_workspace_size(batch: int, num_queries: int, num_heads: int,
                                      num_ctas: int = 0) -> int:
    return int(load_library().mla_decode_grouped_workspace_size(batch, num_queries, num_heads,
                                                                num_ctas))


def mla_decode_grouped(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                       seq_lens: torch.Tensor, forks: int, prefix_pages: torch.Tensor,
                       sm_scale: float, kv_scale: float, out: torch.Tensor, lse: torch.Tensor,
                       workspace: torch.Tensor, num_ctas: int = 0, stream=None) -> None:
    """mla_decode for groups of ``forks`` requests sharing ``prefix_pages[g]`` pages."""
    batch, nq, heads = _decode_shape(q, block_table, seq_lens, out, lse)
    if prefix_pages.dtype != torch.int32 or prefix_pages.numel() * max(forks, 1) < batch:
        _refuse("prefix_pages is int32 [batch / forks]")
    dtype = kv_dtype_code(kv_pages)
    _same_device(_device_of(kv_pages), q, block_table, seq_lens, prefix_pages, out, lse, workspace)
    st = load_library().mla_decode_grouped(
        _ptr(q), _ptr(kv_pages), int(kv_pages.shape[0]), _page_size(kv_pages),
        dtype, _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
        batch, nq, heads, int(forks), _ptr(prefix_pages), float(sm_scale), float(kv_scale),
        int(num_ctas), _ptr(workspace), int(workspace.numel() * workspace.element_size()),
        _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "mla_decode_grouped")


def mla_decode_tree_workspace_size(batch: int, max_nodes: int, num_heads: int,
                                   num_ctas: int = 0) -> int:
    return int(load_library().mla_decode_tree_workspace_size(batch, max_nodes, num_heads, num_ctas))


def _tree_masks(device: int, tree_mask: torch.Tensor, batch: int, nodes: int) -> None:
    """Node masks are contiguous 64-bit words ``[batch, nodes]`` on `device`."""
    if tree_mask.dtype not in (torch.int64, torch.uint64) or tree_mask.shape != (batch, nodes):
        _refuse("tree_mask is int64 or uint64 [batch, nodes]")
    _same_device(device, tree_mask)


def mla_decode_tree(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                    seq_lens: torch.Tensor, tree_mask: torch.Tensor, sm_scale: float,
                    kv_scale: float, out: torch.Tensor, lse: torch.Tensor,
                    workspace: torch.Tensor, num_nodes: torch.Tensor | None = None,
                    num_ctas: int = 0, stream=None) -> None:
    """Attention of a tree of drafted tokens, the last ``num_nodes[b]`` cached tokens of request b.

    ``q`` is ``[batch, max_nodes, heads, 576]``, ``tree_mask`` 64-bit words ``[batch,
    max_nodes]`` (int64 or uint64; bit i of word j: node j sees node i, for a tree its
    ancestors and itself); without ``num_nodes`` every request has ``max_nodes``. Rows of
    nodes that a request does not have get out = 0, lse = -inf. ``kv_pages`` as in
    :func:`kv_dtype_code`; the workspace's size is :func:`mla_decode_tree_workspace_size`.
    """
    batch, nodes, heads = _decode_shape(q, block_table, seq_lens, out, lse)
    dtype = kv_dtype_code(kv_pages)
    device = _device_of(kv_pages)
    _tree_masks(device, tree_mask, batch, nodes)
    _same_device(device, q, block_table, seq_lens, out, lse, workspace)
    if num_nodes is not None:
        _int32(device, num_nodes)
        if num_nodes.numel() != batch:
            _refuse("num_nodes is [batch]")
    st = load_library().mla_decode_tree(
        q.data_ptr(), kv_pages.data_ptr(), kv_pages.shape[0], _page_size(kv_pages), dtype,
        block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), tree_mask.data_ptr(),
        _ptr(num_nodes), batch, nodes, heads, sm_scale, kv_scale, num_ctas, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), out.data_ptr(), lse.data_ptr(),
        _stream(stream, device))
    _check(st, "mla_decode_tree")


def mla_decode_combine(part_out: torch.Tensor, part_lse: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, stream=None) -> None:
    """Merge ``part_out [S, R, 512]`` / ``part_lse [S, R]`` into ``out [R, 512]`` / ``lse [R]``."""
    if part_out.dtype != torch.float32 or part_lse.dtype != torch.float32:
        _refuse("part_out and part_lse are float32 [parts, rows, 512] and [parts, rows]")
    num_parts, rows = int(part_lse.shape[0]), int(part_lse.shape[1])
    if part_out.shape != (num_parts, rows, 512):
        _refuse("part_out is [parts, rows, 512]")
    if out.dtype != torch.bfloat16 or out.numel() != rows * 512:
        _refuse("out is bfloat16 [rows, 512]")
    if lse.dtype != torch.float32 or lse.numel() != rows:
        _refuse("lse is float32 [rows]")
    _same_device(_device_of(out), part_out, part_lse, out, lse)
    st = load_library().mla_decode_combine(_ptr(part_out), _ptr(part_lse), num_parts, rows,
                                           _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "mla_decode_combine")


def mla_kv_check(page_tags: torch.Tensor, block_table: torch.Tensor,
                 expected_tags: torch.Tensor, seq_lens: torch.Tensor,
                 request_status: torch.Tensor, checked_seq_lens: torch.Tensor,
                 stream=None) -> None:
    """Compare each request's expected page tags with the pages' current tags.

    ``page_tags [num_pages]`` and ``expected_tags [batch, max_pages]`` hold 32-bit
    tags (int32 or uint32 tensors; compared as unsigned), ``block_table`` and
    ``seq_lens`` are the decode call's. Writes ``request_status [batch]``
    (MLA_KV_CHECK_* bits, int32) and ``checked_seq_lens [batch]`` (the lengths,
    -1 for every request that failed), to be passed to mla_decode as seq_lens.
    """
    tag_types = (_I32, _U32)
    if page_tags.dtype not in tag_types or page_tags.dim() != 1:
        _refuse("page_tags is int32 or uint32 [num_pages]")
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        _refuse("block_table is int32 [batch, max_pages]")
    batch, max_pages = int(block_table.shape[0]), int(block_table.shape[1])
    if expected_tags.dtype not in tag_types or expected_tags.shape != (batch, max_pages):
        _refuse("expected_tags is int32 or uint32 [batch, max_pages]")
    if seq_lens.dtype != torch.int32 or seq_lens.numel() != batch:
        _refuse("seq_lens is int32 [batch]")
    if request_status.dtype not in tag_types or request_status.numel() != batch:
        _refuse("request_status is int32 or uint32 [batch]")
    if checked_seq_lens.dtype != torch.int32 or checked_seq_lens.numel() != batch:
        _refuse("checked_seq_lens is int32 [batch]")
    _same_device(_device_of(block_table), page_tags, block_table, expected_tags, seq_lens,
                 request_status, checked_seq_lens)
    st = load_library().mla_kv_check(_ptr(page_tags), int(page_tags.numel()), _ptr(block_table),
                                     _ptr(expected_tags), max_pages, _ptr(seq_lens), batch, 64,
                                     _ptr(request_status), _ptr(checked_seq_lens),
                                     _stream(stream))
    _check(st, "mla_kv_check")


def mla_kv_gather(kv_pages: torch.Tensor, kv_scale: float, block_table: torch.Tensor,
                  cu_tokens: torch.Tensor, latent: torch.Tensor, rope: torch.Tensor,
                  starts: torch.Tensor | None = None, stream=None) -> None:
    """Read cached entries back as bfloat16 rows ``latent [n, 512]`` and ``rope [n, 64]``.

    Rows ``cu_tokens[b] .. cu_tokens[b + 1] - 1`` receive tokens ``starts[b]``
    (0 without ``starts``) and on of request b, through ``block_table [batch,
    max_pages]``. Tokens in no page of the cache give zero rows; rows from
    ``cu_tokens[batch]`` on are left as they were. ``kv_pages`` as in
    :func:`kv_dtype_code`.
    """
    dtype, device = kv_dtype_code(kv_pages), _device_of(kv_pages)
    if block_table.dim() != 2:
        _refuse("block_table is [batch, max_pages]")
    batch, max_pages = block_table.shape
    rows = latent.shape[0]
    _int32(device, block_table, cu_tokens)
    if cu_tokens.dim() != 1 or cu_tokens.shape[0] != batch + 1:
        _refuse("cu_tokens is [batch + 1]")
    if starts is not None:
        _int32(device, starts)
        if starts.numel() != batch:
            _refuse("starts is [batch]")
    _entries(latent, rope, rows)
    _same_device(device, latent, rope)
    st = load_library().mla_kv_gather(kv_pages.data_ptr(), kv_pages.shape[0],
                                      _page_size(kv_pages), dtype, kv_scale,
                                      block_table.data_ptr(), max_pages, _ptr(starts),
                                      cu_tokens.data_ptr(), batch, rows, latent.data_ptr(),
                                      rope.data_ptr(), _stream(stream))
    _check(st, "mla_kv_gather")


def mla_kv_alloc(seq_lens: torch.Tensor, new_tokens: torch.Tensor, pages_held: torch.Tensor,
                 free_pages: torch.Tensor, free_count: torch.Tensor, num_pages: int,
                 block_table: torch.Tensor, seq_lens_out: torch.Tensor,
                 pages_held_out: torch.Tensor, free_count_out: torch.Tensor,
                 cu_tokens: torch.Tensor, slot_mapping: torch.Tensor,
                 request_status: torch.Tensor, page_tags: torch.Tensor | None = None,
                 expected_tags: torch.Tensor | None = None, stream=None) -> None:
    """Extend each request by ``new_tokens[b]`` tokens: pages, block-table rows, tags, slots.

    Takes the pages it needs off the end of ``free_pages[:free_count]``, appends
    them to ``block_table`` rows (``pages_held[b]`` entries in use), raises their
    ``page_tags`` and records the new tags in ``expected_tags`` (both or neither),
    and writes ``slot_mapping`` (the new tokens' slots, request by request, -1
    behind the last), ``cu_tokens [batch + 1]`` (first row of each request),
    ``seq_lens_out``, ``pages_held_out`` and ``free_count_out`` (each may be its
    input) and ``request_status`` (MLA_KV_ALLOC_* bits; a refused request gets
    length -1 and slots -1).
    """
    device = _device_of(block_table)
    if block_table.dim() != 2:
        _refuse("block_table is [batch, max_pages]")
    batch, max_pages = block_table.shape
    _int32(device, seq_lens, new_tokens, pages_held, free_pages, free_count, block_table,
           seq_lens_out, pages_held_out, free_count_out, cu_tokens, slot_mapping, request_status)
    if (seq_lens.numel() != batch or new_tokens.numel() != batch or pages_held.numel() != batch
            or pages_held_out.numel() != batch or seq_lens_out.numel() != batch
            or request_status.numel() != batch):
        _refuse("lengths, pages held and status words are [batch]")
    if free_count.numel() != 1 or free_count_out.numel() != 1 or cu_tokens.numel() != batch + 1:
        _refuse("free_count and free_count_out have one element, cu_tokens batch + 1")
    if (page_tags is None) != (expected_tags is None):
        _refuse("page_tags and expected_tags are given together")
    if page_tags is not None:
        _int32(device, page_tags, expected_tags)
        if page_tags.numel() != num_pages or expected_tags.shape != block_table.shape:
            _refuse("page_tags is [num_pages], expected_tags [batch, max_pages]")
    st = load_library().mla_kv_alloc(
        seq_lens.data_ptr(), new_tokens.data_ptr(), batch, 64, pages_held.data_ptr(),
        free_pages.data_ptr(), free_count.data_ptr(), free_pages.numel(), num_pages,
        block_table.data_ptr(), max_pages, _ptr(page_tags), _ptr(expected_tags),
        seq_lens_out.data_ptr(), pages_held_out.data_ptr(), free_count_out.data_ptr(),
        cu_tokens.data_ptr(), slot_mapping.data_ptr(), slot_mapping.numel(),
        request_status.data_ptr(), _stream(stream))
    _check(st, "mla_kv_alloc")


def _row_stride(probs: torch.Tensor) -> int:
    """Elements between the rows of ``[batch, rows, vocab]`` probabilities, evenly apart."""
    batch, rows, vocab = probs.shape
    if vocab != 1 and probs.stride(2) != 1:
        _refuse("a row of probabilities is not contiguous")
    stride = probs.stride(1) if rows > 1 else probs.stride(0) if batch > 1 else vocab
    if stride < vocab or (batch != 1 and probs.stride(0) != rows * stride):
        _refuse("the rows of probabilities are not evenly apart")
    return stride


def mla_verify_drafts(target_probs: torch.Tensor, draft_probs: torch.Tensor | None,
                      draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                      out_tokens: torch.Tensor, num_accepted: torch.Tensor,
                      num_drafts: torch.Tensor | None = None,
                      seq_lens: torch.Tensor | None = None,
                      seq_lens_out: torch.Tensor | None = None, stream=None) -> None:
    """Keep drafted tokens with probability min(1, p / q) and sample the next token.

    ``target_probs [batch, K + 1, vocab]`` and ``draft_probs [batch, K, vocab]``
    (or None: the drafter was certain) are float32 or bfloat16 probabilities whose
    rows may be padded (an even stride), ``draft_tokens [batch, K]``, ``uniforms
    [batch, K + 1]`` float32 in [0, 1): one per draft, the last for the sample.
    ``num_drafts [batch]`` limits a request to fewer than K drafts. Writes
    ``out_tokens [batch, K + 1]`` (kept drafts, next token, then -1),
    ``num_accepted [batch]`` and, given ``seq_lens``, ``seq_lens_out``: the
    lengths without the rejected drafts (may be ``seq_lens`` itself).
    """
    if target_probs.dim() != 3:
        _refuse("target_probs is [batch, drafts + 1, vocab]")
    device = _device_of(target_probs)
    batch, rows, vocab = target_probs.shape
    drafts = rows - 1
    if target_probs.dtype not in (torch.float32, torch.bfloat16):
        _refuse("target_probs is float32 or bfloat16")
    dtype = MLA_PROB_F32 if target_probs.dtype == torch.float32 else MLA_PROB_BF16
    target_stride = _row_stride(target_probs) if batch > 0 else vocab
    draft_stride = vocab
    if draft_probs is not None:
        if draft_probs.dtype != target_probs.dtype or draft_probs.shape != (batch, drafts, vocab):
            _refuse("draft_probs is [batch, drafts, vocab], of target_probs' type")
        if draft_probs.get_device() != device:
            _refuse("draft_probs is on another device")
        if batch > 0 and drafts > 0:
            draft_stride = _row_stride(draft_probs)
    if draft_tokens.shape != (batch, drafts) or out_tokens.shape != (batch, rows):
        _refuse("draft_tokens is [batch, drafts], out_tokens [batch, drafts + 1]")
    if uniforms.dtype != torch.float32 or uniforms.shape != (batch, rows):
        _refuse("uniforms is float32 [batch, drafts + 1]")
    _same_device(device, uniforms)
    if num_accepted.numel() != batch:
        _refuse("num_accepted is [batch]")
    _int32(device, draft_tokens, out_tokens, num_accepted)
    if seq_lens_out is not None and seq_lens is None:
        _refuse("seq_lens_out needs seq_lens")
    for t in (num_drafts, seq_lens, seq_lens_out):
        if t is not None:
            _int32(device, t)
            if t.numel() != batch:
                _refuse("num_drafts, seq_lens and seq_lens_out are [batch]")
    st = load_library().mla_verify_drafts(
        target_probs.data_ptr(), target_stride, _ptr(draft_probs), draft_stride, dtype,
        draft_tokens.data_ptr(), uniforms.data_ptr(), _ptr(num_drafts), _ptr(seq_lens), batch,
        drafts, vocab, out_tokens.data_ptr(), num_accepted.data_ptr(), _ptr(seq_lens_out),
        _stream(stream))
    _check(st, "mla_verify_drafts")


def _float32(device: int, count: int, *tensors) -> None:
    """Each tensor that is given holds `count` contiguous float32 on `device`."""
    for t in tensors:
        if t is not None:
            if t.dtype is not torch.float32 or t.numel() != count:
                _refuse("a setting or uniform is float32, one for each request (or node)")
            _same_device(device, t)


def _prob_dtype(t: torch.Tensor) -> int:
    if t.dtype is torch.float32:
        return MLA_PROB_F32
    if t.dtype is torch.bfloat16:
        return MLA_PROB_BF16
    _refuse("logits and probabilities are float32 or bfloat16")


def mla_logits_to_probs(logits: torch.Tensor, probs: torch.Tensor,
                        temperature: torch.Tensor | None = None,
                        num_rows: torch.Tensor | None = None,
                        node_tokens: torch.Tensor | None = None,
                        tree_mask: torch.Tensor | None = None,
                        token_counts: torch.Tensor | None = None,
                        prompt_mask: torch.Tensor | None = None,
                        repetition: torch.Tensor | None = None,
                        frequency: torch.Tensor | None = None,
                        presence: torch.Tensor | None = None,
                        bias_tokens: torch.Tensor | None = None,
                        biases: torch.Tensor | None = None,
                        allowed: torch.Tensor | None = None, stream=None) -> None:
    """The probabilities that each request's settings make of its rows of logits.

    ``logits`` and ``probs`` are ``[batch, rows, vocab]``, float32 or bfloat16 each, rows evenly
    apart (``probs`` may be ``logits``). ``temperature``, ``repetition``, ``frequency`` and
    ``presence`` are float32 ``[batch]``; ``token_counts`` int32 ``[batch, vocab]`` and
    ``prompt_mask`` 32-bit words ``[batch, ceil(vocab / 32)]`` say which tokens came before;
    ``node_tokens`` int32 and ``tree_mask`` 64-bit words, both ``[batch, rows]``, which drafts come
    before each row as well (bit 0 never counts). ``bias_tokens`` (-1: none) and ``biases`` are
    ``[batch, n]``, ``allowed`` 32-bit words ``[batch, rows, ceil(vocab / 32)]``. Rows from
    ``num_rows[b]`` on are left as they were. The result is what :func:`mla_verify_drafts` and
    :func:`mla_verify_tree` take.
    """
    if logits.dim() != 3 or probs.shape != logits.shape:
        _refuse("logits and probs are [batch, rows, vocab]")
    device = _device_of(logits)
    if probs.get_device() != device:
        _refuse("probs is on another device")
    batch, rows, vocab = logits.shape
    in_type, out_type = _prob_dtype(logits), _prob_dtype(probs)
    in_stride = out_stride = vocab
    if batch > 0 and rows > 0 and vocab > 0:
        in_stride, out_stride = _row_stride(logits), _row_stride(probs)
    _float32(device, batch, temperature, repetition, frequency, presence)
    if num_rows is not None:
        _int32(device, num_rows)
        if num_rows.numel() != batch:
            _refuse("num_rows is [batch]")
    if (node_tokens is None) != (tree_mask is None):
        _refuse("node_tokens and tree_mask are given together")
    if tree_mask is not None:
        _tree_masks(device, tree_mask, batch, rows)
        _int32(device, node_tokens)
        if node_tokens.shape != (batch, rows):
            _refuse("node_tokens is [batch, rows]")
    words = (vocab + 31) // 32
    for t, shape in ((token_counts, (batch, vocab)), (prompt_mask, (batch, words)), (allowed, (batch, rows, words))):
        if t is not None:
            _int32(device, t)
            if t.shape != shape:
                _refuse("token_counts is [batch, vocab], prompt_mask [batch, words], allowed [batch, rows, words]")
    if (bias_tokens is None) != (biases is None):
        _refuse("bias_tokens and biases are given together")
    num_biases = 0
    if biases is not None:
        _int32(device, bias_tokens)
        if bias_tokens.dim() != 2 or bias_tokens.shape[0] != batch:
            _refuse("bias_tokens is [batch, n]")
        num_biases = bias_tokens.shape[1]
        _float32(device, batch * num_biases, biases)
    st = load_library().mla_logits_to_probs(
        logits.data_ptr(), in_stride, in_type, probs.data_ptr(), out_stride, out_type, batch, rows,
        vocab, _ptr(temperature), _ptr(num_rows), _ptr(node_tokens), _ptr(tree_mask),
        _ptr(token_counts), _ptr(prompt_mask), _ptr(repetition), _ptr(frequency), _ptr(presence),
        _ptr(bias_tokens), _ptr(biases), num_biases, _ptr(allowed), _stream(stream, device))
    _check(st, "mla_logits_to_probs")


def mla_verify_tree(target_probs: torch.Tensor, draft_probs: torch.Tensor | None,
                    node_tokens: torch.Tensor, tree_mask: torch.Tensor, uniforms: torch.Tensor,
                    out_tokens: torch.Tensor, path: torch.Tensor, num_accepted: torch.Tensor,
                    num_nodes: torch.Tensor | None = None, seq_lens: torch.Tensor | None = None,
                    seq_lens_out: torch.Tensor | None = None,
                    token_counts: torch.Tensor | None = None, stream=None) -> None:
    """Walk down each request's tree of drafts and sample the token behind the last kept node.

    ``target_probs`` and ``draft_probs`` (which a node's children were drawn from; None: they were
    certain) are ``[batch, N, vocab]``, float32 or bfloat16, rows evenly apart; ``node_tokens`` int32,
    ``tree_mask`` 64-bit words and ``uniforms`` float32 in [0, 1) are ``[batch, N]`` (``uniforms[:, 0]``
    is the sample's). ``num_nodes [batch]`` limits a request to fewer nodes. Writes ``out_tokens
    [batch, N]`` (kept drafts, next token, then -1), ``path [batch, N]`` (0, kept nodes, then -1),
    ``num_accepted [batch]``, given ``seq_lens`` also ``seq_lens_out``, the lengths after
    :func:`mla_kv_compact` (may be ``seq_lens`` itself), and adds the tokens to ``token_counts
    [batch, vocab]``.
    """
    if target_probs.dim() != 3:
        _refuse("target_probs is [batch, nodes, vocab]")
    device = _device_of(target_probs)
    batch, nodes, vocab = target_probs.shape
    dtype = _prob_dtype(target_probs)
    target_stride = draft_stride = vocab
    if batch > 0 and nodes > 0 and vocab > 0:
        target_stride = _row_stride(target_probs)
    if draft_probs is not None:
        if draft_probs.dtype != target_probs.dtype or draft_probs.shape != target_probs.shape:
            _refuse("draft_probs has target_probs' type and shape")
        if draft_probs.get_device() != device:
            _refuse("draft_probs is on another device")
        if batch > 0 and nodes > 0 and vocab > 0:
            draft_stride = _row_stride(draft_probs)
    _tree_masks(device, tree_mask, batch, nodes)
    if node_tokens.shape != (batch, nodes) or out_tokens.shape != (batch, nodes) or path.shape != (batch, nodes):
        _refuse("node_tokens, out_tokens and path are [batch, nodes]")
    if uniforms.shape != (batch, nodes):
        _refuse("uniforms is float32 [batch, nodes]")
    _float32(device, batch * nodes, uniforms)
    if num_accepted.numel() != batch:
        _refuse("num_accepted is [batch]")
    _int32(device, node_tokens, out_tokens, path, num_accepted)
    if seq_lens_out is not None and seq_lens is None:
        _refuse("seq_lens_out needs seq_lens")
    for t in (num_nodes, seq_lens, seq_lens_out):
        if t is not None:
            _int32(device, t)
            if t.numel() != batch:
                _refuse("num_nodes, seq_lens and seq_lens_out are [batch]")
    if token_counts is not None:
        _int32(device, token_counts)
        if token_counts.shape != (batch, vocab):
            _refuse("token_counts is [batch, vocab]")
    st = load_library().mla_verify_tree(
        target_probs.data_ptr(), target_stride, _ptr(draft_probs), draft_stride, dtype,
        node_tokens.data_ptr(), tree_mask.data_ptr(), uniforms.data_ptr(), _ptr(num_nodes),
        _ptr(seq_lens), batch, nodes, vocab, out_tokens.data_ptr(), path.data_ptr(),
        num_accepted.data_ptr(), _ptr(seq_lens_out), _ptr(token_counts), _stream(stream, device))
    _check(st, "mla_verify_tree")


def mla_kv_compact(kv_pages: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                   path: torch.Tensor, num_accepted: torch.Tensor, stream=None) -> None:
    """Move the kept nodes' cache entries behind each request's context, in every layer's cache.

    ``kv_pages`` as in :func:`kv_dtype_code`, or several layers of it: one more dimension in front,
    each layer contiguous. ``seq_lens`` are the lengths after verification, ``path [batch, N]`` and
    ``num_accepted [batch]`` as :func:`mla_verify_tree` writes them.
    """
    # (from the whole tensor's shape and type: taking a layer out of it costs more host time
    # than the launch)
    shape, kind = kv_pages.shape, kv_pages.dtype
    width = shape[-1]
    if width == 576 and (kind is torch.uint8 or kind is torch.bfloat16):
        inner, dtype = 3, MLA_KV_E4M3 if kind is torch.uint8 else MLA_KV_BF16
    elif width == MLA_E2M1_PAGE_BYTES and kind is torch.uint8:
        inner, dtype = 2, MLA_KV_E2M1
    else:
        _refuse("kv_pages are uint8 or bfloat16 [.., num_pages, 64, 576] or uint8 [.., num_pages, 19008]")
    layers, layer_bytes = 1, 0
    if len(shape) == inner + 1:
        layers, layer_bytes = shape[0], kv_pages.stride(0) * kv_pages.element_size()
        if layers == 0 or not (kv_pages.is_contiguous() or kv_pages[0].is_contiguous()):
            _refuse("kv_pages has no layer, or layers that are not contiguous")
    elif len(shape) != inner or not kv_pages.is_contiguous():
        _refuse("kv_pages is not a contiguous cache, nor layers of one")
    device = _device_of(kv_pages)
    if block_table.dim() != 2:
        _refuse("block_table is [batch, max_pages]")
    batch, max_pages = block_table.shape
    if path.dim() != 2 or path.shape[0] != batch:
        _refuse("path is [batch, nodes]")
    if seq_lens.numel() != batch or num_accepted.numel() != batch:
        _refuse("seq_lens and num_accepted are [batch]")
    _int32(device, block_table, seq_lens, path, num_accepted)
    st = load_library().mla_kv_compact(
        kv_pages.data_ptr(), layers, layer_bytes, shape[-inner], 64 if inner == 2 else shape[-2], dtype,
        block_table.data_ptr(), max_pages, seq_lens.data_ptr(), path.data_ptr(),
        num_accepted.data_ptr(), batch, path.shape[1], _stream(stream, device))
    _check(st, "mla_kv_compact")


def mla_decode_static_scratch(q: torch.Tensor, kv_pages: torch.Tensor,
                              block_table: torch.Tensor, seq_lens: torch.Tensor, sm_scale: float,
                              kv_scale: float, out: torch.Tensor, lse: torch.Tensor,
                              device_status: torch.Tensor | None = None, num_ctas: int = 0,
                              stream=None) -> None:
    """mla_decode without a workspace, for callers that cannot allocate device memory.

    The split-KV scratch is a fixed array inside libmla.so (MLA_STATIC_SCRATCH_BYTES),
    shared by every call on a device: calls must not overlap on the GPU. The first
    call on a device looks up the array's address and should precede any stream
    capture. ``device_status`` (int32, one element, optional) receives the call's
    MLA_DEVICE_ERR_* bits.
    """
    batch, nq, heads = _decode_shape(q, block_table, seq_lens, out, lse)
    dtype = kv_dtype_code(kv_pages)
    device = _device_of(kv_pages)
    _same_device(device, q, block_table, seq_lens, out, lse)
    if device_status is not None:
        if device_status.dtype != torch.int32 or device_status.numel() < 1:
            _refuse("device_status is int32, one element")
        _same_device(device, device_status)
    st = load_library().mla_decode_static_scratch(
        _ptr(q), _ptr(kv_pages), int(kv_pages.shape[0]), _page_size(kv_pages),
        dtype, _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
        batch, nq, heads, float(sm_scale), float(kv_scale), int(num_ctas), _ptr(out), _ptr(lse),
        _ptr(device_status), _stream(stream))
    _check(st, "mla_decode_static_scratch")


def read_device_status(workspace: torch.Tensor) -> int:
    """The sticky device status word at the head of a decode workspace (syncs)."""
    return int(workspace[:4].view(torch.int32).item()) & 0xFFFFFFFF
