"""Python binding of libdsa: the C-ABI entry points with the same names, taking
torch CUDA tensors. Argument marshalling only: shape/dtype/device checks, then
``data_ptr()`` and the current stream go to the C call. Every computation runs in
the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import DsaPageArrays, DsaPaging, check

__all__ = ["paging", "dsa_compress", "dsa_compress_append", "dsa_indexer_store",
           "dsa_write_geom", "dsa_decode_append", "dsa_decode_append_fp8", "dsa_score", "dsa_score_prefill", "dsa_select", "dsa_expand",
           "dsa_select_expand", "dsa_expand_tail", "dsa_select_expand_tail",
           "dsa_sparse_mla_decode_workspace", "dsa_sparse_mla_decode",
           "dsa_sparse_mla_decode_noalloc", "dsa_sparse_mla_decode_fp8", "dsa_quantize_latent",
           "dsa_dequantize_latent", "dsa_quantize_latent_fp4", "dsa_dequantize_latent_fp4", "dsa_decode_append_fp4",
           "dsa_sparse_mla_decode_fp4_workspace", "dsa_sparse_mla_decode_fp4_splits",
           "dsa_sparse_mla_decode_fp4",
           "page_arrays", "dsa_pages_workspace", "dsa_pages_free", "dsa_pages_fork",
           "dsa_pages_serve", "dsa_pages_reserve", "dsa_pages_compact", "DsaPageArrays",
           "dsa_frontend_workspace", "dsa_frontend", "dsa_rmsnorm", "dsa_router_logits_workspace",
           "dsa_router_logits", "dsa_route", "dsa_experts_workspace", "dsa_experts",
           "dsa_latent_project_workspace",
           "dsa_latent_project", "dsa_select_k",
           "dsa_validate_config", "dsa_prefetch_l2", "dsa_set_option", "dsa_get_option", "mla_kernel",
           "select_kernel", "project_kernel", "DsaPaging"]


def _ptr(t: Optional[torch.Tensor], dtype=None, name: str = "tensor",
         host_ok: bool = False) -> Optional[int]:
    """Device address of t. With host_ok, pinned host memory is accepted too: under
    unified addressing its address is valid in kernels, which then read or write it
    directly (no copy)."""
    if t is None:
        return None
    if not t.is_cuda and not (host_ok and t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor" + (" or pinned host memory" if host_ok else ""))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def dsa_set_option(option: int, value: int) -> None:
    """Set a process-wide launch option (DSA_OPT_* in include/dsa.h)."""
    check(_lib.load().dsa_set_option(int(option), int(value)))


def dsa_get_option(option: int) -> int:
    """Current value of a launch option (-1 for an unknown option)."""
    return int(_lib.load().dsa_get_option(int(option)))


class mla_kernel:
    """Context manager pinning the sparse-attention kernel: "auto", "tcgen05" (the
    persistent tensor-core split kernel where it supports the shape), "mma" (the
    mma.sync split kernel) or "cluster" (the tensor-core decode kernel that merges a
    row's splits inside a cluster); the previous choice is restored on exit."""

    _VALUES = {"auto": _lib.DSA_MLA_KERNEL_AUTO, "tcgen05": _lib.DSA_MLA_KERNEL_TCGEN05,
               "mma": _lib.DSA_MLA_KERNEL_MMA, "cluster": _lib.DSA_MLA_KERNEL_CLUSTER}

    def __init__(self, which: str):
        if which not in self._VALUES:
            raise ValueError(f"kernel {which!r}: one of {sorted(self._VALUES)}")
        self.value = self._VALUES[which]
        self.prev = None

    def __enter__(self):
        self.prev = dsa_get_option(_lib.DSA_OPT_MLA_KERNEL)
        dsa_set_option(_lib.DSA_OPT_MLA_KERNEL, self.value)
        return self

    def __exit__(self, *exc):
        dsa_set_option(_lib.DSA_OPT_MLA_KERNEL, self.prev)
        return False


class select_kernel:
    """Context manager pinning how clustered rows are selected: "merge" (the
    default) or "radix"; the previous choice is restored on exit."""

    _VALUES = {"merge": _lib.DSA_SELECT_KERNEL_MERGE, "radix": _lib.DSA_SELECT_KERNEL_RADIX}

    def __init__(self, which: str):
        if which not in self._VALUES:
            raise ValueError(f"kernel {which!r}: one of {sorted(self._VALUES)}")
        self.value = self._VALUES[which]
        self.prev = None

    def __enter__(self):
        self.prev = dsa_get_option(_lib.DSA_OPT_SELECT_KERNEL)
        dsa_set_option(_lib.DSA_OPT_SELECT_KERNEL, self.value)
        return self

    def __exit__(self, *exc):
        dsa_set_option(_lib.DSA_OPT_SELECT_KERNEL, self.prev)
        return False


class project_kernel:
    """Context manager pinning the projection kernel: "auto" (the default),
    "tcgen05" or "mma"; the previous choice is restored on exit."""

    _VALUES = {"auto": _lib.DSA_PROJECT_KERNEL_AUTO, "tcgen05": _lib.DSA_PROJECT_KERNEL_TCGEN05,
               "mma": _lib.DSA_PROJECT_KERNEL_MMA}

    def __init__(self, which: str):
        if which not in self._VALUES:
            raise ValueError(f"kernel {which!r}: one of {sorted(self._VALUES)}")
        self.value = self._VALUES[which]
        self.prev = None

    def __enter__(self):
        self.prev = dsa_get_option(_lib.DSA_OPT_PROJECT_KERNEL)
        dsa_set_option(_lib.DSA_OPT_PROJECT_KERNEL, self.value)
        return self

    def __exit__(self, *exc):
        dsa_set_option(_lib.DSA_OPT_PROJECT_KERNEL, self.prev)
        return False


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def paging(seq_lens: torch.Tensor, max_seq_len: int, block_table: Optional[torch.Tensor] = None,
           block_size: int = 0, num_blocks: int = 0) -> DsaPaging:
    """Describe where sequences live (see ``dsa_paging`` in include/dsa.h).

    The tensors must outlive every call that uses the returned descriptor."""
    pg = DsaPaging()
    pg.batch = int(seq_lens.numel())
    pg.max_seq_len = int(max_seq_len)
    pg.seq_lens = _ptr(seq_lens, torch.int32, "seq_lens")
    pg.device = seq_lens.get_device()  # beside the C fields: where its tensors live
    if block_table is not None:
        if block_table.get_device() != pg.device:
            raise ValueError(f"block_table is on {block_table.device}, seq_lens on "
                             f"{seq_lens.device}: one device per descriptor")
        pg.block_table = _ptr(block_table, torch.int32, "block_table")
        pg.max_blocks = int(block_table.shape[1])
        pg.block_size = int(block_size)
        pg.num_blocks = int(num_blocks)
    else:
        pg.block_table = None
        pg.max_blocks = 0
        pg.block_size = 0
        pg.num_blocks = 0
    return pg


def dsa_validate_config(index_kpool: int, index_topk: int, kv_lora_rank: int,
                        local_heads: int) -> None:
    check(_lib.load().dsa_validate_config(index_kpool, index_topk, kv_lora_rank, local_heads))


def dsa_select_k(index_topk: int, kpool: int, n_pools: int) -> int:
    return _lib.load().dsa_select_k(index_topk, kpool, n_pools)


def dsa_compress(k_raw, gate, token_valid, ape, ln_w, ln_b, eps: float, pg: DsaPaging,
                 first_key: int, kpool: int, kpool_out, pool_valid, pool_idx=None, status=None,
                 stream=None) -> None:
    ihd = int(k_raw.shape[-1])
    check(_lib.load().dsa_compress(
        _ptr(k_raw, torch.bfloat16, "k_raw"), _ptr(gate, torch.bfloat16, "gate"),
        _ptr(token_valid, torch.uint8, "token_valid"), _ptr(ape, torch.float32, "ape"),
        _ptr(ln_w, torch.bfloat16, "ln_w"), _ptr(ln_b, torch.bfloat16, "ln_b"), float(eps),
        ctypes.byref(pg), int(first_key), int(kpool), ihd,
        _ptr(kpool_out, torch.bfloat16, "kpool_out"), _ptr(pool_valid, torch.uint8, "pool_valid"),
        _ptr(pool_idx, torch.int32, "pool_idx"), _ptr(status, torch.int32, "status"),
        _stream(stream)))


def dsa_compress_append(k_raw, gate, token_valid, ape, ln_w, ln_b, eps: float, pg: DsaPaging,
                        first_key: int, kpool: int, new_tokens: int, kpool_out, pool_valid,
                        pool_idx=None, status=None, stream=None) -> None:
    """dsa_compress for the pools the last ``new_tokens`` tokens of each sequence
    completed (the lengths are read on the device)."""
    ihd = int(k_raw.shape[-1])
    check(_lib.load().dsa_compress_append(
        _ptr(k_raw, torch.bfloat16, "k_raw"), _ptr(gate, torch.bfloat16, "gate"),
        _ptr(token_valid, torch.uint8, "token_valid"), _ptr(ape, torch.float32, "ape"),
        _ptr(ln_w, torch.bfloat16, "ln_w"), _ptr(ln_b, torch.bfloat16, "ln_b"), float(eps),
        ctypes.byref(pg), int(first_key), int(kpool), ihd, int(new_tokens),
        _ptr(kpool_out, torch.bfloat16, "kpool_out"), _ptr(pool_valid, torch.uint8, "pool_valid"),
        _ptr(pool_idx, torch.int32, "pool_idx"), _ptr(status, torch.int32, "status"),
        _stream(stream)))


def dsa_indexer_store(k_new, gate_new, pg: DsaPaging, seq_lens, k_raw, gate, token_valid,
                      ckv_new=None, ckv=None, status=None, stream=None) -> None:
    """Append one staged token per sequence at its current length (read on the
    device) and advance ``seq_lens`` (the tensor ``pg`` was built from)."""
    batch, ihd = (int(x) for x in k_new.shape)
    if tuple(gate_new.shape) != (batch, ihd):
        raise ValueError(f"gate_new must be [{batch}, {ihd}]")
    kvl = int(ckv_new.shape[-1]) if ckv_new is not None else 0
    check(_lib.load().dsa_indexer_store(
        _ptr(k_new, torch.bfloat16, "k_new"), _ptr(gate_new, torch.bfloat16, "gate_new"),
        _ptr(ckv_new, torch.bfloat16, "ckv_new"), ihd, kvl, ctypes.byref(pg),
        _ptr(seq_lens, torch.int32, "seq_lens"), _ptr(k_raw, torch.bfloat16, "k_raw"),
        _ptr(gate, torch.bfloat16, "gate"), _ptr(token_valid, torch.uint8, "token_valid"),
        _ptr(ckv, torch.bfloat16, "ckv"), _ptr(status, torch.int32, "status"), _stream(stream)))


def dsa_write_geom(seq_lens, row_seq, row_ctx, status=None, stream=None) -> None:
    """row_ctx[r] = seq_lens[row_seq[r]] on the device (row_seq None: r)."""
    check(_lib.load().dsa_write_geom(
        _ptr(seq_lens, torch.int32, "seq_lens"), int(seq_lens.numel()),
        _ptr(row_seq, torch.int32, "row_seq"), int(row_ctx.numel()),
        _ptr(row_ctx, torch.int32, "row_ctx"), _ptr(status, torch.int32, "status"),
        _stream(stream)))


def dsa_decode_append(k_new, gate_new, ape, ln_w, ln_b, eps: float, pg: DsaPaging, seq_lens,
                      first_key: int, kpool: int, k_raw, gate, token_valid, kpool_out, pool_valid,
                      ckv_new=None, ckv=None, pool_idx=None, row_ctx=None, status=None,
                      stream=None, refs=None, serving=None) -> None:
    """dsa_indexer_store + dsa_write_geom + dsa_compress_append(new_tokens=1) in one
    launch (identical results). With ``refs`` (the pool's counts) a sequence whose next
    page is shared, with ``serving`` one whose entry is negative, is left as it is
    (dsa_decode_append_guarded)."""
    batch, ihd = (int(x) for x in k_new.shape)
    if tuple(gate_new.shape) != (batch, ihd):
        raise ValueError(f"gate_new must be [{batch}, {ihd}]")
    kvl = int(ckv_new.shape[-1]) if ckv_new is not None else 0
    if refs is not None or serving is not None:
        _append_guarded(refs, serving, _lib.DSA_LATENT_BF16, k_new, gate_new, ckv_new, ape, ln_w,
                        ln_b, eps, pg, seq_lens, first_key, kpool, kvl, k_raw, gate, token_valid,
                        ckv, None, None, 0, kpool_out, pool_valid, pool_idx, row_ctx, status,
                        stream)
        return
    check(_lib.load().dsa_decode_append(
        _ptr(k_new, torch.bfloat16, "k_new"), _ptr(gate_new, torch.bfloat16, "gate_new"),
        _ptr(ckv_new, torch.bfloat16, "ckv_new"), _ptr(ape, torch.float32, "ape"),
        _ptr(ln_w, torch.bfloat16, "ln_w"), _ptr(ln_b, torch.bfloat16, "ln_b"), float(eps),
        ctypes.byref(pg), _ptr(seq_lens, torch.int32, "seq_lens"), int(first_key), int(kpool),
        ihd, kvl, _ptr(k_raw, torch.bfloat16, "k_raw"), _ptr(gate, torch.bfloat16, "gate"),
        _ptr(token_valid, torch.uint8, "token_valid"), _ptr(ckv, torch.bfloat16, "ckv"),
        _ptr(kpool_out, torch.bfloat16, "kpool_out"), _ptr(pool_valid, torch.uint8, "pool_valid"),
        _ptr(pool_idx, torch.int32, "pool_idx"), _ptr(row_ctx, torch.int32, "row_ctx"),
        _ptr(status, torch.int32, "status"), _stream(stream)))


def dsa_decode_append_fp8(k_new, gate_new, ckv_new, ape, ln_w, ln_b, eps: float, pg: DsaPaging,
                          seq_lens, first_key: int, kpool: int, k_raw, gate, token_valid,
                          ckv_codes, ckv_scales, kpool_out, pool_valid, ckv=None, pool_idx=None,
                          row_ctx=None, status=None, stream=None, refs=None,
                          serving=None) -> None:
    """dsa_decode_append that also encodes the staged latent row into the FP8 cache
    (same codec and bytes as dsa_quantize_latent); the bf16 cache ``ckv`` is optional.
    ``refs`` and ``serving`` as in dsa_decode_append."""
    batch, ihd = (int(x) for x in k_new.shape)
    if tuple(gate_new.shape) != (batch, ihd):
        raise ValueError(f"gate_new must be [{batch}, {ihd}]")
    kvl = int(ckv_new.shape[-1])
    if int(ckv_codes.shape[-1]) != kvl or int(ckv_scales.shape[-1]) != kvl // 128:
        raise ValueError(f"ckv_codes must be [.., {kvl}] and ckv_scales [.., {kvl // 128}]")
    if refs is not None or serving is not None:
        _append_guarded(refs, serving, _lib.DSA_LATENT_FP8, k_new, gate_new, ckv_new, ape, ln_w,
                        ln_b, eps, pg, seq_lens, first_key, kpool, kvl, k_raw, gate, token_valid,
                        ckv, ckv_codes, ckv_scales, 0, kpool_out, pool_valid, pool_idx, row_ctx,
                        status, stream)
        return
    check(_lib.load().dsa_decode_append_fp8(
        _ptr(k_new, torch.bfloat16, "k_new"), _ptr(gate_new, torch.bfloat16, "gate_new"),
        _ptr(ckv_new, torch.bfloat16, "ckv_new"), _ptr(ape, torch.float32, "ape"),
        _ptr(ln_w, torch.bfloat16, "ln_w"), _ptr(ln_b, torch.bfloat16, "ln_b"), float(eps),
        ctypes.byref(pg), _ptr(seq_lens, torch.int32, "seq_lens"), int(first_key), int(kpool),
        ihd, kvl, _ptr(k_raw, torch.bfloat16, "k_raw"), _ptr(gate, torch.bfloat16, "gate"),
        _ptr(token_valid, torch.uint8, "token_valid"), _ptr(ckv, torch.bfloat16, "ckv"),
        _ptr(ckv_codes, torch.uint8, "ckv_codes"), _ptr(ckv_scales, torch.float32, "ckv_scales"),
        _ptr(kpool_out, torch.bfloat16, "kpool_out"), _ptr(pool_valid, torch.uint8, "pool_valid"),
        _ptr(pool_idx, torch.int32, "pool_idx"), _ptr(row_ctx, torch.int32, "row_ctx"),
        _ptr(status, torch.int32, "status"), _stream(stream)))


def dsa_score(qidx, w, row_seq, row_ctx, kpool, pool_valid, pg: DsaPaging, first_key: int,
              kpool_size: int, scale: float, scores, status=None, stream=None) -> None:
    rows, heads, ihd = (int(x) for x in qidx.shape)
    if tuple(w.shape) != (rows, heads):
        raise ValueError(f"w must be [{rows}, {heads}]")
    if scores.dim() != 2 or scores.shape[0] != rows:
        raise ValueError("scores must be [rows, p_stride]")
    check(_lib.load().dsa_score(
        _ptr(qidx, torch.bfloat16, "qidx"), _ptr(w, torch.float32, "w"), rows, heads, ihd,
        _ptr(row_seq, torch.int32, "row_seq"), _ptr(row_ctx, torch.int32, "row_ctx"),
        _ptr(kpool, torch.bfloat16, "kpool"), _ptr(pool_valid, torch.uint8, "pool_valid"),
        ctypes.byref(pg), int(first_key), int(kpool_size), float(scale),
        _ptr(scores, torch.float32, "scores"), int(scores.shape[1]),
        _ptr(status, torch.int32, "status"), _stream(stream)))


def dsa_score_prefill(qidx, w, seq: int, row_ctx, kpool, pool_valid, pg: DsaPaging,
                      first_key: int, kpool_size: int, scale: float, scores, status=None,
                      stream=None) -> None:
    """Index scores of a chunk of query rows of sequence ``seq`` on the tensor cores
    (contiguous pooled-key cache; index_heads in {32, 64, 128})."""
    rows, heads, ihd = (int(x) for x in qidx.shape)
    if tuple(w.shape) != (rows, heads):
        raise ValueError(f"w must be [{rows}, {heads}]")
    if scores.dim() != 2 or scores.shape[0] != rows:
        raise ValueError("scores must be [rows, p_stride]")
    check(_lib.load().dsa_score_prefill(
        _ptr(qidx, torch.bfloat16, "qidx"), _ptr(w, torch.float32, "w"), rows, heads, ihd,
        int(seq), _ptr(row_ctx, torch.int32, "row_ctx"),
        _ptr(kpool, torch.bfloat16, "kpool"), _ptr(pool_valid, torch.uint8, "pool_valid"),
        ctypes.byref(pg), int(first_key), int(kpool_size), float(scale),
        _ptr(scores, torch.float32, "scores"), int(scores.shape[1]),
        _ptr(status, torch.int32, "status"), _stream(stream)))


def dsa_select(scores, index_topk: int, kpool: int, pool_ids, stream=None) -> None:
    rows, p_stride = (int(x) for x in scores.shape)
    sk = dsa_select_k(index_topk, kpool, p_stride)
    if tuple(pool_ids.shape) != (rows, max(sk, 0)):
        raise ValueError(f"pool_ids must be [{rows}, {sk}]")
    check(_lib.load().dsa_select(
        _ptr(scores, torch.float32, "scores"), rows, p_stride, int(index_topk), int(kpool),
        _ptr(pool_ids, torch.int32, "pool_ids"), _stream(stream)))


def dsa_select_expand(scores, index_topk: int, kpool: int, first_key: int, pool_ids, token_ids,
                      stream=None) -> None:
    """dsa_select and dsa_expand in one launch (identical results)."""
    rows, p_stride = (int(x) for x in scores.shape)
    sk = dsa_select_k(index_topk, kpool, p_stride)
    if tuple(pool_ids.shape) != (rows, max(sk, 0)):
        raise ValueError(f"pool_ids must be [{rows}, {sk}]")
    if token_ids.dim() != 2 or token_ids.shape[0] != rows:
        raise ValueError("token_ids must be [rows, out_width]")
    check(_lib.load().dsa_select_expand(
        _ptr(scores, torch.float32, "scores"), rows, p_stride, int(index_topk), int(kpool),
        int(first_key), int(token_ids.shape[1]), _ptr(pool_ids, torch.int32, "pool_ids"),
        _ptr(token_ids, torch.int32, "token_ids"), _stream(stream)))


def dsa_expand(pool_ids, first_key: int, kpool: int, token_ids, stream=None) -> None:
    rows, sk = (int(x) for x in pool_ids.shape)
    if token_ids.dim() != 2 or token_ids.shape[0] != rows:
        raise ValueError("token_ids must be [rows, out_width]")
    check(_lib.load().dsa_expand(
        _ptr(pool_ids, torch.int32, "pool_ids"), rows, sk, int(first_key), int(kpool),
        int(token_ids.shape[1]), _ptr(token_ids, torch.int32, "token_ids"), _stream(stream)))


def dsa_expand_tail(pool_ids, first_key: int, kpool: int, index_topk: int, row_ctx, token_ids,
                    stream=None) -> None:
    """dsa_expand with always_select_tail: the trailing partial pool's tokens of
    each row (row_ctx [rows] i32) follow the pools from position index_topk on."""
    rows, sk = (int(x) for x in pool_ids.shape)
    if token_ids.dim() != 2 or token_ids.shape[0] != rows:
        raise ValueError("token_ids must be [rows, out_width]")
    if tuple(row_ctx.shape) != (rows,):
        raise ValueError(f"row_ctx must be [{rows}]")
    check(_lib.load().dsa_expand_tail(
        _ptr(pool_ids, torch.int32, "pool_ids"), rows, sk, int(first_key), int(kpool),
        int(index_topk), _ptr(row_ctx, torch.int32, "row_ctx"), int(token_ids.shape[1]),
        _ptr(token_ids, torch.int32, "token_ids"), _stream(stream)))


def dsa_select_expand_tail(scores, index_topk: int, kpool: int, first_key: int, row_ctx,
                           pool_ids, token_ids, stream=None) -> None:
    """dsa_select and dsa_expand_tail in one launch (identical results)."""
    rows, p_stride = (int(x) for x in scores.shape)
    sk = dsa_select_k(index_topk, kpool, p_stride)
    if tuple(pool_ids.shape) != (rows, max(sk, 0)):
        raise ValueError(f"pool_ids must be [{rows}, {sk}]")
    if token_ids.dim() != 2 or token_ids.shape[0] != rows:
        raise ValueError("token_ids must be [rows, out_width]")
    if tuple(row_ctx.shape) != (rows,):
        raise ValueError(f"row_ctx must be [{rows}]")
    check(_lib.load().dsa_select_expand_tail(
        _ptr(scores, torch.float32, "scores"), rows, p_stride, int(index_topk), int(kpool),
        int(first_key), _ptr(row_ctx, torch.int32, "row_ctx"), int(token_ids.shape[1]),
        _ptr(pool_ids, torch.int32, "pool_ids"), _ptr(token_ids, torch.int32, "token_ids"),
        _stream(stream)))


def dsa_sparse_mla_decode_workspace(rows: int, heads: int, out_width: int, hidden: int,
                                    with_o_absorb: bool, kv_lora_rank: int = 512) -> int:
    n = ctypes.c_size_t(0)
    check(_lib.load().dsa_sparse_mla_decode_workspace(
        int(rows), int(heads), int(kv_lora_rank), int(out_width), int(hidden),
        1 if with_o_absorb else 0, ctypes.byref(n)))
    return int(n.value)


def dsa_sparse_mla_decode(qlat, row_seq, ckv, pg: DsaPaging, token_ids, softmax_scale: float,
                          o_absorb=None, y=None, olat=None, status=None, workspace=None,
                          stream=None) -> None:
    rows, heads, kvl = (int(x) for x in qlat.shape)
    ow = int(token_ids.shape[1])
    hidden = int(o_absorb.shape[0]) if o_absorb is not None else 0
    if o_absorb is not None and tuple(o_absorb.shape) != (hidden, heads * kvl):
        raise ValueError(f"o_absorb must be [hidden, {heads * kvl}]")
    if y is not None and tuple(y.shape) != (rows, hidden):
        raise ValueError(f"y must be [{rows}, {hidden}]")
    if olat is not None and tuple(olat.shape) != (rows, heads, kvl):
        raise ValueError(f"olat must be [{rows}, {heads}, {kvl}]")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(_lib.load().dsa_sparse_mla_decode(
        _ptr(qlat, torch.bfloat16, "qlat"), rows, heads, kvl,
        _ptr(row_seq, torch.int32, "row_seq"), _ptr(ckv, torch.bfloat16, "ckv"),
        ctypes.byref(pg), _ptr(token_ids, torch.int32, "token_ids"), ow, float(softmax_scale),
        _ptr(o_absorb, torch.bfloat16, "o_absorb"), hidden,
        _ptr(y, torch.bfloat16, "y", host_ok=True),
        _ptr(olat, torch.float32, "olat"), _ptr(status, torch.int32, "status"),
        _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream)))


def dsa_sparse_mla_decode_fp8(qlat, row_seq, ckv_codes, ckv_scales, pg: DsaPaging, token_ids,
                              softmax_scale: float, o_absorb=None, y=None, olat=None,
                              status=None, workspace=None, stream=None) -> None:
    """dsa_sparse_mla_decode over an FP8 latent cache (E4M3 codes + per-128-channel
    power-of-two scales, see dsa_quantize_latent)."""
    rows, heads, kvl = (int(x) for x in qlat.shape)
    ow = int(token_ids.shape[1])
    hidden = int(o_absorb.shape[0]) if o_absorb is not None else 0
    if o_absorb is not None and tuple(o_absorb.shape) != (hidden, heads * kvl):
        raise ValueError(f"o_absorb must be [hidden, {heads * kvl}]")
    if y is not None and tuple(y.shape) != (rows, hidden):
        raise ValueError(f"y must be [{rows}, {hidden}]")
    if olat is not None and tuple(olat.shape) != (rows, heads, kvl):
        raise ValueError(f"olat must be [{rows}, {heads}, {kvl}]")
    if ckv_codes.shape[-1] != kvl or ckv_scales.shape[-1] != kvl // 128:
        raise ValueError("ckv_codes must be [..., kvl] and ckv_scales [..., kvl/128]")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(_lib.load().dsa_sparse_mla_decode_fp8(
        _ptr(qlat, torch.bfloat16, "qlat"), rows, heads, kvl,
        _ptr(row_seq, torch.int32, "row_seq"), _ptr(ckv_codes, torch.uint8, "ckv_codes"),
        _ptr(ckv_scales, torch.float32, "ckv_scales"), ctypes.byref(pg),
        _ptr(token_ids, torch.int32, "token_ids"), ow, float(softmax_scale),
        _ptr(o_absorb, torch.bfloat16, "o_absorb"), hidden, _ptr(y, torch.bfloat16, "y", host_ok=True),
        _ptr(olat, torch.float32, "olat"), _ptr(status, torch.int32, "status"),
        _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream)))


def dsa_quantize_latent(x, codes, scales, stream=None) -> None:
    """FP8 latent cache from bf16 rows: codes [..., kvl] u8, scales [..., kvl/128] f32."""
    kvl = int(x.shape[-1])
    rows = x.numel() // kvl
    if codes.numel() != x.numel() or scales.numel() != rows * (kvl // 128):
        raise ValueError("codes must match x and scales hold kvl/128 per row")
    check(_lib.load().dsa_quantize_latent(
        _ptr(x, torch.bfloat16, "x"), rows, kvl, _ptr(codes, torch.uint8, "codes"),
        _ptr(scales, torch.float32, "scales"), _stream(stream)))


# -- FP4 latent cache ------------------------------------------------------

_FP4_BLOCK = 16  # channels under one scale


def _fp4_cache(codes, scales) -> int:
    """Channels of an FP4 latent cache (codes [.., kvl/2], scales [.., kvl/16])."""
    kvl = 2 * codes.size(-1)
    if scales.size(-1) * _FP4_BLOCK != kvl or scales.numel() * 8 != codes.numel():
        raise ValueError("codes must be [.., kvl/2] and scales [.., kvl/16] of the same rows")
    return kvl


def _fp4_covers(codes, kvl: int, pg: DsaPaging) -> None:
    """The cache holds every row that the paging descriptor can name."""
    need = pg.num_blocks * pg.block_size if pg.block_table else pg.batch * pg.max_seq_len
    if codes.numel() * 2 < need * kvl:
        raise ValueError(f"the cache holds {codes.numel() * 2 // kvl} rows, the paging "
                         f"descriptor names {need}")


def _dev_ptr(t: Optional[torch.Tensor], dtype, dev: int, name: str) -> Optional[int]:
    """_ptr for the calls whose tensors must all live on one device, ``dev``."""
    if t is None:
        return None
    if t.get_device() == dev and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return t.data_ptr()
    p = _ptr(t, dtype, name)
    raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}: one device per call ({p:#x})")


# The current device and its current stream by their raw handles: the GPU work of these
# calls is often shorter than making a Stream object takes.
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _run(dev: int, stream, fn, *args) -> None:
    """One library call with device ``dev`` current, on its current stream by default."""
    if _current_device() != dev:
        with torch.cuda.device(dev):
            check(fn(*args, _stream(stream)))
        return
    rc = fn(*args, _current_stream(dev) if stream is None else _stream(stream))
    if rc:
        check(rc)


def _described(d, dev: int, name: str) -> None:
    """The tensors behind descriptor ``d`` (paging, page_arrays) are on device ``dev``."""
    at = getattr(d, "device", dev)
    if at != dev:
        raise ValueError(f"{name} describes tensors on cuda:{at}, not on cuda:{dev}: one device "
                         "per call")


def _device_of(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def dsa_quantize_latent_fp4(x, codes, scales, cache_exp: int = 0, stream=None) -> None:
    """FP4 latent cache from bf16 rows: codes [..., kvl/2] u8 (two E2M1 codes a byte),
    scales [..., kvl/16] u8 (E4M3), under 2^cache_exp (see include/dsa.h)."""
    kvl, n = x.size(-1), x.numel()
    if _fp4_cache(codes, scales) != kvl or codes.numel() * 2 != n:
        raise ValueError("codes [.., kvl/2] and scales [.., kvl/16] must match x [.., kvl]")
    if n == 0:
        return
    dev = _device_of(x, "x")
    _run(dev, stream, _lib.load().dsa_quantize_latent_fp4,
         _dev_ptr(x, torch.bfloat16, dev, "x"), n // kvl, kvl, int(cache_exp),
         _dev_ptr(codes, torch.uint8, dev, "codes"), _dev_ptr(scales, torch.uint8, dev, "scales"))


def dsa_dequantize_latent_fp4(codes, scales, out, cache_exp: int = 0, rows=None, status=None,
                              stream=None) -> None:
    """Rows of an FP4 latent cache back as bf16, exactly: all of them in order, or the
    cache rows named by ``rows`` (i32, one per row of out)."""
    kvl = _fp4_cache(codes, scales)
    if out.size(-1) != kvl:
        raise ValueError(f"out must be [.., {kvl}]")
    n, cache_rows = out.numel() // kvl, codes.numel() * 2 // kvl
    if rows is not None and rows.numel() != n:
        raise ValueError(f"rows must hold {n} row numbers")
    if rows is None and n != cache_rows:
        raise ValueError(f"out must hold the cache's {cache_rows} rows")
    if n == 0:
        return
    dev = _device_of(codes, "codes")
    _run(dev, stream, _lib.load().dsa_dequantize_latent_fp4,
         _dev_ptr(codes, torch.uint8, dev, "codes"), _dev_ptr(scales, torch.uint8, dev, "scales"),
         cache_rows, _dev_ptr(rows, torch.int32, dev, "rows"), n, kvl, int(cache_exp),
         _dev_ptr(out, torch.bfloat16, dev, "out"), _dev_ptr(status, torch.int32, dev, "status"))


def _fp8_rows(codes, scales) -> int:
    """Width of FP8 rows: codes [.., w] with scales [.., w/128] over the same rows."""
    w = codes.size(-1)
    if w < 1 or w % 128 or scales.size(-1) * 128 != w or scales.numel() * 128 != codes.numel():
        raise ValueError("codes must be [.., w] and scales [.., w/128] of the same rows, w a "
                         "multiple of 128")
    return w


def dsa_dequantize_latent(codes, scales, out, rows=None, status=None, stream=None) -> None:
    """Rows of an FP8 latent cache back as bf16, exactly: all of them in order, or the cache
    rows named by ``rows`` (i32, one per row of out)."""
    kvl = _fp8_rows(codes, scales)
    if out.size(-1) != kvl:
        raise ValueError(f"out must be [.., {kvl}]")
    n, cache_rows = out.numel() // kvl, codes.numel() // kvl
    if rows is not None and rows.numel() != n:
        raise ValueError(f"rows must hold {n} row numbers")
    if rows is None and n != cache_rows:
        raise ValueError(f"out must hold the cache's {cache_rows} rows")
    if n == 0:
        return
    dev = _device_of(out, "out")
    _run(dev, stream, _lib.load().dsa_dequantize_latent,
         _dev_ptr(codes, torch.uint8, dev, "codes"), _dev_ptr(scales, torch.float32, dev, "scales"),
         cache_rows, _dev_ptr(rows, torch.int32, dev, "rows"), n, kvl,
         _dev_ptr(out, torch.bfloat16, dev, "out"), _dev_ptr(status, torch.int32, dev, "status"))


def dsa_decode_append_fp4(k_new, gate_new, ckv_new, ape, ln_w, ln_b, eps: float, pg: DsaPaging,
                          seq_lens, first_key: int, kpool: int, k_raw, gate, token_valid,
                          ckv_codes, ckv_scales, cache_exp: int, kpool_out, pool_valid, ckv=None,
                          pool_idx=None, row_ctx=None, status=None, stream=None, refs=None,
                          serving=None) -> None:
    """dsa_decode_append that also encodes the staged latent row into the FP4 cache
    (same codec and bytes as dsa_quantize_latent_fp4); the bf16 cache ``ckv`` is
    optional. ``refs`` and ``serving`` as in dsa_decode_append."""
    batch, ihd = k_new.shape
    if gate_new.shape != k_new.shape:
        raise ValueError(f"gate_new must be [{batch}, {ihd}]")
    kvl = ckv_new.size(-1)
    if (ckv_new.dim() != 2 or ckv_new.size(0) != batch
            or _fp4_cache(ckv_codes, ckv_scales) != kvl):
        raise ValueError(f"ckv_new must be [{batch}, kvl], ckv_codes [.., kvl/2] and "
                         "ckv_scales [.., kvl/16]")
    if batch != pg.batch:
        raise ValueError(f"one staged row per sequence: {batch} rows, {pg.batch} sequences")
    _fp4_covers(ckv_codes, kvl, pg)
    if refs is not None or serving is not None:
        _append_guarded(refs, serving, _lib.DSA_LATENT_FP4, k_new, gate_new, ckv_new, ape, ln_w,
                        ln_b, eps, pg, seq_lens, first_key, kpool, kvl, k_raw, gate, token_valid,
                        ckv, ckv_codes, ckv_scales, cache_exp, kpool_out, pool_valid, pool_idx,
                        row_ctx, status, stream)
        return
    dev = _device_of(k_new, "k_new")
    _described(pg, dev, "pg")
    bf16, u8, i32, f32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
    _run(dev, stream, _lib.load().dsa_decode_append_fp4,
         _dev_ptr(k_new, bf16, dev, "k_new"), _dev_ptr(gate_new, bf16, dev, "gate_new"),
         _dev_ptr(ckv_new, bf16, dev, "ckv_new"), _dev_ptr(ape, f32, dev, "ape"),
         _dev_ptr(ln_w, bf16, dev, "ln_w"), _dev_ptr(ln_b, bf16, dev, "ln_b"), float(eps),
         ctypes.byref(pg), _dev_ptr(seq_lens, i32, dev, "seq_lens"), int(first_key), int(kpool),
         ihd, kvl, _dev_ptr(k_raw, bf16, dev, "k_raw"), _dev_ptr(gate, bf16, dev, "gate"),
         _dev_ptr(token_valid, u8, dev, "token_valid"), _dev_ptr(ckv, bf16, dev, "ckv"),
         _dev_ptr(ckv_codes, u8, dev, "ckv_codes"), _dev_ptr(ckv_scales, u8, dev, "ckv_scales"),
         int(cache_exp), _dev_ptr(kpool_out, bf16, dev, "kpool_out"),
         _dev_ptr(pool_valid, u8, dev, "pool_valid"), _dev_ptr(pool_idx, i32, dev, "pool_idx"),
         _dev_ptr(row_ctx, i32, dev, "row_ctx"), _dev_ptr(status, i32, dev, "status"))


def _append_guarded(refs, serving, latent: int, k_new, gate_new, ckv_new, ape, ln_w, ln_b, eps,
                    pg: DsaPaging, seq_lens, first_key, kpool, kvl: int, k_raw, gate, token_valid,
                    ckv, codes, scales, cache_exp, kpool_out, pool_valid, pool_idx, row_ctx,
                    status, stream) -> None:
    """The dsa_decode_append* of a pool with counts or a serving list."""
    batch, ihd = k_new.shape
    if batch != pg.batch:
        raise ValueError(f"one staged row per sequence: {batch} rows, {pg.batch} sequences")
    if refs is not None and refs.numel() != pg.num_blocks:
        raise ValueError(f"refs must be [{pg.num_blocks}]")
    if serving is not None and serving.numel() != pg.batch:
        raise ValueError(f"serving must be [{pg.batch}]")
    dev = _device_of(k_new, "k_new")
    _described(pg, dev, "pg")
    bf16, u8, i32, f32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
    _run(dev, stream, _lib.load().dsa_decode_append_guarded,
         _dev_ptr(refs, i32, dev, "refs"), _dev_ptr(serving, i32, dev, "serving"), latent,
         _dev_ptr(k_new, bf16, dev, "k_new"), _dev_ptr(gate_new, bf16, dev, "gate_new"),
         _dev_ptr(ckv_new, bf16, dev, "ckv_new"), _dev_ptr(ape, f32, dev, "ape"),
         _dev_ptr(ln_w, bf16, dev, "ln_w"), _dev_ptr(ln_b, bf16, dev, "ln_b"), float(eps),
         ctypes.byref(pg), _dev_ptr(seq_lens, i32, dev, "seq_lens"), int(first_key), int(kpool),
         ihd, kvl, _dev_ptr(k_raw, bf16, dev, "k_raw"), _dev_ptr(gate, bf16, dev, "gate"),
         _dev_ptr(token_valid, u8, dev, "token_valid"), _dev_ptr(ckv, bf16, dev, "ckv"),
         _dev_ptr(codes, u8, dev, "ckv_codes"),
         _dev_ptr(scales, f32 if latent == _lib.DSA_LATENT_FP8 else u8, dev, "ckv_scales"),
         int(cache_exp), _dev_ptr(kpool_out, bf16, dev, "kpool_out"),
         _dev_ptr(pool_valid, u8, dev, "pool_valid"), _dev_ptr(pool_idx, i32, dev, "pool_idx"),
         _dev_ptr(row_ctx, i32, dev, "row_ctx"), _dev_ptr(status, i32, dev, "status"))


def dsa_sparse_mla_decode_fp4_workspace(rows: int, heads: int, out_width: int, hidden: int,
                                        with_o_absorb: bool, kv_lora_rank: int = 512) -> int:
    n = ctypes.c_size_t(0)
    check(_lib.load().dsa_sparse_mla_decode_fp4_workspace(
        int(rows), int(heads), int(kv_lora_rank), int(out_width), int(hidden),
        1 if with_o_absorb else 0, ctypes.byref(n)))
    return int(n.value)


def dsa_sparse_mla_decode_fp4_splits(rows: int, heads: int, out_width: int, cache_rows: int,
                                     kv_lora_rank: int = 512) -> int:
    """Parts that dsa_sparse_mla_decode_fp4 cuts each row's tokens into (more than one: a
    second launch merges them)."""
    n = ctypes.c_int(0)
    check(_lib.load().dsa_sparse_mla_decode_fp4_splits(
        int(rows), int(heads), int(kv_lora_rank), int(out_width), int(cache_rows),
        ctypes.byref(n)))
    return int(n.value)


def dsa_sparse_mla_decode_fp4(qlat, row_seq, ckv_codes, ckv_scales, cache_exp: int,
                              pg: DsaPaging, token_ids, softmax_scale: float, o_absorb=None,
                              y=None, olat=None, status=None, workspace=None,
                              stream=None) -> None:
    """dsa_sparse_mla_decode over an FP4 latent cache (see dsa_quantize_latent_fp4).
    ``olat`` [rows, heads, 512] may be float32 or bfloat16."""
    rows, heads, kvl = qlat.shape
    if token_ids.dim() != 2 or token_ids.size(0) != rows:
        raise ValueError(f"token_ids must be [{rows}, out_width]")
    ow = token_ids.size(1)
    if _fp4_cache(ckv_codes, ckv_scales) != kvl:
        raise ValueError(f"ckv_codes must be [.., {kvl // 2}] and ckv_scales [.., {kvl // 16}]")
    _fp4_covers(ckv_codes, kvl, pg)
    if row_seq is not None and row_seq.numel() != rows:
        raise ValueError(f"row_seq must be [{rows}]")
    hidden = int(o_absorb.shape[0]) if o_absorb is not None else 0
    if o_absorb is not None and tuple(o_absorb.shape) != (hidden, heads * kvl):
        raise ValueError(f"o_absorb must be [hidden, {heads * kvl}]")
    if y is not None and tuple(y.shape) != (rows, hidden):
        raise ValueError(f"y must be [{rows}, {hidden}]")
    if olat is not None and olat.shape != qlat.shape:
        raise ValueError(f"olat must be [{rows}, {heads}, {kvl}]")
    if olat is not None and olat.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"olat must be float32 or bfloat16, got {olat.dtype}")
    dev = _device_of(ckv_codes, "ckv_codes")
    _described(pg, dev, "pg")
    bf16, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    p_olat = _dev_ptr(olat, None, dev, "olat")
    half = olat is not None and olat.dtype is bf16
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(dev, stream, _lib.load().dsa_sparse_mla_decode_fp4,
         _dev_ptr(qlat, bf16, dev, "qlat"), rows, heads, kvl, _dev_ptr(row_seq, i32, dev, "row_seq"),
         _dev_ptr(ckv_codes, u8, dev, "ckv_codes"), _dev_ptr(ckv_scales, u8, dev, "ckv_scales"),
         int(cache_exp), ctypes.byref(pg), _dev_ptr(token_ids, i32, dev, "token_ids"), ow,
         float(softmax_scale), _dev_ptr(o_absorb, bf16, dev, "o_absorb"), hidden,
         _ptr(y, bf16, "y", host_ok=True), None if half else p_olat, p_olat if half else None,
         _dev_ptr(status, i32, dev, "status"), _dev_ptr(workspace, None, dev, "workspace"), ws_bytes)


# -- pages -----------------------------------------------------------------


def page_arrays(caches, num_blocks: int) -> DsaPageArrays:
    """The paged caches that dsa_pages_reserve and dsa_pages_compact copy pages of: each a
    contiguous CUDA tensor [num_blocks, ...] of any type (see ``dsa_page_arrays`` in
    include/dsa.h). They must outlive every call that uses the returned descriptor."""
    caches = list(caches)
    if len(caches) > _lib.DSA_MAX_PAGE_ARRAYS:
        raise ValueError(f"{len(caches)} caches: at most {_lib.DSA_MAX_PAGE_ARRAYS}")
    pa = DsaPageArrays()
    pa.n, pa.num_pages = len(caches), int(num_blocks)
    if caches:
        pa.device = caches[0].get_device()  # beside the C fields: where the caches live
    for i, c in enumerate(caches):
        if c.dim() < 1 or int(c.shape[0]) != int(num_blocks):
            raise ValueError(f"cache {i} must be [{num_blocks}, ...], got {tuple(c.shape)}")
        pa.base[i] = _ptr(c, None, f"cache {i}")
        if c.get_device() != pa.device:
            raise ValueError(f"cache {i} is on {c.device}, cache 0 on cuda:{pa.device}: one "
                             "device per descriptor")
        pa.page_bytes[i] = c.numel() // int(num_blocks) * c.element_size()
    return pa


def dsa_pages_workspace(num_blocks: int, batch: int) -> int:
    n = ctypes.c_size_t(0)
    check(_lib.load().dsa_pages_workspace(int(num_blocks), int(batch), ctypes.byref(n)))
    return int(n.value)


def _pool(pg: DsaPaging, block_table, refs) -> int:
    """The pool's device."""
    if block_table.shape != (pg.batch, pg.max_blocks):
        raise ValueError(f"block_table must be [{pg.batch}, {pg.max_blocks}]")
    if refs.numel() != pg.num_blocks:
        raise ValueError(f"refs must be [{pg.num_blocks}]")
    dev = _device_of(refs, "refs")
    _described(pg, dev, "pg")
    return dev


def dsa_pages_free(seqs, pg: DsaPaging, block_table, seq_lens, refs, status=None,
                   stream=None) -> None:
    """End the listed sequences: their pages lose a reference, their rows become -1 and
    their lengths 0 (-1 entries of ``seqs`` are skipped)."""
    dev = _pool(pg, block_table, refs)
    i32 = torch.int32
    _run(dev, stream, _lib.load().dsa_pages_free,
         _dev_ptr(seqs, i32, dev, "seqs"), seqs.numel(), ctypes.byref(pg),
         _dev_ptr(block_table, i32, dev, "block_table"), _dev_ptr(seq_lens, i32, dev, "seq_lens"),
         _dev_ptr(refs, i32, dev, "refs"), _dev_ptr(status, i32, dev, "status"))


def dsa_pages_fork(parents, children, pg: DsaPaging, block_table, seq_lens, refs, status=None,
                   stream=None) -> None:
    """children[i] becomes a copy of parents[i] that shares its pages (-1 entries of
    ``children`` are skipped)."""
    dev = _pool(pg, block_table, refs)
    if parents.numel() != children.numel():
        raise ValueError("parents and children must have the same length")
    i32 = torch.int32
    _run(dev, stream, _lib.load().dsa_pages_fork,
         _dev_ptr(parents, i32, dev, "parents"), _dev_ptr(children, i32, dev, "children"),
         children.numel(), ctypes.byref(pg), _dev_ptr(block_table, i32, dev, "block_table"),
         _dev_ptr(seq_lens, i32, dev, "seq_lens"), _dev_ptr(refs, i32, dev, "refs"),
         _dev_ptr(status, i32, dev, "status"))


def dsa_pages_serve(seqs, serving, on: bool = True, parents=None, status=None,
                    stream=None) -> None:
    """Entry b of ``serving`` [batch] becomes b (``on``) or -1 for each listed sequence b:
    the list that dsa_pages_reserve takes as ``seqs`` and dsa_decode_append* as
    ``serving``. With ``parents``, ``seqs`` are the children of a dsa_pages_fork."""
    if parents is not None and parents.numel() != seqs.numel():
        raise ValueError("parents and seqs must have the same length")
    dev = _device_of(serving, "serving")
    i32 = torch.int32
    _run(dev, stream, _lib.load().dsa_pages_serve,
         _dev_ptr(parents, i32, dev, "parents"), _dev_ptr(seqs, i32, dev, "seqs"), seqs.numel(),
         serving.numel(), 1 if on else 0, _dev_ptr(serving, i32, dev, "serving"),
         _dev_ptr(status, i32, dev, "status"))


def dsa_pages_reserve(pg: DsaPaging, block_table, refs, new_tokens: int,
                      arrays: Optional[DsaPageArrays], first_key: int = 0, kpool: int = 0,
                      seqs=None, status=None, workspace=None, stream=None) -> None:
    """Room for the next ``new_tokens`` tokens of each listed sequence (all of them by
    default): free pages where none is mapped, private copies of shared ones."""
    dev = _pool(pg, block_table, refs)
    if seqs is not None and seqs.numel() == 0:
        return  # an empty list has no address: to the C call it would mean every sequence
    if arrays is not None:
        _described(arrays, dev, "arrays")
    i32 = torch.int32
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(dev, stream, _lib.load().dsa_pages_reserve,
         _dev_ptr(seqs, i32, dev, "seqs"), 0 if seqs is None else seqs.numel(), ctypes.byref(pg),
         _dev_ptr(block_table, i32, dev, "block_table"), _dev_ptr(refs, i32, dev, "refs"),
         int(new_tokens), int(first_key), int(kpool),
         None if arrays is None else ctypes.byref(arrays), _dev_ptr(status, i32, dev, "status"),
         _dev_ptr(workspace, None, dev, "workspace"), ws_bytes)


def dsa_pages_compact(pg: DsaPaging, block_table, refs, arrays: Optional[DsaPageArrays],
                      remap=None, live=None, status=None, workspace=None, stream=None) -> None:
    """Move the pool's live pages to its front and rewrite the block table."""
    dev = _pool(pg, block_table, refs)
    if remap is not None and remap.numel() != pg.num_blocks:
        raise ValueError(f"remap must be [{pg.num_blocks}]")
    if live is not None and live.numel() != 1:
        raise ValueError("live must hold one number")
    if arrays is not None:
        _described(arrays, dev, "arrays")
    i32 = torch.int32
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(dev, stream, _lib.load().dsa_pages_compact,
         ctypes.byref(pg), _dev_ptr(block_table, i32, dev, "block_table"),
         _dev_ptr(refs, i32, dev, "refs"), None if arrays is None else ctypes.byref(arrays),
         _dev_ptr(remap, i32, dev, "remap"), _dev_ptr(live, i32, dev, "live"),
         _dev_ptr(status, i32, dev, "status"), _dev_ptr(workspace, None, dev, "workspace"), ws_bytes)


def dsa_frontend_workspace(rows: int, hidden: int, n_x: int, q_lora_rank: int, kv_lora_rank: int,
                           ihd: int, index_heads: int, heads: int) -> int:
    n = ctypes.c_size_t(0)
    check(_lib.load().dsa_frontend_workspace(int(rows), int(hidden), int(n_x), int(q_lora_rank),
                                             int(kv_lora_rank), int(ihd), int(index_heads),
                                             int(heads), ctypes.byref(n)))
    return int(n.value)


def dsa_frontend(x, w_x, q_a_norm, kv_a_norm, eps: float, w_q, qlat, qidx, w, k_new, gate_new,
                 ckv_new, status=None, workspace=None, stream=None) -> None:
    """The step's inputs from the hidden state (see dsa_frontend in include/dsa.h):
    w_x packs the five x projections, w_q packs q_absorb over indexer.wq_b."""
    rows, hidden = (int(v) for v in x.shape)
    n_x = int(w_x.shape[0])
    ql, kvl = int(q_a_norm.numel()), int(kv_a_norm.numel())
    _, heads, kvl2 = (int(v) for v in qlat.shape)
    _, hi, ihd = (int(v) for v in qidx.shape)
    if kvl2 != kvl or tuple(w_x.shape) != (n_x, hidden):
        raise ValueError("qlat's width must be kv_lora_rank and w_x [n_x, hidden]")
    if tuple(w_q.shape) != (heads * kvl + hi * ihd, ql):
        raise ValueError("w_q must be [heads*kvl + index_heads*ihd, q_lora]")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(_lib.load().dsa_frontend(
        _ptr(x, torch.bfloat16, "x"), rows, hidden, _ptr(w_x, torch.bfloat16, "w_x"), n_x, ql, kvl,
        ihd, hi, _ptr(q_a_norm, torch.bfloat16, "q_a_norm"),
        _ptr(kv_a_norm, torch.bfloat16, "kv_a_norm"), float(eps),
        _ptr(w_q, torch.bfloat16, "w_q"), heads,
        _ptr(qlat, torch.bfloat16, "qlat"), _ptr(qidx, torch.bfloat16, "qidx"),
        _ptr(w, torch.float32, "w"), _ptr(k_new, torch.bfloat16, "k_new"),
        _ptr(gate_new, torch.bfloat16, "gate_new"), _ptr(ckv_new, torch.bfloat16, "ckv_new"),
        _ptr(status, torch.int32, "status"), _ptr(workspace, None, "workspace"), ws_bytes,
        _stream(stream)))


def dsa_rmsnorm(x, weight, eps: float, out=None, residual=None, residual_out=None, codes=None,
                scales=None, stream=None) -> None:
    """RMS norm of x + residual (x alone without one) into ``out`` (bf16) and/or the FP8 rows
    ``codes``, ``scales``; the sum itself into ``residual_out`` (which may be ``residual``)."""
    shape = x.shape
    width = shape[-1]
    if (weight.numel() != width or (out is not None and out.shape != shape)
            or (residual is not None and residual.shape != shape)
            or (residual_out is not None and residual_out.shape != shape)):
        raise ValueError(f"weight must be [{width}]; out, residual and residual_out must be "
                         f"{tuple(shape)} as x")
    if codes is not None and scales is not None and (codes.shape != shape
                                                     or _fp8_rows(codes, scales) != width):
        raise ValueError(f"codes must be {tuple(shape)} as x")
    dev = _device_of(x, "x")
    bf16 = torch.bfloat16
    _run(dev, stream, _lib.load().dsa_rmsnorm,
         _dev_ptr(x, bf16, dev, "x"), _dev_ptr(residual, bf16, dev, "residual"),
         _dev_ptr(weight, bf16, dev, "weight"), x.numel() // width if width else 0, width,
         eps, _dev_ptr(residual_out, bf16, dev, "residual_out"),
         _dev_ptr(out, bf16, dev, "out"), _dev_ptr(codes, torch.uint8, dev, "codes"),
         _dev_ptr(scales, torch.float32, dev, "scales"))


def dsa_router_logits_workspace(rows: int, hidden: int, n: int) -> int:
    b = ctypes.c_size_t(0)
    check(_lib.load().dsa_router_logits_workspace(int(rows), int(hidden), int(n), ctypes.byref(b)))
    return int(b.value)


def dsa_router_logits(x, w, logits, status=None, workspace=None, stream=None) -> None:
    """logits = x @ w.T with f32 results (x, w bf16; w's rows padded to a multiple of 64)."""
    rows, hidden = x.shape
    n = w.size(0)
    if w.shape != (n, hidden) or logits.shape != (rows, n):
        raise ValueError(f"w must be [n, {hidden}] and logits [{rows}, n]")
    dev = _device_of(x, "x")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(dev, stream, _lib.load().dsa_router_logits,
         _dev_ptr(x, torch.bfloat16, dev, "x"), rows, hidden, _dev_ptr(w, torch.bfloat16, dev, "w"),
         n, _dev_ptr(logits, torch.float32, dev, "logits"),
         _dev_ptr(status, torch.int32, dev, "status"), _dev_ptr(workspace, None, dev, "workspace"),
         ws_bytes)


_ROUTE_SCORE = {"sigmoid": _lib.DSA_ROUTE_SIGMOID, "softmax": _lib.DSA_ROUTE_SOFTMAX}


def dsa_route(logits, topk: int, ids, weights, n_experts: Optional[int] = None,
              score: str = "sigmoid", bias=None, n_group: int = 1, topk_group: int = 1,
              group_top: int = 2, renorm: bool = True, scale: float = 1.0, shared: int = 0,
              stream=None) -> None:
    """The ``topk`` experts of each row of logits and their weights, then ``shared`` ones that
    every row takes (see dsa_route in include/dsa.h). The row's first ``n_experts`` logits
    count (all of them by default)."""
    rows, ld = logits.shape
    n = ld if n_experts is None else int(n_experts)
    if n > ld:
        raise ValueError(f"logits hold {ld} of {n} experts")
    if score not in _ROUTE_SCORE:
        raise ValueError(f"score {score!r}: one of {sorted(_ROUTE_SCORE)}")
    if bias is not None and bias.numel() != n:
        raise ValueError(f"bias must be [{n}]")
    width = (rows, int(topk) + int(shared))
    if ids.shape != width or weights.shape != width:
        raise ValueError(f"ids and weights must be {list(width)}")
    dev = _device_of(logits, "logits")
    f32 = torch.float32
    _run(dev, stream, _lib.load().dsa_route,
         _dev_ptr(logits, f32, dev, "logits"), rows, n, ld, _ROUTE_SCORE[score],
         _dev_ptr(bias, f32, dev, "bias"), int(n_group), int(topk_group), int(group_top), int(topk),
         1 if renorm else 0, float(scale), int(shared), _dev_ptr(ids, torch.int32, dev, "ids"),
         _dev_ptr(weights, f32, dev, "weights"))


def dsa_experts_workspace(rows: int, topk: int, n_experts: int, hidden: int, inter: int,
                          fp8: bool = False) -> int:
    b = ctypes.c_size_t(0)
    check(_lib.load().dsa_experts_workspace(int(rows), int(topk), int(n_experts), int(hidden),
                                            int(inter), 1 if fp8 else 0, ctypes.byref(b)))
    return int(b.value)


def dsa_experts(x, ids, weights, w13, w2, y, x_scales=None, w13_scales=None, w2_scales=None,
                status=None, workspace=None, stream=None) -> None:
    """The weighted sum of each row's experts' gated products (see dsa_experts in
    include/dsa.h): x, w13, w2 in bf16, or FP8 codes (u8) with their scales."""
    rows, hidden = x.shape
    topk = ids.size(-1)
    n, _, inter = w2.shape
    if w13.shape != (n, 2 * inter, hidden) or w2.size(1) != hidden:
        raise ValueError(f"w13 must be [n, 2 inter, {hidden}] and w2 [n, {hidden}, inter]")
    if ids.shape != (rows, topk) or weights.shape != (rows, topk):
        raise ValueError(f"ids and weights must be [{rows}, topk]")
    if y.shape != (rows, hidden):
        raise ValueError(f"y must be [{rows}, {hidden}]")
    dt = torch.bfloat16
    if x_scales is not None or w13_scales is not None or w2_scales is not None:
        if x_scales is None or w13_scales is None or w2_scales is None:
            raise ValueError("FP8 takes the scales of x, w13 and w2, bf16 none")
        dt = torch.uint8
        if (x_scales.shape != (rows, hidden // 128) or w13_scales.shape != (n, 2 * inter, hidden // 128)
                or w2_scales.shape != (n, hidden, inter // 128)):
            raise ValueError("the scales must be [.., width/128] of the same rows as the codes")
    dev = _device_of(x, "x")
    f32 = torch.float32
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(dev, stream, _lib.load().dsa_experts,
         _dev_ptr(x, dt, dev, "x"), _dev_ptr(x_scales, f32, dev, "x_scales"), rows, hidden,
         _dev_ptr(ids, torch.int32, dev, "ids"), _dev_ptr(weights, f32, dev, "weights"), topk,
         _dev_ptr(w13, dt, dev, "w13"), _dev_ptr(w13_scales, f32, dev, "w13_scales"),
         _dev_ptr(w2, dt, dev, "w2"), _dev_ptr(w2_scales, f32, dev, "w2_scales"), n, inter,
         _dev_ptr(y, torch.bfloat16, dev, "y"), _dev_ptr(status, torch.int32, dev, "status"),
         _dev_ptr(workspace, None, dev, "workspace"), ws_bytes)


def dsa_latent_project_workspace(rows: int, heads: int, hidden: int,
                                 kv_lora_rank: int = 512) -> int:
    n = ctypes.c_size_t(0)
    check(_lib.load().dsa_latent_project_workspace(int(rows), int(heads), int(kv_lora_rank),
                                                   int(hidden), ctypes.byref(n)))
    return int(n.value)


def dsa_prefetch_l2(t: torch.Tensor, nbytes: Optional[int] = None, stream=None) -> None:
    """Bring the first nbytes of device tensor t (all of it by default) into L2: a hint
    issued beside latency-bound work, e.g. on a second stream."""
    total = t.numel() * t.element_size()
    n = total if nbytes is None else min(int(nbytes), total)
    check(_lib.load().dsa_prefetch_l2(_ptr(t, None, "t"), n, _stream(stream)))


def dsa_latent_project(olat, o_absorb, y, status=None, workspace=None, stream=None) -> None:
    """y = bf16(o_absorb @ bf16(olat)) per row; olat [rows, heads, 512] f32."""
    rows, heads, kvl = (int(x) for x in olat.shape)
    hidden = int(o_absorb.shape[0])
    if tuple(o_absorb.shape) != (hidden, heads * kvl) or tuple(y.shape) != (rows, hidden):
        raise ValueError("o_absorb must be [hidden, heads*kvl] and y [rows, hidden]")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(_lib.load().dsa_latent_project(
        _ptr(olat, torch.float32, "olat"), rows, heads, kvl, _ptr(o_absorb, torch.bfloat16, "o_absorb"),
        hidden, _ptr(y, torch.bfloat16, "y", host_ok=True), _ptr(status, torch.int32, "status"),
        _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream)))


def dsa_sparse_mla_decode_noalloc(qlat, row_seq, ckv, pg: DsaPaging, token_ids,
                                  softmax_scale: float, o_absorb=None, y=None, olat=None,
                                  status=None, stream=None) -> None:
    """dsa_sparse_mla_decode without a workspace: the library's fixed scratch array
    is used instead (for hosts that cannot allocate device memory; see
    include/dsa.h). Calls whose GPU work overlaps in time must be serialised."""
    rows, heads, kvl = (int(x) for x in qlat.shape)
    ow = int(token_ids.shape[1])
    hidden = int(o_absorb.shape[0]) if o_absorb is not None else 0
    check(_lib.load().dsa_sparse_mla_decode_noalloc(
        _ptr(qlat, torch.bfloat16, "qlat"), rows, heads, kvl,
        _ptr(row_seq, torch.int32, "row_seq"), _ptr(ckv, torch.bfloat16, "ckv"),
        ctypes.byref(pg), _ptr(token_ids, torch.int32, "token_ids"), ow, float(softmax_scale),
        _ptr(o_absorb, torch.bfloat16, "o_absorb"), hidden, _ptr(y, torch.bfloat16, "y", host_ok=True),
        _ptr(olat, torch.float32, "olat"), _ptr(status, torch.int32, "status"),
        _stream(stream)))
