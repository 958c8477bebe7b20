"""Thin PyTorch binding of libidx (include/idx.h).

Every function checks tensor dtypes, devices and shapes, then passes raw
device pointers and the current CUDA stream to the C entry point of the same
name.  All arithmetic happens in the library's kernels; if the library is
missing the import fails loudly (there is no fallback).
"""
from __future__ import annotations

import collections
import ctypes
import math
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libidx.so")

IDX_OK = 0
STATUS_NAMES = {0: "IDX_OK", 1: "IDX_ERR_INVALID_ARG", 2: "IDX_ERR_UNSUPPORTED_DEVICE",
                3: "IDX_ERR_WORKSPACE_TOO_SMALL", 4: "IDX_ERR_CUDA"}
HEAD_DIM = 128
PAGE_SIZE = 64
PAGE_BYTES = PAGE_SIZE * 68

# Every symbol include/idx.h declares, with (restype, argtypes).
_P = ctypes.c_void_p
_I64, _I32, _SZ = ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_F32, _F64 = ctypes.c_float, ctypes.c_double
SIGNATURES = {
    "idx_version": (ctypes.c_int, []),
    "idx_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "idx_last_error_detail": (ctypes.c_char_p, []),
    "idx_arch_supported": (ctypes.c_int, [ctypes.c_int, ctypes.c_int]),
    "idx_check_device": (ctypes.c_int, [ctypes.c_int]),
    "idx_quant_insert": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _I64, _I32, _P, _P]),
    "idx_quant_q": (ctypes.c_int, [_P, _I64, _P, _P, _P]),
    "idx_paged_mqa_logits": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _I64, _I32, _P, _I32,
                                            _P, _P, _P, _I64, ctypes.c_int, _P, _P]),
    "idx_mqa_logits": (ctypes.c_int, [_P, _P, _I64, _I32, _P, _P, _I64, _P, _P, _P, _P, _I64,
                                      ctypes.c_int, _P, _P]),
    "idx_topk_rows": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _I32, _P, _P]),
    "idx_paged_logits_topk_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "idx_paged_logits_topk": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _I64, _I32, _P, _I32,
                                             _P, _P, _I32, _P, _P, _SZ, _P, _P]),
    "idx_gather_k": (ctypes.c_int, [_P, _I64, _I32, _P, _I32, _P, _P, _I32, _P, _P, _I64, _P,
                                    _P]),
    "idx_paged_logits_topk_noalloc": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _I64, _I32, _P,
                                                     _I32, _P, _P, _I32, _P, _P, _P]),
    "idx_paged_decode_step_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "idx_paged_decode_step": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _I64, _I32, _P, _I32,
                                             _P, _P, _I32, _P, _P, _SZ, _P, _P]),
    "idx_mqa_logits_topk_workspace_bytes": (_SZ, [_I64, _I64, _I32]),
    "idx_mqa_logits_topk": (ctypes.c_int, [_P, _P, _I64, _I32, _P, _P, _I64, _P, _P, _P, _I32, _P,
                                           _P, _SZ, _P, _P]),
    "idx_rope_quant_q": (ctypes.c_int, [_P, _I64, _I32, _P, _P, _P, _I32, _I32, _P, _P, _P, _P]),
    "idx_kpool_insert": (ctypes.c_int, [_P, _P, _P, _P, _I64, _I32, _P, _I64, _I32, _P, _P, _P]),
    "idx_copy_async": (ctypes.c_int, [_P, _P, _SZ, _P]),
    "idx_plan_step": (ctypes.c_int, [_P, _P, _I32, _P, _I32, _P, _I32, _P, _P, _I64, _I32, _P, _P,
                                     _P, _P, _P, _I64, _P, _P]),
    "idx_rope_table": (ctypes.c_int, [_I64, _I64, _I32, _F64, _I32, _F64, _F64, _F64, _F64, _F64,
                                      _P, _P, _P]),
    "idx_qk_norm_rope_insert": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64,
                                               _I64, _I32, _I32, _P, _P, _F32, _P, _P, _P, _I64,
                                               _I32, _I32, _P, _P, _P, _P, _P]),
    "idx_paged_attention_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "idx_paged_attention_form": (ctypes.c_int, [_I32] * 11 + [_P]),
    "idx_paged_attention": (ctypes.c_int, [_P, _I64, _I64, _I32, _I32, _I32, _I32, _P, _P, _I32,
                                           _P, _P, _I32, _F32, _F32, _I32, _P, _P, _P, _SZ, _P,
                                           _P]),
}


class KvCacheStruct(ctypes.Structure):
    """idx_kv_cache of include/idx.h."""
    _fields_ = ([(n, _P) for n in ("k", "v", "k_scale", "v_scale")]
                + [(n, _I64) for n in ("num_blocks", "k_block_stride", "k_head_stride",
                                       "k_token_stride", "v_block_stride", "v_head_stride",
                                       "v_token_stride")]
                + [(n, _I32) for n in ("page_size", "heads", "head_dim", "dtype")])


class IdxError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {detail}")
        self.status = status
        self.detail = detail


def load_library(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: the CUDA library must be built first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = load_library()


def _check(fn: str, status: int):
    if status != IDX_OK:
        raise IdxError(fn, status, lib.idx_last_error_detail().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, name, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def new_errors(device=None) -> torch.Tensor:
    """A zeroed idx_device_errors struct: int32 [bad_inputs, timeouts]."""
    return torch.zeros(2, dtype=torch.int32, device=device or "cuda")


def arch_supported(major: int, minor: int) -> bool:
    return lib.idx_arch_supported(major, minor) == IDX_OK


def check_device(device: int = 0) -> None:
    _check("idx_check_device", lib.idx_check_device(device))


def new_cache(num_blocks: int, device=None) -> torch.Tensor:
    return torch.zeros((num_blocks, PAGE_BYTES), dtype=torch.uint8, device=device or "cuda")


def quant_insert(k: torch.Tensor, slot_mapping: torch.Tensor, kcache: torch.Tensor,
                 errors: torch.Tensor | None = None, stream=None) -> None:
    """Quantise k ([N, >=128] bf16, row-major, rows may be strided) to MXFP4 and
    scatter into kcache ([num_blocks, 4352] uint8) at slot_mapping ([N] int64)."""
    _need(k, torch.bfloat16, "k", contiguous=False)
    _need(slot_mapping, torch.int64, "slot_mapping")
    _need(kcache, torch.uint8, "kcache")
    if k.dim() != 2 or k.stride(1) != 1 or k.shape[1] < HEAD_DIM:
        raise ValueError("k must be [N, >=128] with unit stride in the last dim")
    n = k.shape[0]
    if slot_mapping.numel() != n:
        raise ValueError("slot_mapping must have one entry per row of k")
    if kcache.dim() != 2 or kcache.shape[1] != PAGE_BYTES:
        raise ValueError("kcache must be [num_blocks, 4352]")
    stride = k.stride(0) if n > 1 else max(k.stride(0), HEAD_DIM)
    _check("idx_quant_insert", lib.idx_quant_insert(
        _ptr(k), n, stride, _ptr(slot_mapping), _ptr(kcache), kcache.shape[0], PAGE_SIZE,
        _ptr(errors), _stream(stream)))


def quant_q(q: torch.Tensor, out_vals=None, out_scales=None, stream=None):
    """q [..., 128] bf16 -> (vals [rows, 64] uint8, scales [rows, 4] uint8)."""
    _need(q, torch.bfloat16, "q")
    if q.shape[-1] != HEAD_DIM:
        raise ValueError("q must end in 128")
    rows = q.numel() // HEAD_DIM
    vals = out_vals if out_vals is not None else torch.empty((rows, 64), dtype=torch.uint8,
                                                             device=q.device)
    scales = out_scales if out_scales is not None else torch.empty((rows, 4), dtype=torch.uint8,
                                                                   device=q.device)
    _check("idx_quant_q", lib.idx_quant_q(_ptr(q), rows, _ptr(vals), _ptr(scales),
                                          _stream(stream)))
    return vals, scales


def rope_quant_q(q: torch.Tensor, positions: torch.Tensor, cos: torch.Tensor | None,
                 sin: torch.Tensor | None, rot_dim: int, out_vals=None, out_scales=None,
                 errors=None, stream=None):
    """Rotary embedding of q ([T, H, 128] bf16) by table rows positions ([T]
    int32) of cos/sin ([num_pos, rot_dim/2] fp32), fused with the MXFP4
    quantisation: (vals [T*H, 64] uint8, scales [T*H, 4] uint8)."""
    _need(q, torch.bfloat16, "q")
    _need(positions, torch.int32, "positions")
    if q.dim() != 3 or q.shape[2] != HEAD_DIM:
        raise ValueError("q must be [T, H, 128]")
    T, H = q.shape[0], q.shape[1]
    if positions.numel() != T:
        raise ValueError("positions must have one entry per token")
    num_pos = 0
    if rot_dim > 0:
        _need(cos, torch.float32, "cos")
        _need(sin, torch.float32, "sin")
        if cos.shape != sin.shape or cos.dim() != 2 or cos.shape[1] != rot_dim // 2:
            raise ValueError("cos/sin must be [num_pos, rot_dim / 2]")
        num_pos = cos.shape[0]
    rows = T * H
    vals = out_vals if out_vals is not None else torch.empty((rows, 64), dtype=torch.uint8,
                                                             device=q.device)
    scales = out_scales if out_scales is not None else torch.empty((rows, 4), dtype=torch.uint8,
                                                                   device=q.device)
    _check("idx_rope_quant_q", lib.idx_rope_quant_q(
        _ptr(q), T, H, _ptr(positions), _ptr(cos) if rot_dim > 0 else None,
        _ptr(sin) if rot_dim > 0 else None, num_pos, rot_dim, _ptr(vals), _ptr(scales),
        _ptr(errors), _stream(stream)))
    return vals, scales


def kpool_insert(k: torch.Tensor, gate: torch.Tensor, ape: torch.Tensor,
                 slot_mapping: torch.Tensor, kcache: torch.Tensor, pooled=None, errors=None,
                 stream=None) -> None:
    """K-pool compressed insert: pools of kpool = ape.shape[0] keys of k
    ([n, 128] bf16) weighted by a softmax of gate ([n, 128] fp32) plus ape
    ([kpool, 128] fp32), written as MXFP4 keys at the pool-granular
    slot_mapping ([n] int64) of kcache; pooled ([n, 128] fp32, optional)
    receives the pooled vectors of the written rows."""
    _need(k, torch.bfloat16, "k")
    _need(gate, torch.float32, "gate")
    _need(ape, torch.float32, "ape")
    _need(slot_mapping, torch.int64, "slot_mapping")
    _need(kcache, torch.uint8, "kcache")
    n = k.shape[0]
    if k.dim() != 2 or k.shape[1] != HEAD_DIM or gate.shape != k.shape:
        raise ValueError("k and gate must be [n, 128]")
    if ape.dim() != 2 or ape.shape[1] != HEAD_DIM or slot_mapping.numel() != n:
        raise ValueError("ape must be [kpool, 128] and slot_mapping [n]")
    if pooled is not None:
        _need(pooled, torch.float32, "pooled")
        if pooled.shape != k.shape:
            raise ValueError("pooled must be [n, 128]")
    _check("idx_kpool_insert", lib.idx_kpool_insert(
        _ptr(k), _ptr(gate), _ptr(ape), _ptr(slot_mapping), n, ape.shape[0], _ptr(kcache),
        kcache.shape[0], PAGE_SIZE, _ptr(pooled), _ptr(errors), _stream(stream)))


def _paged_common(q_vals, q_scales, weights, kcache, block_table, context_lens, next_n, H):
    _need(q_vals, torch.uint8, "q_vals")
    _need(q_scales, torch.uint8, "q_scales")
    _need(weights, torch.float32, "weights")
    _need(kcache, torch.uint8, "kcache")
    _need(block_table, torch.int32, "block_table")
    _need(context_lens, torch.int32, "context_lens")
    B = context_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks]")
    if weights.numel() != B * next_n * H or q_vals.numel() != B * next_n * H * 64:
        raise ValueError("q/weights do not match B * next_n * H")
    return B, block_table.shape[1]


def paged_mqa_logits(q_vals, q_scales, weights, kcache, block_table, context_lens, next_n: int,
                     H: int, ld: int | None = None, clean: bool = False, out=None, errors=None,
                     stream=None):
    B, max_blocks = _paged_common(q_vals, q_scales, weights, kcache, block_table, context_lens,
                                  next_n, H)
    if ld is None:
        ld = max_blocks * PAGE_SIZE
    logits = out if out is not None else torch.empty((B * next_n, ld), dtype=torch.float32,
                                                     device=q_vals.device)
    _check("idx_paged_mqa_logits", lib.idx_paged_mqa_logits(
        _ptr(q_vals), _ptr(q_scales), B, next_n, H, _ptr(kcache), kcache.shape[0], PAGE_SIZE,
        _ptr(block_table), max_blocks, _ptr(context_lens), _ptr(weights), _ptr(logits), ld,
        1 if clean else 0, _ptr(errors), _stream(stream)))
    return logits


def paged_logits_topk_workspace_bytes(B: int, next_n: int, max_blocks: int, k: int) -> int:
    return int(lib.idx_paged_logits_topk_workspace_bytes(B, next_n, max_blocks, PAGE_SIZE, k))


def new_paged_topk_workspace(B: int, next_n: int, max_blocks: int, k: int, device=None):
    n = paged_logits_topk_workspace_bytes(B, next_n, max_blocks, k)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def paged_logits_topk(q_vals, q_scales, weights, kcache, block_table, context_lens, next_n: int,
                      H: int, k: int = 2048, workspace=None, out=None, errors=None, stream=None):
    B, max_blocks = _paged_common(q_vals, q_scales, weights, kcache, block_table, context_lens,
                                  next_n, H)
    if workspace is None:
        workspace = new_paged_topk_workspace(B, next_n, max_blocks, k, q_vals.device)
    _need(workspace, torch.uint8, "workspace")
    idx = out if out is not None else torch.empty((B * next_n, k), dtype=torch.int32,
                                                  device=q_vals.device)
    _check("idx_paged_logits_topk", lib.idx_paged_logits_topk(
        _ptr(q_vals), _ptr(q_scales), B, next_n, H, _ptr(kcache), kcache.shape[0], PAGE_SIZE,
        _ptr(block_table), max_blocks, _ptr(context_lens), _ptr(weights), k, _ptr(idx),
        _ptr(workspace), workspace.numel(), _ptr(errors), _stream(stream)))
    return idx


def paged_logits_topk_noalloc(q_vals, q_scales, weights, kcache, block_table, context_lens,
                              next_n: int, H: int, k: int = 2048, out=None, errors=None,
                              stream=None):
    """idx_paged_logits_topk_noalloc: the fused decode path with the library's
    built-in 32 MiB scratch instead of a caller workspace (for callers that
    cannot allocate device memory)."""
    B, max_blocks = _paged_common(q_vals, q_scales, weights, kcache, block_table, context_lens,
                                  next_n, H)
    idx = out if out is not None else torch.empty((B * next_n, k), dtype=torch.int32,
                                                  device=q_vals.device)
    _check("idx_paged_logits_topk_noalloc", lib.idx_paged_logits_topk_noalloc(
        _ptr(q_vals), _ptr(q_scales), B, next_n, H, _ptr(kcache), kcache.shape[0], PAGE_SIZE,
        _ptr(block_table), max_blocks, _ptr(context_lens), _ptr(weights), k, _ptr(idx),
        _ptr(errors), _stream(stream)))
    return idx


def paged_decode_step_workspace_bytes(B: int, next_n: int, H: int, max_blocks: int,
                                      k: int) -> int:
    return int(lib.idx_paged_decode_step_workspace_bytes(B, next_n, H, max_blocks, PAGE_SIZE, k))


def paged_decode_step(k_new, q, weights, kcache, block_table, context_lens, next_n: int, H: int,
                      k: int = 2048, workspace=None, out=None, errors=None, stream=None):
    """One decode step: insert the step's new keys (k_new [B*next_n, 128] bf16,
    at positions L_b - next_n + j through the block table), quantise its query
    heads (q [B*next_n, H, 128] bf16) and return the top-k of every row
    ([B*next_n, k] int32), in two launches."""
    _need(k_new, torch.bfloat16, "k_new")
    _need(q, torch.bfloat16, "q")
    _need(weights, torch.float32, "weights")
    _need(kcache, torch.uint8, "kcache")
    _need(block_table, torch.int32, "block_table")
    _need(context_lens, torch.int32, "context_lens")
    B = context_lens.numel()
    max_blocks = block_table.shape[1]
    if k_new.numel() != B * next_n * HEAD_DIM or q.numel() != B * next_n * H * HEAD_DIM:
        raise ValueError("k_new / q do not match B * next_n (* H) rows of 128")
    if weights.numel() != B * next_n * H:
        raise ValueError("weights must be [B * next_n, H]")
    if workspace is None:
        n = paged_decode_step_workspace_bytes(B, next_n, H, max_blocks, k)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    _need(workspace, torch.uint8, "workspace")
    idx = out if out is not None else torch.empty((B * next_n, k), dtype=torch.int32,
                                                  device=q.device)
    _check("idx_paged_decode_step", lib.idx_paged_decode_step(
        _ptr(k_new), _ptr(q), B, next_n, H, _ptr(kcache), kcache.shape[0], PAGE_SIZE,
        _ptr(block_table), max_blocks, _ptr(context_lens), _ptr(weights), k, _ptr(idx),
        _ptr(workspace), workspace.numel(), _ptr(errors), _stream(stream)))
    return idx


def mqa_logits(q_vals, q_scales, weights, k_vals, k_scales, row_start, row_end, H: int,
               ld: int | None = None, clean: bool = False, out=None, errors=None, stream=None):
    _need(q_vals, torch.uint8, "q_vals")
    _need(q_scales, torch.uint8, "q_scales")
    _need(k_vals, torch.uint8, "k_vals")
    _need(k_scales, torch.uint8, "k_scales")
    _need(weights, torch.float32, "weights")
    _need(row_start, torch.int32, "row_start")
    _need(row_end, torch.int32, "row_end")
    T = row_end.numel()
    S = k_vals.numel() // 64
    if ld is None:
        ld = S
    logits = out if out is not None else torch.empty((T, ld), dtype=torch.float32,
                                                     device=q_vals.device)
    _check("idx_mqa_logits", lib.idx_mqa_logits(
        _ptr(q_vals), _ptr(q_scales), T, H, _ptr(k_vals), _ptr(k_scales), S, _ptr(weights),
        _ptr(row_start), _ptr(row_end), _ptr(logits), ld, 1 if clean else 0, _ptr(errors),
        _stream(stream)))
    return logits


def mqa_logits_topk_workspace_bytes(T: int, S: int, k: int) -> int:
    return int(lib.idx_mqa_logits_topk_workspace_bytes(T, S, k))


def mqa_logits_topk(q_vals, q_scales, weights, k_vals, k_scales, row_start, row_end, H: int,
                    k: int = 2048, workspace=None, out=None, errors=None, stream=None):
    """Prefill logits + top-k of every row without a logits tensor:
    [T, k] int32 positions relative to row_start (-1 padded)."""
    _need(q_vals, torch.uint8, "q_vals")
    _need(q_scales, torch.uint8, "q_scales")
    _need(k_vals, torch.uint8, "k_vals")
    _need(k_scales, torch.uint8, "k_scales")
    _need(weights, torch.float32, "weights")
    _need(row_start, torch.int32, "row_start")
    _need(row_end, torch.int32, "row_end")
    T = row_end.numel()
    S = k_vals.numel() // 64
    if workspace is None:
        workspace = torch.empty(max(mqa_logits_topk_workspace_bytes(T, S, k), 256),
                                dtype=torch.uint8, device=q_vals.device)
    _need(workspace, torch.uint8, "workspace")
    idx = out if out is not None else torch.empty((T, k), dtype=torch.int32, device=q_vals.device)
    _check("idx_mqa_logits_topk", lib.idx_mqa_logits_topk(
        _ptr(q_vals), _ptr(q_scales), T, H, _ptr(k_vals), _ptr(k_scales), S, _ptr(weights),
        _ptr(row_start), _ptr(row_end), k, _ptr(idx), _ptr(workspace), workspace.numel(),
        _ptr(errors), _stream(stream)))
    return idx


def topk_rows(logits, row_end, k: int = 2048, row_start=None, out=None, stream=None):
    _need(logits, torch.float32, "logits", contiguous=False)
    _need(row_end, torch.int32, "row_end")
    if row_start is not None:
        _need(row_start, torch.int32, "row_start")
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be 2-D with unit column stride")
    rows = logits.shape[0]
    idx = out if out is not None else torch.empty((rows, k), dtype=torch.int32,
                                                  device=logits.device)
    _check("idx_topk_rows", lib.idx_topk_rows(_ptr(logits), rows, logits.stride(0),
                                              _ptr(row_start), _ptr(row_end), k, _ptr(idx),
                                              _stream(stream)))
    return idx


def gather_k(kcache, block_table, seq_lens, out_offsets, out_rows: int, errors=None,
             stream=None):
    _need(kcache, torch.uint8, "kcache")
    _need(block_table, torch.int32, "block_table")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(out_offsets, torch.int64, "out_offsets")
    B = seq_lens.numel()
    vals = torch.empty((out_rows, 64), dtype=torch.uint8, device=kcache.device)
    scales = torch.empty((out_rows, 4), dtype=torch.uint8, device=kcache.device)
    _check("idx_gather_k", lib.idx_gather_k(
        _ptr(kcache), kcache.shape[0], PAGE_SIZE, _ptr(block_table), block_table.shape[1],
        _ptr(seq_lens), _ptr(out_offsets), B, _ptr(vals), _ptr(scales), out_rows,
        _ptr(errors), _stream(stream)))
    return vals, scales


def copy_async(dst: torch.Tensor, src: torch.Tensor, stream=None) -> None:
    """Copy src into dst (both contiguous, the same number of bytes; each a CUDA
    tensor of the current device or a pinned CPU tensor) with the GPU's SMs,
    enqueued on `stream`."""
    for t, name in ((dst, "dst"), (src, "src")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{name} must be a CUDA tensor or a pinned CPU tensor")
    n = dst.numel() * dst.element_size()
    if src.numel() * src.element_size() != n:
        raise ValueError("dst and src must hold the same number of bytes")
    _check("idx_copy_async", lib.idx_copy_async(_ptr(dst), _ptr(src), n, _stream(stream)))


# ---------------------------------------------------------------- serving operators

ROPE_SCALINGS = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3}

StepPlan = collections.namedtuple(
    "StepPlan", "context_lens query_start slot_mapping positions token_seq pool_head")


class _NoServing:
    """In the place of the compiled part where it is missing or does not load: the
    other entries, which need ctypes alone, work; every serving call fails."""

    def __init__(self, why: Exception):
        self._why = why

    def __getattr__(self, name):
        raise RuntimeError(
            f"{name}: the serving binding is missing or does not load: build it first "
            "(python -c 'import __graft_entry__ as g; g.build()')") from self._why


def _load_serving():
    try:
        from . import _serving
    except ImportError as e:
        return _NoServing(e)
    _serving.set_errors(IdxError, torch.OutOfMemoryError)
    return _serving


# Checks, allocation and marshalling of the serving entries (csrc/serving_py.cpp).
# Outputs and workspaces are allocated on the stream of the call: their memory
# can then neither be taken from work still pending on another stream nor be
# reused before the call is done.
_serving = _load_serving()


def _call(fn, stream, *args):
    if stream is None:
        return fn(*args)
    with torch.cuda.stream(stream):
        return fn(*args)


def plan_step(cached_lens, new_lens, block_table, free_pages, pool_head, num_tokens: int,
              num_blocks: int, page_size: int = PAGE_SIZE, out: StepPlan | None = None,
              errors=None, stream=None) -> StepPlan:
    """Block tables, slot maps and positions of a step from request lengths.

    cached_lens, new_lens [B] int32; block_table [B, max_blocks] int32 (the
    entries of newly opened pages are written); free_pages [num_free] int32,
    taken from entry pool_head ([1] int32) on.  Returns the step's context_lens
    [B], query_start [B+1], slot_mapping [num_tokens] (int64), positions and
    token_seq [num_tokens], and the advanced pool_head [1] (all int32 but the
    slots); num_tokens may exceed the step's tokens (slot -1, position 0 and
    request -1 past them).  `out`: an earlier plan to write into; its
    context_lens may be cached_lens (advanced in place), other arrays must not
    overlap."""
    return StepPlan(*_call(_serving.plan_step, stream, cached_lens, new_lens, block_table,
                           free_pages, pool_head, num_tokens, num_blocks, page_size, out, errors))


def rope_table(num_pos: int, rot_dim: int, base: float = 10000.0, scaling: str | None = None,
               factor: float = 1.0, orig_len: int = 0, beta_fast: float = 32.0,
               beta_slow: float = 1.0, mscale: float | None = None, pos0: int = 0, out=None,
               stream=None):
    """Rotary tables (cos, sin), each [num_pos, rot_dim/2] fp32, for positions
    pos0 on.  scaling: None, "linear", "ntk" or "yarn" (which needs orig_len,
    the length the frequencies were trained for).  mscale multiplies every
    entry; by default 1, or 0.1 ln(factor) + 1 with "yarn" and a factor above 1."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(filter(None, ROPE_SCALINGS))} or None")
    if mscale is None:
        mscale = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1.0 else 1.0
    cos, sin = (None, None) if out is None else out
    return _call(_serving.rope_table, stream, num_pos, rot_dim, base, ROPE_SCALINGS[scaling],
                 factor, orig_len, beta_fast, beta_slow, mscale, pos0, cos, sin)


def new_kv_cache(num_blocks: int, heads: int, head_dim: int, dtype=torch.bfloat16,
                 page_size: int = PAGE_SIZE, device=None):
    """A zeroed paged key-value cache: (k, v), each [num_blocks, heads,
    page_size, head_dim] of bf16, fp16 or float8_e4m3fn."""
    raw = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
    return tuple(torch.zeros((num_blocks, heads, page_size, head_dim), dtype=raw,
                             device=device or "cuda").view(dtype) for _ in range(2))


def qk_norm_rope_insert(q, k, v, q_weight, k_weight, eps: float, positions, cos, sin,
                        rot_dim: int, slot_mapping, k_cache, v_cache, interleaved: bool = False,
                        k_scale=None, v_scale=None, q_out=None, errors=None, stream=None):
    """RMS norm of every query and key head (weights [D] fp32; None: no norm),
    rotary turn of their first rot_dim dimensions by table rows positions, and
    the insert of keys and values into the paged cache at slot_mapping (-1:
    none), in one pass.  q [N, Hq, D], k and v [N, Hkv, D] bf16 or fp16, which
    may be slices of one projection; caches [num_blocks, Hkv, page_size, D] of
    the same type or float8_e4m3fn (codes hold x / scale).  Returns the turned
    queries [N, Hq, D] (q_out; q itself where it is contiguous is allowed)."""
    return _call(_serving.qk_norm_rope_insert, stream, q, k, v, q_weight, k_weight, eps,
                 positions, cos, sin, rot_dim, slot_mapping, k_cache, v_cache, interleaved,
                 k_scale, v_scale, q_out, errors)


def paged_attention_workspace_bytes(B: int, next_n: int, Hq: int, Hkv: int,
                                    head_dim: int) -> int:
    return int(lib.idx_paged_attention_workspace_bytes(B, next_n, Hq, Hkv, head_dim))


AttentionForm = collections.namedtuple("AttentionForm", "split warps rows row_tiles unit places")


def paged_attention_form(B: int, next_n: int, Hq: int, Hkv: int, head_dim: int,
                         cache_dtype=torch.bfloat16, page_size: int = PAGE_SIZE, max_blocks: int = 1,
                         topk: int = 0, window: int = 0, sms: int | None = None) -> AttentionForm:
    """How paged_attention shares out a call of these sizes on a device of `sms` SMs
    (None: the current device): items cut along their keys over all CTAs and joined
    (split), or whole by teams of `warps` warps; items' query rows, items a kv head's
    rows make, keys by which a split item is cut, and items or CTAs that run at once."""
    if sms is None:
        sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    kinds = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}
    if cache_dtype not in kinds:
        raise TypeError("cache_dtype must be bfloat16, float16 or float8_e4m3fn")
    form = (ctypes.c_int32 * 6)()
    _check("idx_paged_attention_form",
           lib.idx_paged_attention_form(B, next_n, Hq, Hkv, head_dim, kinds[cache_dtype], page_size,
                                        max_blocks, topk, window, sms, form))
    return AttentionForm(bool(form[0]), *form[1:])


def paged_attention(q, k_cache, v_cache, block_table, context_lens, next_n: int = 1,
                    scale: float | None = None, softcap: float = 0.0, window: int = 0, topk=None,
                    k_scale=None, v_scale=None, workspace=None, out=None, lse=None,
                    return_lse: bool = False, errors=None, stream=None):
    """Attention of next_n new tokens per request over the paged cache.

    q [B*next_n, Hq, D]; caches [num_blocks, Hkv, page_size, D] (any strides
    with a unit last one); block_table [B, max_blocks], context_lens [B] int32
    (new tokens counted).  topk [B*next_n, k] int32: only the listed positions
    (negative: none), as paged_logits_topk returns them; otherwise the whole
    context, or its last `window` positions.  scale defaults to D^-0.5; softcap
    > 0 bounds scores by softcap * tanh(score / softcap).  Returns out
    [B*next_n, Hq, D] of q's type, with return_lse also ln sum exp of the
    scores ([B*next_n, Hq] fp32)."""
    o, l = _call(_serving.paged_attention, stream, q, k_cache, v_cache, block_table, context_lens,
                 next_n, scale, softcap, window, topk, k_scale, v_scale, workspace, out, lse,
                 return_lse, errors)
    return (o, l) if return_lse else o
