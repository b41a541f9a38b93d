"""Thin ctypes binding over libpkv.so (C ABI in include/pkv.h).

Argument marshalling only: shapes are read from the tensors, outputs are
allocated with PyTorch when the caller passes none, and every computation
runs in the library's CUDA kernels on the caller's current stream. There is
no fallback: if ``libpkv.so`` is missing or fails to load, every call raises.
Tensors live on the GPU, except that the decode calls also take q,
batch_idx, seq_lens, k_new, v_new, out and lse as pinned host tensors, which
the kernels read or write over the host link (no copy).

Functions keep the names of the C entry points: ``pkv_append``,
``pkv_append_rope``, ``pkv_decode_workspace_size``, ``pkv_decode_attention``,
``pkv_decode_append_attention``, ``pkv_decode_attention_static_scratch``,
``pkv_prefill_attention``, ``pkv_prefill_paged_attention``,
``pkv_mixed_workspace_size``, ``pkv_mixed_attention``,
``pkv_stage_from_host``, ``pkv_tree_workspace_size``, ``pkv_tree_attention``,
``pkv_verify_tree``, ``pkv_commit_path``, ``pkv_update_workspace_size``,
``pkv_update_pages``, ``pkv_compact_workspace_size``, ``pkv_compact_pages``,
``pkv_rotate``, ``pkv_latent_append``, ``pkv_latent_gather``,
``pkv_latent_decode_workspace_size``, ``pkv_latent_decode_attention``,
``pkv_latent_prefill_attention``, ``pkv_status_string``, ``pkv_status_from_device_error`` and
``pkv_last_cuda_error_string``.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpkv.so")

PKV_OK = 0
STATUS_NAMES = {0: "PKV_OK", 1: "PKV_ERR_ARG", 2: "PKV_ERR_ALIGN",
                3: "PKV_ERR_BAD_PAGE", 4: "PKV_ERR_WORKSPACE", 5: "PKV_ERR_CUDA",
                6: "PKV_ERR_DEVICE", 7: "PKV_ERR_BAD_INPUT"}
DEV_ERR_BAD_PAGE = 0x1
DEV_ERR_BAD_SLOT = 0x2
DEV_ERR_BAD_POS = 0x4
DEV_ERR_LAYOUT = 0x8
DEV_ERR_TIMEOUT = 0x10
DEV_ERR_BAD_TREE = 0x20
DEV_ERR_NO_PAGES = 0x40
DEV_ERR_BAD_PROBS = 0x80
MAX_TREE_NODES = 64
LATENT_DIM = 512       # a cache row of shared latents: the latent,
LATENT_ROTATED = 64    # then the rotated part
LATENT_ROW = LATENT_DIM + LATENT_ROTATED
LATENT_KEY = 128       # expanded: a head's own part of a key
LATENT_VALUE = 128     # expanded: a head's value

EXPORTED = ("pkv_append", "pkv_append_rope", "pkv_decode_workspace_size", "pkv_decode_attention",
            "pkv_decode_append_attention", "pkv_decode_attention_static_scratch",
            "pkv_prefill_paged_attention",
            "pkv_prefill_attention", "pkv_mixed_workspace_size", "pkv_mixed_attention",
            "pkv_stage_from_host", "pkv_tree_workspace_size", "pkv_tree_attention",
            "pkv_verify_tree", "pkv_commit_path", "pkv_update_workspace_size",
            "pkv_update_pages", "pkv_compact_workspace_size", "pkv_compact_pages",
            "pkv_rotate", "pkv_latent_append", "pkv_latent_gather",
            "pkv_latent_decode_workspace_size", "pkv_latent_decode_attention",
            "pkv_latent_prefill_attention", "pkv_status_string",
            "pkv_status_from_device_error", "pkv_last_cuda_error_string")


class PkvError(RuntimeError):
    """A libpkv call returned a status other than PKV_OK."""

    def __init__(self, func: str, status: int):
        self.status = status
        detail = status_string(status)
        if status == 5:
            detail += ": " + load_library().pkv_last_cuda_error_string().decode()
        super().__init__(f"{func}: {STATUS_NAMES.get(status, status)} ({detail})")


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("max_batch", ctypes.c_int), ("max_blocks", ctypes.c_int)]


_lib = None


def load_library() -> ctypes.CDLL:
    """Loads the in-tree libpkv.so (built by ``paged_kv_gqa_pkv_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m paged_kv_gqa_pkv_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32p, f32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    c_int, c_float, c_size = ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    desc_p = ctypes.POINTER(CacheDesc)
    lib.pkv_append.argtypes = [desc_p, vp, vp, i32p, vp, vp, i32p, i32p, c_int, i32p, vp]
    lib.pkv_append.restype = c_int
    lib.pkv_append_rope.argtypes = [desc_p, vp, vp, i32p, vp, vp, i32p, i32p, c_int, f32p, f32p,
                                    c_int, f32p, c_float, i32p, vp]
    lib.pkv_append_rope.restype = c_int
    lib.pkv_decode_workspace_size.argtypes = [desc_p, c_int, c_int, c_int]
    lib.pkv_decode_workspace_size.restype = c_size
    lib.pkv_decode_attention.argtypes = [desc_p, vp, vp, i32p, vp, c_int, i32p, i32p, c_int,
                                         c_float, vp, f32p, vp, c_size, i32p, vp]
    lib.pkv_decode_attention.restype = c_int
    lib.pkv_decode_append_attention.argtypes = [desc_p, vp, vp, i32p, vp, c_int, vp, vp, i32p,
                                                i32p, c_int, c_float, vp, f32p, vp, c_size, i32p,
                                                vp]
    lib.pkv_decode_append_attention.restype = c_int
    lib.pkv_prefill_paged_attention.argtypes = [desc_p, vp, vp, i32p, vp, c_int, i32p, i32p,
                                                c_int, c_float, vp, f32p, i32p, vp]
    lib.pkv_prefill_paged_attention.restype = c_int
    lib.pkv_prefill_attention.argtypes = [vp, vp, vp, c_int, c_int, c_int, i32p, i32p, c_int,
                                          c_float, vp, f32p, i32p, vp]
    lib.pkv_prefill_attention.restype = c_int
    lib.pkv_decode_attention_static_scratch.argtypes = [desc_p, vp, vp, i32p, vp, c_int, i32p,
                                                        i32p, c_int, c_float, vp, f32p, i32p,
                                                        vp]
    lib.pkv_decode_attention_static_scratch.restype = c_int
    lib.pkv_mixed_workspace_size.argtypes = [desc_p, c_int, c_int]
    lib.pkv_mixed_workspace_size.restype = c_size
    lib.pkv_mixed_attention.argtypes = [desc_p, vp, vp, i32p, vp, c_int, i32p, i32p, c_int,
                                        c_float, vp, f32p, vp, c_size, i32p, vp]
    lib.pkv_mixed_attention.restype = c_int
    lib.pkv_stage_from_host.argtypes = [vp, vp, c_size, vp]
    lib.pkv_stage_from_host.restype = c_int
    lib.pkv_tree_workspace_size.argtypes = [desc_p, c_int, c_int, c_int]
    lib.pkv_tree_workspace_size.restype = c_size
    lib.pkv_tree_attention.argtypes = [desc_p, vp, vp, i32p, vp, c_int, i32p, i32p, i32p, i32p,
                                       c_int, c_int, c_float, vp, f32p, vp, c_size, i32p, vp]
    lib.pkv_tree_attention.restype = c_int
    lib.pkv_verify_tree.argtypes = [vp, vp, c_int, c_int, i32p, i32p, i32p, f32p, f32p, c_int,
                                    c_int, i32p, i32p, i32p, i32p, vp]
    lib.pkv_verify_tree.restype = c_int
    lib.pkv_commit_path.argtypes = [desc_p, vp, vp, i32p, i32p, i32p, i32p, i32p, c_int, c_int,
                                    i32p, i32p, vp]
    lib.pkv_commit_path.restype = c_int
    lib.pkv_update_workspace_size.argtypes = [desc_p, c_int]
    lib.pkv_update_workspace_size.restype = c_size
    lib.pkv_update_pages.argtypes = [desc_p, vp, vp, i32p, i32p, i32p, i32p, i32p, i32p, c_int,
                                     vp, c_size, i32p, vp]
    lib.pkv_update_pages.restype = c_int
    lib.pkv_compact_workspace_size.argtypes = [desc_p]
    lib.pkv_compact_workspace_size.restype = c_size
    lib.pkv_compact_pages.argtypes = [desc_p, vp, vp, i32p, i32p, i32p, vp, c_size, i32p, vp]
    lib.pkv_compact_pages.restype = c_int
    i64 = ctypes.c_int64
    lib.pkv_rotate.argtypes = [vp, i64, i64, vp, i64, i64, c_int, c_int, c_int, c_int, i32p, f32p,
                               f32p, c_int, i32p, vp]
    lib.pkv_rotate.restype = c_int
    lib.pkv_latent_append.argtypes = [desc_p, vp, i32p, vp, i64, i32p, i32p, c_int, f32p, f32p,
                                      c_int, c_int, f32p, c_float, i32p, vp]
    lib.pkv_latent_append.restype = c_int
    lib.pkv_latent_gather.argtypes = [desc_p, vp, i32p, i32p, i32p, c_int, c_int, vp, i32p, vp]
    lib.pkv_latent_gather.restype = c_int
    lib.pkv_latent_decode_workspace_size.argtypes = [desc_p, c_int, c_int, c_int]
    lib.pkv_latent_decode_workspace_size.restype = c_size
    lib.pkv_latent_decode_attention.argtypes = [desc_p, vp, i32p, vp, c_int, i32p, i32p, c_int,
                                                c_int, c_float, vp, f32p, vp, c_size, i32p, vp]
    lib.pkv_latent_decode_attention.restype = c_int
    lib.pkv_latent_prefill_attention.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, i64,
                                                 c_int, i32p, i32p, c_int, c_int, c_int, c_float, vp,
                                                 f32p, i32p, vp]
    lib.pkv_latent_prefill_attention.restype = c_int
    lib.pkv_status_string.argtypes = [c_int]
    lib.pkv_status_string.restype = ctypes.c_char_p
    lib.pkv_last_cuda_error_string.argtypes = []
    lib.pkv_last_cuda_error_string.restype = ctypes.c_char_p
    lib.pkv_status_from_device_error.argtypes = [ctypes.c_int32]
    lib.pkv_status_from_device_error.restype = c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().pkv_status_string(int(status)).decode()


pkv_status_string = status_string


def pkv_status_from_device_error(dev_err_word: int) -> int:
    """Status for a dev_err word read back after the stream synchronised:
    PKV_OK when 0, PKV_ERR_BAD_PAGE when the bad-page bit is set, else
    PKV_ERR_BAD_INPUT."""
    return int(load_library().pkv_status_from_device_error(int(dev_err_word)))


def pkv_last_cuda_error_string() -> str:
    """Text of the CUDA error behind the last PKV_ERR_CUDA of this process."""
    return load_library().pkv_last_cuda_error_string().decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int, host_ok: bool = False):
    """A contiguous tensor of `dtype` and rank `ndim` on the GPU, or (with
    host_ok) in pinned host memory, which the decode kernels read over the
    host link."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    where_ok = t.is_cuda or (host_ok and t.device.type == "cpu" and t.is_pinned())
    if t.dtype != dtype or t.dim() != ndim or not where_ok or not t.is_contiguous():
        kind = "CUDA or pinned host" if host_ok else "CUDA"
        raise ValueError(f"{name}: expected a contiguous {kind} {dtype} tensor of rank {ndim}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def cache_desc(k_pool: torch.Tensor, page_table: torch.Tensor, page_size: int) -> CacheDesc:
    rows, hkv, d = k_pool.shape
    if rows % page_size:
        raise ValueError("pool rows must be a multiple of page_size")
    return CacheDesc(rows // page_size, page_size, hkv, d, page_table.shape[0],
                     page_table.shape[1])


def _check(func: str, status: int):
    if status != PKV_OK:
        raise PkvError(func, status)


def pkv_append(k_pool, v_pool, page_table, k_new, v_new, batch_idx, input_pos,
               page_size: int, dev_err=None, stream=None) -> None:
    """Writes k_new/v_new [N, H_kv, D] into the pools through the page table."""
    for name, t, dt, nd in (("k_pool", k_pool, torch.bfloat16, 3),
                            ("v_pool", v_pool, torch.bfloat16, 3),
                            ("page_table", page_table, torch.int32, 2),
                            ("k_new", k_new, torch.bfloat16, 3),
                            ("v_new", v_new, torch.bfloat16, 3),
                            ("batch_idx", batch_idx, torch.int32, 1),
                            ("input_pos", input_pos, torch.int32, 1)):
        _need(t, name, dt, nd)
    desc = cache_desc(k_pool, page_table, page_size)
    st = load_library().pkv_append(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), _ptr(k_new),
        _ptr(v_new), _ptr(batch_idx), _ptr(input_pos), int(batch_idx.numel()),
        _ptr(dev_err), _stream(stream))
    _check("pkv_append", st)


def pkv_append_rope(k_pool, v_pool, page_table, k_new, v_new, batch_idx, input_pos,
                    page_size: int, rope_cos, rope_sin, k_norm_weight=None,
                    k_norm_eps: float = 1e-6, dev_err=None, stream=None) -> None:
    """pkv_append with the rotary embedding (and, given ``k_norm_weight``
    fp32 [D], the per-head k_norm before it) applied to K; rope_cos/rope_sin
    are fp32 [L, D/2] tables indexed by position."""
    for name, t, dt, nd in (("k_pool", k_pool, torch.bfloat16, 3),
                            ("v_pool", v_pool, torch.bfloat16, 3),
                            ("page_table", page_table, torch.int32, 2),
                            ("k_new", k_new, torch.bfloat16, 3),
                            ("v_new", v_new, torch.bfloat16, 3),
                            ("batch_idx", batch_idx, torch.int32, 1),
                            ("input_pos", input_pos, torch.int32, 1),
                            ("rope_cos", rope_cos, torch.float32, 2),
                            ("rope_sin", rope_sin, torch.float32, 2)):
        _need(t, name, dt, nd)
    if rope_cos.shape != rope_sin.shape or rope_cos.shape[1] * 2 != k_new.shape[2]:
        raise ValueError("rope tables must both be [L, D/2]")
    if k_norm_weight is not None:
        _need(k_norm_weight, "k_norm_weight", torch.float32, 1)
        if k_norm_weight.shape[0] != k_new.shape[2]:
            raise ValueError("k_norm_weight must be [D]")
    desc = cache_desc(k_pool, page_table, page_size)
    st = load_library().pkv_append_rope(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), _ptr(k_new),
        _ptr(v_new), _ptr(batch_idx), _ptr(input_pos), int(batch_idx.numel()), _ptr(rope_cos),
        _ptr(rope_sin), int(rope_cos.shape[0]), _ptr(k_norm_weight), float(k_norm_eps),
        _ptr(dev_err), _stream(stream))
    _check("pkv_append_rope", st)


def pkv_decode_workspace_size(k_pool, page_table, page_size: int, batch: int,
                              num_q_heads: int, max_seq_len: int = 0) -> int:
    desc = cache_desc(k_pool, page_table, page_size)
    n = load_library().pkv_decode_workspace_size(ctypes.byref(desc), batch, num_q_heads,
                                                 max_seq_len)
    if n == 0 and batch > 0:
        raise PkvError("pkv_decode_workspace_size", 1)
    return int(n)


def pkv_decode_attention(k_pool, v_pool, page_table, q, batch_idx, seq_lens,
                         page_size: int, scale: float, out=None, lse=None,
                         workspace=None, dev_err=None, stream=None):
    """Split-KV GQA decode. q [B, Hq, D] bf16 -> (out [B, Hq, D] bf16,
    lse [B, Hq] fp32). q, batch_idx and seq_lens may be pinned host tensors,
    and out/lse pinned host tensors too; the outputs default to the pools'
    device."""
    _need(q, "q", torch.bfloat16, 3, host_ok=True)
    for name, t, dt, nd, h in (("k_pool", k_pool, torch.bfloat16, 3, False),
                               ("v_pool", v_pool, torch.bfloat16, 3, False),
                               ("page_table", page_table, torch.int32, 2, False),
                               ("batch_idx", batch_idx, torch.int32, 1, True),
                               ("seq_lens", seq_lens, torch.int32, 1, True)):
        _need(t, name, dt, nd, host_ok=h)
    B, hq, d = q.shape
    if out is None:
        out = torch.empty((B, hq, d), dtype=torch.bfloat16, device=k_pool.device)
    if lse is None:
        lse = torch.empty((B, hq), dtype=torch.float32, device=k_pool.device)
    desc = cache_desc(k_pool, page_table, page_size)
    lib = load_library()
    if workspace is None:
        n = lib.pkv_decode_workspace_size(ctypes.byref(desc), B, hq, 0)
        workspace = torch.empty(max(int(n), 256), dtype=torch.uint8, device=k_pool.device)
    st = lib.pkv_decode_attention(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), _ptr(q), hq,
        _ptr(batch_idx), _ptr(seq_lens), B, float(scale), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_err),
        _stream(stream))
    _check("pkv_decode_attention", st)
    return out, lse


def pkv_decode_append_attention(k_pool, v_pool, page_table, q, k_new, v_new, batch_idx,
                                seq_lens, page_size: int, scale: float, out=None, lse=None,
                                workspace=None, dev_err=None, stream=None):
    """One decode step in one call: row b's new token (k_new/v_new
    [B, Hkv, D] bf16) is written to position seq_lens[b] - 1 of its slot and
    attended with the rest. Returns (out [B, Hq, D] bf16, lse [B, Hq] fp32)."""
    _need(q, "q", torch.bfloat16, 3, host_ok=True)
    for name, t, dt, nd, h in (("k_pool", k_pool, torch.bfloat16, 3, False),
                               ("v_pool", v_pool, torch.bfloat16, 3, False),
                               ("k_new", k_new, torch.bfloat16, 3, True),
                               ("v_new", v_new, torch.bfloat16, 3, True),
                               ("page_table", page_table, torch.int32, 2, False),
                               ("batch_idx", batch_idx, torch.int32, 1, True),
                               ("seq_lens", seq_lens, torch.int32, 1, True)):
        _need(t, name, dt, nd, host_ok=h)
    B, hq, d = q.shape
    if k_new.shape != (B, k_pool.shape[1], d) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [B, Hkv, D]")
    if out is None:
        out = torch.empty((B, hq, d), dtype=torch.bfloat16, device=k_pool.device)
    if lse is None:
        lse = torch.empty((B, hq), dtype=torch.float32, device=k_pool.device)
    desc = cache_desc(k_pool, page_table, page_size)
    lib = load_library()
    if workspace is None:
        n = lib.pkv_decode_workspace_size(ctypes.byref(desc), B, hq, 0)
        workspace = torch.empty(max(int(n), 256), dtype=torch.uint8, device=k_pool.device)
    st = lib.pkv_decode_append_attention(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), _ptr(q), hq,
        _ptr(k_new), _ptr(v_new), _ptr(batch_idx), _ptr(seq_lens), B, float(scale), _ptr(out),
        _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_err),
        _stream(stream))
    _check("pkv_decode_append_attention", st)
    return out, lse


def pkv_prefill_paged_attention(k_pool, v_pool, page_table, q, batch_idx, input_pos,
                                page_size: int, scale: float, out=None, lse=None, dev_err=None,
                                stream=None):
    """Chunked prefill over the paged cache: token i of q [T, Hq, D] attends
    its slot's keys 0..input_pos[i] through the page table (its own chunk
    appended first). Returns (out [T, Hq, D] bf16, lse [T, Hq] fp32)."""
    _need(q, "q", torch.bfloat16, 3)
    for name, t, dt, nd in (("k_pool", k_pool, torch.bfloat16, 3),
                            ("v_pool", v_pool, torch.bfloat16, 3),
                            ("page_table", page_table, torch.int32, 2),
                            ("batch_idx", batch_idx, torch.int32, 1),
                            ("input_pos", input_pos, torch.int32, 1)):
        _need(t, name, dt, nd)
    T, hq, d = q.shape
    if out is None:
        out = torch.empty((T, hq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, hq), dtype=torch.float32, device=q.device)
    desc = cache_desc(k_pool, page_table, page_size)
    st = load_library().pkv_prefill_paged_attention(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), _ptr(q), hq,
        _ptr(batch_idx), _ptr(input_pos), T, float(scale), _ptr(out), _ptr(lse), _ptr(dev_err),
        _stream(stream))
    _check("pkv_prefill_paged_attention", st)
    return out, lse


def pkv_mixed_workspace_size(k_pool, page_table, page_size: int, n_tokens: int,
                             num_q_heads: int) -> int:
    desc = cache_desc(k_pool, page_table, page_size)
    n = load_library().pkv_mixed_workspace_size(ctypes.byref(desc), n_tokens, num_q_heads)
    if n == 0:
        raise PkvError("pkv_mixed_workspace_size", 1)
    return int(n)


def pkv_mixed_attention(k_pool, v_pool, page_table, q, batch_idx, input_pos, page_size: int,
                        scale: float, out=None, lse=None, workspace=None, dev_err=None,
                        stream=None):
    """A step of prefill chunks and decode tokens in one call: the results of
    ``pkv_prefill_paged_attention`` (token i of q [T, Hq, D] attends its
    slot's keys 0..input_pos[i]), with the decode tokens served by the
    split-KV decode kernels. Returns (out [T, Hq, D] bf16, lse [T, Hq] fp32)."""
    _need(q, "q", torch.bfloat16, 3)
    for name, t, dt, nd in (("k_pool", k_pool, torch.bfloat16, 3),
                            ("v_pool", v_pool, torch.bfloat16, 3),
                            ("page_table", page_table, torch.int32, 2),
                            ("batch_idx", batch_idx, torch.int32, 1),
                            ("input_pos", input_pos, torch.int32, 1)):
        _need(t, name, dt, nd)
    T, hq, d = q.shape
    if out is None:
        out = torch.empty((T, hq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, hq), dtype=torch.float32, device=q.device)
    desc = cache_desc(k_pool, page_table, page_size)
    lib = load_library()
    if workspace is None:
        n = lib.pkv_mixed_workspace_size(ctypes.byref(desc), T, hq)
        workspace = torch.empty(max(int(n), 256), dtype=torch.uint8, device=q.device)
    st = lib.pkv_mixed_attention(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), _ptr(q), hq,
        _ptr(batch_idx), _ptr(input_pos), T, float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_err), _stream(stream))
    _check("pkv_mixed_attention", st)
    return out, lse


def pkv_decode_attention_static_scratch(k_pool, v_pool, page_table, q, batch_idx, seq_lens,
                                        page_size: int, scale: float, out=None, lse=None,
                                        dev_err=None, stream=None):
    """Decode for callers that cannot allocate device memory: same result as
    ``pkv_decode_attention``, with the library's built-in 8 MiB scratch array
    instead of a caller workspace (calls must not overlap on the GPU)."""
    _need(q, "q", torch.bfloat16, 3, host_ok=True)
    for name, t, dt, nd, h in (("k_pool", k_pool, torch.bfloat16, 3, False),
                               ("v_pool", v_pool, torch.bfloat16, 3, False),
                               ("page_table", page_table, torch.int32, 2, False),
                               ("batch_idx", batch_idx, torch.int32, 1, True),
                               ("seq_lens", seq_lens, torch.int32, 1, True)):
        _need(t, name, dt, nd, host_ok=h)
    B, hq, d = q.shape
    if out is None:
        out = torch.empty((B, hq, d), dtype=torch.bfloat16, device=k_pool.device)
    if lse is None:
        lse = torch.empty((B, hq), dtype=torch.float32, device=k_pool.device)
    desc = cache_desc(k_pool, page_table, page_size)
    st = load_library().pkv_decode_attention_static_scratch(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), _ptr(q), hq,
        _ptr(batch_idx), _ptr(seq_lens), B, float(scale), _ptr(out), _ptr(lse), _ptr(dev_err),
        _stream(stream))
    _check("pkv_decode_attention_static_scratch", st)
    return out, lse


def pkv_prefill_attention(q, k, v, batch_idx, input_pos, scale: float, out=None,
                          lse=None, dev_err=None, stream=None):
    """Packed document-causal prefill. q [T, Hq, D], k/v [T, H_kv, D] bf16 ->
    (out [T, Hq, D] bf16, lse [T, Hq] fp32)."""
    for name, t, dt, nd in (("q", q, torch.bfloat16, 3), ("k", k, torch.bfloat16, 3),
                            ("v", v, torch.bfloat16, 3),
                            ("batch_idx", batch_idx, torch.int32, 1),
                            ("input_pos", input_pos, torch.int32, 1)):
        _need(t, name, dt, nd)
    T, hq, d = q.shape
    if out is None:
        out = torch.empty((T, hq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, hq), dtype=torch.float32, device=q.device)
    st = load_library().pkv_prefill_attention(
        _ptr(q), _ptr(k), _ptr(v), hq, k.shape[1], d, _ptr(batch_idx), _ptr(input_pos), T,
        float(scale), _ptr(out), _ptr(lse), _ptr(dev_err), _stream(stream))
    _check("pkv_prefill_attention", st)
    return out, lse


def pkv_stage_from_host(dst: torch.Tensor, src: torch.Tensor, stream=None) -> None:
    """Copies the bytes of ``src`` (pinned host memory) into ``dst`` (a CUDA
    tensor of the same byte size) with the GPU's own loads, on the current
    stream. Both contiguous, 16-byte aligned, size a multiple of 16 bytes."""
    for name, t in (("dst", dst), ("src", src)):
        if not isinstance(t, torch.Tensor) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor")
    if not dst.is_cuda:
        raise ValueError("dst must be a CUDA tensor")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("dst and src must hold the same number of bytes")
    st = load_library().pkv_stage_from_host(_ptr(dst), _ptr(src), nbytes, _stream(stream))
    _check("pkv_stage_from_host", st)


def _tensor(name: str, t, dtype: torch.dtype, shape, dev: int) -> int:
    """The address of a contiguous CUDA tensor of `dtype` and `shape` on device
    `dev`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {list(shape)} on "
                     f"cuda:{dev}, got {t.dtype} {list(t.shape)} on {t.device}"
                     f"{'' if t.is_contiguous() else ', not contiguous'}")


def _cache(k_pool, v_pool, page_table, page_size: int):
    """Device, descriptor and addresses of a call's cache."""
    _need(k_pool, "k_pool", torch.bfloat16, 3)
    dev, shape = k_pool.get_device(), k_pool.shape
    v = _tensor("v_pool", v_pool, torch.bfloat16, shape, dev)
    _need(page_table, "page_table", torch.int32, 2)
    if page_table.get_device() != dev:
        raise ValueError(f"page_table: expected a tensor on cuda:{dev}, got {page_table.device}")
    return dev, cache_desc(k_pool, page_table, page_size), k_pool.data_ptr(), v, page_table.data_ptr()


def _result(name: str, t, like: torch.Tensor, dev: int, stream, shape=None, dtype=None):
    """The caller's output tensor, or a new one, and its address: of the type and
    shape of the (checked) input `like`, or of those given. A new one is in the
    memory of the stream that writes it, so that nothing else can reuse it
    meanwhile."""
    if t is not None:
        return t, _tensor(name, t, dtype or like.dtype, like.shape if shape is None else shape, dev)
    if stream is not None:
        with torch.cuda.stream(stream):
            return _result(name, None, like, dev, None, shape, dtype)
    t = torch.empty_like(like) if shape is None else \
        torch.empty(shape, dtype=dtype, device=like.device)
    return t, t.data_ptr()


def _dev_err(t, dev: int) -> Optional[int]:
    return None if t is None else _tensor("dev_err", t, torch.int32, t.shape, dev)


# The handle of the current stream without the stream object around it (a few
# microseconds less per call), where this PyTorch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# PyTorch's caching allocator without a tensor around the memory: a workspace
# that lives for one call costs 2.5 us this way and 5.7 as a tensor, which it is
# where this PyTorch does not have them.
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_delete = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)
if _raw_delete is None:
    _raw_alloc = None


def _handle(name: str, dev: int, stream) -> int:
    """The handle of `stream`, or of the current stream of device `dev`."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"{name}: the stream is on {stream.device}, the tensors on cuda:{dev}")
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def _run(name: str, dev: int, stream, fn, *args) -> None:
    """Calls fn(*args, stream) with `dev` current, on `stream` or the device's
    current one."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            _run(name, dev, stream, fn, *args)
        return
    st = fn(*args, _handle(name, dev, stream))
    if st != PKV_OK:
        raise PkvError(name, st)


def _run_with(workspace, size, name: str, dev: int, stream, err, fn, *args) -> None:
    """_run of fn(*args, workspace, its bytes, err, stream) with the caller's
    workspace, or one of size() bytes that goes back to the stream's memory."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            _run_with(workspace, size, name, dev, stream, err, fn, *args)
        return
    handle = _handle(name, dev, stream)
    if workspace is None and _raw_alloc is None:
        with torch.cuda.stream(stream):   # (None: the current one)
            workspace = torch.empty(max(size(), 256), dtype=torch.uint8, device=f"cuda:{dev}")
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or \
                not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous CUDA tensor on cuda:{dev}")
        st = fn(*args, workspace.data_ptr(), workspace.nbytes, err, handle)
    else:
        nbytes = max(size(), 256)
        ptr = _raw_alloc(nbytes, handle)
        try:
            st = fn(*args, ptr, nbytes, err, handle)
        finally:
            _raw_delete(ptr)
    if st != PKV_OK:
        raise PkvError(name, st)


def pkv_tree_workspace_size(k_pool, page_table, page_size: int, batch: int, n_nodes: int,
                            num_q_heads: int) -> int:
    desc = cache_desc(k_pool, page_table, page_size)
    n = load_library().pkv_tree_workspace_size(ctypes.byref(desc), batch, n_nodes, num_q_heads)
    if n == 0:
        raise PkvError("pkv_tree_workspace_size", 1)
    return int(n)


def pkv_tree_attention(k_pool, v_pool, page_table, q, parents, tree_lens, batch_idx, ctx_lens,
                       page_size: int, scale: float, out=None, lse=None, workspace=None,
                       dev_err=None, stream=None):
    """Attention of a tree of drafted tokens per sequence: node i of row b of
    q [B, N, Hq, D] attends the ctx_lens[b] committed tokens of slot
    batch_idx[b], itself and its ancestors by parents [B, N]; the nodes' own
    K/V are in the pools at positions ctx_lens[b] + node (appended first).
    Returns (out [B, N, Hq, D] bf16, lse [B, N, Hq] fp32)."""
    dev, desc, k, v, table = _cache(k_pool, v_pool, page_table, page_size)
    _need(q, "q", torch.bfloat16, 4)
    B, N, hq, d = q.shape
    if d != desc.head_dim:
        raise ValueError("q and the pools must have one head dim")
    i32, nodes, rows = torch.int32, (B, N), (B,)
    args = (_tensor("q", q, torch.bfloat16, q.shape, dev), hq,
            _tensor("parents", parents, i32, nodes, dev),
            _tensor("tree_lens", tree_lens, i32, rows, dev),
            _tensor("batch_idx", batch_idx, i32, rows, dev),
            _tensor("ctx_lens", ctx_lens, i32, rows, dev), B, N, float(scale))
    out, out_p = _result("out", out, q, dev, stream)
    lse, lse_p = _result("lse", lse, q, dev, stream, (B, N, hq), torch.float32)
    lib = load_library()
    desc_p = ctypes.byref(desc)
    _run_with(workspace, lambda: lib.pkv_tree_workspace_size(desc_p, B, N, hq),
              "pkv_tree_attention", dev, stream, _dev_err(dev_err, dev), lib.pkv_tree_attention,
              desc_p, k, v, table, *args, out_p, lse_p)
    return out, lse


_PROBS_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def pkv_verify_tree(target_probs, draft_tokens, parents, tree_lens, u_accept, u_sample,
                    draft_probs=None, path=None, tokens=None, n_accepted=None, dev_err=None,
                    stream=None):
    """Acceptance of drafted tokens against the target's probabilities
    target_probs [B, N, V] (fp32 or bf16), from the random numbers u_accept
    [B, N] and u_sample [B]; draft_probs is like target_probs, or None for
    guessed tokens. Returns (path [B, N], tokens [B, N], n_accepted [B])
    int32: the accepted nodes, their tokens and the next one."""
    kind = target_probs.dtype if isinstance(target_probs, torch.Tensor) else None
    if kind not in _PROBS_TYPES:
        raise ValueError("target_probs must be an fp32 or bf16 tensor")
    _need(target_probs, "target_probs", kind, 3)
    dev = target_probs.get_device()
    B, N, V = target_probs.shape
    i32, nodes, rows = torch.int32, (B, N), (B,)
    args = (target_probs.data_ptr(),
            None if draft_probs is None else
            _tensor("draft_probs", draft_probs, kind, target_probs.shape, dev),
            _PROBS_TYPES[kind], V, _tensor("draft_tokens", draft_tokens, i32, nodes, dev),
            _tensor("parents", parents, i32, nodes, dev),
            _tensor("tree_lens", tree_lens, i32, rows, dev),
            _tensor("u_accept", u_accept, torch.float32, nodes, dev),
            _tensor("u_sample", u_sample, torch.float32, rows, dev), B, N)
    path, path_p = _result("path", path, parents, dev, stream)
    tokens, tokens_p = _result("tokens", tokens, parents, dev, stream)
    n_accepted, n_p = _result("n_accepted", n_accepted, tree_lens, dev, stream)
    _run("pkv_verify_tree", dev, stream, load_library().pkv_verify_tree, *args, path_p, tokens_p,
         n_p, _dev_err(dev_err, dev))
    return path, tokens, n_accepted


def pkv_commit_path(k_pool, v_pool, page_table, path, n_accepted, batch_idx, ctx_lens,
                    page_size: int, new_lens=None, dev_err=None, stream=None):
    """Moves the K/V rows of the accepted nodes path[b, :n_accepted[b]] from
    positions ctx_lens[b] + node to ctx_lens[b], ctx_lens[b] + 1, ... in
    place. Returns new_lens [B] = ctx_lens + n_accepted (``new_lens`` may be
    ctx_lens itself, with several layers in the last one's call)."""
    dev, desc, k, v, table = _cache(k_pool, v_pool, page_table, page_size)
    _need(path, "path", torch.int32, 2)
    B, N = path.shape
    i32, rows = torch.int32, (B,)
    args = (_tensor("path", path, i32, (B, N), dev),
            _tensor("n_accepted", n_accepted, i32, rows, dev),
            _tensor("batch_idx", batch_idx, i32, rows, dev),
            _tensor("ctx_lens", ctx_lens, i32, rows, dev), B, N)
    new_lens, new_p = _result("new_lens", new_lens, ctx_lens, dev, stream)
    _run("pkv_commit_path", dev, stream, load_library().pkv_commit_path, ctypes.byref(desc), k, v,
         table, *args, new_p, _dev_err(dev_err, dev))
    return new_lens


def pkv_update_workspace_size(k_pool, page_table, page_size: int, n: int) -> int:
    desc = cache_desc(k_pool, page_table, page_size)
    size = load_library().pkv_update_workspace_size(ctypes.byref(desc), n)
    if size == 0:
        raise PkvError("pkv_update_workspace_size", 1)
    return int(size)


def pkv_update_pages(k_pool, v_pool, page_table, page_refs, dst_slots, src_slots, keep_lens,
                     new_lens, page_size: int, workspace=None, dev_err=None,
                     stream=None) -> None:
    """Fork, reserve, copy on write, truncate and free, in place: slot
    dst_slots[i] gets the first keep_lens[i] tokens of slot src_slots[i] (pages
    shared) and pages of its own for the positions up to new_lens[i].
    page_refs [num_pages] counts the table entries that use each page (0: free).
    A call moves the rows of one layer's pools. Layers that share page_table and
    page_refs make all calls but the last on clones of both, taken before the
    first: on the updated state a layer's rows would stay behind."""
    dev, desc, k, v, table = _cache(k_pool, v_pool, page_table, page_size)
    _need(dst_slots, "dst_slots", torch.int32, 1)
    n = dst_slots.shape[0]
    i32, rows = torch.int32, (n,)
    args = (_tensor("page_refs", page_refs, i32, (desc.num_pages,), dev),
            _tensor("dst_slots", dst_slots, i32, rows, dev),
            _tensor("src_slots", src_slots, i32, rows, dev),
            _tensor("keep_lens", keep_lens, i32, rows, dev),
            _tensor("new_lens", new_lens, i32, rows, dev), n)
    lib = load_library()
    desc_p = ctypes.byref(desc)
    _run_with(workspace, lambda: lib.pkv_update_workspace_size(desc_p, n), "pkv_update_pages", dev,
              stream, _dev_err(dev_err, dev), lib.pkv_update_pages, desc_p, k, v, table, *args)


def pkv_compact_workspace_size(k_pool, page_table, page_size: int) -> int:
    desc = cache_desc(k_pool, page_table, page_size)
    size = load_library().pkv_compact_workspace_size(ctypes.byref(desc))
    if size == 0:
        raise PkvError("pkv_compact_workspace_size", 1)
    return int(size)


def pkv_compact_pages(k_pool, v_pool, page_table, page_refs, page_size: int, num_live=None,
                      workspace=None, dev_err=None, stream=None):
    """Moves the live pages to the low end of the pool (K/V rows, table
    entries and counts), in place. Returns num_live [1], how many there are.
    Layers that share page_table and page_refs: as for ``pkv_update_pages``."""
    dev, desc, k, v, table = _cache(k_pool, v_pool, page_table, page_size)
    refs = _tensor("page_refs", page_refs, torch.int32, (desc.num_pages,), dev)
    num_live, live_p = _result("num_live", num_live, page_refs, dev, stream, (1,), torch.int32)
    lib = load_library()
    desc_p = ctypes.byref(desc)
    _run_with(workspace, lambda: lib.pkv_compact_workspace_size(desc_p), "pkv_compact_pages", dev,
              stream, _dev_err(dev_err, dev), lib.pkv_compact_pages, desc_p, k, v, table, refs,
              live_p)
    return num_live


def _rope_tables(cos, sin, half: int, dev: int):
    """The addresses of a call's cosines and sines, fp32 [L, half], and L."""
    _need(cos, "rope_cos", torch.float32, 2)
    if cos.shape[1] != half:
        raise ValueError(f"rope tables must be [L, {half}], got {list(cos.shape)}")
    return (_tensor("rope_cos", cos, torch.float32, cos.shape, dev),
            _tensor("rope_sin", sin, torch.float32, cos.shape, dev), cos.shape[0])


def _strided(name: str, t, dev, shape=None) -> int:
    """The address of a bf16 CUDA tensor whose last dim is contiguous and whose other strides
    are free."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16 or not t.is_cuda or (dev is not None and t.get_device() != dev) or \
            (shape is not None and t.shape != shape) or (t.shape[-1] > 1 and t.stride(-1) != 1):
        want = "" if shape is None else f" of shape {list(shape)}"
        raise ValueError(f"{name}: expected a bfloat16 CUDA tensor{want} with a contiguous last dim, "
                         f"got {t.dtype} {list(t.shape)} with strides {list(t.stride())} on {t.device}")
    return t.data_ptr()


def pkv_rotate(x, positions, rope_cos, rope_sin, interleaved: bool = False, out=None, dev_err=None,
               stream=None):
    """The rotary embedding of x [T, H, dims] bf16, a view of any token and head
    stride (a slice ``q[..., a:b]`` rotates part of each head), by the fp32 tables
    [L, dims / 2] at ``positions`` [T]. Pairs are the halves' (x_j, x_{j + dims/2}) or,
    interleaved, neighbours (x_{2j}, x_{2j+1}). ``out`` is a view like x, x itself for a
    rotation in place, or None for a new tensor. Returns it."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a tensor [T, H, dims]")
    x_p = _strided("x", x, None)
    dev = x.get_device()
    T, H, dims = x.shape
    if dims % 2 or dims == 0 or H == 0:
        raise ValueError("x must be [T, H, dims] with at least one head and an even number of dims")
    pos = _tensor("positions", positions, torch.int32, (T,), dev)
    cos, sin, L = _rope_tables(rope_cos, rope_sin, dims // 2, dev)
    if out is None:
        out, out_p = _result("out", None, x, dev, stream, (T, H, dims), torch.bfloat16)
    else:
        out_p = _strided("out", out, dev, x.shape)
    _run("pkv_rotate", dev, stream, load_library().pkv_rotate, x_p, x.stride(0), x.stride(1), out_p,
         out.stride(0), out.stride(1), T, H, dims, int(bool(interleaved)), pos, cos, sin, L,
         _dev_err(dev_err, dev))
    return out


@functools.lru_cache(maxsize=64)
def _latent_desc(rows: int, row: int, page_size: int, max_batch: int, max_blocks: int):
    """A latent cache's descriptor and its address, by the cache's sizes."""
    if page_size <= 0 or rows % page_size:
        raise ValueError("pool rows must be a multiple of page_size")
    desc = CacheDesc(rows // page_size, page_size, 1, row, max_batch, max_blocks)
    return desc, ctypes.byref(desc)


def latent_cache_desc(pool: torch.Tensor, page_table: torch.Tensor, page_size: int) -> CacheDesc:
    """The descriptor of a paged cache of shared latents, pool [num_pages * page_size, 576]."""
    # (the caller's own: the one that calls share stays here)
    return CacheDesc.from_buffer_copy(_latent_desc(*pool.shape, int(page_size), *page_table.shape)[0])


def _latent_cache(pool, page_table, page_size: int):
    """Device, descriptor and addresses of a call's latent cache."""
    _need(pool, "pool", torch.bfloat16, 2)
    _need(page_table, "page_table", torch.int32, 2)
    dev = pool.get_device()
    if page_table.get_device() != dev:
        raise ValueError(f"page_table: expected a tensor on cuda:{dev}, got {page_table.device}")
    desc_p = _latent_desc(*pool.shape, int(page_size), *page_table.shape)[1]
    return dev, desc_p, pool.data_ptr(), page_table.data_ptr()


def pkv_latent_append(pool, page_table, x_new, batch_idx, input_pos, page_size: int, rope_cos,
                      rope_sin, norm_weight=None, norm_eps: float = 1e-6, interleaved: bool = False,
                      dev_err=None, stream=None) -> None:
    """Writes new tokens' rows x_new [N, 576] bf16 (a view of any token stride that is a multiple of 8,
    also where N is 1: the latent, then the position part) into the pool [num_pages * page_size, 576] through the page
    table: the latent normalised with ``norm_weight`` fp32 [512] if given, the position
    part rotated by the fp32 tables [L, 32] at input_pos [N]."""
    dev, desc_p, pool_p, table = _latent_cache(pool, page_table, page_size)
    if not isinstance(x_new, torch.Tensor) or x_new.dim() != 2 or x_new.shape[1] != LATENT_ROW:
        raise ValueError(f"x_new must be a tensor [N, {LATENT_ROW}]")
    x_p = _strided("x_new", x_new, dev)
    n = x_new.shape[0]
    b = _tensor("batch_idx", batch_idx, torch.int32, (n,), dev)
    pos = _tensor("input_pos", input_pos, torch.int32, (n,), dev)
    cos, sin, L = _rope_tables(rope_cos, rope_sin, LATENT_ROTATED // 2, dev)
    w = None if norm_weight is None else \
        _tensor("norm_weight", norm_weight, torch.float32, (LATENT_DIM,), dev)
    _run("pkv_latent_append", dev, stream, load_library().pkv_latent_append, desc_p,
         pool_p, table, x_p, x_new.stride(0), b, pos, n, cos, sin, L, int(bool(interleaved)), w,
         float(norm_eps), _dev_err(dev_err, dev))


def pkv_latent_gather(pool, page_table, slots, starts, total: int, page_size: int, out=None,
                      dev_err=None, stream=None):
    """The cached rows of sequences, one after another: row starts[b] + t of the result
    [total, 576] is the row of position t of slot slots[b], t < starts[b + 1] - starts[b].
    Rows that no sequence covers stay as they were. Returns ``out`` (a new one if None)."""
    dev, desc_p, pool_p, table = _latent_cache(pool, page_table, page_size)
    _need(slots, "slots", torch.int32, 1)
    n = slots.shape[0]
    slots_p = _tensor("slots", slots, torch.int32, (n,), dev)
    starts_p = _tensor("starts", starts, torch.int32, (n + 1,), dev)
    out, out_p = _result("out", out, pool, dev, stream, (int(total), pool.shape[1]), torch.bfloat16)
    _run("pkv_latent_gather", dev, stream, load_library().pkv_latent_gather, desc_p, pool_p,
         table, slots_p, starts_p, n, int(total), out_p, _dev_err(dev_err, dev))
    return out


def pkv_latent_decode_workspace_size(pool, page_table, page_size: int, batch: int, n_q: int,
                                     num_heads: int) -> int:
    desc = latent_cache_desc(pool, page_table, page_size)
    n = load_library().pkv_latent_decode_workspace_size(ctypes.byref(desc), batch, n_q, num_heads)
    if n == 0:
        raise PkvError("pkv_latent_decode_workspace_size", 1)
    return int(n)


def pkv_latent_decode_attention(pool, page_table, q, batch_idx, seq_lens, page_size: int,
                                scale: float, out=None, lse=None, workspace=None, dev_err=None,
                                stream=None):
    """Attention of new tokens over a paged cache of shared latents (the absorbed form). q
    [B, n_q, H, 576] bf16, or [B, H, 576] for one token a row: row b's tokens are the last
    n_q of the seq_lens[b] positions of slot batch_idx[b], each sees the rows up to its own
    (appended first). Returns (out [B, n_q, H, 512] bf16, lse [B, n_q, H] fp32), without the
    n_q axis where q has none."""
    dev, desc_p, pool_p, table = _latent_cache(pool, page_table, page_size)
    if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4) or q.shape[-1] != LATENT_ROW:
        raise ValueError(f"q must be a tensor [B, n_q, H, {LATENT_ROW}] or [B, H, {LATENT_ROW}]")
    q_p = _tensor("q", q, torch.bfloat16, q.shape, dev)
    B, H = q.shape[0], q.shape[-2]
    n_q = q.shape[1] if q.dim() == 4 else 1
    args = (q_p, H, _tensor("batch_idx", batch_idx, torch.int32, (B,), dev),
            _tensor("seq_lens", seq_lens, torch.int32, (B,), dev), B, n_q, float(scale))
    out, out_p = _result("out", out, q, dev, stream, (*q.shape[:-1], LATENT_DIM), torch.bfloat16)
    lse, lse_p = _result("lse", lse, q, dev, stream, q.shape[:-1], torch.float32)
    lib = load_library()
    _run_with(workspace, lambda: lib.pkv_latent_decode_workspace_size(desc_p, B, n_q, H),
              "pkv_latent_decode_attention", dev, stream, _dev_err(dev_err, dev),
              lib.pkv_latent_decode_attention, desc_p, pool_p, table, *args, out_p, lse_p)
    return out, lse


def pkv_latent_prefill_attention(q, k_own, k_rot, v, q_starts, k_starts, scale: float, out=None,
                                 lse=None, dev_err=None, stream=None):
    """Causal attention of packed sequences in the expanded form of shared latents. q [Tq, H,
    192], k_own and v [Tk, H, 128], k_rot [Tk, 64], bf16, views of any token and head stride
    (multiples of 8): sequence s has the queries q_starts[s] : q_starts[s + 1] and the keys
    k_starts[s] : k_starts[s + 1], a cached prefix first; its last query sees all of them.
    Returns (out [Tq, H, 128] bf16, lse [Tq, H] fp32); rows of no sequence stay as they were."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.shape[2] != LATENT_KEY + LATENT_ROTATED:
        raise ValueError(f"q must be a tensor [Tq, H, {LATENT_KEY + LATENT_ROTATED}]")
    q_p = _strided("q", q, None)
    dev = q.get_device()
    Tq, H, _ = q.shape
    if not isinstance(k_own, torch.Tensor) or k_own.dim() != 3:
        raise ValueError(f"k_own must be a tensor [Tk, H, {LATENT_KEY}]")
    Tk = k_own.shape[0]
    k_p = _strided("k_own", k_own, dev, (Tk, H, LATENT_KEY))
    r_p = _strided("k_rot", k_rot, dev, (Tk, LATENT_ROTATED))
    v_p = _strided("v", v, dev, (Tk, H, LATENT_VALUE))
    _need(q_starts, "q_starts", torch.int32, 1)
    n = q_starts.shape[0] - 1
    if n < 0:
        raise ValueError("q_starts must be [n_seqs + 1]")
    qs = _tensor("q_starts", q_starts, torch.int32, (n + 1,), dev)
    ks = _tensor("k_starts", k_starts, torch.int32, (n + 1,), dev)
    out, out_p = _result("out", out, q, dev, stream, (Tq, H, LATENT_VALUE), torch.bfloat16)
    lse, lse_p = _result("lse", lse, q, dev, stream, (Tq, H), torch.float32)
    _run("pkv_latent_prefill_attention", dev, stream, load_library().pkv_latent_prefill_attention, q_p,
         q.stride(0), q.stride(1), k_p, k_own.stride(0), k_own.stride(1), r_p, k_rot.stride(0), v_p,
         v.stride(0), v.stride(1), H, qs, ks, n, Tq, Tk, float(scale), out_p, lse_p,
         _dev_err(dev_err, dev))
    return out, lse
