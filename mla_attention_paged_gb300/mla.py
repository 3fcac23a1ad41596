"""Thin ctypes binding of libmla (include/mla.h).

Argument marshalling only: every step of the attention runs in the CUDA kernels behind the
C ABI.  PyTorch supplies device memory and the current stream.  If ``libmla.so`` has not
been built, importing this module raises; there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla.so")

MLA_OK = 0
MLA_ERR_INVALID_ARG = 1
MLA_ERR_UNSUPPORTED = 2
MLA_ERR_WORKSPACE_TOO_SMALL = 3
MLA_ERR_CUDA = 4
MLA_ERR_TIMEOUT = 5
MLA_ERR_DEVICE_ARG = 6
MLA_KV_BF16 = 0
MLA_KV_E4M3 = 1
MLA_KV_INT8 = 2
MLA_KV_INT8_PAGE = 3
MLA_KV_FP4 = 4

# Every function include/mla.h declares; each is given its C signature in _load().
EXPORTED = ["mla_decode_plan", "mla_decode", "mla_decode_partial", "mla_decode_combine", "mla_decode_noalloc",
            "mla_decode_int8_paged",
            "mla_prefill_varlen", "mla_prefill_paged", "mla_get_status", "mla_status_string", "mla_version", "mla_set_profile_events",
            "mla_profile_elapsed_ms", "mla_selftest_wait_timeout", "mla_kv_append", "mla_kv_evict",
            "mla_decode_tree_plan", "mla_decode_tree", "mla_key_mass_workspace", "mla_key_mass", "mla_kv_gather",
            "mla_page_fork", "mla_page_free", "mla_page_compact_workspace", "mla_page_compact"]


class MlaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what} failed: {status_string(code)} ({code})")


class DecodePlan(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("q_len", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("num_pages", ctypes.c_int64), ("num_sms", ctypes.c_int32),
                ("rows", ctypes.c_int32), ("head_groups", ctypes.c_int32), ("chunk_tokens", ctypes.c_int32),
                ("max_splits", ctypes.c_int32), ("max_seq_len", ctypes.c_int32), ("split_major", ctypes.c_int32), ("num_splits", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_size_t)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmla.so is not built at {LIB_PATH}; run `python -m mla_attention_paged_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.mla_decode_plan.restype = i32
    lib.mla_decode_plan.argtypes = [i32, P, i32, i32, i32, i32, i64, i32, i32, ctypes.POINTER(DecodePlan)]
    lib.mla_decode.restype = i32
    lib.mla_decode.argtypes = [ctypes.POINTER(DecodePlan), P, P, P, P, i32, i32, f32, f32, P, P, P, sz, P]
    lib.mla_decode_partial.restype = i32
    lib.mla_decode_partial.argtypes = [ctypes.POINTER(DecodePlan), P, P, P, P, i32, i32, f32, f32, P, P, P, sz, P]
    lib.mla_decode_combine.restype = i32
    lib.mla_decode_noalloc.restype = i32
    lib.mla_decode_noalloc.argtypes = [ctypes.POINTER(DecodePlan), P, P, P, P, i32, i32, f32, f32, P, P, P]
    lib.mla_decode_combine.argtypes = [ctypes.POINTER(DecodePlan), P, i32, i32, P, P, P, sz, P]
    lib.mla_decode_int8_paged.restype = i32
    lib.mla_decode_int8_paged.argtypes = [ctypes.POINTER(DecodePlan), P, P, P, P, P, i32, i32, f32, f32, P, P, P,
                                          sz, P]
    lib.mla_prefill_varlen.restype = i32
    lib.mla_prefill_varlen.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, P, P, P]
    lib.mla_prefill_paged.restype = i32
    lib.mla_prefill_paged.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i64, i32, i32, f32, P, P, P]
    lib.mla_decode_tree_plan.restype = i32
    lib.mla_decode_tree_plan.argtypes = lib.mla_decode_plan.argtypes
    lib.mla_decode_tree.restype = i32
    lib.mla_decode_tree.argtypes = [ctypes.POINTER(DecodePlan), P, P, P, P, P, P, i32, i32, f32, f32, P, P, P, sz, P]
    lib.mla_key_mass_workspace.restype = i32
    lib.mla_key_mass_workspace.argtypes = [ctypes.POINTER(DecodePlan), ctypes.POINTER(sz)]
    lib.mla_key_mass.restype = i32
    lib.mla_key_mass.argtypes = [ctypes.POINTER(DecodePlan), P, P, P, P, P, P, P, i32, i32, f32, f32, f32, P, i64, P, sz, P]
    lib.mla_kv_append.restype = i32
    lib.mla_kv_append.argtypes = [P, i64, i64, P, i64, i64, i32, i32, P, P, i64, P, f32, P, i32, P, P, i32, i32, P, i64,
                                  i32, f32, P]
    lib.mla_page_fork.restype = i32
    lib.mla_page_fork.argtypes = [P, i64, i32, i32, P, P, i32, P, i32, P, P, P, P, i32, P]
    lib.mla_page_free.restype = i32
    lib.mla_page_free.argtypes = [P, i32, P, i32, i32, P, i64, P, P, i32, P, P, P]
    lib.mla_page_compact_workspace.restype = i32
    lib.mla_page_compact_workspace.argtypes = [i64, ctypes.POINTER(sz)]
    lib.mla_page_compact.restype = i32
    lib.mla_page_compact.argtypes = [P, i64, i32, i32, P, P, i32, P, i32, P, P, P, sz, P]
    lib.mla_kv_gather.restype = i32
    lib.mla_kv_gather.argtypes = [P, i64, i32, i32, f32, P, P, i32, P, i32, i32, P, i64, P]
    lib.mla_kv_evict.restype = i32
    lib.mla_kv_evict.argtypes = [P, i64, i32, i32, P, i32, P, P, P, i64, P, i32, i32, i32, i32, i32, i32, P, i64, P, P,
                                 i64, P]
    lib.mla_get_status.restype = i32
    lib.mla_get_status.argtypes = [P]
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_status_string.argtypes = [i32]
    lib.mla_version.restype = i32
    lib.mla_set_profile_events.restype = i32
    lib.mla_set_profile_events.argtypes = [P, P]
    lib.mla_profile_elapsed_ms.restype = i32
    lib.mla_selftest_wait_timeout.restype = i32
    lib.mla_selftest_wait_timeout.argtypes = [P]
    lib.mla_profile_elapsed_ms.argtypes = [P, P, ctypes.POINTER(ctypes.c_float)]
    return lib


lib = _load()


def status_string(code: int) -> str:
    return lib.mla_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != MLA_OK:
        raise MlaError(code, what)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _stream_handle(stream):
    if stream is None:
        if torch.cuda.is_initialized():
            return _raw_stream(_current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


_POOL_DTYPE = {MLA_KV_BF16: (torch.bfloat16,), MLA_KV_E4M3: (torch.uint8, torch.float8_e4m3fn),
               MLA_KV_INT8: (torch.int8,), MLA_KV_INT8_PAGE: (torch.int8,), MLA_KV_FP4: (torch.uint8,)}
FP4_ROW_BYTES = 336  # a latent row of a 4-bit pool (include/mla.h)
_ROW_BYTES = {MLA_KV_BF16: 1152, MLA_KV_E4M3: 576, MLA_KV_INT8: 576, MLA_KV_INT8_PAGE: 576, MLA_KV_FP4: FP4_ROW_BYTES}


def _refuse(what: str, why: str):
    raise MlaError(MLA_ERR_INVALID_ARG, f"{what} ({why})")


def _want(what, dev, name, t, dtype, shape=None):
    """One tensor argument: on CUDA device number `dev`, contiguous, of `dtype` and (unless None) `shape`."""
    if t.get_device() != dev or dev < 0:
        _refuse(what, f"{name} is on {t.device}")
    if t.dtype is not dtype:
        _refuse(what, f"{name} is {t.dtype}")
    if shape is not None and t.shape != shape:
        _refuse(what, f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_contiguous():
        _refuse(what, f"{name} is not contiguous")
    return t.data_ptr()


def _want_rows(what, dev, name, t, dtype, rows):
    """A contiguous [rows, any] tensor: its address and row length."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows:
        _refuse(what, f"{name} has shape {tuple(shape)}")
    return _want(what, dev, name, t, dtype), shape[1]


def _want_pool(what, kv_pages, kv_dtype):
    """The latent pool: its device number, address, pages and page size."""
    dev, shape, dtype = kv_pages.get_device(), kv_pages.shape, kv_pages.dtype
    if len(shape) != 3 or shape[2] != (FP4_ROW_BYTES if kv_dtype == MLA_KV_FP4 else 576):
        _refuse(what, f"kv_pages has shape {tuple(shape)}")
    if dtype not in _POOL_DTYPE.get(kv_dtype, ()):
        _refuse(what, f"kv_pages is {dtype} for kv_dtype {kv_dtype}")
    return dev, _want(what, dev, "kv_pages", kv_pages, dtype), shape[0], shape[1]


def _hold_pool(what, plan, kv_pages):
    """The tensor holds all of the plan's num_pages pages in its format, as the header asks: of another format it would be
    read as other rows, and with fewer bytes past its end."""
    kind, bytes_ = plan.kv_dtype, kv_pages.numel() * kv_pages.element_size()
    if bytes_ < plan.num_pages * plan.page_size * _ROW_BYTES.get(kind, 0) or (kv_pages.shape[-1] == FP4_ROW_BYTES) != (kind == MLA_KV_FP4):
        _refuse(what, f"kv_pages is {kv_pages.dtype} {tuple(kv_pages.shape)}, not the plan's {plan.num_pages} pages of kv_dtype {kind}")


def _want_workspace(what, dev, workspace):
    if workspace is None:
        return None, 0
    return _want(what, dev, "workspace", workspace, workspace.dtype), workspace.numel() * workspace.element_size()


# The current stream's handle without a Stream object around it (2.8 us a call; this 0.1).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device  # (0.1 us against 0.2)
_CURRENT = contextlib.nullcontext()


def _on(stream):
    """The context in which a call allocates: what it makes belongs to the stream that uses it."""
    return _CURRENT if stream is None else torch.cuda.stream(stream)


def _call(what, dev, stream, fn, *args):
    """fn(*args, stream) on CUDA device number `dev`: its current stream unless one is given."""
    if stream is not None and stream.device_index != dev:
        _refuse(what, f"the stream is on device {stream.device_index}")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _call(what, dev, stream, fn, *args)
    rc = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc != MLA_OK:
        raise MlaError(rc, what)


def decode_plan(seq_lens_host, q_len: int, num_heads: int, page_size: int, max_pages_per_seq: int,
                num_pages: int, kv_dtype: int = MLA_KV_BF16, num_sms: int = 0) -> DecodePlan:
    """Plan a decode launch from HOST sequence lengths (drafts included)."""
    lens = torch.as_tensor(seq_lens_host, dtype=torch.int32).cpu().contiguous()
    plan = DecodePlan()
    rc = lib.mla_decode_plan(int(lens.numel()), ctypes.c_void_p(lens.data_ptr()), int(q_len), int(num_heads),
                             int(page_size), int(max_pages_per_seq), int(num_pages), int(kv_dtype), int(num_sms),
                             ctypes.byref(plan))
    _check(rc, "mla_decode_plan")
    return plan


def decode_tree_plan(seq_lens_host, q_len: int, num_heads: int, page_size: int, max_pages_per_seq: int,
                     num_pages: int, kv_dtype: int = MLA_KV_BF16, num_sms: int = 0) -> DecodePlan:
    """Plan a decode_tree launch (q_len <= 64 drafts) from HOST sequence lengths (drafts included)."""
    lens = torch.as_tensor(seq_lens_host, dtype=torch.int32).cpu().contiguous()
    plan = DecodePlan()
    rc = lib.mla_decode_tree_plan(int(lens.numel()), ctypes.c_void_p(lens.data_ptr()), int(q_len), int(num_heads),
                                  int(page_size), int(max_pages_per_seq), int(num_pages), int(kv_dtype), int(num_sms),
                                  ctypes.byref(plan))
    _check(rc, "mla_decode_tree_plan")
    return plan


def workspace_for(plan: DecodePlan, device) -> torch.Tensor | None:
    """Allocate (with torch) a workspace of the size the plan asks for."""
    if plan.workspace_bytes == 0:
        return None
    return torch.empty(int(plan.workspace_bytes), dtype=torch.uint8, device=device)


def decode(plan: DecodePlan, q: torch.Tensor, kv_pages: torch.Tensor, page_table: torch.Tensor,
           seq_lens: torch.Tensor, scale: float, kv_scale: float = 1.0, out=None, lse=None, workspace=None,
           stream=None):
    """mla_decode through the C ABI.  Returns (out [B,T,H,512] bf16, lse [B,T,H] fp32)."""
    _hold_pool("mla_decode", plan, kv_pages)
    B, T, H, D = q.shape
    if out is None:
        out = torch.empty(B, T, H, 512, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(B, T, H, dtype=torch.float32, device=q.device)
    if workspace is None and plan.workspace_bytes:
        workspace = workspace_for(plan, q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.mla_decode(ctypes.byref(plan), _ptr(q), _ptr(kv_pages), _ptr(page_table), _ptr(seq_lens), int(T),
                        int(H), float(scale), float(kv_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                        int(ws_bytes), _stream_handle(stream))
    _check(rc, "mla_decode")
    return out, lse


def decode_int8_paged(plan: DecodePlan, q: torch.Tensor, kv_pages: torch.Tensor, page_scales: torch.Tensor,
                      page_table: torch.Tensor, seq_lens: torch.Tensor, scale: float, kv_scale: float, out=None,
                      lse=None, workspace=None, stream=None):
    """mla_decode_int8_paged through the C ABI: an int8 pool with one fp32 scale per page
    (page_scales [num_pages] on the device).  Returns (out [B,T,H,512] bf16, lse [B,T,H] fp32)."""
    _hold_pool("mla_decode_int8_paged", plan, kv_pages)
    B, T, H, D = q.shape
    if out is None:
        out = torch.empty(B, T, H, 512, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(B, T, H, dtype=torch.float32, device=q.device)
    if workspace is None and plan.workspace_bytes:
        workspace = workspace_for(plan, q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.mla_decode_int8_paged(ctypes.byref(plan), _ptr(q), _ptr(kv_pages), _ptr(page_scales), _ptr(page_table),
                                   _ptr(seq_lens), int(T), int(H), float(scale), float(kv_scale), _ptr(out),
                                   _ptr(lse), _ptr(workspace), int(ws_bytes), _stream_handle(stream))
    _check(rc, "mla_decode_int8_paged")
    return out, lse


def decode_partial(plan: DecodePlan, q: torch.Tensor, kv_pages: torch.Tensor, page_table: torch.Tensor,
                   seq_lens: torch.Tensor, scale: float, kv_scale: float = 1.0, out=None, lse=None,
                   workspace=None, stream=None):
    """mla_decode_partial through the C ABI (stage 1 of decode): returns (out, lse, workspace);
    multi-split requests are finished by decode_combine with the same out/lse/workspace."""
    _hold_pool("mla_decode_partial", plan, kv_pages)
    B, T, H, D = q.shape
    if out is None:
        out = torch.empty(B, T, H, 512, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(B, T, H, dtype=torch.float32, device=q.device)
    if workspace is None and plan.workspace_bytes:
        workspace = workspace_for(plan, q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.mla_decode_partial(ctypes.byref(plan), _ptr(q), _ptr(kv_pages), _ptr(page_table), _ptr(seq_lens),
                                int(T), int(H), float(scale), float(kv_scale), _ptr(out), _ptr(lse),
                                _ptr(workspace), int(ws_bytes), _stream_handle(stream))
    _check(rc, "mla_decode_partial")
    return out, lse, workspace


def decode_combine(plan: DecodePlan, seq_lens: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, workspace=None,
                   stream=None):
    """mla_decode_combine through the C ABI (stage 2 of decode): merges the split partials
    left in `workspace` by decode_partial into out/lse."""
    B, T, H, _ = out.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.mla_decode_combine(ctypes.byref(plan), _ptr(seq_lens), int(T), int(H), _ptr(out), _ptr(lse),
                                _ptr(workspace), int(ws_bytes), _stream_handle(stream))
    _check(rc, "mla_decode_combine")
    return out, lse


def decode_noalloc(plan: DecodePlan, q: torch.Tensor, kv_pages: torch.Tensor, page_table: torch.Tensor,
                   seq_lens: torch.Tensor, scale: float, kv_scale: float = 1.0, out=None, lse=None, stream=None):
    """mla_decode_noalloc through the C ABI: decode with the split-KV scratch in the
    library's fixed 32 MiB device buffer instead of a workspace.  Returns (out, lse)."""
    _hold_pool("mla_decode_noalloc", plan, kv_pages)
    B, T, H, D = q.shape
    if out is None:
        out = torch.empty(B, T, H, 512, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(B, T, H, dtype=torch.float32, device=q.device)
    rc = lib.mla_decode_noalloc(ctypes.byref(plan), _ptr(q), _ptr(kv_pages), _ptr(page_table), _ptr(seq_lens),
                                int(T), int(H), float(scale), float(kv_scale), _ptr(out), _ptr(lse),
                                _stream_handle(stream))
    _check(rc, "mla_decode_noalloc")
    return out, lse


def prefill_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                   cu_seqlens_kv: torch.Tensor, prefix_lens: torch.Tensor, max_seqlen_q: int, scale: float,
                   out=None, lse=None, stream=None):
    """mla_prefill_varlen through the C ABI.  Returns (out [Nq,H,128] bf16, lse [Nq,H] fp32)."""
    Nq, H, _ = q.shape
    if out is None:
        out = torch.empty(Nq, H, v.shape[2], dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(Nq, H, dtype=torch.float32, device=q.device)
    rc = lib.mla_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv), _ptr(prefix_lens),
                                int(prefix_lens.numel()), int(H), int(max_seqlen_q), int(Nq), int(k.shape[0]),
                                float(scale), _ptr(out), _ptr(lse), _stream_handle(stream))
    _check(rc, "mla_prefill_varlen")
    return out, lse


def prefill_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                  cu_seqlens_q: torch.Tensor, kv_lens: torch.Tensor, max_seqlen_q: int, scale: float, out=None,
                  lse=None, stream=None):
    """mla_prefill_paged through the C ABI: the varlen prefill with K/V read through a page
    table from [num_pages, page_size, H, 192 | 128] pools.  Returns (out, lse)."""
    Nq, H, _ = q.shape
    num_pages, page_size = k_pages.shape[0], k_pages.shape[1]
    if out is None:
        out = torch.empty(Nq, H, v_pages.shape[3], dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(Nq, H, dtype=torch.float32, device=q.device)
    rc = lib.mla_prefill_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(cu_seqlens_q),
                               _ptr(kv_lens), int(kv_lens.numel()), int(H), int(page_size), int(page_table.shape[1]),
                               int(num_pages), int(max_seqlen_q), int(Nq), float(scale), _ptr(out), _ptr(lse),
                               _stream_handle(stream))
    _check(rc, "mla_prefill_paged")
    return out, lse


def decode_tree(plan: DecodePlan, q: torch.Tensor, kv_pages: torch.Tensor, page_table: torch.Tensor,
                seq_lens: torch.Tensor, tree_mask: torch.Tensor, scale: float, kv_scale: float = 1.0, page_scales=None,
                out=None, lse=None, workspace=None, *, stream=None):
    """mla_decode_tree through the C ABI: decode of a tree of drafts.  tree_mask [B,T] int64 (its 64
    bits): bit u of [b, t] = draft t sees draft u.  Returns (out [B,T,H,512] bf16, lse [B,T,H] fp32)."""
    what = "mla_decode_tree"
    dev, pool, pages, page_size = _want_pool(what, kv_pages, plan.kv_dtype)
    B, T, H = plan.batch, plan.q_len, plan.num_heads
    if pages != plan.num_pages or page_size != plan.page_size:
        _refuse(what, f"kv_pages has shape {tuple(kv_pages.shape)}, not the plan's")
    if out is None or lse is None or workspace is None:
        with _on(stream):
            if out is None:
                out = torch.empty(B, T, H, 512, dtype=torch.bfloat16, device=kv_pages.device)
            if lse is None:
                lse = torch.empty(B, T, H, dtype=torch.float32, device=kv_pages.device)
            if workspace is None:
                workspace = workspace_for(plan, kv_pages.device)
    ws, ws_bytes = _want_workspace(what, dev, workspace)
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    _call(what, dev, stream, lib.mla_decode_tree, plan, _want(what, dev, "q", q, bf16, (B, T, H, 576)), pool,
          None if page_scales is None else _want(what, dev, "page_scales", page_scales, f32, (plan.num_pages,)),
          _want(what, dev, "page_table", page_table, i32, (B, plan.max_pages_per_seq)),
          _want(what, dev, "seq_lens", seq_lens, i32, (B,)),
          _want(what, dev, "tree_mask", tree_mask, torch.int64, (B, T)), T, H, scale, kv_scale,
          _want(what, dev, "out", out, bf16, (B, T, H, 512)), _want(what, dev, "lse", lse, f32, (B, T, H)), ws, ws_bytes)
    return out, lse


def kv_append(q: torch.Tensor | None, kv: torch.Tensor | None, positions: torch.Tensor, slots: torch.Tensor | None,
              cos_sin: torch.Tensor, kv_pages: torch.Tensor | None, kv_weight=None, q_weight=None, eps: float = 1e-6,
              interleaved: bool = True, kv_dtype: int = MLA_KV_BF16, kv_scale: float = 1.0, q_out=None, *, stream=None):
    """mla_kv_append through the C ABI: norm and rotate a step's queries [N,H,q_dim] and latent
    keys [N,576], and write the keys into pool rows ``slots`` [N] int64 (negative: not stored).
    q (and q_out) may be strided views with a dense last dimension; q None: keys only, kv None:
    queries only.  Returns q_out (allocated when not given)."""
    what = "mla_kv_append"
    some = q if q is not None else kv
    if some is None:
        _refuse(what, "neither q nor kv")
    dev, n = some.get_device(), some.shape[0]
    bf16 = torch.bfloat16
    if cos_sin.dim() != 2 or cos_sin.shape[1] != 64:
        _refuse(what, f"cos_sin has shape {tuple(cos_sin.shape)}")
    table, pos = _want(what, dev, "cos_sin", cos_sin, torch.float32), _want(what, dev, "positions", positions, torch.int32, (n,))
    qa = (None, 0, 0, None, 0, 0, 0, 0, None)
    if q is not None:
        shape = q.shape
        if q_out is None:
            with _on(stream):
                q_out = torch.empty(shape, dtype=bf16, device=q.device)
        if q_out.get_device() != dev or dev < 0 or q.dtype is not bf16 or q_out.dtype is not bf16 or len(shape) != 3 or q_out.shape != shape:
            _refuse(what, f"q is {q.dtype} {tuple(shape)} on {q.device}, q_out {q_out.dtype} {tuple(q_out.shape)} on {q_out.device}")
        qt, qh, dense = q.stride()
        ot, oh, out_dense = q_out.stride()
        if dense != 1 or out_dense != 1:
            _refuse(what, "the last dimension of q or q_out is not dense")
        H, D = shape[1], shape[2]
        qa = (q.data_ptr(), qt, qh, q_out.data_ptr(), ot, oh, H, D,
              None if q_weight is None else _want(what, dev, "q_weight", q_weight, bf16, (D,)))
    ka, pool, rows, slot = (None, 0, None), None, 0, None
    if kv is not None:
        if kv_pages is None or slots is None:
            _refuse(what, "kv without kv_pages and slots")
        pool_dev, pool, pages, page_size = _want_pool(what, kv_pages, kv_dtype)
        if kv.get_device() != dev or pool_dev != dev or kv.dtype is not bf16 or kv.shape != (n, 576) or kv.stride(1) != 1:
            _refuse(what, f"kv is {kv.dtype} {tuple(kv.shape)} on {kv.device}")
        slot = _want(what, dev, "slots", slots, torch.int64, (n,))
        ka = (kv.data_ptr(), kv.stride(0), None if kv_weight is None else _want(what, dev, "kv_weight", kv_weight, bf16, (512,)))
        rows = pages * page_size
    _call(what, dev, stream, lib.mla_kv_append, *qa, *ka, eps, table, cos_sin.shape[0], pos, slot, n, 1 if interleaved else 0,
          pool, rows, kv_dtype, kv_scale)
    return q_out


def kv_gather(kv_pages: torch.Tensor, page_table: torch.Tensor, cu_rows: torch.Tensor, out: torch.Tensor,
              kv_dtype: int = MLA_KV_BF16, kv_scale: float = 1.0, page_scales=None, *, stream=None) -> torch.Tensor:
    """mla_kv_gather through the C ABI: the latent rows of each request, out of the pages, into rows
    cu_rows[b] .. cu_rows[b+1]-1 of out [N,576] bf16 (its rows may be strided).  cu_rows [B+1] int32 on
    the device.  Returns out."""
    what = "mla_kv_gather"
    dev, pool, pages, page_size = _want_pool(what, kv_pages, kv_dtype)
    B = cu_rows.numel() - 1
    if out.get_device() != dev or out.dtype is not torch.bfloat16 or out.dim() != 2 or out.shape[1] != 576 or out.stride(1) != 1:
        _refuse(what, f"out is {out.dtype} {tuple(out.shape)} on {out.device}")
    _call(what, dev, stream, lib.mla_kv_gather, pool, pages, page_size, kv_dtype, kv_scale,
          None if page_scales is None else _want(what, dev, "page_scales", page_scales, torch.float32, (pages,)),
          *_want_rows(what, dev, "page_table", page_table, torch.int32, B), _want(what, dev, "cu_rows", cu_rows, torch.int32, (B + 1,)),
          B, out.shape[0], out.data_ptr(), out.stride(0) if out.shape[0] > 1 else 576)
    return out


def key_mass_workspace_for(plan: DecodePlan, device) -> torch.Tensor | None:
    """Allocate (with torch) a workspace of the size key_mass needs under this plan."""
    need = ctypes.c_size_t()
    _check(lib.mla_key_mass_workspace(ctypes.byref(plan), ctypes.byref(need)), "mla_key_mass_workspace")
    return torch.empty(need.value, dtype=torch.uint8, device=device) if need.value else None


def key_mass(plan: DecodePlan, q: torch.Tensor, kv_pages: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
             lse: torch.Tensor, mass: torch.Tensor, scale: float, kv_scale: float = 1.0, tree_mask=None, page_scales=None,
             decay: float = 1.0, workspace=None, *, stream=None) -> torch.Tensor:
    """mla_key_mass through the C ABI: mass [B, >= max_seq_len] fp32 becomes decay * mass + the
    attention weight each key received in the step whose lse [B,T,H] this is.  Returns mass."""
    what = "mla_key_mass"
    dev, pool, pages, page_size = _want_pool(what, kv_pages, plan.kv_dtype)
    B, T, H = plan.batch, plan.q_len, plan.num_heads
    if pages != plan.num_pages or page_size != plan.page_size:
        _refuse(what, f"kv_pages has shape {tuple(kv_pages.shape)}, not the plan's")
    if workspace is None and plan.rows > 128:  # (fewer need none)
        with _on(stream):
            workspace = key_mass_workspace_for(plan, kv_pages.device)
    ws, ws_bytes = _want_workspace(what, dev, workspace)
    i32, f32 = torch.int32, torch.float32
    mass_ptr, stride = _want_rows(what, dev, "mass", mass, f32, B)
    _call(what, dev, stream, lib.mla_key_mass, plan, _want(what, dev, "q", q, torch.bfloat16, (B, T, H, 576)), pool,
          None if page_scales is None else _want(what, dev, "page_scales", page_scales, f32, (plan.num_pages,)),
          _want(what, dev, "page_table", page_table, i32, (B, plan.max_pages_per_seq)),
          _want(what, dev, "seq_lens", seq_lens, i32, (B,)),
          None if tree_mask is None else _want(what, dev, "tree_mask", tree_mask, torch.int64, (B, T)),
          _want(what, dev, "lse", lse, f32, (B, T, H)), T, H, scale, kv_scale, decay, mass_ptr, stride, ws, ws_bytes)
    return mass


def kv_evict(kv_pages: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, keep_lens: torch.Tensor,
             mass: torch.Tensor, dst_page_table: torch.Tensor, sink: int, recent: int, max_seq_len: int, max_keep: int,
             kv_dtype: int = MLA_KV_BF16, kept=None, new_lens=None, mass_out=None, *, stream=None):
    """mla_kv_evict through the C ABI: keep the heaviest keys of each request (its first ``sink``
    and last ``recent`` always) and copy their rows, in order, into the pages of
    ``dst_page_table``.  mass [B, >= max_seq_len] fp32.  Returns (kept [B,max_keep] int32, new_lens
    [B] int32, mass_out [B, >= max_keep] fp32)."""
    what = "mla_kv_evict"
    dev, pool, pages, page_size = _want_pool(what, kv_pages, kv_dtype)
    B = seq_lens.numel()
    i32, f32 = torch.int32, torch.float32
    with _on(stream):
        if kept is None:
            kept = torch.zeros(B, max_keep, dtype=i32, device=kv_pages.device)
        if new_lens is None:
            new_lens = torch.zeros(B, dtype=i32, device=kv_pages.device)
        if mass_out is None:
            mass_out = torch.zeros(B, max_keep, dtype=f32, device=kv_pages.device)
    table, dst = _want_rows(what, dev, "page_table", page_table, i32, B), _want_rows(what, dev, "dst_page_table", dst_page_table, i32, B)
    _call(what, dev, stream, lib.mla_kv_evict, pool, pages, page_size, kv_dtype, *table,
          _want(what, dev, "seq_lens", seq_lens, i32, (B,)), _want(what, dev, "keep_lens", keep_lens, i32, (B,)),
          *_want_rows(what, dev, "mass", mass, f32, B), *dst, B, sink, recent, max_seq_len, max_keep,
          *_want_rows(what, dev, "kept", kept, i32, B), _want(what, dev, "new_lens", new_lens, i32, (B,)),
          *_want_rows(what, dev, "mass_out", mass_out, f32, B))
    return kept, new_lens, mass_out


def page_fork(kv_pages: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor, parents: torch.Tensor,
              children: torch.Tensor, new_pages: torch.Tensor, kv_dtype: int = MLA_KV_BF16, page_scales=None, *, stream=None) -> None:
    """mla_page_fork through the C ABI: slots ``children`` [n] become copies of slots ``parents`` [n]: full
    pages shared, a partial last one copied to ``new_pages`` [n].  page_table [slots, any], seq_lens
    [slots] and refs [num_pages], all int32, are changed in place."""
    what = "mla_page_fork"
    dev, pool, pages, page_size = _want_pool(what, kv_pages, kv_dtype)
    i32, n, slots = torch.int32, parents.numel(), seq_lens.numel()
    _call(what, dev, stream, lib.mla_page_fork, pool, pages, page_size, kv_dtype,
          None if page_scales is None else _want(what, dev, "page_scales", page_scales, torch.float32, (pages,)),
          *_want_rows(what, dev, "page_table", page_table, i32, slots), _want(what, dev, "seq_lens", seq_lens, i32, (slots,)), slots,
          _want(what, dev, "refs", refs, i32, (pages,)), _want(what, dev, "parents", parents, i32, (n,)),
          _want(what, dev, "children", children, i32, (n,)), _want(what, dev, "new_pages", new_pages, i32, (n,)), n)


def page_free(page_table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor, slots: torch.Tensor, keep_lens: torch.Tensor,
              page_size: int, freed=None, num_freed=None, *, stream=None):
    """mla_page_free through the C ABI: slots ``slots`` [n] shrink to ``keep_lens`` [n] (0: they end).  seq_lens and
    refs [num_pages] are changed in place.  Returns (freed [num_pages] int32: the pages that came free,
    ascending, and zeros behind them where it is allocated here; num_freed [1] int32)."""
    what = "mla_page_free"
    dev, i32, n = refs.get_device(), torch.int32, slots.numel()
    pages = refs.numel()
    if dev >= 0 and (freed is None or num_freed is None):
        with _on(stream):
            freed = torch.zeros(pages, dtype=i32, device=refs.device) if freed is None else freed
            num_freed = torch.zeros(1, dtype=i32, device=refs.device) if num_freed is None else num_freed
    r = _want(what, dev, "refs", refs, i32, (pages,))
    _call(what, dev, stream, lib.mla_page_free, *_want_rows(what, dev, "page_table", page_table, i32, seq_lens.numel()),
          _want(what, dev, "seq_lens", seq_lens, i32, (seq_lens.numel(),)), seq_lens.numel(), page_size, r, pages,
          _want(what, dev, "slots", slots, i32, (n,)), _want(what, dev, "keep_lens", keep_lens, i32, (n,)), n,
          _want(what, dev, "freed", freed, i32, (pages,)), _want(what, dev, "num_freed", num_freed, i32, (1,)))
    return freed, num_freed


def page_compact_workspace_for(num_pages: int, device) -> torch.Tensor:
    """Allocate (with torch) a workspace of the size page_compact needs for a pool of num_pages pages."""
    need = ctypes.c_size_t()
    _check(lib.mla_page_compact_workspace(int(num_pages), ctypes.byref(need)), "mla_page_compact_workspace")
    return torch.empty(need.value, dtype=torch.uint8, device=device)


def page_compact(kv_pages: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor,
                 kv_dtype: int = MLA_KV_BF16, num_live=None, workspace=None, page_scales=None, *, stream=None) -> torch.Tensor:
    """mla_page_compact through the C ABI: the pages that anything refers to move to 0 .. num_live - 1;
    page_table, refs and page_scales follow in place.  Returns num_live [1] int32."""
    what = "mla_page_compact"
    dev, pool, pages, page_size = _want_pool(what, kv_pages, kv_dtype)
    if dev >= 0 and (num_live is None or workspace is None):
        with _on(stream):
            num_live = torch.zeros(1, dtype=torch.int32, device=kv_pages.device) if num_live is None else num_live
            workspace = page_compact_workspace_for(pages, kv_pages.device) if workspace is None else workspace
    ws, ws_bytes = _want_workspace(what, dev, workspace)
    i32, slots = torch.int32, seq_lens.numel()
    _call(what, dev, stream, lib.mla_page_compact, pool, pages, page_size, kv_dtype,
          None if page_scales is None else _want(what, dev, "page_scales", page_scales, torch.float32, (pages,)),
          *_want_rows(what, dev, "page_table", page_table, i32, slots), _want(what, dev, "seq_lens", seq_lens, i32, (slots,)), slots,
          _want(what, dev, "refs", refs, i32, (pages,)), _want(what, dev, "num_live", num_live, i32, (1,)), ws, ws_bytes)
    return num_live


def set_profile_events(start=None, stop=None) -> None:
    """Record torch.cuda.Event pairs around the main kernel of later calls (this thread)."""
    lib.mla_set_profile_events(ctypes.c_void_p(start.cuda_event) if start is not None else None,
                               ctypes.c_void_p(stop.cuda_event) if stop is not None else None)


def profile_elapsed_ms(start, stop) -> float:
    """Milliseconds between two torch.cuda.Event objects recorded through the hook."""
    ms = ctypes.c_float()
    _check(lib.mla_profile_elapsed_ms(ctypes.c_void_p(start.cuda_event), ctypes.c_void_p(stop.cuda_event),
                                      ctypes.byref(ms)), "mla_profile_elapsed_ms")
    return ms.value


def selftest_wait_timeout(stream=None) -> None:
    """Enqueue the watchdog self-test kernel (its bounded wait must expire)."""
    _check(lib.mla_selftest_wait_timeout(_stream_handle(stream)), "mla_selftest_wait_timeout")


def get_status(stream=None) -> int:
    """Read and clear the device status word (synchronises the stream)."""
    return lib.mla_get_status(_stream_handle(stream))
