"""Python binding of the C ABI in include/kivi.h (argument marshalling only).

Every step of the hot path runs in the CUDA library ``lib/libkivi.so``; this
module only converts torch tensors into device pointers and the current CUDA
stream into a ``cudaStream_t``.  PyTorch is used for device memory and streams.
There is no fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libkivi.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "kivi.h")

STATUS = {0: "KIVI_OK", 1: "KIVI_ERR_ARG", 2: "KIVI_ERR_ALIGN", 3: "KIVI_ERR_UNSUPPORTED",
          4: "KIVI_ERR_CAPACITY", 5: "KIVI_ERR_WORKSPACE", 6: "KIVI_ERR_CUDA"}
KIVI_OK, KIVI_ERR_ARG, KIVI_ERR_ALIGN, KIVI_ERR_UNSUPPORTED, KIVI_ERR_CAPACITY, KIVI_ERR_WORKSPACE, KIVI_ERR_CUDA = range(7)


class KiviError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call}: {STATUS.get(status, status)}")
        self.status = status


class kivi_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("G", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("value_residual", ctypes.c_int32), ("value_group", ctypes.c_int32),
                ("max_tokens", ctypes.c_int64)]


class kivi_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_meta", ctypes.c_void_p), ("k_res", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_meta", ctypes.c_void_p), ("v_res", ctypes.c_void_p),
                ("n_tokens", ctypes.c_int64)]


class kivi_paged_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("G", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("value_residual", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("num_pages", ctypes.c_int64)]


class kivi_paged_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_meta", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_meta", ctypes.c_void_p), ("k_res", ctypes.c_void_p), ("v_res", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p)]


class kivi_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class kivi_page_pool(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("ref_counts", ctypes.c_void_p), ("info", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libkivi.so (built by ``bit_asymmetric_kv_gb300.build``); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m bit_asymmetric_kv_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, D, C = ctypes.c_void_p, ctypes.POINTER(kivi_dims), ctypes.POINTER(kivi_cache)
        i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.kivi_buffer_bytes.argtypes = [D, ctypes.POINTER(sz)]
        L.kivi_quantize_prefill.argtypes = [D, C, P, P, i64, P]
        L.kivi_append_token.argtypes = [D, C, P, P, P]
        L.kivi_prefill_attention.argtypes = [D, C, P, i32, P, P, i64, ctypes.c_float, P, P]
        L.kivi_prefill_attention.restype = ctypes.c_int
        L.kivi_decode_splits.argtypes = [D, i32, i64]
        L.kivi_decode_workspace_bytes.argtypes = [D, i32, i64]
        L.kivi_decode_workspace_bytes.restype = sz
        L.kivi_decode_attention.argtypes = [D, C, P, i32, ctypes.c_float, P, P, sz, P]
        L.kivi_dequantize_debug.argtypes = [D, C, P, P, P]
        L.kivi_decode_attention_noalloc.argtypes = [D, C, P, i32, ctypes.c_float, P, P]
        L.kivi_decode_attention_noalloc.restype = ctypes.c_int
        L.kivi_decode_attention_noalloc_max_workspace.argtypes = []
        L.kivi_decode_attention_noalloc_max_workspace.restype = sz
        L.kivi_decode_fp16_workspace_bytes.argtypes = [i32, i32, i32, i32, i64]
        L.kivi_decode_fp16_workspace_bytes.restype = sz
        L.kivi_decode_attention_fp16.argtypes = [i32, i32, i32, i32, i64, P, P, P, ctypes.c_float, P, P, sz, P]
        L.kivi_decode_attention_fp16.restype = ctypes.c_int
        L.kivi_decode_step.argtypes = [D, C, P, P, P, i32, ctypes.c_float, P, P, sz, P]
        L.kivi_decode_step.restype = ctypes.c_int
        PD, PC = ctypes.POINTER(kivi_paged_dims), ctypes.POINTER(kivi_paged_cache)
        L.kivi_paged_buffer_bytes.argtypes = [PD, ctypes.POINTER(sz)]
        L.kivi_paged_prefill.argtypes = [PD, PC, i32, P, P, i64, P]
        L.kivi_paged_append_token.argtypes = [PD, PC, P, P, P]
        L.kivi_paged_decode_workspace_bytes.argtypes = [PD, i32]
        L.kivi_paged_decode_workspace_bytes.restype = sz
        L.kivi_paged_decode_attention.argtypes = [PD, PC, P, i32, ctypes.c_float, P, P, sz, P]
        L.kivi_paged_decode_step.argtypes = [PD, PC, P, P, P, i32, ctypes.c_float, P, P, sz, P]
        L.kivi_paged_decode_attention_window.argtypes = [PD, PC, P, i32, ctypes.c_float, i32, i32, P, P, sz, P]
        L.kivi_paged_decode_step_window.argtypes = [PD, PC, P, P, P, i32, ctypes.c_float, i32, i32, P, P, sz, P]
        for name in ("kivi_paged_buffer_bytes", "kivi_paged_prefill", "kivi_paged_append_token",
                     "kivi_paged_decode_attention", "kivi_paged_decode_step", "kivi_paged_decode_attention_window",
                     "kivi_paged_decode_step_window"):
            getattr(L, name).restype = ctypes.c_int
        PR, PP = ctypes.POINTER(kivi_rows), ctypes.POINTER(kivi_page_pool)
        L.kivi_prefill_attention_packed.argtypes = [i32, i32, i32, i32, P, i64, PR, PR, PR, ctypes.c_float, PR, P]
        L.kivi_prefill_attention_window.argtypes = [i32, i32, i32, i32, P, i64, P, i64, PR, PR, PR, ctypes.c_float, i32,
                                                    i32, PR, P]
        L.kivi_paged_prefill_packed.argtypes = [PD, PC, P, i64, PR, PR, P]
        L.kivi_paged_extend_packed.argtypes = [PD, PC, P, i64, PR, PR, P]
        L.kivi_paged_read.argtypes = [PD, PC, P, i64, P, i32, PR, PR, P]
        L.kivi_paged_pool_workspace_bytes.argtypes = [PD]
        L.kivi_paged_pool_workspace_bytes.restype = sz
        for name in ("kivi_paged_reserve", "kivi_paged_reorder", "kivi_paged_compact"):
            getattr(L, name).argtypes = [PD, PC, PP, P, P, sz, P]
        L.kivi_paged_reserve_window.argtypes = [PD, PC, PP, P, i32, i32, P, sz, P]
        L.kivi_paged_reserve_window.restype = ctypes.c_int
        for name in ("kivi_prefill_attention_packed", "kivi_prefill_attention_window", "kivi_paged_prefill_packed",
                     "kivi_paged_extend_packed", "kivi_paged_read", "kivi_paged_reserve",
                     "kivi_paged_reorder", "kivi_paged_compact"):
            getattr(L, name).restype = ctypes.c_int
        L.kivi_status_string.argtypes = [ctypes.c_int]
        L.kivi_status_string.restype = ctypes.c_char_p
        for name in ("kivi_buffer_bytes", "kivi_quantize_prefill", "kivi_append_token", "kivi_decode_splits",
                     "kivi_decode_attention", "kivi_dequantize_debug"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int, call: str) -> None:
    if status != KIVI_OK:
        raise KiviError(status, call)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _f16(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.float16 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous CUDA float16 tensor")
    return t


def make_dims(B: int, Hkv: int, G: int, max_tokens: int, D: int = 128, bits: int = 2,
              value_residual: bool = False, value_group: int = 0) -> kivi_dims:
    return kivi_dims(B, Hkv, D, G, bits, int(value_residual), int(value_group), max_tokens)


def kivi_buffer_bytes(dims: kivi_dims) -> list[int]:
    out = (ctypes.c_size_t * 6)()
    _check(lib().kivi_buffer_bytes(ctypes.byref(dims), out), "kivi_buffer_bytes")
    return list(out)


@dataclass
class Cache:
    """Caller-owned device buffers of one quantized KV cache (layouts in include/kivi.h)."""

    dims: kivi_dims
    k_codes: torch.Tensor  # int32 [B, Hkv, T, D*bits/32]   (uint32 bit patterns)
    k_meta: torch.Tensor   # int32 [B, Hkv, T/G, D]    ({s, z} fp16 pairs)
    k_res: torch.Tensor    # fp16  [B, Hkv, G, D]
    v_codes: torch.Tensor  # int32 [B, Hkv, T, D*bits/32]
    v_meta: torch.Tensor   # int32 [B, Hkv, T], or [B, Hkv, T, D/vg] with value channel groups
    c: kivi_cache
    v_res: torch.Tensor | None = None  # fp16 [B, Hkv, G, D] with a value residual

    @property
    def n_tokens(self) -> int:
        return int(self.c.n_tokens)

    @classmethod
    def allocate(cls, B: int, Hkv: int, G: int, max_tokens: int, device="cuda", D: int = 128,
                 value_residual: bool = False, bits: int = 2, value_group: int = 0) -> "Cache":
        dims = make_dims(B, Hkv, G, max_tokens, D, bits=bits, value_residual=value_residual,
                         value_group=value_group)
        kivi_buffer_bytes(dims)  # validates the geometry
        T = max_tokens
        W = D * bits // 32  # words of a packed token row
        kc = torch.empty((B, Hkv, T, W), dtype=torch.int32, device=device)
        km = torch.empty((B, Hkv, T // G, D), dtype=torch.int32, device=device)
        kr = torch.empty((B, Hkv, G, D), dtype=torch.float16, device=device)
        vc = torch.empty((B, Hkv, T, W), dtype=torch.int32, device=device)
        vg = value_group or D
        vm = torch.empty((B, Hkv, T) if vg == D else (B, Hkv, T, D // vg), dtype=torch.int32, device=device)
        vr = torch.empty((B, Hkv, G, D), dtype=torch.float16, device=device) if value_residual else None
        c = kivi_cache(kc.data_ptr(), km.data_ptr(), kr.data_ptr(), vc.data_ptr(), vm.data_ptr(),
                       0 if vr is None else vr.data_ptr(), 0)
        return cls(dims, kc, km, kr, vc, vm, c, vr)


def kivi_quantize_prefill(cache: Cache, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """k, v: fp16 [B, Hkv, n, D] on the device."""
    _f16(k, "k"), _f16(v, "v")
    n = k.shape[2]
    _check(lib().kivi_quantize_prefill(ctypes.byref(cache.dims), ctypes.byref(cache.c), _ptr(k), _ptr(v), n,
                                       _stream(stream)), "kivi_quantize_prefill")


def kivi_prefill_attention(cache: Cache | None, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                           softmax_scale: float, out: torch.Tensor | None = None, dims: kivi_dims | None = None,
                           stream=None) -> torch.Tensor:
    """Causal prompt attention (q fp16 [B, Hq, n, D], k, v fp16 [B, Hkv, n, D] on the
    device) with the cache quantized from the same k, v in the same kernel; with
    cache=None (and the cache geometry in `dims`) the attention alone."""
    _f16(q, "q"), _f16(k, "k"), _f16(v, "v")
    if out is None:
        out = torch.empty_like(q)
    _f16(out, "out")
    B, Hq, n, D = q.shape
    if cache is not None:
        d, c = ctypes.byref(cache.dims), ctypes.byref(cache.c)
    else:
        if dims is None:
            raise ValueError("attention alone needs the geometry in `dims`")
        d, c = ctypes.byref(dims), None
    _check(lib().kivi_prefill_attention(d, c, _ptr(q), Hq, _ptr(k), _ptr(v), n, float(softmax_scale), _ptr(out),
                                        _stream(stream)), "kivi_prefill_attention")
    return out


def kivi_append_token(cache: Cache, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
    """k_new, v_new: fp16 [B, Hkv, D] on the device."""
    _f16(k_new, "k_new"), _f16(v_new, "v_new")
    _check(lib().kivi_append_token(ctypes.byref(cache.dims), ctypes.byref(cache.c), _ptr(k_new), _ptr(v_new),
                                   _stream(stream)), "kivi_append_token")


def kivi_decode_splits(dims: kivi_dims, Hq: int, n_tokens: int) -> int:
    return int(lib().kivi_decode_splits(ctypes.byref(dims), Hq, n_tokens))


def kivi_decode_workspace_bytes(dims: kivi_dims, Hq: int, n_tokens: int) -> int:
    return int(lib().kivi_decode_workspace_bytes(ctypes.byref(dims), Hq, n_tokens))


def workspace(cache: Cache, Hq: int, n_tokens: int | None = None, device="cuda") -> torch.Tensor:
    """Allocate a decode workspace for this cache (uint8 device tensor)."""
    n = cache.n_tokens if n_tokens is None else n_tokens
    nbytes = kivi_decode_workspace_bytes(cache.dims, Hq, n)
    if nbytes == 0:
        raise KiviError(KIVI_ERR_ARG, "kivi_decode_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def kivi_decode_attention(cache: Cache, q: torch.Tensor, softmax_scale: float, out: torch.Tensor | None = None,
                          ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q: fp16 [B, Hq, D] -> out fp16 [B, Hq, D]."""
    _f16(q, "q")
    Hq = q.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(cache, Hq, device=q.device)
    _check(lib().kivi_decode_attention(ctypes.byref(cache.dims), ctypes.byref(cache.c), _ptr(q), Hq,
                                       float(softmax_scale), _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                       _stream(stream)), "kivi_decode_attention")
    return out


def kivi_decode_attention_noalloc(cache: Cache, q: torch.Tensor, softmax_scale: float,
                                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kivi_decode_attention with the workspace taken from the library's built-in
    array (for callers that cannot allocate device memory); q: fp16 [B, Hq, D]."""
    _f16(q, "q")
    if out is None:
        out = torch.empty_like(q)
    _check(lib().kivi_decode_attention_noalloc(ctypes.byref(cache.dims), ctypes.byref(cache.c), _ptr(q), q.shape[1],
                                               float(softmax_scale), _ptr(out), _stream(stream)),
           "kivi_decode_attention_noalloc")
    return out


def kivi_decode_attention_noalloc_max_workspace() -> int:
    return int(lib().kivi_decode_attention_noalloc_max_workspace())


def kivi_decode_step(cache: Cache, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor, softmax_scale: float,
                     out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Append (k_new, v_new fp16 [B, Hkv, D]) then attend with q fp16 [B, Hq, D]."""
    _f16(k_new, "k_new"), _f16(v_new, "v_new"), _f16(q, "q")
    Hq = q.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(cache, Hq, n_tokens=cache.n_tokens + 1, device=q.device)
    _check(lib().kivi_decode_step(ctypes.byref(cache.dims), ctypes.byref(cache.c), _ptr(k_new), _ptr(v_new), _ptr(q),
                                  Hq, float(softmax_scale), _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)), "kivi_decode_step")
    return out


def kivi_dequantize_debug(cache: Cache, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Dequantized cache as fp32 [B, Hkv, n_tokens, D] (keys, values)."""
    d = cache.dims
    shape = (d.B, d.Hkv, cache.n_tokens, d.D)
    k = torch.empty(shape, dtype=torch.float32, device=cache.k_codes.device)
    v = torch.empty(shape, dtype=torch.float32, device=cache.k_codes.device)
    _check(lib().kivi_dequantize_debug(ctypes.byref(d), ctypes.byref(cache.c), _ptr(k), _ptr(v), _stream(stream)),
           "kivi_dequantize_debug")
    return k, v


def kivi_decode_fp16_workspace_bytes(B: int, Hq: int, Hkv: int, n: int, D: int = 128) -> int:
    return int(lib().kivi_decode_fp16_workspace_bytes(B, Hq, Hkv, D, n))


def kivi_decode_attention_fp16(k: torch.Tensor, v: torch.Tensor, q: torch.Tensor, softmax_scale: float,
                               out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                               stream=None) -> torch.Tensor:
    """Decode attention over an unquantized fp16 cache: k, v [B, Hkv, n, D], q [B, Hq, D]."""
    _f16(k, "k"), _f16(v, "v"), _f16(q, "q")
    B, Hkv, n, D = k.shape
    Hq = q.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        nbytes = kivi_decode_fp16_workspace_bytes(B, Hq, Hkv, n, D)
        if nbytes == 0:
            raise KiviError(KIVI_ERR_ARG, "kivi_decode_fp16_workspace_bytes")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _check(lib().kivi_decode_attention_fp16(B, Hq, Hkv, D, n, _ptr(k), _ptr(v), _ptr(q), float(softmax_scale),
                                            _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "kivi_decode_attention_fp16")
    return out


def kivi_status_string(status: int) -> str:
    return lib().kivi_status_string(status).decode()


# ---------------------------------------------------------------------------------------
# paged cache
# ---------------------------------------------------------------------------------------
def make_paged_dims(B: int, Hkv: int, G: int, page_tokens: int, max_pages_per_seq: int, num_pages: int,
                    D: int = 128, bits: int = 2, value_residual: bool = False) -> kivi_paged_dims:
    return kivi_paged_dims(B, Hkv, D, G, bits, int(value_residual), page_tokens, max_pages_per_seq, num_pages)


def kivi_paged_buffer_bytes(dims: kivi_paged_dims) -> list[int]:
    out = (ctypes.c_size_t * 8)()
    _check(lib().kivi_paged_buffer_bytes(ctypes.byref(dims), out), "kivi_paged_buffer_bytes")
    return list(out)


@dataclass
class PagedCache:
    """Caller-owned device buffers of a paged cache (layouts in include/kivi.h): a
    page pool, per-sequence residual keys, the block table and the lengths."""

    dims: kivi_paged_dims
    k_codes: torch.Tensor      # int32 [num_pages, Hkv, P, D/16]
    k_meta: torch.Tensor       # int32 [num_pages, Hkv, P/G, D]
    v_codes: torch.Tensor      # int32 [num_pages, Hkv, P, D/16]
    v_meta: torch.Tensor       # int32 [num_pages, Hkv, P]
    k_res: torch.Tensor        # fp16  [B, Hkv, G, D]
    block_table: torch.Tensor  # int32 [B, max_pages_per_seq]
    seq_lens: torch.Tensor     # int32 [B]
    c: kivi_paged_cache
    v_res: torch.Tensor | None = None  # fp16 [B, Hkv, G, D] with a value residual

    @classmethod
    def allocate(cls, B: int, Hkv: int, G: int, page_tokens: int, max_pages_per_seq: int, num_pages: int,
                 device="cuda", D: int = 128, value_residual: bool = False, bits: int = 2) -> "PagedCache":
        dims = make_paged_dims(B, Hkv, G, page_tokens, max_pages_per_seq, num_pages, D, bits=bits,
                               value_residual=value_residual)
        kivi_paged_buffer_bytes(dims)  # validates the geometry
        P = page_tokens
        W = D * bits // 32  # words of a packed token row
        kc = torch.empty((num_pages, Hkv, P, W), dtype=torch.int32, device=device)
        km = torch.empty((num_pages, Hkv, P // G, D), dtype=torch.int32, device=device)
        vc = torch.empty((num_pages, Hkv, P, W), dtype=torch.int32, device=device)
        vm = torch.empty((num_pages, Hkv, P), dtype=torch.int32, device=device)
        kr = torch.empty((B, Hkv, G, D), dtype=torch.float16, device=device)
        vr = torch.empty((B, Hkv, G, D), dtype=torch.float16, device=device) if value_residual else None
        bt = torch.zeros((B, max_pages_per_seq), dtype=torch.int32, device=device)
        sl = torch.zeros((B,), dtype=torch.int32, device=device)
        c = kivi_paged_cache(kc.data_ptr(), km.data_ptr(), vc.data_ptr(), vm.data_ptr(), kr.data_ptr(),
                             0 if vr is None else vr.data_ptr(), bt.data_ptr(), sl.data_ptr())
        return cls(dims, kc, km, vc, vm, kr, bt, sl, c, vr)


def kivi_paged_prefill(cache: PagedCache, seq: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Prompt of sequence `seq`: k, v fp16 [Hkv, n, D] on the device."""
    _f16(k, "k"), _f16(v, "v")
    _check(lib().kivi_paged_prefill(ctypes.byref(cache.dims), ctypes.byref(cache.c), seq, _ptr(k), _ptr(v),
                                    k.shape[1], _stream(stream)), "kivi_paged_prefill")


def kivi_paged_append_token(cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
    """k_new, v_new: fp16 [B, Hkv, D] on the device."""
    _f16(k_new, "k_new"), _f16(v_new, "v_new")
    _check(lib().kivi_paged_append_token(ctypes.byref(cache.dims), ctypes.byref(cache.c), _ptr(k_new), _ptr(v_new),
                                         _stream(stream)), "kivi_paged_append_token")


def kivi_paged_decode_workspace_bytes(dims: kivi_paged_dims, Hq: int) -> int:
    return int(lib().kivi_paged_decode_workspace_bytes(ctypes.byref(dims), Hq))


def paged_workspace(cache: PagedCache, Hq: int, device="cuda") -> torch.Tensor:
    nbytes = kivi_paged_decode_workspace_bytes(cache.dims, Hq)
    if nbytes == 0:
        raise KiviError(KIVI_ERR_ARG, "kivi_paged_decode_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def kivi_paged_decode_attention(cache: PagedCache, q: torch.Tensor, softmax_scale: float,
                                out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """q: fp16 [B, Hq, D] -> out fp16 [B, Hq, D], each sequence over its own length."""
    _f16(q, "q")
    Hq = q.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = paged_workspace(cache, Hq, device=q.device)
    _check(lib().kivi_paged_decode_attention(ctypes.byref(cache.dims), ctypes.byref(cache.c), _ptr(q), Hq,
                                             float(softmax_scale), _ptr(out), _ptr(ws),
                                             ws.numel() * ws.element_size(), _stream(stream)),
           "kivi_paged_decode_attention")
    return out


def kivi_paged_decode_step(cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                           softmax_scale: float, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """Append (k_new, v_new fp16 [B, Hkv, D]) at every sequence's length, attend with
    q fp16 [B, Hq, D], advance the lengths."""
    _f16(k_new, "k_new"), _f16(v_new, "v_new"), _f16(q, "q")
    Hq = q.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = paged_workspace(cache, Hq, device=q.device)
    _check(lib().kivi_paged_decode_step(ctypes.byref(cache.dims), ctypes.byref(cache.c), _ptr(k_new), _ptr(v_new),
                                        _ptr(q), Hq, float(softmax_scale), _ptr(out), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)), "kivi_paged_decode_step")
    return out


# ---------------------------------------------------------------------------------------
# packed prompts, and pages handed out on the device
# ---------------------------------------------------------------------------------------
def _run(call: str, device: torch.device, stream, *args) -> None:
    """Call `call` of the library with `device` current, on the given stream (a torch stream or a
    cudaStream_t) or the device's current one.  Switching the device costs more than the call, so it is
    switched only when it is not the current one."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device.index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    fn = getattr(_lib or lib(), call)
    if torch._C._cuda_getDevice() == device.index:  # the tensors on it have initialised CUDA
        status = fn(*args, int(stream))
    else:
        with torch.cuda.device(device):
            status = fn(*args, int(stream))
    if status != KIVI_OK:
        raise KiviError(status, call)


def _allocating_on(device: torch.device, stream):
    """Context in which tensors are made for use on the given stream."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device) if int(stream) else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _rows(t: torch.Tensor, name: str, device: torch.device) -> kivi_rows:
    """kivi_rows of an fp16 CUDA tensor [tokens, heads, D] with contiguous channels.  The stride of an
    axis of one element says nothing, and torch may hold any number there."""
    stride = t.stride()
    if t.dtype is not torch.float16 or not t.is_cuda or len(stride) != 3 or (stride[2] != 1 and t.numel()):
        raise TypeError(f"{name}: expected a CUDA float16 tensor [tokens, heads, D] with contiguous channels")
    if t.get_device() != device.index:
        raise ValueError(f"{name}: expected a tensor on {device}")
    T, H, D = t.shape
    return kivi_rows(t.data_ptr(), stride[0] if T > 1 else max(D, 128), stride[1] if H > 1 else max(D, 128))


def _i32(t: torch.Tensor, name: str, numel: int, device: torch.device) -> int:
    """Address of a contiguous int32 tensor of `numel` elements on `device`."""
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous() or t.numel() != numel:
        raise TypeError(f"{name}: expected a contiguous CUDA int32 tensor of {numel} elements")
    if t.get_device() != device.index:
        raise ValueError(f"{name}: expected a tensor on {device}")
    return t.data_ptr()


def kivi_prefill_attention_packed(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                                  softmax_scale: float, out: torch.Tensor | None = None,
                                  stream=None) -> torch.Tensor:
    """Causal attention of prompts packed into one token axis: q fp16 [T, Hq, D], k, v fp16 [T, Hkv, D] on
    the device, any token and head strides that are multiples of 8 (views of one projection, or
    transposed head-major tensors); sequence s is rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1
    (int32 [n_seqs + 1] on the device).  Rows of no sequence are not written (zero in an `out` made
    here)."""
    dev = q.device
    rq, rk, rv = _rows(q, "q", dev), _rows(k, "k", dev), _rows(v, "v", dev)
    shape, kv = q.shape, k.shape
    T, Hq, D = shape
    if kv != v.shape or kv[0] != T or kv[2] != D:
        raise ValueError(f"q {list(shape)}, k {list(kv)}, v {list(v.shape)} do not fit together")
    bounds = cu_seqlens.numel()
    if bounds < 2:
        raise ValueError("cu_seqlens holds at least two bounds")
    cu = _i32(cu_seqlens, "cu_seqlens", bounds, dev)
    if out is None:
        with _allocating_on(dev, stream):
            out = torch.zeros(shape, dtype=torch.float16, device=dev)
    elif out.shape != shape:
        raise ValueError(f"out: expected shape {list(shape)}")
    ro = _rows(out, "out", dev)
    if T:
        _run("kivi_prefill_attention_packed", dev, stream, Hq, kv[1], D, bounds - 1, cu, T, rq, rk, rv,
             float(softmax_scale), ro)
    return out


def _count(x: int, name: str, least: int) -> int:
    """A number of positions as the ABI's int32: at least `least`; one beyond int32 sees what the largest does."""
    if x < least:
        raise ValueError(f"{name}: expected at least {least}")
    return min(int(x), 2**31 - 1)


def kivi_prefill_attention_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                                  window: int, sinks: int, softmax_scale: float,
                                  cu_seqlens_kv: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                  stream=None) -> torch.Tensor:
    """kivi_prefill_attention_packed in which position p sees the positions p - window + 1 .. p and the
    first `sinks`.  With cu_seqlens_kv (int32 [n_seqs + 1]) k and v have a token axis of their own,
    [Tk, Hkv, D], and the queries of a sequence are its last tokens; a query before the first key
    gets zeros."""
    dev = q.device
    rq = _rows(q, "q", dev)
    shape, kv = q.shape, k.shape
    T, Hq, D = shape
    if kv != v.shape or len(kv) != 3 or kv[2] != D or (cu_seqlens_kv is None and kv[0] != T):
        raise ValueError(f"q {list(shape)}, k {list(kv)}, v {list(v.shape)} do not fit together")
    rk, rv = _rows(k, "k", dev), _rows(v, "v", dev)
    bounds = cu_seqlens.numel()
    if bounds < 2:
        raise ValueError("cu_seqlens holds at least two bounds")
    cu = _i32(cu_seqlens, "cu_seqlens", bounds, dev)
    cu_kv = None if cu_seqlens_kv is None else _i32(cu_seqlens_kv, "cu_seqlens_kv", bounds, dev)
    window, sinks = _count(window, "window", 1), _count(sinks, "sinks", 0)
    if out is None:
        with _allocating_on(dev, stream):
            out = torch.zeros(shape, dtype=torch.float16, device=dev)
    elif out.shape != shape:
        raise ValueError(f"out: expected shape {list(shape)}")
    ro = _rows(out, "out", dev)
    if T:
        _run("kivi_prefill_attention_window", dev, stream, Hq, kv[1], D, bounds - 1, cu, T, cu_kv, kv[0], rq, rk, rv,
             float(softmax_scale), window, sinks, ro)
    return out


def _heads(t: torch.Tensor, name: str, cache: PagedCache, heads: int | None = None) -> torch.Tensor:
    """An fp16 tensor [B, heads, D] of one token a sequence, contiguous and on the cache's device."""
    d, shape = cache.dims, t.shape
    _f16(t, name)
    if t.get_device() != cache.k_codes.get_device():
        raise ValueError(f"{name}: expected a tensor on {cache.k_codes.device}")
    if len(shape) != 3 or shape[0] != d.B or shape[2] != d.D or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name}: {list(shape)}, expected [{d.B}, {heads or 'heads'}, {d.D}]")
    return t


def _decode_window(call: str, cache: PagedCache, new: list, q: torch.Tensor, window: int, sinks: int,
                   softmax_scale: float, out: torch.Tensor | None, ws: torch.Tensor | None, stream) -> torch.Tensor:
    dev, Hq = cache.k_codes.device, _heads(q, "q", cache).shape[1]
    window, sinks = _count(window, "window", 1), _count(sinks, "sinks", 0)
    if out is None or ws is None:
        with _allocating_on(dev, stream):
            out = torch.empty_like(q) if out is None else out
            ws = paged_workspace(cache, Hq, device=dev) if ws is None else ws
    _heads(out, "out", cache, Hq)
    if ws.get_device() != dev.index or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor on {dev}")
    _run(call, dev, stream, cache.dims, cache.c, *new, q.data_ptr(), Hq, float(softmax_scale), window, sinks,
         out.data_ptr(), ws.data_ptr(), ws.nbytes)
    return out


def kivi_paged_decode_attention_window(cache: PagedCache, q: torch.Tensor, window: int, sinks: int,
                                       softmax_scale: float, out: torch.Tensor | None = None,
                                       ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kivi_paged_decode_attention in which a sequence's newest token sees its newest `window` tokens and its
    first `sinks`; pages that hold none of these are not read."""
    return _decode_window("kivi_paged_decode_attention_window", cache, [], q, window, sinks, softmax_scale, out, ws,
                          stream)


def kivi_paged_decode_step_window(cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                                  window: int, sinks: int, softmax_scale: float, out: torch.Tensor | None = None,
                                  ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kivi_paged_decode_step in which the appended token sees the newest `window` tokens, itself among them,
    and the first `sinks`."""
    new = [_heads(t, name, cache, cache.dims.Hkv).data_ptr() for t, name in ((k_new, "k_new"), (v_new, "v_new"))]
    return _decode_window("kivi_paged_decode_step_window", cache, new, q, window, sinks, softmax_scale, out, ws, stream)


def kivi_paged_prefill_packed(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                              stream=None) -> None:
    """Prompts of all sequences of a paged batch, packed: k, v fp16 [T, Hkv, D] (strides as for
    kivi_prefill_attention_packed), cu_seqlens int32 [B + 1]; an empty sequence is left as it is."""
    dev, cu, rk, rv = _pack(cache, cu_seqlens, k, v, "k", "v")
    if k.shape[0]:
        _run("kivi_paged_prefill_packed", dev, stream, cache.dims, cache.c, cu, k.shape[0], rk, rv)


def _pack(cache: PagedCache, cu_seqlens: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_name: str, v_name: str):
    """(device, bounds, rows of k, rows of v) of a paged batch's packed keys and values."""
    d, dev = cache.dims, cache.k_codes.device
    rk, rv = _rows(k, k_name, dev), _rows(v, v_name, dev)
    if k.shape != v.shape or tuple(k.shape[1:]) != (d.Hkv, d.D):
        raise ValueError(f"{k_name} {list(k.shape)}, {v_name} {list(v.shape)}: expected [tokens, {d.Hkv}, {d.D}]")
    return dev, _i32(cu_seqlens, "cu_seqlens", d.B + 1, dev), rk, rv


def kivi_paged_extend_packed(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                             stream=None) -> None:
    """New tokens of all sequences of a paged batch, packed, behind what the sequences hold: k, v fp16
    [T, Hkv, D] (strides as for kivi_prefill_attention_packed), cu_seqlens int32 [B + 1]; the lengths grow."""
    dev, cu, rk, rv = _pack(cache, cu_seqlens, k, v, "k", "v")
    if k.shape[0]:
        _run("kivi_paged_extend_packed", dev, stream, cache.dims, cache.c, cu, k.shape[0], rk, rv)


def kivi_paged_read(cache: PagedCache, cu_seqlens: torch.Tensor, take: torch.Tensor | None, k_out: torch.Tensor,
                    v_out: torch.Tensor, first: int = 0, stream=None) -> None:
    """The first `first` and the newest tokens of every sequence, take[s] of them together (int32 [B] on the
    device; None: as many as it has rows), as fp16 rows cu_seqlens[s] .. of k_out and v_out [T, Hkv, D] (strides
    as for kivi_prefill_attention_packed); the rows behind them are left as they were."""
    dev, cu, rk, rv = _pack(cache, cu_seqlens, k_out, v_out, "k_out", "v_out")
    at = None if take is None else _i32(take, "take", cache.dims.B, dev)
    first = _count(first, "first", 0)
    if k_out.shape[0]:
        _run("kivi_paged_read", dev, stream, cache.dims, cache.c, cu, k_out.shape[0], at, first, rk, rv)


def kivi_paged_pool_workspace_bytes(dims: kivi_paged_dims) -> int:
    return int(lib().kivi_paged_pool_workspace_bytes(ctypes.byref(dims)))


@dataclass
class PagePool:
    """The reference counts of a paged cache's pages, what the last call did, and the workspace of the
    page calls (include/kivi.h)."""

    ref_counts: torch.Tensor  # int32 [num_pages]; a page is free when its count is not positive
    info: torch.Tensor        # int32 [4]
    ws: torch.Tensor          # uint8
    c: kivi_page_pool

    @classmethod
    def allocate(cls, cache: PagedCache) -> "PagePool":
        """A pool with every page free: the cache's block table is emptied."""
        pool = cls.adopt(cache, torch.zeros(cache.dims.num_pages, dtype=torch.int32, device=cache.k_codes.device))
        cache.block_table.fill_(-1)
        return pool

    @classmethod
    def adopt(cls, cache: PagedCache, ref_counts: torch.Tensor, info: torch.Tensor | None = None) -> "PagePool":
        """A pool over pages that the cache's block table holds already, with their counts."""
        dev = cache.k_codes.device
        nbytes = kivi_paged_pool_workspace_bytes(cache.dims)
        if nbytes == 0:
            raise KiviError(KIVI_ERR_UNSUPPORTED, "kivi_paged_pool_workspace_bytes")
        _i32(ref_counts, "ref_counts", cache.dims.num_pages, dev)
        if info is None:
            info = torch.zeros(4, dtype=torch.int32, device=dev)
        _i32(info, "info", 4, dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        c = kivi_page_pool(cache.block_table.data_ptr(), ref_counts.data_ptr(), info.data_ptr())
        return cls(ref_counts, info, ws, c)


def _pool_call(name: str, cache: PagedCache, pool: PagePool, array: torch.Tensor, what: str, numel: int,
               stream) -> None:
    dev = cache.k_codes.device
    at = _i32(array, what, numel, dev)
    _run(name, dev, stream, cache.dims, cache.c, pool.c, at, pool.ws.data_ptr(), pool.ws.numel())


def kivi_paged_reserve(cache: PagedCache, pool: PagePool, extra: torch.Tensor, stream=None) -> None:
    """Pages for extra[b] more tokens of every sequence b (int32 [B] on the device; <= 0: none)."""
    _pool_call("kivi_paged_reserve", cache, pool, extra, "extra", cache.dims.B, stream)


def kivi_paged_reserve_window(cache: PagedCache, pool: PagePool, extra: torch.Tensor, window: int, sinks: int,
                              stream=None) -> None:
    """kivi_paged_reserve for attention with a sliding window and sinks: of the sequences with extra[b] > 0, pages
    that no token to come sees are given back first, and their table entries get none."""
    dev = cache.k_codes.device
    at = _i32(extra, "extra", cache.dims.B, dev)
    _run("kivi_paged_reserve_window", dev, stream, cache.dims, cache.c, pool.c, at, _count(window, "window", 1),
         _count(sinks, "sinks", 0), pool.ws.data_ptr(), pool.ws.numel())


def kivi_paged_reorder(cache: PagedCache, pool: PagePool, parent: torch.Tensor, stream=None) -> None:
    """Sequence b becomes what sequence parent[b] was (int32 [B] on the device; -1: empty)."""
    _pool_call("kivi_paged_reorder", cache, pool, parent, "parent", cache.dims.B, stream)


def kivi_paged_compact(cache: PagedCache, pool: PagePool, new_ids: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """Move the pages in use to the low ids; the new id of every page (int32 [num_pages], -1: free)."""
    if new_ids is None:
        with _allocating_on(cache.k_codes.device, stream):
            new_ids = torch.empty_like(pool.ref_counts)
    _pool_call("kivi_paged_compact", cache, pool, new_ids, "new_ids", cache.dims.num_pages, stream)
    return new_ids
