"""Paged grouped-query attention at head_dim 512 for GB300 (sm_103a): Python binding.

This module only marshals arguments into the C ABI of ``libpaged_attn.so`` (declared in
include/paged_attn.h); every step of the computation runs in the library's CUDA kernels.  The
calls of a serving step go through a compiled module (csrc/binding.cpp), the others through
ctypes.
Tensors must already live on the GPU.  If the library has not been built, the calls raise
instead of falling back to anything else.

    out, lse = paged_attn_decode(q, kv_cache, kv_indptr, kv_indices, kv_last_page_len,
                                 num_kv_heads=4, head_dim_vo=512, page_size=64,
                                 sm_scale=512 ** -0.5)
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import Optional, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libpaged_attn.so")
BINDING_PATH = os.path.join(HERE, "_build", "_binding.so")

PA_KV_BF16, PA_KV_FP8_E4M3, PA_KV_NVFP4, PA_KV_INT8_BLOCK, PA_KV_FP8_BLOCK = 0, 1, 2, 3, 4
PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_ALIGNMENT = 0, -1, -2, -3
PA_ERR_SMEM, PA_ERR_CUDA, PA_ERR_DEVICE, PA_ERR_SCRATCH = -4, -5, -6, -7
PA_NOALLOC_SCRATCH_BYTES = 32 << 20

# every symbol include/paged_attn.h declares
EXPORTED = ("paged_attn_decode", "paged_attn_prefill", "paged_attn_status_string",
            "paged_attn_release_workspace", "paged_attn_check_device_error",
            "paged_attn_set_decode_chunk_pages", "paged_attn_set_decode_direct", "paged_attn_last_variant",
            "paged_attn_profile_begin", "paged_attn_profile_end", "paged_attn_decode_noalloc",
            "paged_attn_set_prefill_dequant_limit", "paged_attn_set_prefill_cta_pairs",
            "paged_attn_append_kv", "paged_attn_prefill_custom_mask", "paged_attn_set_prefill_split_kv",
            "paged_attn_debug_set_error_word", "paged_attn_append_kv_block", "paged_attn_resize_tables",
            "paged_attn_build_tables")

_lib = None


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {paged_attn_status_string(status)} (status {status})")


class _Scales(ctypes.Structure):
    _fields_ = [("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("sf", ctypes.c_void_p),
                ("block_scales", ctypes.c_void_p), ("block_tokens", ctypes.c_int)]


def load(path: Optional[str] = None):
    """Load libpaged_attn.so (build it with ``python -m paged_gqa_attention_hd512_gb300.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library not built: {p} is missing")
    lib = ctypes.CDLL(p)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.paged_attn_decode.restype = i32
    lib.paged_attn_decode.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, i32,
                                      i32, ctypes.POINTER(_Scales), vp, vp, vp]
    lib.paged_attn_decode_noalloc.restype = i32
    lib.paged_attn_decode_noalloc.argtypes = list(lib.paged_attn_decode.argtypes)
    lib.paged_attn_prefill.restype = i32
    lib.paged_attn_prefill.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                       f32, i32, i32, i32, ctypes.POINTER(_Scales), vp, vp, vp]
    lib.paged_attn_append_kv.restype = i32
    lib.paged_attn_append_kv.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                         vp, vp, vp, vp]
    lib.paged_attn_append_kv_block.restype = i32
    lib.paged_attn_append_kv_block.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                               vp, i32, vp]
    lib.paged_attn_resize_tables.restype = i32
    lib.paged_attn_resize_tables.argtypes = [vp, i32, i32, i32, vp, vp, vp, i32, i32, vp, i32, vp, vp]
    lib.paged_attn_build_tables.restype = i32
    lib.paged_attn_build_tables.argtypes = [vp, i32, i32, i32, vp, vp, vp, i32, i32, i32, vp, vp, i32, vp, vp, vp, vp,
                                            i32, vp]
    lib.paged_attn_prefill_custom_mask.restype = i32
    lib.paged_attn_prefill_custom_mask.argtypes = list(lib.paged_attn_prefill.argtypes[:-1]) + [vp, vp, vp]
    lib.paged_attn_status_string.restype = ctypes.c_char_p
    lib.paged_attn_status_string.argtypes = [i32]
    lib.paged_attn_release_workspace.restype = i32
    lib.paged_attn_check_device_error.restype = i32
    lib.paged_attn_check_device_error.argtypes = [ctypes.POINTER(ctypes.c_int)]
    lib.paged_attn_debug_set_error_word.restype = i32
    lib.paged_attn_debug_set_error_word.argtypes = [i32, i32]
    lib.paged_attn_set_decode_chunk_pages.restype = i32
    lib.paged_attn_set_decode_chunk_pages.argtypes = [i32]
    lib.paged_attn_set_decode_direct.restype = i32
    lib.paged_attn_set_decode_direct.argtypes = [i32]
    lib.paged_attn_set_prefill_dequant_limit.restype = i32
    lib.paged_attn_set_prefill_dequant_limit.argtypes = [ctypes.c_longlong]
    lib.paged_attn_set_prefill_cta_pairs.restype = i32
    lib.paged_attn_set_prefill_cta_pairs.argtypes = [i32]
    lib.paged_attn_set_prefill_split_kv.restype = i32
    lib.paged_attn_set_prefill_split_kv.argtypes = [i32]
    lib.paged_attn_last_variant.restype = i32
    lib.paged_attn_last_variant.argtypes = [ctypes.c_char_p, i32]
    lib.paged_attn_profile_begin.restype = i32
    lib.paged_attn_profile_begin.argtypes = [i32]
    lib.paged_attn_profile_end.restype = i32
    lib.paged_attn_profile_end.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float)]
    if path is None:
        _lib = lib
    return lib


_binding = None


def _load_binding():
    """The compiled binding of the serving calls (built with the library)."""
    global _binding
    if _binding is None:
        load()
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"Python binding not built: {BINDING_PATH} is missing")
        loader = importlib.machinery.ExtensionFileLoader("_binding", BINDING_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_binding", loader))
        loader.exec_module(module)
        _binding = module
    return _binding


def paged_attn_status_string(status: int) -> str:
    return load().paged_attn_status_string(status).decode()


def _ptr(t: Optional[torch.Tensor]):
    """The device address of a contiguous CUDA tensor (an int; ctypes passes it as a
    pointer), None for None."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


# the current stream's handle without building a Stream object (2.9 us a call on the GB300's
# host, against 0.1); torch.cuda.current_stream() where a torch build lacks it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _x2(kv_dtype: int) -> int:
    return {PA_KV_BF16: 4, PA_KV_FP8_E4M3: 2, PA_KV_NVFP4: 1, PA_KV_INT8_BLOCK: 2, PA_KV_FP8_BLOCK: 2}[kv_dtype]


def _typed(t: torch.Tensor, dtype: torch.dtype, numel: int, what: str):
    """_ptr(t) of a tensor that must have this dtype and at least numel elements."""
    if t.dtype != dtype or t.numel() < numel:
        raise ValueError(f"{what}: expected at least {numel} elements of {dtype}, got {t.numel()} of {t.dtype}")
    return _ptr(t)


def _block_scales(block_scales, block_tokens, num_pages, num_kv_heads, page_size):
    """The pointer of a block_scales pool, after checking that it covers the pages."""
    if block_scales is None or not 1 <= block_tokens <= page_size:
        raise ValueError("the block dtypes need block_scales and 1 <= block_tokens <= page_size")
    return _typed(block_scales, torch.float32, num_pages * 2 * num_kv_heads * (page_size // block_tokens),
                  "block_scales")


def _scales(kv_dtype, k_scale, v_scale, sf, block_scales, block_tokens, num_pages, num_kv_heads, page_size):
    sc = _Scales(None, None, None)
    if kv_dtype in (PA_KV_INT8_BLOCK, PA_KV_FP8_BLOCK):
        sc.block_scales = _block_scales(block_scales, block_tokens, num_pages, num_kv_heads, page_size)
        sc.block_tokens = block_tokens
    elif kv_dtype != PA_KV_BF16:
        sc.k_scale = _ptr(k_scale)
        sc.v_scale = _ptr(v_scale)
        sc.sf = _ptr(sf)
    return sc


def _num_pages(kv_cache, num_kv_heads, head_dim_qk, head_dim_vo, page_size, kv_dtype):
    page_bytes = num_kv_heads * page_size * (head_dim_qk + head_dim_vo) * _x2(kv_dtype) // 2
    return (kv_cache.numel() * kv_cache.element_size()) // page_bytes


def paged_attn_decode(q: torch.Tensor, kv_cache: torch.Tensor, kv_indptr: torch.Tensor,
                      kv_indices: torch.Tensor, kv_last_page_len: torch.Tensor, *,
                      num_kv_heads: int, head_dim_vo: int, page_size: int, sm_scale: float,
                      window_left: int = -1, kv_dtype: int = PA_KV_BF16,
                      k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                      sf: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, num_pages: Optional[int] = None,
                      stream=None, return_lse: bool = True, block_scales: Optional[torch.Tensor] = None,
                      block_tokens: int = 0) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Decode: q [batch, Hq, head_dim_qk] bf16 -> out [batch, Hq, head_dim_vo] bf16, lse [batch, Hq].
    block_scales [num_pages, 2, Hkv, page_size / block_tokens] (fp32) for the block dtypes."""
    st, out, lse = (_binding or _load_binding()).decode(
        q, kv_cache, kv_indptr, kv_indices, kv_last_page_len, out, lse, return_lse, stream, num_kv_heads, head_dim_vo,
        page_size, sm_scale, window_left, kv_dtype, k_scale, v_scale, sf, block_scales, block_tokens, num_pages)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_decode")
    return out, lse


def paged_attn_decode_noalloc(q: torch.Tensor, kv_cache: torch.Tensor, kv_indptr: torch.Tensor,
                              kv_indices: torch.Tensor, kv_last_page_len: torch.Tensor, *, out: torch.Tensor,
                              lse: Optional[torch.Tensor], num_kv_heads: int, head_dim_vo: int, page_size: int,
                              sm_scale: float, window_left: int = -1, kv_dtype: int = PA_KV_BF16,
                              k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                              sf: Optional[torch.Tensor] = None, num_pages: Optional[int] = None,
                              stream=None, block_scales: Optional[torch.Tensor] = None,
                              block_tokens: int = 0) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Decode for callers that cannot allocate device memory: the library uses only its
    fixed scratch array, and the caller passes ``out`` (and ``lse``) already allocated.
    Overlapping calls race on that array; serialise them."""
    batch, hq, dqk = q.shape
    if num_pages is None:
        num_pages = _num_pages(kv_cache, num_kv_heads, dqk, head_dim_vo, page_size, kv_dtype)
    sc = _scales(kv_dtype, k_scale, v_scale, sf, block_scales, block_tokens, num_pages, num_kv_heads, page_size)
    st = load().paged_attn_decode_noalloc(_ptr(q), _ptr(kv_cache), _ptr(kv_indptr), _ptr(kv_indices),
                                          _ptr(kv_last_page_len), batch, num_pages, hq, num_kv_heads, dqk,
                                          head_dim_vo, page_size, float(sm_scale), window_left, kv_dtype,
                                          ctypes.byref(sc), _ptr(out), _ptr(lse), _stream(stream))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_decode_noalloc")
    return out, lse


def paged_attn_prefill(q: torch.Tensor, qo_indptr: torch.Tensor, kv_cache: torch.Tensor,
                       kv_indptr: torch.Tensor, kv_indices: torch.Tensor,
                       kv_last_page_len: torch.Tensor, *, num_kv_heads: int, head_dim_vo: int,
                       page_size: int, sm_scale: float, window_left: int = -1, causal: bool = True,
                       kv_dtype: int = PA_KV_BF16, k_scale: Optional[torch.Tensor] = None,
                       v_scale: Optional[torch.Tensor] = None, sf: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       num_pages: Optional[int] = None, stream=None,
                       return_lse: bool = True, custom_mask: Optional[torch.Tensor] = None,
                       mask_indptr: Optional[torch.Tensor] = None, block_scales: Optional[torch.Tensor] = None,
                       block_tokens: int = 0) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Prefill: q [total_q, Hq, head_dim_qk] bf16 -> out [total_q, Hq, head_dim_vo] bf16.
    custom_mask (uint8 bits) with mask_indptr (int64 byte offsets per sequence) selects
    paged_attn_prefill_custom_mask.  block_scales as for paged_attn_decode."""
    st, out, lse = (_binding or _load_binding()).prefill(
        q, qo_indptr, kv_cache, kv_indptr, kv_indices, kv_last_page_len, bool(causal), custom_mask, mask_indptr, out,
        lse, return_lse, stream, num_kv_heads, head_dim_vo, page_size, sm_scale, window_left, kv_dtype, k_scale,
        v_scale, sf, block_scales, block_tokens, num_pages)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_prefill" if custom_mask is None else "paged_attn_prefill_custom_mask")
    return out, lse


def paged_attn_append_kv(k_new: torch.Tensor, v_new: torch.Tensor, append_indptr: torch.Tensor,
                         kv_cache: torch.Tensor, kv_indptr: torch.Tensor, kv_indices: torch.Tensor,
                         kv_last_page_len: torch.Tensor, *, page_size: int, kv_dtype: int = PA_KV_BF16,
                         k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                         sf: Optional[torch.Tensor] = None, num_pages: Optional[int] = None,
                         stream=None) -> None:
    """Write k_new [total_new, Hkv, head_dim_qk] / v_new [total_new, Hkv, head_dim_vo] (bf16)
    as the last tokens of each sequence, converted to the cache's element type."""
    total_new, hkv, dqk = k_new.shape
    dvo = v_new.shape[2]
    batch = append_indptr.numel() - 1
    if num_pages is None:
        num_pages = _num_pages(kv_cache, hkv, dqk, dvo, page_size, kv_dtype)
    st = load().paged_attn_append_kv(_ptr(k_new), _ptr(v_new), _ptr(append_indptr), total_new, _ptr(kv_cache),
                                     _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_last_page_len), batch,
                                     num_pages, hkv, dqk, dvo, page_size, kv_dtype, _ptr(k_scale),
                                     _ptr(v_scale), _ptr(sf), _stream(stream))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_append_kv")


def paged_attn_append_kv_block(k_new: torch.Tensor, v_new: torch.Tensor, append_indptr: torch.Tensor,
                               kv_cache: torch.Tensor, kv_indptr: torch.Tensor, kv_indices: torch.Tensor,
                               kv_last_page_len: torch.Tensor, block_scales: torch.Tensor, *, page_size: int,
                               block_tokens: int, kv_dtype: int = PA_KV_INT8_BLOCK, num_pages: Optional[int] = None,
                               stream=None) -> None:
    """Write k_new [total_new, Hkv, head_dim_qk] / v_new [total_new, Hkv, head_dim_vo] (bf16) as
    8-bit codes of the last tokens of each sequence, and the scales of the blocks they fall
    into: block_scales [num_pages, 2, Hkv, page_size / block_tokens] (fp32)."""
    st = (_binding or _load_binding()).append_kv_block(
        k_new, v_new, append_indptr, kv_cache, kv_indptr, kv_indices, kv_last_page_len, block_scales, page_size,
        block_tokens, kv_dtype, num_pages, stream)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_append_kv_block")


def paged_attn_resize_tables(block_table: torch.Tensor, row_ids: Optional[torch.Tensor], kv_lens: torch.Tensor,
                             deltas: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor, *,
                             page_size: int, stream=None) -> None:
    """Change the length of sequence b (row row_ids[b] of block_table [rows, max_pages], or row b)
    by deltas[b] tokens, moving pages between its row and the free list (free_pages, the first
    free_count[0] entries free); kv_lens [rows] and free_count [1] are updated.  All int32."""
    st = (_binding or _load_binding()).resize_tables(block_table, row_ids, kv_lens, deltas, free_pages, free_count,
                                                     page_size, stream)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_resize_tables")


def paged_attn_build_tables(block_table: torch.Tensor, row_ids: Optional[torch.Tensor], kv_lens: torch.Tensor,
                            new_counts: torch.Tensor, *, page_size: int, num_pages: int, max_indices: int,
                            num_tokens: int, out: Optional[Tuple[torch.Tensor, ...]] = None,
                            stream=None) -> Tuple[torch.Tensor, ...]:
    """Page table of a batch, its last new_counts[b] tokens per sequence being new:
    (kv_indptr [batch + 1], kv_indices [max_indices], kv_last_page_len [batch], new_indptr
    [batch + 1], slot_map int64 [num_tokens], positions [num_tokens]), int32 but for slot_map.
    max_indices and num_tokens are capacities; ``out`` gives the six tensors to write."""
    st, out = (_binding or _load_binding()).build_tables(block_table, row_ids, kv_lens, new_counts, page_size,
                                                         num_pages, max_indices, num_tokens, out, stream)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_build_tables")
    return out


def paged_attn_release_workspace() -> None:
    st = load().paged_attn_release_workspace()
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_release_workspace")


def paged_attn_check_device_error() -> int:
    """Synchronise and return the device error word (0 = none); raises on a CUDA error."""
    code = ctypes.c_int(0)
    st = load().paged_attn_check_device_error(ctypes.byref(code))
    if st not in (PA_OK, PA_ERR_DEVICE):
        raise PagedAttnError(st, "paged_attn_check_device_error")
    return code.value


def paged_attn_debug_set_error_word(target: int, code: int) -> None:
    """Test hook: store ``code`` in the workspace's (0) or the no-alloc array's (1) device
    error word."""
    st = load().paged_attn_debug_set_error_word(target, code)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_debug_set_error_word")


def paged_attn_set_decode_chunk_pages(pages: int) -> None:
    st = load().paged_attn_set_decode_chunk_pages(pages)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_set_decode_chunk_pages")


def paged_attn_set_decode_direct(mode: int) -> None:
    """Single-launch decode: -1 where the library's rule applies (default), 0 never, 1
    whenever every (sequence, kv head) item fits one round of CTAs."""
    st = load().paged_attn_set_decode_direct(mode)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_set_decode_direct")


def paged_attn_set_prefill_dequant_limit(nbytes: int) -> None:
    """Largest bf16 copy of FP8 / NVFP4 pages the prefill may build (0: convert inside the
    kernel; negative: the library default)."""
    st = load().paged_attn_set_prefill_dequant_limit(nbytes)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_set_prefill_dequant_limit")


def paged_attn_set_prefill_cta_pairs(mode: int) -> None:
    """1: bf16 prefill on CTA pairs whenever two-CTA clusters fit; 0 or -1 (default): one
    CTA per query tile."""
    st = load().paged_attn_set_prefill_cta_pairs(mode)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_set_prefill_cta_pairs")


def paged_attn_set_prefill_split_kv(mode: int) -> None:
    """-1 (default): prefills that leave SMs idle may split long KV ranges; 0: never."""
    st = load().paged_attn_set_prefill_split_kv(mode)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_set_prefill_split_kv")


def paged_attn_last_variant() -> str:
    buf = ctypes.create_string_buffer(64)
    load().paged_attn_last_variant(buf, 64)
    return buf.value.decode()


def paged_attn_profile_begin(max_launches: int) -> None:
    st = load().paged_attn_profile_begin(max_launches)
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_profile_begin")


def paged_attn_profile_end() -> Tuple[int, float]:
    """(recorded launches, summed device milliseconds of the main kernel)."""
    n, ms = ctypes.c_int(0), ctypes.c_float(0.0)
    st = load().paged_attn_profile_end(ctypes.byref(n), ctypes.byref(ms))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_profile_end")
    return n.value, ms.value


def case_args(case) -> dict:
    """Keyword arguments of a synth.Case (already on the GPU) for the two calls."""
    kw = dict(num_kv_heads=case.Hkv, head_dim_vo=case.d_vo, page_size=case.page_size,
              sm_scale=case.sm_scale, window_left=case.window_left, kv_dtype=case.kv_dtype,
              num_pages=case.num_pages)
    if case.kv_dtype != PA_KV_BF16:
        dev = case.q.device
        kw["k_scale"] = torch.tensor([case.k_scale], dtype=torch.float32, device=dev)
        kw["v_scale"] = torch.tensor([case.v_scale], dtype=torch.float32, device=dev)
        if case.kv_dtype == PA_KV_NVFP4:
            kw["sf"] = case.sf
    if case.phase == "prefill" and getattr(case, "mask", None) is not None:
        kw["custom_mask"] = case.mask
        kw["mask_indptr"] = case.mask_indptr
    return kw


def run_case(case, **extra):
    """Run the call that matches case.phase on a synth.Case that lives on the GPU."""
    kw = case_args(case)
    kw.update(extra)
    if case.phase == "decode":
        return paged_attn_decode(case.q, case.kv_cache, case.kv_indptr, case.kv_indices,
                                 case.kv_last_page_len, **kw)
    return paged_attn_prefill(case.q, case.qo_indptr, case.kv_cache, case.kv_indptr, case.kv_indices,
                              case.kv_last_page_len, causal=bool(case.causal), **kw)
