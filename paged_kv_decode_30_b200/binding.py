"""ctypes binding of the C ABI in ``include/paged_decode_attn.h``.

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the CUDA stream, and the library does every step of the
computation. If the shared library is missing, loading raises; there is no
fallback implementation.
"""

from __future__ import annotations

import ctypes
import os
import sys
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libpaged_decode_attn.so")

PDA_KV_BF16 = 0
PDA_KV_FP8_E4M3 = 1
PDA_KV_NVFP4 = 2
PDA_CAUSAL_OFF = -1
PDA_CAUSAL_BOTTOM_RIGHT = -2
PDA_FLAG_NO_PDL = 1
PDA_FLAG_TENSOR_CORES = 2
PDA_FLAG_CUDA_CORES = 4
PDA_FLAG_FUSED_MERGE = 8
PDA_FLAG_NATIVE_FP8_QK = 16
# Size of the library's fixed workspace array used by paged_decode_attn_no_alloc.
PDA_NO_ALLOC_WORKSPACE_BYTES = 16 * 1024 * 1024

STATUS = {
    0: "PDA_OK", 1: "PDA_ERR_INVALID_ARG", 2: "PDA_ERR_UNSUPPORTED",
    3: "PDA_ERR_MISALIGNED", 4: "PDA_ERR_WORKSPACE", 5: "PDA_ERR_CUDA",
    6: "PDA_ERR_BAD_PAGE", 7: "PDA_ERR_TIMEOUT",
}

# Every symbol the header declares (checked by the CPU test suite).
EXPORTED = (
    "paged_decode_attn", "paged_decode_attn_no_alloc", "paged_decode_attn_workspace_bytes",
    "pda_choose_num_splits", "pda_merge_states", "pda_status_string",
    "pda_last_device_error", "pda_abi_version", "pda_plan_kernel", "pda_hbm_read_probe",
    "paged_kv_append", "paged_latent_append", "paged_latent_gather", "paged_latent_decode",
    "paged_latent_decode_workspace_bytes", "latent_prefill_attn",
)
PDA_KERNEL_SPLIT_FMA = 0
PDA_KERNEL_SPLIT_TMA = 1
KERNEL_NAMES = {PDA_KERNEL_SPLIT_FMA: "split_fma_kernel", PDA_KERNEL_SPLIT_TMA: "split_tma_kernel"}


class PdaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class PdaAppendParams(ctypes.Structure):
    """Mirror of ``pda_append_params``."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_new", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("kv_scale", ctypes.c_float),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
    ]


class PdaParams(ctypes.Structure):
    """Mirror of ``pda_params``."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("causal_offset", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("kv_scale", ctypes.c_float),
        ("max_kv_len", ctypes.c_int32),
        ("num_splits", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("num_splits_out", ctypes.POINTER(ctypes.c_int32)),
        ("sinks", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
    ]


class PdaLatentRowsParams(ctypes.Structure):
    """Mirror of ``pda_latent_rows_params``."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("total_rows", ctypes.c_int32),
        ("latent_dim", ctypes.c_int32),
        ("rope_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("latent_stride", ctypes.c_int64),
        ("rope_stride", ctypes.c_int64),
        ("latent_scales", ctypes.c_void_p),
    ]


class PdaLatentParams(ctypes.Structure):
    """Mirror of ``pda_latent_params``."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("latent_dim", ctypes.c_int32),
        ("rope_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("causal_offset", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("latent_scales", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class PdaLatentPrefillParams(ctypes.Structure):
    """Mirror of ``pda_latent_prefill_params``."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("total_q", ctypes.c_int32),
        ("total_kv", ctypes.c_int32),
        ("max_q_len", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("rope_dim", ctypes.c_int32),
        ("k_rope_stride", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("causal_offset", ctypes.c_int32),
        ("window", ctypes.c_int32),
    ]


_lib = None
# What works without tensors (load, planning, sizes) works without torch. The latent
# calls, in which an import statement shows, use this name, set by the first of them.
torch = sys.modules.get("torch")


def _with_torch():
    global torch
    import torch


def load(path: Optional[str] = None):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if path is None and _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build it with `python -m paged_kv_decode_30_b200.build`"
            " (there is no CPU fallback)")
    lib = ctypes.CDLL(p)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    pp = ctypes.POINTER(PdaParams)
    lib.paged_decode_attn.restype = i32
    lib.paged_decode_attn.argtypes = [vp, vp, vp, vp, vp, pp, vp, vp, vp]
    lib.paged_decode_attn_no_alloc.restype = i32
    lib.paged_decode_attn_no_alloc.argtypes = [vp, vp, vp, vp, vp, pp, vp, vp, vp]
    lib.paged_decode_attn_workspace_bytes.restype = ctypes.c_size_t
    lib.paged_decode_attn_workspace_bytes.argtypes = [pp]
    lib.pda_choose_num_splits.restype = i32
    lib.pda_choose_num_splits.argtypes = [pp, i32]
    lib.pda_merge_states.restype = i32
    lib.pda_merge_states.argtypes = [vp, vp, i32, i64, i32, vp, vp, vp, i32, vp]
    lib.pda_status_string.restype = ctypes.c_char_p
    lib.pda_status_string.argtypes = [i32]
    lib.pda_last_device_error.restype = i32
    lib.pda_last_device_error.argtypes = [vp]
    lib.pda_abi_version.restype = i32
    lib.pda_abi_version.argtypes = []
    lib.pda_plan_kernel.restype = i32
    lib.pda_plan_kernel.argtypes = [pp]
    lib.paged_kv_append.restype = i32
    lib.paged_kv_append.argtypes = [vp, vp, vp, vp, ctypes.POINTER(PdaAppendParams), vp, vp, vp]
    lib.pda_hbm_read_probe.restype = i32
    lib.pda_hbm_read_probe.argtypes = [vp, ctypes.c_size_t, vp, vp]
    rp = ctypes.POINTER(PdaLatentRowsParams)
    lib.paged_latent_append.restype = i32
    lib.paged_latent_append.argtypes = [vp, vp, vp, vp, vp, rp, vp, vp, vp]
    lib.paged_latent_gather.restype = i32
    lib.paged_latent_gather.argtypes = [vp, vp, vp, vp, vp, rp, vp, vp, vp]
    lp = ctypes.POINTER(PdaLatentParams)
    lib.paged_latent_decode.restype = i32
    lib.paged_latent_decode.argtypes = [vp, vp, vp, vp, vp, lp, vp, vp, vp]
    lib.paged_latent_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.paged_latent_decode_workspace_bytes.argtypes = [lp]
    lib.latent_prefill_attn.restype = i32
    lib.latent_prefill_attn.argtypes = [vp, vp, vp, vp, vp, ctypes.POINTER(PdaLatentPrefillParams),
                                        vp, vp, vp]
    if path is None:
        _lib = lib
    return lib


def make_params(*, batch, q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                max_pages_per_seq, num_pages, scale, causal_offset=PDA_CAUSAL_OFF,
                window=0, kv_dtype=PDA_KV_BF16, kv_scale=1.0, max_kv_len=0,
                num_splits=0, flags=0) -> PdaParams:
    p = PdaParams()
    p.batch, p.q_len = batch, q_len
    p.num_q_heads, p.num_kv_heads = num_q_heads, num_kv_heads
    p.head_dim, p.page_size = head_dim, page_size
    p.max_pages_per_seq, p.num_pages = max_pages_per_seq, num_pages
    p.scale = scale
    p.causal_offset, p.window = causal_offset, window
    p.kv_dtype, p.kv_scale = kv_dtype, kv_scale
    p.max_kv_len, p.num_splits, p.flags = max_kv_len, num_splits, flags
    p.workspace = None
    p.workspace_bytes = 0
    return p


def status_string(status: int) -> str:
    return load().pda_status_string(status).decode()


def choose_num_splits(params: PdaParams, num_sms: int) -> int:
    return load().pda_choose_num_splits(ctypes.byref(params), num_sms)


def plan_kernel(params: PdaParams) -> int:
    """PDA_KERNEL_SPLIT_FMA or PDA_KERNEL_SPLIT_TMA (-1: invalid params)."""
    return load().pda_plan_kernel(ctypes.byref(params))


def hbm_read_probe(buf, sink, stream=None):
    """Read every byte of the CUDA tensor ``buf`` once (bandwidth probe);
    ``sink`` is an 8-byte CUDA tensor the kernel XORs into."""
    st = load().pda_hbm_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                   _stream_handle(stream))
    if st != 0:
        raise PdaError(st, "pda_hbm_read_probe")


def workspace_bytes(params: PdaParams) -> int:
    return load().paged_decode_attn_workspace_bytes(ctypes.byref(params))


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream or None


def _params_for(q, k_pages, v_pages, page_table, kv_lens, k_scales, v_scales, **kw):
    """pda_params for CUDA tensors (checks they are contiguous CUDA tensors);
    the KV dtype follows the pools: bf16, uint8 e4m3 codes, or uint8 NVFP4
    codes when block-scale pools are given."""
    import torch
    B, q_len, Hq, D = q.shape
    for t in (q, k_pages, v_pages, page_table, kv_lens):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all inputs must be contiguous CUDA tensors")
    if k_scales is not None or v_scales is not None:
        for t in (k_scales, v_scales):
            if t is None or not t.is_cuda or not t.is_contiguous() or t.dtype != torch.uint8:
                raise ValueError("k_scales and v_scales must be contiguous uint8 CUDA tensors")
        kv_dtype = PDA_KV_NVFP4
    else:
        kv_dtype = PDA_KV_FP8_E4M3 if k_pages.dtype == torch.uint8 else PDA_KV_BF16
    params = make_params(
        batch=B, q_len=q_len, num_q_heads=Hq, head_dim=D, page_size=k_pages.shape[2],
        max_pages_per_seq=page_table.shape[1], num_pages=k_pages.shape[0],
        kv_dtype=kv_dtype, **kw)
    if kv_dtype == PDA_KV_NVFP4:
        params.k_scales = k_scales.data_ptr()
        params.v_scales = v_scales.data_ptr()
    return params


def paged_decode_attn(q, k_pages, v_pages, page_table, kv_lens, *, num_kv_heads,
                      scale, causal_offset=PDA_CAUSAL_OFF, window=0, kv_scale=1.0,
                      max_kv_len=0, num_splits=0, flags=0, out=None, lse=None,
                      workspace=None, stream=None, with_lse=True, sinks=None,
                      library_workspace=False, k_scales=None, v_scales=None):
    """Run the library on CUDA tensors; returns (out, lse, num_splits_used).

    q [B, q_len, Hq, D] bf16; k/v_pages [num_pages, Hkv, P, D] bf16 or uint8
    (e4m3 codes), or with k_scales / v_scales (uint8 [num_pages, Hkv, P,
    D/16] e4m3 block scales) uint8 [num_pages, Hkv, P, D/2] NVFP4 codes;
    page_table int32 [B, max_pages]; kv_lens int32 [B];
    sinks: optional float32 CUDA tensor [Hq] of attention-sink logits.
    ``workspace``: a CUDA uint8 tensor (any contents; reusable across calls),
    or None to let the binding allocate exactly what the call needs.
    ``library_workspace``: pass no workspace, so the library uses (and grows
    in stream order) the buffer it owns on the device.
    """
    import torch
    lib = load()
    B, q_len, Hq, D = q.shape
    params = _params_for(q, k_pages, v_pages, page_table, kv_lens, k_scales, v_scales,
                         num_kv_heads=num_kv_heads, scale=scale, causal_offset=causal_offset,
                         window=window, kv_scale=kv_scale, max_kv_len=max_kv_len,
                         num_splits=num_splits, flags=flags)
    if out is None:
        out = torch.empty((B, q_len, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None and with_lse:
        lse = torch.empty((B, q_len, Hq), dtype=torch.float32, device=q.device)
    if workspace is None and not library_workspace:
        need = lib.paged_decode_attn_workspace_bytes(ctypes.byref(params))
        if need == ctypes.c_size_t(-1).value:
            raise PdaError(1, "paged_decode_attn_workspace_bytes")
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if workspace is not None:
        params.workspace = workspace.data_ptr()
        params.workspace_bytes = workspace.numel() * workspace.element_size()
    if sinks is not None:
        if not (sinks.is_cuda and sinks.dtype == torch.float32 and sinks.numel() == Hq):
            raise ValueError("sinks must be a float32 CUDA tensor of num_q_heads entries")
        params.sinks = sinks.data_ptr()
    used = ctypes.c_int32(0)
    params.num_splits_out = ctypes.pointer(used)
    st = lib.paged_decode_attn(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(kv_lens),
        ctypes.byref(params), _ptr(out), _ptr(lse), _stream_handle(stream))
    if st != 0:
        raise PdaError(st, "paged_decode_attn")
    return out, lse, used.value


def paged_decode_attn_no_alloc(q, k_pages, v_pages, page_table, kv_lens, *,
                               num_kv_heads, scale, causal_offset=PDA_CAUSAL_OFF,
                               window=0, kv_scale=1.0, max_kv_len=0, num_splits=0,
                               flags=0, out=None, lse=None, stream=None, sinks=None,
                               k_scales=None, v_scales=None):
    """The allocation-free entry point: the call's whole workspace goes to
    the library's fixed device array (see the C header). Same arguments as
    paged_decode_attn minus ``workspace``. ``out`` and ``lse`` are allocated
    here by torch only when the caller passes None."""
    import torch
    lib = load()
    B, q_len, Hq, D = q.shape
    params = _params_for(q, k_pages, v_pages, page_table, kv_lens, k_scales, v_scales,
                         num_kv_heads=num_kv_heads, scale=scale, causal_offset=causal_offset,
                         window=window, kv_scale=kv_scale, max_kv_len=max_kv_len,
                         num_splits=num_splits, flags=flags)
    if out is None:
        out = torch.empty((B, q_len, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, q_len, Hq), dtype=torch.float32, device=q.device)
    for t in (out, lse):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float32:
            raise ValueError("out and lse must be contiguous float32 CUDA tensors")
    if sinks is not None:
        if not (sinks.is_cuda and sinks.dtype == torch.float32 and sinks.numel() == Hq):
            raise ValueError("sinks must be a float32 CUDA tensor of num_q_heads entries")
        params.sinks = sinks.data_ptr()
    used = ctypes.c_int32(0)
    params.num_splits_out = ctypes.pointer(used)
    st = lib.paged_decode_attn_no_alloc(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(kv_lens),
        ctypes.byref(params), _ptr(out), _ptr(lse), _stream_handle(stream))
    if st != 0:
        raise PdaError(st, "paged_decode_attn_no_alloc")
    return out, lse, used.value


def paged_kv_append(k_new, v_new, page_table, kv_lens, k_pages, v_pages, *, kv_scale=1.0,
                    stream=None, k_scales=None, v_scales=None):
    """Write new K/V rows (bf16 [B, num_new, Hkv, D]) into the pools at
    positions kv_lens[b] + t (kv_lens is not advanced). Pools of uint8 are
    e4m3 codes quantised with kv_scale, or, with k_scales / v_scales (uint8
    block-scale pools), NVFP4 codes; bf16 pools get the bits."""
    import torch
    B, T, Hkv, D = k_new.shape
    kv_dtype = PDA_KV_FP8_E4M3 if k_pages.dtype == torch.uint8 else PDA_KV_BF16
    tensors = [k_new, v_new, page_table, kv_lens, k_pages, v_pages]
    if k_scales is not None or v_scales is not None:
        kv_dtype = PDA_KV_NVFP4
        tensors += [k_scales, v_scales]
    for t_ in tensors:
        if t_ is None or not t_.is_cuda or not t_.is_contiguous():
            raise ValueError("all inputs must be contiguous CUDA tensors")
    p = PdaAppendParams(B, T, Hkv, D, k_pages.shape[2], page_table.shape[1], k_pages.shape[0],
                        kv_dtype, kv_scale, _ptr(k_scales), _ptr(v_scales))
    st = load().paged_kv_append(_ptr(k_new), _ptr(v_new), _ptr(page_table), _ptr(kv_lens),
                                ctypes.byref(p), _ptr(k_pages), _ptr(v_pages),
                                _stream_handle(stream))
    if st != 0:
        raise PdaError(st, "paged_kv_append")


def merge_states(o_parts, lse_parts, *, out=None, lse=None, sinks=None, stream=None):
    """LSE merge: o_parts [S, rows, D] fp32, lse_parts [S, rows] fp32; sinks
    optional fp32 [Hq] (row r uses sinks[r % Hq])."""
    import torch
    S, rows, D = o_parts.shape
    if out is None:
        out = torch.empty((rows, D), dtype=torch.float32, device=o_parts.device)
    if lse is None:
        lse = torch.empty((rows,), dtype=torch.float32, device=o_parts.device)
    st = load().pda_merge_states(_ptr(o_parts), _ptr(lse_parts), S, rows, D,
                                 _ptr(out), _ptr(lse), _ptr(sinks),
                                 0 if sinks is None else sinks.numel(), _stream_handle(stream))
    if st != 0:
        raise PdaError(st, "pda_merge_states")
    return out, lse


def _check(name, t, dtype, shape, device, rows=False):
    """Raise ValueError unless t is a tensor of this type and shape on `device`,
    contiguous (``rows``: unit stride within a row is enough)."""
    if t.dtype is dtype and t.shape == shape and t.device == device and (
            t.is_contiguous() or (rows and t.stride(-1) == 1)):
        return
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, not {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _sizes(name, t, dims):
    """The sizes of a tensor that must have `dims` dimensions."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {t.dim()}")
    return t.shape


def _current_stream(device, stream=None):
    """The CUDA stream handle of a call on tensors of `device`: the given stream,
    or the current one. The library works on the current device, so tensors of
    another are refused."""
    if device.type != "cuda" or device.index != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on {device}, which is not the current CUDA device")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
        return stream.cuda_stream or None
    # (the handle itself: the Stream object around it costs two microseconds; and a
    # CUDA tensor is there, so that nothing is left to initialise)
    return torch._C._cuda_getCurrentRawStream(device.index) or None


def _check_mask(causal_offset, window):
    """Refuse what would not arrive: the library's fields have 32 bits."""
    if not -0x80000000 <= min(causal_offset, window) <= max(causal_offset, window) <= 0x7FFFFFFF:
        raise ValueError("causal_offset and window must fit 32 bits")


def _on(stream, call, *args, **kw):
    """`call` with `stream` as the current stream, so that what it allocates is ordered
    on that stream (a block that the caller's stream gave back may still be in use
    there). The allocator learns that both streams use the results."""
    if torch is None:
        _with_torch()
    caller = torch.cuda.current_stream(args[0].device)
    with torch.cuda.stream(stream):
        res = call(*args, **kw)
    for t in (*res, kw.get("workspace")):
        if t is not None:
            t.record_stream(caller)
            t.record_stream(stream)
    return res


def _row_stride(t):
    """Elements between the rows of a [rows, width] tensor (one row has none:
    its width, which any row count accepts)."""
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def _latent_pools(latent_pages, rope_pages, latent_scales, page_table):
    """Check the pools of a latent cache and its page table. Returns their device,
    (num_pages, page_size, latent_dim), rope_dim, (batch, max_pages) and KV dtype."""
    if torch is None:
        _with_torch()
    dev = latent_pages.device
    pools = _sizes("latent_pages", latent_pages, 3)
    num_pages, page, _ = pools
    rope_dim = _sizes("rope_pages", rope_pages, 3)[2]
    table = _sizes("page_table", page_table, 2)
    fp8 = latent_pages.dtype is torch.uint8
    # (one expression for what fits, the checks one by one for what does not: these
    # calls are short, and a Python call a tensor shows)
    if not ((fp8 or latent_pages.dtype is torch.bfloat16) and rope_pages.dtype is torch.bfloat16
            and page_table.dtype is torch.int32 and rope_pages.shape == (num_pages, page, rope_dim)
            and rope_pages.device == dev and page_table.device == dev
            and latent_pages.is_contiguous() and rope_pages.is_contiguous()
            and page_table.is_contiguous()):
        _check("latent_pages", latent_pages, torch.uint8 if fp8 else torch.bfloat16, pools, dev)
        _check("rope_pages", rope_pages, torch.bfloat16, (num_pages, page, rope_dim), dev)
        _check("page_table", page_table, torch.int32, table, dev)
    if fp8:
        if latent_scales is None:
            raise ValueError("uint8 latent_pages need latent_scales")
        _check("latent_scales", latent_scales, torch.uint8, (num_pages, page), dev)
    elif latent_scales is not None:
        raise ValueError("latent_scales go with uint8 latent_pages")
    return dev, pools, rope_dim, table, PDA_KV_FP8_E4M3 if fp8 else PDA_KV_BF16


def _latent_rows(latent, rope, row_offsets, page_table, starts, latent_pages, rope_pages,
                 latent_scales):
    dev, (num_pages, page, width), rope_dim, (batch, max_pages), kv_dtype = _latent_pools(
        latent_pages, rope_pages, latent_scales, page_table)
    rows = _sizes("latent", latent, 2)[0]
    c_strides = latent.stride()
    if not (latent.dtype is torch.bfloat16 and rope.dtype is torch.bfloat16
            and row_offsets.dtype is torch.int32 and latent.shape == (rows, width)
            and rope.shape == (rows, rope_dim) and row_offsets.shape == (batch + 1,)
            and latent.device == dev and rope.device == dev and row_offsets.device == dev
            and c_strides[1] == 1 and (r_strides := rope.stride())[1] == 1
            and row_offsets.is_contiguous()):
        _check("latent", latent, torch.bfloat16, (rows, width), dev, rows=True)
        _check("rope", rope, torch.bfloat16, (rows, rope_dim), dev, rows=True)
        _check("row_offsets", row_offsets, torch.int32, (batch + 1,), dev)
    if starts is not None and not (starts.dtype is torch.int32 and starts.shape == (batch,)
                                   and starts.device == dev and starts.is_contiguous()):
        _check("kv_lens / starts", starts, torch.int32, (batch,), dev)
    if rows < 2:  # one row has no stride: its width, which any row count accepts
        c_strides, r_strides = (width,), (rope_dim,)
    return PdaLatentRowsParams(batch, rows, width, rope_dim, page, max_pages, num_pages, kv_dtype,
                               c_strides[0], r_strides[0],
                               None if latent_scales is None else latent_scales.data_ptr())


def paged_latent_append(latent, rope, row_offsets, page_table, kv_lens, latent_pages, rope_pages,
                        *, latent_scales=None, stream=None):
    """Write ragged new rows into a latent cache: rows row_offsets[b] ..
    row_offsets[b + 1] of latent (bf16 [rows, R]) and rope (bf16 [rows, Dr])
    go to positions kv_lens[b], kv_lens[b] + 1, ... of sequence b (kv_lens is
    not advanced). latent_pages [num_pages, P, R] bf16 takes the bits; uint8
    takes e4m3 codes, and latent_scales (uint8 [num_pages, P]) each row's
    power-of-two scale. latent and rope may be column slices of one tensor."""
    p = _latent_rows(latent, rope, row_offsets, page_table, kv_lens, latent_pages, rope_pages,
                     latent_scales)
    st = load().paged_latent_append(latent.data_ptr(), rope.data_ptr(), row_offsets.data_ptr(),
                                    page_table.data_ptr(), _ptr(kv_lens), p,
                                    latent_pages.data_ptr(), rope_pages.data_ptr(),
                                    _current_stream(latent.device, stream))
    if st != 0:
        raise PdaError(st, "paged_latent_append")


def paged_latent_gather(latent_pages, rope_pages, page_table, row_offsets, *, total_rows=None,
                        starts=None, latent_scales=None, latent=None, rope=None, stream=None):
    """Read rows of a latent cache back as bf16: positions starts[b] (default
    0), starts[b] + 1, ... of sequence b become rows row_offsets[b] ..
    row_offsets[b + 1] of the outputs. Returns (latent [rows, R], rope [rows,
    Dr]): the given ones (rows behind row_offsets[B] are left alone), or new
    ones of total_rows rows."""
    if stream is not None:
        return _on(stream, paged_latent_gather, latent_pages, rope_pages, page_table, row_offsets,
                   total_rows=total_rows, starts=starts, latent_scales=latent_scales, latent=latent,
                   rope=rope)
    if latent is None or rope is None:
        if total_rows is None:
            raise ValueError("total_rows is needed to allocate the outputs")
        if latent is None:
            latent = rope_pages.new_empty((total_rows, _sizes("latent_pages", latent_pages, 3)[2]))
        if rope is None:
            rope = rope_pages.new_empty((total_rows, _sizes("rope_pages", rope_pages, 3)[2]))
    p = _latent_rows(latent, rope, row_offsets, page_table, starts, latent_pages, rope_pages,
                     latent_scales)
    st = load().paged_latent_gather(latent_pages.data_ptr(), rope_pages.data_ptr(),
                                    page_table.data_ptr(), row_offsets.data_ptr(), _ptr(starts), p,
                                    latent.data_ptr(), rope.data_ptr(),
                                    _current_stream(latent.device))
    if st != 0:
        raise PdaError(st, "paged_latent_gather")
    return latent, rope


def paged_latent_decode(q, latent_pages, rope_pages, page_table, kv_lens, *, scale,
                        causal_offset=PDA_CAUSAL_OFF, window=0, latent_scales=None, out=None,
                        lse=None, with_lse=True, workspace=None, library_workspace=False, flags=0,
                        stream=None):
    """Decode attention over a latent cache in the absorbed form; returns
    (out, lse). q bf16 [B, q_len, H, R + Dr] holds each head's query against
    the latents and its rotated part; out bf16 [B, q_len, H, R] is the weighted
    sum of latents, lse fp32 [B, q_len, H]. Pools as for paged_latent_append;
    masks and workspace as for paged_decode_attn."""
    if stream is not None:
        return _on(stream, paged_latent_decode, q, latent_pages, rope_pages, page_table, kv_lens,
                   scale=scale, causal_offset=causal_offset, window=window,
                   latent_scales=latent_scales, out=out, lse=lse, with_lse=with_lse,
                   workspace=workspace, library_workspace=library_workspace, flags=flags)
    lib = load()
    dev, (num_pages, page, width), rope_dim, (B, max_pages), kv_dtype = _latent_pools(
        latent_pages, rope_pages, latent_scales, page_table)
    _, q_len, H, _ = _sizes("q", q, 4)
    if not (q.dtype is torch.bfloat16 and kv_lens.dtype is torch.int32
            and q.shape == (B, q_len, H, width + rope_dim) and kv_lens.shape == (B,)
            and q.device == dev and kv_lens.device == dev
            and q.is_contiguous() and kv_lens.is_contiguous()):
        _check("q", q, torch.bfloat16, (B, q_len, H, width + rope_dim), dev)
        _check("kv_lens", kv_lens, torch.int32, (B,), dev)
    _check_mask(causal_offset, window)
    handle = _current_stream(dev)
    if out is None:
        out = q.new_empty((B, q_len, H, width))
    else:
        _check("out", out, torch.bfloat16, (B, q_len, H, width), dev)
    if lse is not None:
        _check("lse", lse, torch.float32, (B, q_len, H), dev)
    elif with_lse:
        lse = q.new_empty((B, q_len, H), dtype=torch.float32)
    p = PdaLatentParams(B, q_len, H, width, rope_dim, page, max_pages, num_pages, scale,
                        causal_offset, window, kv_dtype, flags, _ptr(latent_scales), None, 0)
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    elif not library_workspace:
        need = lib.paged_latent_decode_workspace_bytes(p)
        if need == ctypes.c_size_t(-1).value:
            need = 0  # the call below says what is wrong
        if need:
            workspace = q.new_empty(need, dtype=torch.uint8)
    if workspace is not None:
        p.workspace = workspace.data_ptr()
        p.workspace_bytes = workspace.nbytes
    st = lib.paged_latent_decode(q.data_ptr(), latent_pages.data_ptr(), rope_pages.data_ptr(),
                                 page_table.data_ptr(), kv_lens.data_ptr(), p, out.data_ptr(),
                                 _ptr(lse), handle)
    if st != 0:
        raise PdaError(st, "paged_latent_decode")
    return out, lse


def latent_prefill_attn(q, kv, k_rope, q_offsets, kv_offsets, *, scale,
                        causal_offset=PDA_CAUSAL_BOTTOM_RIGHT, window=0, max_q_len=None, out=None,
                        lse=None, with_lse=True, stream=None):
    """Attention over an expanded latent cache, ragged; returns (out, lse).
    q bf16 [total_q, H, D + Dr]; kv bf16 [total_kv, H, 2 D], each head's keys
    then its values (the up-projection's output); k_rope bf16 [total_kv, Dr],
    shared by the heads; q_offsets, kv_offsets int32 [B + 1]. ``max_q_len``:
    a bound on the query rows of a sequence (default total_q; a tighter one
    launches fewer idle CTAs; rows past it are not computed). out bf16 [total_q, H, D], lse fp32 [total_q, H]."""
    if stream is not None:
        return _on(stream, latent_prefill_attn, q, kv, k_rope, q_offsets, kv_offsets, scale=scale,
                   causal_offset=causal_offset, window=window, max_q_len=max_q_len, out=out,
                   lse=lse, with_lse=with_lse)
    if torch is None:
        _with_torch()
    lib = load()
    dev = q.device
    total_q, H, width = _sizes("q", q, 3)
    total_kv, _, D2 = _sizes("kv", kv, 3)
    D = D2 // 2
    B = _sizes("q_offsets", q_offsets, 1)[0] - 1
    _check("q", q, torch.bfloat16, (total_q, H, width), dev)
    _check("kv", kv, torch.bfloat16, (total_kv, H, 2 * D), dev)
    _check("k_rope", k_rope, torch.bfloat16, (total_kv, width - D), dev, rows=True)
    _check("q_offsets", q_offsets, torch.int32, (B + 1,), dev)
    _check("kv_offsets", kv_offsets, torch.int32, (B + 1,), dev)
    _check_mask(causal_offset, window)
    handle = _current_stream(dev)
    if out is None:
        out = q.new_empty((total_q, H, D))
    else:
        _check("out", out, torch.bfloat16, (total_q, H, D), dev)
    if lse is not None:
        _check("lse", lse, torch.float32, (total_q, H), dev)
    elif with_lse:
        lse = q.new_empty((total_q, H), dtype=torch.float32)
    p = PdaLatentPrefillParams(B, total_q, total_kv, total_q if max_q_len is None else min(max_q_len, total_q), H,
                               D, width - D, _row_stride(k_rope), scale, causal_offset, window)
    st = lib.latent_prefill_attn(q.data_ptr(), kv.data_ptr(), k_rope.data_ptr(), q_offsets.data_ptr(),
                                 kv_offsets.data_ptr(), p, out.data_ptr(), _ptr(lse), handle)
    if st != 0:
        raise PdaError(st, "latent_prefill_attn")
    return out, lse


def last_device_error(stream=None) -> int:
    """Synchronise the stream and return (then clear) the device error word."""
    return load().pda_last_device_error(_stream_handle(stream))
