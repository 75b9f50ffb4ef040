"""GB300-native sparse MLA attention forward.

A thin Python binding over the C ABI of libsmla (include/smla.h): the
functions below carry the C names, take torch tensors that already live on the
GPU, check dtypes and shapes, and pass raw pointers and sizes through ctypes.
Every step of the computation runs in the library's CUDA kernels; there is no
fallback of any kind.  If libsmla.so has not been built (``build.build()``,
or ``__graft_entry__.build()``), every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

_lib = None
_lock = threading.Lock()

SMLA_KV_BF16 = 0
SMLA_KV_FP8_E4M3 = 1
SMLA_KV_FP8_E4M3_GROUP128 = 2
SMLA_KV_FP8_DS_MLA = 3            # 656-byte rows: 512 E4M3 | 4 fp32 scales | 64 bf16
SMLA_KV_FP8_E4M3_GROUP4_KPE = 4   # E4M3 [S, 576], k_scale [S, 4], one kpe scale
SMLA_KV_FP8_E4M3_BLOCK = 5        # E4M3 [S, d_qk], one fp32 scale per cache block
DS_MLA_ROW_BYTES = 656

SMLA_OK = 0
STATUS_NAMES = {0: "SMLA_OK", 1: "SMLA_ERR_INVALID_ARG",
                2: "SMLA_ERR_UNSUPPORTED", 3: "SMLA_ERR_CUDA",
                4: "SMLA_ERR_TIMEOUT", 5: "SMLA_ERR_BAD_INDEX",
                6: "SMLA_ERR_WORKSPACE"}


class SmlaError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}")
        self.code = code


def library_path() -> str:
    return _build.LIB


def load():
    """Load libsmla.so (raises if it is missing: there is no fallback)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(
                f"libsmla.so not built at {path}; run "
                "python -m sparse_mla_attention_02_gb300.build")
        lib = ctypes.CDLL(path)
        P, I, I64, F, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                            ctypes.c_float, ctypes.c_size_t)
        fwd_args = [P, P, I, P, P, P, I, I, I, I, I, I64, F, P, P]
        lib.smla_fwd.argtypes = fwd_args + [P]
        lib.smla_fwd.restype = I
        lib.smla_fwd_ws.argtypes = fwd_args + [P, SZ, P]
        lib.smla_fwd_ws.restype = I
        lib.smla_cache_write_e4m3_group.argtypes = [P, P, P, I, I, I64, P, P, P]
        lib.smla_cache_write_e4m3_group.restype = I
        lib.smla_cache_append.argtypes = [P, I64, P, I64, P, I64, I, P, I64, I64, P, I64, I64,
                                          I, P, P, P, I, I, I, I, I, I, I, I64, P, P, F, P]
        lib.smla_cache_append.restype = I
        lib.smla_fwd_window.argtypes = [P, P, I, P, P, P, P, I, I, I, I, I, I, I, I, I, I, I, I64,
                                        F, P, P, P, SZ, P]
        lib.smla_fwd_window.restype = I
        lib.smla_fwd_window_workspace_size.argtypes = [I] * 11
        lib.smla_fwd_window_workspace_size.restype = SZ
        lib.smla_fwd_partial.argtypes = fwd_args + [P]
        lib.smla_fwd_partial.restype = I
        lib.smla_fwd_paged.argtypes = [P, P, I, P, P, P, P, I, I, I, I, P, I, I, I,
                                       I, I, I64, F, P, P, P, SZ, P]
        lib.smla_fwd_paged.restype = I
        lib.smla_fwd_split_q.argtypes = [P, P, P, I, P, F, P, P, I, I, I, I, I, I64, F,
                                         P, P, P, SZ, P]
        lib.smla_fwd_split_q.restype = I
        lib.smla_fwd_host.argtypes = fwd_args + [I, P, SZ, P]
        lib.smla_fwd_host.restype = I
        lib.smla_fwd_host_workspace_size.argtypes = [I, I, I, I, I, I, I]
        lib.smla_fwd_host_workspace_size.restype = SZ
        lib.smla_workspace_size.argtypes = [I, I, I, I, I, I]
        lib.smla_workspace_size.restype = SZ
        lib.smla_plan_info.argtypes = [I, I, I, I, I, I, ctypes.POINTER(I),
                                       ctypes.POINTER(I), ctypes.POINTER(SZ)]
        lib.smla_plan_info.restype = I
        lib.smla_plan_info_for.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(I),
                                           ctypes.POINTER(I), ctypes.POINTER(SZ)]
        lib.smla_plan_info_for.restype = I
        lib.smla_combine.argtypes = [P, P, I, I64, I, P, P, P]
        lib.smla_combine.restype = I
        lib.smla_get_device_status.argtypes = [ctypes.POINTER(I), I]
        lib.smla_get_device_status.restype = I
        lib.smla_test_set_stall.argtypes = [I, I]
        lib.smla_test_set_stall.restype = I
        lib.smla_status_string.argtypes = [I]
        lib.smla_status_string.restype = ctypes.c_char_p
        lib.smla_version.argtypes = []
        lib.smla_version.restype = I
        _lib = lib
        return lib


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, device, stream):
    """Memory that a call on ``stream`` (None: the current one) writes and the
    current stream may read.  It comes from ``stream``'s memory: the current stream's
    may have held a tensor that work still queued there reads.  Once let go it is
    used again only when both streams are done with it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _check(code, what):
    if code != SMLA_OK:
        raise SmlaError(code, what)


def _require(cond, what):
    """Argument check of the binding (kept under ``python -O``)."""
    if not cond:
        raise ValueError(what)


def _kv_slots(kv_cache, kv_dtype, k_scale, d_qk, num_slots):
    """Check the cache and its scales; return the slot count."""
    import torch
    _require(kv_cache.is_cuda and kv_cache.is_contiguous(),
             "kv_cache must be a contiguous device tensor")
    if kv_dtype == SMLA_KV_BF16:
        _require(kv_cache.dtype == torch.bfloat16, "a bf16 cache must be torch.bfloat16")
    else:
        _require(kv_cache.dtype == torch.uint8, "an E4M3 cache must be torch.uint8 bytes")
    if kv_dtype in (SMLA_KV_FP8_E4M3, SMLA_KV_FP8_E4M3_GROUP128, SMLA_KV_FP8_E4M3_GROUP4_KPE):
        _require(k_scale is not None and k_scale.dtype == torch.float32 and
                 k_scale.is_cuda and k_scale.is_contiguous(),
                 "this cache format needs k_scale, a contiguous fp32 device tensor")
    row = DS_MLA_ROW_BYTES if kv_dtype == SMLA_KV_FP8_DS_MLA else d_qk
    return kv_cache.numel() // row if num_slots is None else int(num_slots)


def _idx_checks(indices, valid_len, T):
    import torch
    _require(indices.is_cuda and indices.dtype == torch.int32 and indices.is_contiguous()
             and indices.dim() == 2 and indices.shape[0] == T,
             "indices must be a contiguous int32 device tensor [T, topk]")
    if valid_len is not None:
        _require(valid_len.is_cuda and valid_len.dtype == torch.int32 and
                 valid_len.is_contiguous() and valid_len.shape == (T,),
                 "valid_len must be a contiguous int32 device tensor [T]")


def _in_args(q, kv_cache, kv_dtype, k_scale, indices, valid_len, sm_scale,
             num_slots):
    """The input arguments of the forward entry points, checked."""
    import torch
    _require(q.is_cuda and q.dtype == torch.bfloat16 and q.is_contiguous() and q.dim() == 3,
             "q must be a contiguous bf16 device tensor [T, h, d_qk]")
    T, h, d_qk = q.shape
    S = _kv_slots(kv_cache, kv_dtype, k_scale, d_qk, num_slots)
    _idx_checks(indices, valid_len, T)
    return [_p(q), _p(kv_cache), int(kv_dtype), _p(k_scale), _p(indices),
            _p(valid_len), T, h, d_qk, 512, indices.shape[1], S, float(sm_scale)]


def _fwd_args(q, kv_cache, kv_dtype, k_scale, indices, valid_len, sm_scale,
              out, lse, num_slots, stream):
    import torch
    _require(q.is_cuda and q.dtype == torch.bfloat16 and q.is_contiguous() and q.dim() == 3,
             "q must be a contiguous bf16 device tensor [T, h, d_qk]")
    T, h, d_qk = q.shape
    S = _kv_slots(kv_cache, kv_dtype, k_scale, d_qk, num_slots)
    _idx_checks(indices, valid_len, T)
    topk = indices.shape[1]
    d_v = 512
    if out is None:
        out = _empty((T, h, d_v), torch.bfloat16, q.device, stream)
    _require(out.dtype == torch.bfloat16 and out.is_contiguous() and out.shape == (T, h, d_v),
             "out must be contiguous bf16 [T, h, 512]")
    if lse is not None:
        _require(lse.dtype == torch.float32 and lse.is_contiguous() and lse.shape == (T, h),
                 "lse must be contiguous fp32 [T, h]")
    args = [_p(q), _p(kv_cache), int(kv_dtype), _p(k_scale), _p(indices),
            _p(valid_len), T, h, d_qk, d_v, topk, S, float(sm_scale),
            _p(out), _p(lse)]
    return args, out, lse


def smla_fwd(q, kv_cache, kv_dtype, k_scale, indices, valid_len, sm_scale,
             out=None, lse=None, want_lse=True, num_slots=None, stream=None):
    """Sparse MLA forward through ``smla_fwd`` (library-owned workspace).

    q bf16 [T,h,d_qk]; kv_cache bf16 or uint8 [S,d_qk]; k_scale f32 or None;
    indices int32 [T,topk]; valid_len int32 [T] or None.
    Returns (out bf16 [T,h,512], lse f32 [T,h] or None)."""
    import torch
    lib = load()
    if lse is None and want_lse:
        lse = _empty(q.shape[:2], torch.float32, q.device, stream)
    args, out, lse = _fwd_args(q, kv_cache, kv_dtype, k_scale, indices,
                               valid_len, sm_scale, out, lse, num_slots, stream)
    _check(lib.smla_fwd(*args, _stream(stream)), "smla_fwd")
    return out, lse


def smla_fwd_split_q(q_nope, q_pe, kv_cache, kv_dtype, k_scale, indices, valid_len,
                     sm_scale, kpe_scale=1.0, out=None, lse=None, want_lse=True,
                     num_slots=None, workspace=None, stream=None):
    """``smla_fwd_split_q``: the forward on q_nope bf16 [T,h,512] and q_pe
    bf16 [T,h,d_qk-512] (or None: q_nope is the concatenated q), with the
    rope scale kpe_scale for SMLA_KV_FP8_E4M3_GROUP4_KPE.
    Returns (out bf16 [T,h,512], lse f32 [T,h] or None)."""
    import torch
    lib = load()
    _require(q_nope.is_cuda and q_nope.dtype == torch.bfloat16 and q_nope.is_contiguous(),
             "q_nope must be a contiguous bf16 device tensor")
    if q_pe is None:
        T, h, d_qk = q_nope.shape
    else:
        T, h, d_nope = q_nope.shape
        _require(d_nope == 512 and q_pe.shape[:2] == (T, h),
                 "q_nope must be [T, h, 512] and q_pe [T, h, d_qk - 512]")
        _require(q_pe.is_cuda and q_pe.dtype == torch.bfloat16 and q_pe.is_contiguous(),
                 "q_pe must be a contiguous bf16 device tensor")
        d_qk = 512 + q_pe.shape[2]
    S = _kv_slots(kv_cache, kv_dtype, k_scale, d_qk, num_slots)
    _idx_checks(indices, valid_len, T)
    if out is None:
        out = _empty((T, h, 512), torch.bfloat16, q_nope.device, stream)
    _require(out.dtype == torch.bfloat16 and out.is_contiguous() and out.shape == (T, h, 512),
             "out must be contiguous bf16 [T, h, 512]")
    if lse is None and want_lse:
        lse = _empty((T, h), torch.float32, q_nope.device, stream)
    if lse is not None:
        _require(lse.dtype == torch.float32 and lse.is_contiguous() and lse.shape == (T, h),
                 "lse must be contiguous fp32 [T, h]")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.smla_fwd_split_q(_p(q_nope), _p(q_pe), _p(kv_cache), int(kv_dtype),
                                _p(k_scale), float(kpe_scale), _p(indices), _p(valid_len),
                                T, h, d_qk, 512, indices.shape[1], S, float(sm_scale),
                                _p(out), _p(lse), _p(workspace), nbytes, _stream(stream)),
           "smla_fwd_split_q")
    return out, lse


def smla_cache_write_e4m3_group(kv_c, k_pe, slot_mapping, kv_cache, scales,
                                stream=None):
    """``smla_cache_write_e4m3_group``: quantize token rows [kv_c | k_pe]
    (bf16 [N,512] and [N,64], or k_pe None for 512-channel rows) into the
    E4M3 cache (uint8 [S, d_qk]) with one fp32 scale per (slot, 128-channel
    group) (scales [S, ceil(d_qk/128)]) at rows slot_mapping (int32 [N];
    negative = skip)."""
    import torch
    lib = load()
    N = kv_c.shape[0]
    for x in (kv_c, k_pe):
        if x is not None:
            _require(x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous(),
                     "kv_c and k_pe must be contiguous bf16 device tensors")
    _require(kv_c.shape == (N, 512), "kv_c must be [N, 512]")
    d_qk = 512 if k_pe is None else 512 + k_pe.shape[1]
    _require(slot_mapping.dtype == torch.int32 and slot_mapping.shape == (N,),
             "slot_mapping must be int32 [N]")
    _require(kv_cache.dtype == torch.uint8 and kv_cache.dim() == 2 and kv_cache.shape[1] == d_qk,
             "kv_cache must be uint8 [S, d_qk]")
    _require(scales.dtype == torch.float32 and
             scales.shape == (kv_cache.shape[0], (d_qk + 127) // 128),
             "scales must be fp32 [S, ceil(d_qk / 128)]")
    _check(lib.smla_cache_write_e4m3_group(_p(kv_c), _p(k_pe), _p(slot_mapping), N, d_qk,
                                           kv_cache.shape[0], _p(kv_cache), _p(scales),
                                           _stream(stream)), "smla_cache_write_e4m3_group")
    return kv_cache, scales


def _batch_args(query_start, seq_lens, block_table, block_size, block_stride_rows, index, i32):
    """Check a ragged batch's descriptors (on CUDA device ``index``); return the
    C arguments."""
    if not (query_start.dtype is i32 and seq_lens.dtype is i32 and block_table.dtype is i32 and
            query_start.is_contiguous() and seq_lens.is_contiguous() and
            block_table.is_contiguous()):
        raise ValueError("query_start, seq_lens and block_table must be contiguous int32 tensors")
    if not query_start.get_device() == seq_lens.get_device() == block_table.get_device() == index:
        raise ValueError("query_start, seq_lens and block_table must be on the inputs' device")
    shape = block_table.shape
    if len(shape) != 2:
        raise ValueError("block_table must be [num_reqs, stride]")
    R, width = shape
    if query_start.shape != (R + 1,) or seq_lens.shape != (R,):
        raise ValueError("query_start must be [num_reqs + 1] and seq_lens [num_reqs]")
    if block_size < 1 or (block_stride_rows != 0 and block_stride_rows < block_size):
        raise ValueError("block_size must be positive and block_stride_rows 0 or at least "
                         "block_size")
    return (query_start.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), R, width,
            block_size, block_stride_rows)


def _device_stream(t, what, stream):
    """The CUDA device and the raw stream of a call on tensor ``t``.  The library
    works on the current device: tensors of another are refused."""
    import torch
    index = t.get_device()                    # (-1: a host tensor)
    if index < 0 or index != torch._C._cuda_getDevice():
        raise ValueError(what + " must be on the current CUDA device")
    # (torch.cuda.current_stream() builds a Stream object, 3 us a call; a tensor's
    # index costs half of its device)
    return index, (torch._C._cuda_getCurrentRawStream(index) if stream is None
                   else stream.cuda_stream)


def _cache_rows(kv_cache, kv_dtype, k_scale, d_qk, num_slots, rows_per_scale, index):
    """Check a paged cache and its scales; return (slots, k_scale's address)."""
    import torch
    if not 0 <= kv_dtype <= SMLA_KV_FP8_E4M3_BLOCK:
        raise ValueError("kv_dtype must be an SMLA_KV_* value")
    row = DS_MLA_ROW_BYTES if kv_dtype == SMLA_KV_FP8_DS_MLA else d_qk
    if not (kv_cache.dtype is (torch.bfloat16 if kv_dtype == SMLA_KV_BF16 else torch.uint8) and
            kv_cache.is_contiguous() and kv_cache.get_device() == index):
        raise ValueError("kv_cache must be a contiguous tensor on the inputs' device, bfloat16 "
                         "for a bf16 cache and uint8 for the E4M3 formats")
    if row < 1 or (kv_cache.dim() > 1 and kv_cache.shape[-1] != row):
        raise ValueError("kv_cache must have the rows of the format, as its last dimension or "
                         "one behind the other")
    S = kv_cache.numel() // row
    if num_slots is not None:
        if num_slots > S:
            raise ValueError("num_slots is larger than kv_cache")
        S = int(num_slots)
    if kv_dtype == SMLA_KV_BF16 or kv_dtype == SMLA_KV_FP8_DS_MLA:
        return S, None
    need = (1 if kv_dtype == SMLA_KV_FP8_E4M3 else
            -(-S // rows_per_scale) if kv_dtype == SMLA_KV_FP8_E4M3_BLOCK else
            4 * S if kv_dtype == SMLA_KV_FP8_E4M3_GROUP4_KPE else S * ((d_qk + 127) // 128))
    if not (k_scale is not None and k_scale.dtype is torch.float32 and
            k_scale.is_contiguous() and k_scale.get_device() == index and
            k_scale.numel() >= need):
        raise ValueError("k_scale must be a contiguous fp32 tensor on the inputs' device with a "
                         "value for every scale of the format")
    return S, k_scale.data_ptr()


def smla_cache_append(kv_c, k_pe, cos_sin, query_start, seq_lens, block_table, block_size,
                      kv_cache, kv_dtype, k_scale=None, kpe_scale=1.0, interleaved=True,
                      q_pe=None, q_out=None, block_stride_rows=0, num_slots=None, stream=None):
    """``smla_cache_append``: write a step's rows [kv_c | rope(k_pe)] into the
    paged cache and rotate the step's queries.

    kv_c bf16 [N,512], k_pe bf16 [N,64] (rows may be strided) or None for
    512-channel rows; cos_sin fp32 [positions,64] = cos 32 | sin 32;
    query_start int32 [R+1], seq_lens int32 [R] (lengths after the append),
    block_table int32 [R,stride]; kv_cache and k_scale as ``kv_dtype`` says
    (SMLA_KV_FP8_E4M3_BLOCK: fp32, one scale per cache block); q_pe bf16
    [N,h,64] (strided) or None, q_out likewise (None: in place).
    Returns (kv_cache, q_out)."""
    import torch
    lib = _lib or load()
    bf16 = torch.bfloat16
    index, raw_stream = _device_stream(kv_c, "kv_c", stream)
    shape = kv_c.shape
    if not (kv_c.dtype is bf16 and len(shape) == 2 and shape[1] == 512 and kv_c.stride(1) == 1):
        raise ValueError("kv_c must be a bf16 tensor [N, 512] with contiguous rows")
    N = shape[0]
    one = N < 2                               # a single token's stride says nothing
    pe = cs = None
    pe_stride = cs_rows = 0
    d_qk = 512
    if k_pe is not None:
        if not (k_pe.dtype is bf16 and k_pe.shape == (N, 64) and k_pe.stride(1) == 1 and
                k_pe.get_device() == index):
            raise ValueError("k_pe must be a bf16 tensor [N, 64] with contiguous rows")
        if not (cos_sin is not None and cos_sin.dtype is torch.float32 and cos_sin.dim() == 2 and
                cos_sin.shape[1] == 64 and cos_sin.is_contiguous() and
                cos_sin.get_device() == index):
            raise ValueError("cos_sin must be a contiguous fp32 tensor [positions, 64]")
        d_qk = 576
        pe, pe_stride = k_pe.data_ptr(), 64 if one else k_pe.stride(0)
        cs, cs_rows = cos_sin.data_ptr(), cos_sin.shape[0]
    elif cos_sin is not None or q_pe is not None:
        raise ValueError("cos_sin and q_pe go with k_pe")
    if q_out is not None and q_pe is None:
        raise ValueError("q_out goes with q_pe")
    batch = _batch_args(query_start, seq_lens, block_table, block_size, block_stride_rows, index,
                        torch.int32)
    S, scale = _cache_rows(kv_cache, kv_dtype, k_scale, d_qk, num_slots,
                           block_stride_rows or block_size, index)
    q_args = (None, 0, 0, None, 0, 0, 0)
    if q_pe is not None:
        if q_out is None:
            q_out = q_pe
        h = q_pe.shape[1] if q_pe.dim() == 3 else 0
        strides = []
        for x in (q_pe, q_out):
            if not (x.dtype is bf16 and x.shape == (N, h, 64) and x.get_device() == index):
                raise ValueError("q_pe and q_out must be bf16 tensors [N, h, 64]")
            s0, s1, s2 = x.stride()
            if s2 != 1:
                raise ValueError("q_pe and q_out must have contiguous channels")
            strides.append((x.data_ptr(), 64 if one else s0, 64 if h < 2 else s1))
        q_args = (*strides[0], *strides[1], h)
    code = lib.smla_cache_append(
        kv_c.data_ptr(), 512 if one else kv_c.stride(0), pe, pe_stride, cs, cs_rows, interleaved,
        *q_args, *batch, N, d_qk, kv_dtype, S, kv_cache.data_ptr(), scale, kpe_scale, raw_stream)
    if code:
        raise SmlaError(code, "smla_cache_append")
    return kv_cache, q_out


def smla_fwd_window_workspace_size(num_reqs, T, h, d_qk, kv_dtype, block_table_stride,
                                   block_size, window=0, sinks=0, max_seq_len=None,
                                   d_v=512) -> int:
    return int(load().smla_fwd_window_workspace_size(
        num_reqs, T, h, d_qk, d_v, kv_dtype, block_table_stride, block_size, window, sinks,
        max_seq_len or 0))


def smla_fwd_window(q, kv_cache, kv_dtype, k_scale, query_start, seq_lens, block_table,
                    block_size, sm_scale, window=0, sinks=0, max_seq_len=None,
                    block_stride_rows=0, out=None, lse=None, want_lse=True, num_slots=None,
                    workspace=None, stream=None):
    """``smla_fwd_window``: causal attention of a ragged batch over its paged
    cache, through a sliding window (0: none) with ``sinks`` first positions
    that stay visible.

    q bf16 [T,h,d_qk]; kv_cache bf16 or uint8 [S,d_qk] (SMLA_KV_BF16,
    SMLA_KV_FP8_E4M3 or SMLA_KV_FP8_E4M3_BLOCK); query_start int32 [R+1],
    seq_lens int32 [R], block_table int32 [R,stride] as for
    ``smla_cache_append``; max_seq_len: a bound on seq_lens that sizes the
    split plan; workspace: a uint8 device tensor of at least
    smla_fwd_window_workspace_size bytes, or None to allocate one.
    Returns (out bf16 [T,h,512], lse f32 [T,h] or None); rows behind the last
    request are not written."""
    import torch
    lib = _lib or load()
    index, raw_stream = _device_stream(q, "q", stream)
    bf16 = torch.bfloat16
    if not (q.dtype is bf16 and q.dim() == 3 and q.is_contiguous()):
        raise ValueError("q must be a contiguous bf16 device tensor [T, h, d_qk]")
    T, h, d_qk = q.shape
    batch = _batch_args(query_start, seq_lens, block_table, block_size, block_stride_rows, index,
                        torch.int32)
    S, scale = _cache_rows(kv_cache, kv_dtype, k_scale, d_qk, num_slots,
                           block_stride_rows or block_size, index)
    if out is None:
        out = _empty((T, h, 512), bf16, q.device, stream)
    elif not (out.dtype is bf16 and out.shape == (T, h, 512) and out.is_contiguous() and
              out.get_device() == index):
        raise ValueError("out must be contiguous bf16 [T, h, 512]")
    if lse is None:
        if want_lse:
            lse = _empty((T, h), torch.float32, q.device, stream)
    elif not (lse.dtype is torch.float32 and lse.shape == (T, h) and lse.is_contiguous() and
              lse.get_device() == index):
        raise ValueError("lse must be contiguous fp32 [T, h]")
    limit = max_seq_len or 0
    if workspace is None:
        ws = None
        nbytes = lib.smla_fwd_window_workspace_size(batch[3], T, h, d_qk, 512, kv_dtype, batch[4],
                                                    block_size, window, sinks, limit)
        if nbytes:
            workspace = _empty((nbytes,), torch.uint8, q.device, stream)
            ws = workspace.data_ptr()
    else:
        if not (workspace.get_device() == index and workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous tensor on the inputs' device")
        nbytes = workspace.numel() * workspace.element_size()
        ws = workspace.data_ptr()
    code = lib.smla_fwd_window(
        q.data_ptr(), kv_cache.data_ptr(), kv_dtype, scale, *batch, window, sinks, limit, T, h,
        d_qk, 512, S, sm_scale, out.data_ptr(), None if lse is None else lse.data_ptr(), ws,
        nbytes, raw_stream)
    if code:
        raise SmlaError(code, "smla_fwd_window")
    return out, lse


def smla_fwd_partial(q, kv_cache, kv_dtype, k_scale, indices, valid_len,
                     sm_scale, out=None, lse=None, num_slots=None, stream=None):
    """``smla_fwd_partial``: normalised fp32 O [T,h,512] and LSE [T,h] for an
    LSE-weighted merge (smla_combine).  Returns (out, lse)."""
    import torch
    lib = load()
    T, h, _ = q.shape
    if out is None:
        out = _empty((T, h, 512), torch.float32, q.device, stream)
    if lse is None:
        lse = _empty((T, h), torch.float32, q.device, stream)
    _require(out.dtype == torch.float32 and out.is_contiguous() and out.shape == (T, h, 512),
             "out must be contiguous fp32 [T, h, 512]")
    _require(lse.dtype == torch.float32 and lse.is_contiguous() and lse.shape == (T, h),
             "lse must be contiguous fp32 [T, h]")
    args = _in_args(q, kv_cache, kv_dtype, k_scale, indices, valid_len,
                    sm_scale, num_slots) + [_p(out), _p(lse)]
    _check(lib.smla_fwd_partial(*args, _stream(stream)), "smla_fwd_partial")
    return out, lse


def smla_fwd_paged(q, kv_cache, kv_dtype, k_scale, token_indices, req_id,
                   block_table, block_size, sm_scale, valid_len=None,
                   block_stride_rows=0, out=None, lse=None, want_lse=True,
                   num_slots=None, workspace=None, stream=None):
    """``smla_fwd_paged``: the forward on request-local top-k indices.

    token_indices int32 [T,topk] (positions in the token's request, -1 =
    none); req_id int32 [T]; block_table int32 [num_reqs, stride]; the slot
    of position e is block_table[req, e // block_size] * block_stride_rows +
    e % block_size (block_stride_rows 0 = block_size).  workspace: a uint8
    device tensor (caller-owned, as smla_fwd_ws) or None (library-owned).
    Returns (out, lse) as smla_fwd."""
    import torch
    lib = load()
    if lse is None and want_lse:
        lse = _empty(q.shape[:2], torch.float32, q.device, stream)
    args, out, lse = _fwd_args(q, kv_cache, kv_dtype, k_scale, token_indices,
                               valid_len, sm_scale, out, lse, num_slots, stream)
    for x in (req_id, block_table):
        _require(x.is_cuda and x.dtype == torch.int32 and x.is_contiguous(),
                 "req_id and block_table must be contiguous int32 device tensors")
    _require(req_id.shape == (args[6],) and block_table.dim() == 2,
             "req_id must be [T] and block_table [num_reqs, stride]")
    ws_p = None if workspace is None else _p(workspace)
    ws_n = 0 if workspace is None else workspace.numel()
    pargs = args[:4] + [args[4], _p(req_id), _p(block_table),
                        int(block_table.shape[0]), int(block_table.shape[1]),
                        int(block_size), int(block_stride_rows), args[5]] + args[6:]
    _check(lib.smla_fwd_paged(*pargs, ws_p, ws_n, _stream(stream)),
           "smla_fwd_paged")
    return out, lse


def smla_workspace_size(T, h, d_qk, topk, kv_dtype, d_v=512) -> int:
    return int(load().smla_workspace_size(T, h, d_qk, d_v, topk, kv_dtype))


KERNEL_NAMES = {0: "cuda_core", 1: "tc_heads", 2: "tc_keys", 3: "tc_keys_fp8"}


def smla_plan_info(T, h, d_qk, topk, kv_dtype, d_v=512) -> dict:
    """``smla_plan_info``: the kernel family, top-k splits and workspace a
    forward of this shape uses on the current device."""
    lib = load()
    k, s, n = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_size_t(0)
    _check(lib.smla_plan_info(T, h, d_qk, d_v, topk, kv_dtype, ctypes.byref(k),
                              ctypes.byref(s), ctypes.byref(n)), "smla_plan_info")
    return {"kernel": KERNEL_NAMES[k.value], "splits": s.value,
            "workspace_bytes": n.value}


def smla_plan_info_for(T, h, d_qk, topk, kv_dtype, num_sms, d_v=512) -> dict:
    """``smla_plan_info_for``: the same plan for a device with ``num_sms``
    SMs, without a device query (works on a host without a GPU)."""
    lib = load()
    k, s, n = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_size_t(0)
    _check(lib.smla_plan_info_for(T, h, d_qk, d_v, topk, kv_dtype, num_sms, ctypes.byref(k),
                                  ctypes.byref(s), ctypes.byref(n)), "smla_plan_info_for")
    return {"kernel": KERNEL_NAMES[k.value], "splits": s.value,
            "workspace_bytes": n.value}


def smla_fwd_ws(q, kv_cache, kv_dtype, k_scale, indices, valid_len, sm_scale,
                workspace, out=None, lse=None, want_lse=True, num_slots=None,
                stream=None):
    """``smla_fwd_ws``: as smla_fwd with a caller-owned workspace tensor
    (uint8 on the device, at least smla_workspace_size bytes)."""
    import torch
    lib = load()
    if lse is None and want_lse:
        lse = _empty(q.shape[:2], torch.float32, q.device, stream)
    args, out, lse = _fwd_args(q, kv_cache, kv_dtype, k_scale, indices,
                               valid_len, sm_scale, out, lse, num_slots, stream)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.smla_fwd_ws(*args, _p(workspace), nbytes, _stream(stream)),
           "smla_fwd_ws")
    return out, lse


def smla_fwd_host_workspace_size(T, h, d_qk, topk, kv_dtype, d_v=512,
                                 chunk_tokens=0) -> int:
    return int(load().smla_fwd_host_workspace_size(T, h, d_qk, d_v, topk,
                                                   kv_dtype, chunk_tokens))


def smla_fwd_host(q, kv_cache, kv_dtype, k_scale, indices, valid_len, sm_scale,
                  out=None, lse=None, want_lse=True, num_slots=None,
                  chunk_tokens=0, workspace=None, stream=None):
    """``smla_fwd_host``: q, indices, valid_len, out and lse are CPU tensors
    (pin them for overlap); kv_cache and k_scale are device tensors.  The
    copies and the forward are queued on ``stream`` (and the library's copy
    streams); synchronise the stream before reading ``out``/``lse``.
    ``workspace``: a device uint8 tensor of at least
    smla_fwd_host_workspace_size(...) bytes, or None to allocate one."""
    import torch
    lib = load()
    T, h, d_qk = q.shape
    d_v = 512
    if q.device.type != "cpu" or indices.device.type != "cpu" or \
            (valid_len is not None and valid_len.device.type != "cpu"):
        raise ValueError("smla_fwd_host: q, indices, valid_len live in host memory")
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [T, h, d_qk]")
    if indices.dtype != torch.int32 or not indices.is_contiguous() or \
            indices.dim() != 2 or indices.shape[0] != T:
        raise ValueError("indices must be contiguous int32 [T, topk]")
    if valid_len is not None and (valid_len.dtype != torch.int32 or
                                  valid_len.shape != (T,) or
                                  not valid_len.is_contiguous()):
        raise ValueError("valid_len must be contiguous int32 [T]")
    topk = indices.shape[1]
    S = _kv_slots(kv_cache, kv_dtype, k_scale, d_qk, num_slots)
    if out is None:
        out = torch.empty((T, h, d_v), dtype=torch.bfloat16, pin_memory=True)
    if lse is None and want_lse:
        lse = torch.empty((T, h), dtype=torch.float32, pin_memory=True)
    for t in (out, lse):
        if t is not None and (t.device.type != "cpu" or not t.is_contiguous()):
            raise ValueError("out / lse must be contiguous host tensors")
    nbytes = smla_fwd_host_workspace_size(T, h, d_qk, topk, kv_dtype, d_v,
                                          chunk_tokens)
    if workspace is None:
        workspace = _empty((max(nbytes, 1),), torch.uint8, kv_cache.device, stream)
    _check(lib.smla_fwd_host(_p(q), _p(kv_cache), kv_dtype, _p(k_scale),
                             _p(indices), _p(valid_len), T, h, d_qk, d_v, topk,
                             S, float(sm_scale), _p(out), _p(lse),
                             int(chunk_tokens), _p(workspace),
                             workspace.numel(), _stream(stream)),
           "smla_fwd_host")
    return out, lse


def smla_combine(o_parts, lse_parts, out=None, lse=None, stream=None):
    """``smla_combine``: o_parts f32 [P, rows, 512], lse_parts f32 [P, rows]."""
    import torch
    lib = load()
    P, rows, d_v = o_parts.shape
    _require(o_parts.dtype == torch.float32 and o_parts.is_contiguous(),
             "o_parts must be contiguous fp32 [P, rows, 512]")
    _require(lse_parts.dtype == torch.float32 and lse_parts.is_contiguous() and
             lse_parts.shape == (P, rows), "lse_parts must be contiguous fp32 [P, rows]")
    if out is None:
        out = _empty((rows, d_v), torch.bfloat16, o_parts.device, stream)
    if lse is None:
        lse = _empty((rows,), torch.float32, o_parts.device, stream)
    _check(lib.smla_combine(_p(o_parts), _p(lse_parts), P, rows, d_v, _p(out),
                            _p(lse), _stream(stream)), "smla_combine")
    return out, lse


def smla_get_device_status(clear=True) -> int:
    v = ctypes.c_int(0)
    _check(load().smla_get_device_status(ctypes.byref(v), int(clear)),
           "smla_get_device_status")
    return v.value


def smla_test_set_stall(stall: bool, wait_limit_us: int = 0) -> None:
    """Tests of the timeout path only: while ``stall`` is set, tensor-core
    launches on the current device leave out each unit's first batch of
    score MMAs, so a bounded wait runs out after ``wait_limit_us`` (0 = the
    default limit) and the launch reports SMLA_ERR_TIMEOUT."""
    _check(load().smla_test_set_stall(int(bool(stall)), int(wait_limit_us)),
           "smla_test_set_stall")


def smla_status_string(code: int) -> str:
    return load().smla_status_string(int(code)).decode()
