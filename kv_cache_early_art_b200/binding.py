"""ctypes binding of libart (include/art.h): argument marshalling only.

Every step of the attention walk runs in the CUDA library; this module turns
torch tensors into ``art_tensor_t`` descriptors, passes the current CUDA
stream, and raises ``ArtError`` on a non-zero status.  There is no CPU
fallback: importing fails when ``libart.so`` has not been built, and calls
with tensors that are not on a CUDA device are refused.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import struct
from importlib.machinery import ExtensionFileLoader
from typing import Optional

import torch

from .build import marshal_path

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libart.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libart.so is not built ({LIB_PATH}); run `python -m kv_cache_early_art_b200.build` "
                      "or __graft_entry__.build()")

_lib = ctypes.CDLL(LIB_PATH)


class _NoMarshal:
    """Stands in for the _marshal module where it cannot be loaded: the cache
    operators raise, the walk and the orders, which do not use it, run."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(self._why)


def _load_marshal():
    """The _marshal module of this torch and Python."""
    path = marshal_path()
    if not os.path.exists(path):
        return _NoMarshal(f"the cache operators need {os.path.basename(path)}, which is not built; run "
                          "`python -m kv_cache_early_art_b200.build` or __graft_entry__.build()")
    name = __package__ + "._marshal"
    spec = importlib.util.spec_from_file_location(name, path, loader=ExtensionFileLoader(name, path))
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        return _NoMarshal(f"the cache operators need {os.path.basename(path)}, which cannot be loaded: {e}")
    return module


_marshal = _load_marshal()

F32, BF16, I32 = 0, 1, 2
_DTYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.int32: I32}

STATUS = {
    0: "ART_OK", -1: "ART_ERR_NULL", -2: "ART_ERR_SHAPE", -3: "ART_ERR_DTYPE", -4: "ART_ERR_UNSUPPORTED",
    -5: "ART_ERR_PARAM", -6: "ART_ERR_LAUNCH", -7: "ART_ERR_DEVICE_TIMEOUT", -8: "ART_ERR_BAD_INDEX",
    -9: "ART_ERR_SCRATCH_SIZE",
}
ENGINE_AUTO, ENGINE_CUDA, ENGINE_MMA = 0, 1, 2


class ArtTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class ArtLaunchInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("engine", "cluster_size", "grid", "threads", "stages",
                                               "compute_warps", "window", "smem_bytes", "prefetch", "merge_cta",
                                               "ring_slots")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class ArtParams(ctypes.Structure):
    _fields_ = [(n, ArtTensor) for n in ("q", "k_cache", "v_cache", "page_table", "block_order", "seq_lens",
                                         "out", "stop_block")] + [
        ("eps_m", ctypes.c_float), ("eps_d", ctypes.c_float), ("P", ctypes.c_int32),
        ("min_blocks", ctypes.c_int32), ("sm_scale", ctypes.c_float),
        ("eps_m_per_seq", ctypes.c_void_p), ("eps_d_per_seq", ctypes.c_void_p),
        ("P_per_seq", ctypes.c_void_p), ("min_blocks_per_seq", ctypes.c_void_p),
        ("blocks_fetched", ctypes.c_void_p), ("device_status", ctypes.c_void_p),
        ("engine", ctypes.c_int32), ("cluster_size", ctypes.c_int32), ("stages", ctypes.c_int32),
        ("compute_warps", ctypes.c_int32), ("window", ctypes.c_int32), ("timeout_ns", ctypes.c_int64),
        ("debug_flags", ctypes.c_int32), ("info", ctypes.POINTER(ArtLaunchInfo)), ("prefetch", ctypes.c_int32),
        ("detector_off", ctypes.c_int32), ("merge_cta", ctypes.c_int32), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_int64)]


def _struct_format(cls) -> str:
    """struct-module format of a ctypes Structure, padding included, read
    from the structure's own field offsets (so it always matches art.h as the
    ctypes declaration does)."""
    codes = {ctypes.c_void_p: "Q", ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f"}
    parts, off = [], 0
    for name, ty in cls._fields_:
        fo = getattr(cls, name).offset
        if fo > off:
            parts.append(f"{fo - off}x")
            off = fo
        if isinstance(ty, type) and issubclass(ty, ctypes.Structure):
            parts.append(_struct_format(ty))
        elif isinstance(ty, type) and issubclass(ty, ctypes.Array):
            parts.append(f"{ty._length_}{codes[ty._type_]}")
        else:
            parts.append(codes.get(ty, "Q"))  # pointers are 8-byte addresses
        off += ctypes.sizeof(ty)
    if ctypes.sizeof(cls) > off:
        parts.append(f"{ctypes.sizeof(cls) - off}x")
    return "".join(parts)


# art_params_t packed in one call: building the nested ctypes structures field
# by field cost ~23 us of host time per call, packing them ~10 us
_PARAMS = struct.Struct("<" + _struct_format(ArtParams))
assert _PARAMS.size == ctypes.sizeof(ArtParams)


_P = ctypes.POINTER
_lib.art_decode_attention.argtypes = [_P(ArtTensor)] * 6 + [ctypes.c_float, ctypes.c_float, ctypes.c_int32,
                                                            ctypes.c_int32, _P(ArtTensor), _P(ArtTensor),
                                                            ctypes.c_void_p]
_lib.art_decode_attention.restype = ctypes.c_int
_lib.art_decode_attention_ex.argtypes = [_P(ArtParams), ctypes.c_void_p]
_lib.art_decode_attention_ex.restype = ctypes.c_int
_lib.art_decode_attention_multi.argtypes = [_P(ArtParams), ctypes.c_int32, ctypes.c_void_p]
_lib.art_decode_attention_multi.restype = ctypes.c_int
_lib.art_build_order_sink_recency.argtypes = [_P(ArtTensor), ctypes.c_int32, _P(ArtTensor), ctypes.c_void_p]
_lib.art_build_order_sink_recency.restype = ctypes.c_int
_lib.art_page_summary.argtypes = [_P(ArtTensor)] * 4 + [ctypes.c_void_p, ctypes.c_void_p]
_lib.art_page_summary.restype = ctypes.c_int
_lib.art_build_order_importance.argtypes = [_P(ArtTensor)] * 4 + [ctypes.c_int32, ctypes.c_float] + [
    _P(ArtTensor)] * 2 + [ctypes.c_void_p, ctypes.c_void_p]
_lib.art_build_order_importance.restype = ctypes.c_int
_lib.art_workspace_bytes.argtypes = [_P(ArtParams)]
_lib.art_workspace_bytes.restype = ctypes.c_int64
_lib.art_decode_attention_no_alloc.argtypes = [_P(ArtParams), ctypes.c_void_p]
_lib.art_decode_attention_no_alloc.restype = ctypes.c_int
_lib.art_strerror.argtypes = [ctypes.c_int]
_lib.art_strerror.restype = ctypes.c_char_p
_lib.art_version.argtypes = []
_lib.art_version.restype = ctypes.c_int32


class ArtRope(ctypes.Structure):
    """art_rope_t: the rotary angles of one model (made by art_rope_init)."""
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("amplitude", ctypes.c_float), ("turns", ctypes.c_uint64 * 128)]


class ArtAppendParams(ctypes.Structure):
    _fields_ = [(n, ArtTensor) for n in ("q", "k", "v", "q_out", "k_cache", "v_cache", "page_table", "slots",
                                         "positions", "token_seq", "mass")] + [
        ("rope", ctypes.c_void_p), ("device_status", ctypes.c_void_p)]


class ArtSplitParams(ctypes.Structure):
    _fields_ = [(n, ArtTensor) for n in ("q", "k_cache", "v_cache", "page_table", "seq_lens", "out", "lse", "mass")] + [
        ("sm_scale", ctypes.c_float), ("reserved", ctypes.c_int32), ("device_status", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class ArtEvictParams(ctypes.Structure):
    _fields_ = [(n, ArtTensor) for n in ("k_cache", "v_cache", "page_table", "seq_lens", "mass", "new_page_table",
                                         "new_mass", "new_seq_lens", "kept")] + [
        ("budget", ctypes.c_int32), ("sink", ctypes.c_int32), ("recent", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("device_status", ctypes.c_void_p)]


# what follows the tensors in the parameter structures; the tensors themselves
# are described by _marshal
_APPEND_TAIL, _SPLIT_TAIL, _EVICT_TAIL = struct.Struct("<QQ"), struct.Struct("<fiQQq"), struct.Struct("<iiiiQ")
assert (11 * ctypes.sizeof(ArtTensor) + _APPEND_TAIL.size, 8 * ctypes.sizeof(ArtTensor) + _SPLIT_TAIL.size,
        9 * ctypes.sizeof(ArtTensor) + _EVICT_TAIL.size) == tuple(
            ctypes.sizeof(c) for c in (ArtAppendParams, ArtSplitParams, ArtEvictParams))
_FN = {}
for _name in ("art_rope_append", "art_decode_attention_split", "art_cache_evict"):
    getattr(_lib, _name).argtypes = [ctypes.c_char_p, ctypes.c_void_p]
    getattr(_lib, _name).restype = ctypes.c_int
    _FN[_name] = ctypes.cast(getattr(_lib, _name), ctypes.c_void_p).value
_lib.art_split_workspace_bytes.argtypes = [ctypes.c_char_p]
_lib.art_split_workspace_bytes.restype = ctypes.c_int64
_FN["art_split_workspace_bytes"] = ctypes.cast(_lib.art_split_workspace_bytes, ctypes.c_void_p).value
_lib.art_evict_cluster_size.argtypes = [ctypes.c_char_p]
_lib.art_evict_cluster_size.restype = ctypes.c_int32
_lib.art_rope_init.argtypes = [_P(ArtRope)] + [ctypes.c_int32] * 3 + [
    ctypes.c_double, ctypes.c_int32, ctypes.c_double, ctypes.c_int32] + [ctypes.c_double] * 3
_lib.art_rope_init.restype = ctypes.c_int
_lib.art_rope_init_freqs.argtypes = [_P(ArtRope)] + [ctypes.c_int32] * 3 + [_P(ctypes.c_double), ctypes.c_double]
_lib.art_rope_init_freqs.restype = ctypes.c_int


class ArtError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({art_strerror(status)})")


def art_strerror(status: int) -> str:
    return _lib.art_strerror(int(status)).decode()


def art_version() -> int:
    return int(_lib.art_version())


def _tensor_fields(t):
    """The eleven art_tensor_t values of a tensor (all zero for None)."""
    if t is None:
        return (0,) * 11
    n = t.dim()
    sh, sd = tuple(t.shape), t.stride()
    if n < 4:
        pad = (0,) * (4 - n)
        sh, sd = sh + pad, sd + pad
    return (t.data_ptr() if t.numel() else 0, _DTYPE.get(t.dtype, -1), n) + sh + sd


def _addr(t):
    return t.data_ptr() if t is not None else 0


def descriptor(t: torch.Tensor) -> ArtTensor:
    """art_tensor_t over a tensor's storage (no copy)."""
    d = ArtTensor()
    d.data = t.data_ptr() if t.numel() else None
    d.dtype = _DTYPE.get(t.dtype, -1)
    d.ndim = t.dim()
    for i in range(t.dim()):
        d.shape[i] = t.shape[i]
        d.stride[i] = t.stride(i)
    return d


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libart runs on the GPU only: every tensor must be on a CUDA device")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None and device is not None and device.index is not None:
            return _raw_stream(device.index)  # the same handle, without building a Stream object
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str):
    if status != 0:
        raise ArtError(status, where)


def art_decode_attention(q, k_cache, v_cache, page_table, block_order, seq_lens, eps_m, eps_d, P, min_blocks,
                         out=None, stop_block=None, stream=None):
    """One ART decode-attention step (art_decode_attention in art.h).
    block_order=None walks the default order (sink block, then newest first).
    Returns (out [B,Hq,d] fp32, stop_block [B,Hkv] int32)."""
    _need_cuda(q, k_cache, v_cache, page_table, block_order, seq_lens, out, stop_block)
    B, Hq, d = q.shape
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    if stop_block is None:
        stop_block = torch.empty(B, k_cache.shape[1], dtype=torch.int32, device=q.device)
    ds = [descriptor(t) if t is not None else None
          for t in (q, k_cache, v_cache, page_table, block_order, seq_lens, out, stop_block)]
    refs = [ctypes.byref(x) if x is not None else None for x in ds]
    st = _lib.art_decode_attention(*refs[:6], float(eps_m), float(eps_d), int(P), int(min_blocks), refs[6],
                                   refs[7], _stream(stream, q.device))
    _check(st, "art_decode_attention")
    return out, stop_block


def _params(q, k_cache, v_cache, page_table, block_order, seq_lens, out, stop_block, eps_m, eps_d, P, min_blocks,
            sm_scale, eps_m_per_seq, eps_d_per_seq, P_per_seq, min_blocks_per_seq, blocks_fetched, device_status,
            engine, cluster_size, stages, compute_warps, window, timeout_ns, debug_flags, prefetch, detector_off=0,
            merge_cta=0, want_info=True):
    """Fill art_params_t (argument marshalling only); returns (params, info)."""
    per = [eps_m_per_seq, eps_d_per_seq, P_per_seq, min_blocks_per_seq, blocks_fetched, device_status]
    _need_cuda(q, k_cache, v_cache, page_table, block_order, seq_lens, out, stop_block, *per)
    for t, dt in zip(per, (torch.float32, torch.float32, torch.int32, torch.int32, torch.int32, torch.int32)):
        if t is not None and (t.dtype != dt or not t.is_contiguous()):
            raise ValueError(f"per-sequence/accounting arrays must be contiguous {dt}")
    p = ArtParams.from_buffer_copy(_PARAMS.pack(
        *_tensor_fields(q), *_tensor_fields(k_cache), *_tensor_fields(v_cache), *_tensor_fields(page_table),
        *_tensor_fields(block_order), *_tensor_fields(seq_lens), *_tensor_fields(out), *_tensor_fields(stop_block),
        float(eps_m), float(eps_d), int(P), int(min_blocks), float(sm_scale),
        _addr(eps_m_per_seq), _addr(eps_d_per_seq), _addr(P_per_seq), _addr(min_blocks_per_seq),
        _addr(blocks_fetched), _addr(device_status), int(engine), int(cluster_size), int(stages),
        int(compute_warps), int(window), int(timeout_ns), int(debug_flags), 0, int(prefetch), int(detector_off),
        int(merge_cta), 0, 0))
    info = None
    if want_info:
        info = ArtLaunchInfo()
        p.info = ctypes.pointer(info)
    return p, info


def art_decode_attention_ex(q, k_cache, v_cache, page_table, block_order, seq_lens, *, eps_m=0.0, eps_d=0.0,
                            P=0, min_blocks=0, sm_scale=0.0, eps_m_per_seq=None, eps_d_per_seq=None,
                            P_per_seq=None, min_blocks_per_seq=None, blocks_fetched=None, device_status=None,
                            engine=0, cluster_size=0, stages=0, compute_warps=0, window=0, timeout_ns=0,
                            debug_flags=0, prefetch=0, detector_off=0, merge_cta=0, workspace=None, out=None,
                            stop_block=None, stream=None, want_info=False):
    """art_decode_attention_ex in art.h.  Per-sequence arrays are device
    tensors of length B (float32 thresholds, int32 P / min_blocks);
    workspace a device tensor (any dtype, 256-byte aligned) or None.
    Returns (out, stop_block) or (out, stop_block, launch_info_dict)."""
    B, Hq, d = q.shape
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    if stop_block is None:
        stop_block = torch.empty(B, k_cache.shape[1], dtype=torch.int32, device=q.device)
    p, info = _params(q, k_cache, v_cache, page_table, block_order, seq_lens, out, stop_block, eps_m, eps_d, P,
                      min_blocks, sm_scale, eps_m_per_seq, eps_d_per_seq, P_per_seq, min_blocks_per_seq,
                      blocks_fetched, device_status, engine, cluster_size, stages, compute_warps, window,
                      timeout_ns, debug_flags, prefetch, detector_off, merge_cta, want_info=want_info)
    if workspace is not None:
        _need_cuda(workspace)
        p.workspace = workspace.data_ptr()
        p.workspace_bytes = workspace.numel() * workspace.element_size()
    st = _lib.art_decode_attention_ex(ctypes.byref(p), _stream(stream, q.device))
    _check(st, "art_decode_attention_ex")
    if want_info:
        return out, stop_block, info.as_dict()
    return out, stop_block


def art_decode_attention_multi(q, k_cache, v_cache, page_table, block_order, seq_lens, *, eps_m=0.0, eps_d=0.0,
                               P=0, min_blocks=0, sm_scale=0.0, eps_m_per_seq=None, eps_d_per_seq=None,
                               P_per_seq=None, min_blocks_per_seq=None, blocks_fetched=None, device_status=None,
                               engine=0, cluster_size=0, stages=0, compute_warps=0, window=0, timeout_ns=0,
                               debug_flags=0, prefetch=0, detector_off=0, merge_cta=0, out=None, stop_block=None,
                               stream=None, want_info=False):
    """art_decode_attention_multi in art.h: q [B, T, Hq, d], T query tokens
    per sequence sharing one walk.  Returns (out [B, T, Hq, d],
    stop_block [B, T, Hkv]) or those plus the launch info dict."""
    B, T, Hq, d = q.shape
    if out is None:
        out = torch.empty(B, T, Hq, d, dtype=torch.float32, device=q.device)
    if stop_block is None:
        stop_block = torch.empty(B, T, k_cache.shape[1], dtype=torch.int32, device=q.device)
    p, info = _params(q, k_cache, v_cache, page_table, block_order, seq_lens, out, stop_block, eps_m, eps_d, P,
                      min_blocks, sm_scale, eps_m_per_seq, eps_d_per_seq, P_per_seq, min_blocks_per_seq,
                      blocks_fetched, device_status, engine, cluster_size, stages, compute_warps, window,
                      timeout_ns, debug_flags, prefetch, detector_off, merge_cta, want_info=want_info)
    st = _lib.art_decode_attention_multi(ctypes.byref(p), int(T), _stream(stream, q.device))
    _check(st, "art_decode_attention_multi")
    if want_info:
        return out, stop_block, info.as_dict()
    return out, stop_block


def art_workspace_bytes(q, k_cache, v_cache, page_table, block_order, seq_lens, **options):
    """art_workspace_bytes in art.h: the workspace art_decode_attention_ex can
    use for this problem (0 when its workspace walk does not apply)."""
    B, Hq, d = q.shape
    out = options.pop("out", None)
    stop_block = options.pop("stop_block", None)
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    if stop_block is None:
        stop_block = torch.empty(B, k_cache.shape[1], dtype=torch.int32, device=q.device)
    kw = dict(eps_m=0.0, eps_d=0.0, P=0, min_blocks=0, sm_scale=0.0, eps_m_per_seq=None, eps_d_per_seq=None,
              P_per_seq=None, min_blocks_per_seq=None, blocks_fetched=None, device_status=None, engine=0,
              cluster_size=0, stages=0, compute_warps=0, window=0, timeout_ns=0, debug_flags=0, prefetch=0,
              detector_off=0, merge_cta=0)
    kw.update(options)
    p, _ = _params(q, k_cache, v_cache, page_table, block_order, seq_lens, out, stop_block, want_info=False, **kw)
    n = int(_lib.art_workspace_bytes(ctypes.byref(p)))
    if n < 0:
        raise ArtError(n, "art_workspace_bytes")
    return n


def art_decode_attention_no_alloc(q, k_cache, v_cache, page_table, block_order, seq_lens, *, eps_m=0.0, eps_d=0.0,
                                  P=0, min_blocks=0, sm_scale=0.0, eps_m_per_seq=None, eps_d_per_seq=None,
                                  P_per_seq=None, min_blocks_per_seq=None, blocks_fetched=None, device_status=None,
                                  engine=0, cluster_size=0, stages=0, compute_warps=0, window=0, timeout_ns=0,
                                  prefetch=0, detector_off=0, out=None, stop_block=None, stream=None,
                                  want_info=False):
    """art_decode_attention_no_alloc in art.h: the workspace walk with the
    library's own fixed scratch array, for callers that cannot allocate
    device memory (pass out and stop_block to allocate nothing here either).
    Returns (out, stop_block) or those plus the launch info dict."""
    B, Hq, d = q.shape
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    if stop_block is None:
        stop_block = torch.empty(B, k_cache.shape[1], dtype=torch.int32, device=q.device)
    p, info = _params(q, k_cache, v_cache, page_table, block_order, seq_lens, out, stop_block, eps_m, eps_d, P,
                      min_blocks, sm_scale, eps_m_per_seq, eps_d_per_seq, P_per_seq, min_blocks_per_seq,
                      blocks_fetched, device_status, engine, cluster_size, stages, compute_warps, window,
                      timeout_ns, 0, prefetch, detector_off, 0, want_info=want_info)
    st = _lib.art_decode_attention_no_alloc(ctypes.byref(p), _stream(stream, q.device))
    _check(st, "art_decode_attention_no_alloc")
    if want_info:
        return out, stop_block, info.as_dict()
    return out, stop_block


def art_build_order_sink_recency(seq_lens, page, block_order=None, max_blocks=None, stream=None):
    """Default walk order [0, N-1, ..., 1] (-1 padded) on the device."""
    _need_cuda(seq_lens, block_order)
    if block_order is None:
        if max_blocks is None:
            raise ValueError("give block_order or max_blocks")
        block_order = torch.empty(seq_lens.shape[0], int(max_blocks), dtype=torch.int32, device=seq_lens.device)
    a, b = descriptor(seq_lens), descriptor(block_order)
    st = _lib.art_build_order_sink_recency(ctypes.byref(a), int(page), ctypes.byref(b), _stream(stream))
    _check(st, "art_build_order_sink_recency")
    return block_order


def _status_ptr(device_status):
    if device_status is None:
        return None
    _need_cuda(device_status)
    if device_status.dtype != torch.int32 or device_status.numel() < 1:
        raise ValueError("device_status must be an int32 device tensor")
    return device_status.data_ptr()


def art_page_summary(k_cache, page_table, seq_lens, summary=None, *, dtype=torch.float32, device_status=None,
                     stream=None):
    """Mean key of every referenced page, per kv-head (art_page_summary in
    art.h).  Returns summary [num_pages, Hkv, d] (float32 or bfloat16)."""
    _need_cuda(k_cache, page_table, seq_lens, summary)
    if summary is None:
        NP, Hkv, _, d = k_cache.shape
        summary = torch.zeros(NP, Hkv, d, dtype=dtype, device=k_cache.device)
    ds = [descriptor(t) for t in (k_cache, page_table, seq_lens, summary)]
    st = _lib.art_page_summary(*[ctypes.byref(x) for x in ds], _status_ptr(device_status), _stream(stream))
    _check(st, "art_page_summary")
    return summary


def art_build_order_importance(q, summary, page_table, seq_lens, page, *, sm_scale=0.0, block_scores=None,
                               block_order=None, device_status=None, stream=None):
    """Importance-first walk order (art_build_order_importance in art.h).
    Returns (block_order [B, max_blocks] int32, block_scores [B, max_blocks] float32)."""
    _need_cuda(q, summary, page_table, seq_lens, block_scores, block_order)
    B, mb = page_table.shape
    if block_scores is None:
        block_scores = torch.empty(B, mb, dtype=torch.float32, device=q.device)
    if block_order is None:
        block_order = torch.empty(B, mb, dtype=torch.int32, device=q.device)
    ds = [descriptor(t) for t in (q, summary, page_table, seq_lens, block_scores, block_order)]
    r = [ctypes.byref(x) for x in ds]
    st = _lib.art_build_order_importance(*r[:4], int(page), float(sm_scale), r[4], r[5],
                                         _status_ptr(device_status), _stream(stream))
    _check(st, "art_build_order_importance")
    return block_order, block_scores


# ---- the cache: rows written, attended exactly, thinned ----------------------

_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}


def _run(name, stream, tensors, others, tail):
    """Call an entry point with the tensors' device current; all of them must
    be on one CUDA device."""
    if stream is not None:
        stream = _stream(stream)
    st = _marshal.call(_FN[name], name, stream, tensors, others, tail)
    if st != 0:
        raise ArtError(st, name)


def _allocating(stream, like):
    """Where a call runs on a stream of its own, what it allocates belongs to
    that stream, on the device of `like`: a Stream of it, or a raw handle (0 and
    1 name the device's default stream; ExternalStream would take 0 as a request
    for some stream of torch's own)."""
    _need_cuda(like)
    device = like.device
    if not isinstance(stream, torch.cuda.Stream) or stream.device != device:
        handle = _stream(stream)
        stream = (torch.cuda.default_stream(device) if handle in (0, 1)
                  else torch.cuda.ExternalStream(handle, device=device))
    return torch.cuda.stream(stream)


def art_rope_init(head_dim, *, rot_dim=None, layout="half", base=10000.0, scaling="none", factor=1.0, original_len=0,
                  low_turns=1.0, high_turns=32.0, amplitude=1.0, inv_freq=None):
    """The rotary angles of a model (art_rope_init in art.h): rot_dim of the
    head_dim channels (default all) in layout "half" or "interleaved", angles
    stretched by scaling "none", "linear", "ntk" or "by_parts".  inv_freq
    gives the rot_dim / 2 frequencies (radians a position) instead of base and
    scaling.  Returns an ArtRope, a host structure to keep for
    art_rope_append."""
    rot_dim = head_dim if rot_dim is None else rot_dim
    if layout not in _ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_ROPE_LAYOUTS)}")
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALINGS)}")
    rope = ArtRope()
    if inv_freq is not None:
        f = [float(x) for x in inv_freq]
        if len(f) != rot_dim // 2:
            raise ValueError("inv_freq needs rot_dim / 2 entries")
        arr = (ctypes.c_double * max(1, len(f)))(*f)
        _check(_lib.art_rope_init_freqs(ctypes.byref(rope), int(head_dim), int(rot_dim), _ROPE_LAYOUTS[layout], arr,
                                        float(amplitude)), "art_rope_init_freqs")
        return rope
    _check(_lib.art_rope_init(ctypes.byref(rope), int(head_dim), int(rot_dim), _ROPE_LAYOUTS[layout], float(base),
                              _ROPE_SCALINGS[scaling], float(factor), int(original_len), float(low_turns),
                              float(high_turns), float(amplitude)), "art_rope_init")
    return rope


def art_rope_append(rope, q, k, v, k_cache, v_cache, page_table, slots, *, positions=None, token_seq=None, mass=None,
                    q_out=None, device_status=None, stream=None):
    """Rotate the queries and keys of new tokens and write keys and values
    into the paged cache (art_rope_append in art.h).  q [T, Hq, d],
    k, v [T, Hkv, d], slots [T] int32 cache rows; positions default to the
    slots, token_seq to token i = sequence i.  Returns the rotated queries
    (q_out, which may be q; a padding token's row is left as it was, so it holds
    anything in one allocated here)."""
    if q_out is None:
        if stream is None:
            q_out = _marshal.empty_as(q, -2, 0)
        else:
            with _allocating(stream, q):
                q_out = _marshal.empty_as(q, -2, 0)
    _run("art_rope_append", stream, (q, k, v, q_out, k_cache, v_cache, page_table, slots, positions, token_seq, mass),
         (device_status,), _APPEND_TAIL.pack(ctypes.addressof(rope), _status_ptr(device_status) or 0))
    return q_out


def art_split_workspace_bytes(q, k_cache, v_cache, page_table, seq_lens, *, mass=None):
    """art_split_workspace_bytes in art.h: the workspace
    art_decode_attention_split needs for tensors of these shapes."""
    n = _marshal.query(_FN["art_split_workspace_bytes"], (q, k_cache, v_cache, page_table, seq_lens, None, None, mass),
                       _SPLIT_TAIL.pack(0.0, 0, 0, 0, 0))
    if n < 0:
        raise ArtError(n, "art_split_workspace_bytes")
    return n


def art_decode_attention_split(q, k_cache, v_cache, page_table, seq_lens, *, sm_scale=0.0, mass=None, out=None, lse=None,
                               workspace=None, device_status=None, stream=None):
    """Exact attention of one new token per sequence, split over the cache's
    length (art_decode_attention_split in art.h).  mass [B, Hkv, width]
    float32, if given, gains the weight every cached token received.
    workspace: a contiguous device tensor (any dtype, 256-byte aligned) of at
    least art_split_workspace_bytes, by default allocated for the call.  Returns
    (out [B, Hq, d] float32, lse [B, Hq] float32); out may be given as
    bfloat16."""
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous: its bytes are written from the first on")
    if stream is not None and (out is None or lse is None or workspace is None):
        with _allocating(stream, q):
            out, lse, workspace = _split_buffers(q, k_cache, v_cache, page_table, seq_lens, mass, out, lse, workspace)
    else:
        out, lse, workspace = _split_buffers(q, k_cache, v_cache, page_table, seq_lens, mass, out, lse, workspace)
    _run("art_decode_attention_split", stream, (q, k_cache, v_cache, page_table, seq_lens, out, lse, mass),
         (workspace, device_status),
         _SPLIT_TAIL.pack(sm_scale, 0, _status_ptr(device_status) or 0, _addr(workspace),
                          workspace.numel() * workspace.element_size() if workspace is not None else 0))
    return out, lse


def _split_buffers(q, k_cache, v_cache, page_table, seq_lens, mass, out, lse, workspace):
    if workspace is None:
        n = art_split_workspace_bytes(q, k_cache, v_cache, page_table, seq_lens, mass=mass)
        if n > 0:
            workspace = _marshal.empty(q, -1, n)
    if out is None:
        out = _marshal.empty_as(q, F32, 0)
    if lse is None:
        lse = _marshal.empty_as(q, F32, 1)
    return out, lse, workspace


def art_cache_evict(k_cache, v_cache, page_table, seq_lens, mass, budget, *, sink=0, recent=0, new_page_table=None,
                    new_mass=None, new_seq_lens=None, kept=None, device_status=None, stream=None):
    """Keep at most budget tokens of every (sequence, kv-head): the first
    sink, the last recent and the heaviest others, in their order
    (art_cache_evict in art.h).  Rows and masses move in place, or to
    new_page_table's pages and to new_mass.  Returns (new_seq_lens [B] int32,
    kept [B, Hkv, budget] int32: old row of every kept token, -1 behind)."""
    if stream is not None and (new_seq_lens is None or kept is None):
        with _allocating(stream, mass):
            new_seq_lens, kept = _evict_buffers(seq_lens, mass, budget, new_seq_lens, kept)
    else:
        new_seq_lens, kept = _evict_buffers(seq_lens, mass, budget, new_seq_lens, kept)
    _run("art_cache_evict", stream,
         (k_cache, v_cache, page_table, seq_lens, mass, new_page_table, new_mass, new_seq_lens, kept), (device_status,),
         _EVICT_TAIL.pack(budget, sink, recent, 0, _status_ptr(device_status) or 0))
    return new_seq_lens, kept


def _evict_buffers(seq_lens, mass, budget, new_seq_lens, kept):
    B, Hkv, _ = mass.shape
    if new_seq_lens is None:
        new_seq_lens = _marshal.empty(mass, I32, B)
    if kept is None:
        kept = _marshal.empty(mass, I32, B, Hkv, max(0, budget))
    return new_seq_lens, kept


def raw_library():
    """The loaded ctypes library (for ABI tests)."""
    return _lib
