"""ctypes binding of the C ABI in include/sdpa.h (argument marshalling only).

Every step of the computation runs in the CUDA kernels of libsdpa_gb300.so;
this module only checks tensor properties, fills ``sdpa_params_t``, hands
device pointers and the current CUDA stream to the library, and turns status
codes into exceptions.  There is no CPU path: if the library cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libsdpa_gb300.so")

SDPA_F32, SDPA_F16, SDPA_BF16 = 0, 1, 2
SDPA_FLAG_SHARED_GPU = 0x1
SDPA_FLAG_BOOL_MASK = 0x2
SDPA_FLAG_STRIDES = 0x4
STATUS = {0: "SDPA_OK", 1: "SDPA_ERR_INVALID_ARGUMENT", 2: "SDPA_ERR_UNSUPPORTED",
          3: "SDPA_ERR_MISALIGNED", 4: "SDPA_ERR_WORKSPACE_TOO_SMALL", 5: "SDPA_ERR_CUDA",
          6: "SDPA_ERR_TIMEOUT", 7: "SDPA_ERR_PAGE_TABLE", 8: "SDPA_ERR_POSITION"}
KERNELS = {0: "none", 1: "prefill_tc", 2: "prefill_f32", 3: "decode_splitkv", 4: "no_keys",
           5: "prefill_tc_f32"}

# Every symbol include/sdpa.h declares.
EXPORTS = ("sdpa_workspace_size", "sdpa_select_kernel", "sdpa_forward", "sdpa_status_string",
           "sdpa_device_status", "sdpa_debug_set_wait_limit_ns", "sdpa_abi_version",
           "sdpa_forward_decode_noalloc", "sdpa_last_launch_count",
           "sdpa_backward_workspace_size", "sdpa_backward", "sdpa_debug_set_option",
           "sdpa_host_staging_size", "sdpa_forward_host", "sdpa_paged_write",
           "sdpa_paged_workspace_size", "sdpa_paged_forward", "sdpa_paged_scores",
           "sdpa_paged_evict", "sdpa_rope_table", "sdpa_rope", "sdpa_paged_append",
           "sdpa_paged_append_fp4", "sdpa_paged_forward_fp4")

# sdpa_debug_option_t
DEBUG_OPTIONS = {"decode_splits": 0, "decode_cluster": 1, "decode_drop_last": 2,
                 "prefill_split": 3, "decode_vector": 4, "paged_simt": 5, "paged_ctas": 6}


class SdpaParams(ctypes.Structure):
    """Mirror of sdpa_params_t."""
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("seq_len_q", ctypes.c_int32),
                ("seq_len_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64 * 4),
                ("sinks", ctypes.c_void_p), ("kv_capacity", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("seq_lens_q", ctypes.c_void_p),
                ("seq_lens_kv", ctypes.c_void_p), ("q_stride", ctypes.c_int64 * 3),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("o_stride", ctypes.c_int64 * 3)]


class SdpaPagedParams(ctypes.Structure):
    """Mirror of sdpa_paged_params_t."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("page_table", ctypes.c_void_p), ("page_table_stride", ctypes.c_int64),
                ("cu_seqlens_q", ctypes.c_void_p), ("seq_lens_kv", ctypes.c_void_p),
                ("sinks", ctypes.c_void_p), ("q_stride", ctypes.c_int64 * 2),
                ("o_stride", ctypes.c_int64 * 2), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3)]


class SdpaRotation(ctypes.Structure):
    """Mirror of sdpa_rotation_t."""
    _fields_ = [("table", ctypes.c_void_p), ("table_len", ctypes.c_int64),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("positions", ctypes.c_void_p)]


class SdpaRopeParams(ctypes.Structure):
    """Mirror of sdpa_rope_params_t."""
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("seq_len", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("transpose", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("rotation", SdpaRotation), ("position_stride", ctypes.c_int64),
                ("q_stride", ctypes.c_int64 * 3), ("k_stride", ctypes.c_int64 * 3),
                ("q_out_stride", ctypes.c_int64 * 3), ("k_out_stride", ctypes.c_int64 * 3)]


class SdpaFp4Cache(ctypes.Structure):
    """Mirror of sdpa_fp4_cache_t."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("k_scale_stride", ctypes.c_int64 * 3), ("v_scale_stride", ctypes.c_int64 * 3),
                ("k_gain", ctypes.c_void_p), ("v_gain", ctypes.c_void_p)]


class SdpaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__("%s%s" % (STATUS.get(status, str(status)), (": " + what) if what else ""))


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load (once) and return the ctypes handle of libsdpa_gb300.so."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError("libsdpa_gb300.so is not built (run __graft_entry__.build())")
            lib = ctypes.CDLL(path)
            P = ctypes.POINTER(SdpaParams)
            lib.sdpa_workspace_size.argtypes = [P]
            lib.sdpa_workspace_size.restype = ctypes.c_size_t
            lib.sdpa_select_kernel.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
            lib.sdpa_select_kernel.restype = ctypes.c_int
            lib.sdpa_forward.argtypes = [P, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_size_t, ctypes.c_void_p]
            lib.sdpa_forward.restype = ctypes.c_int
            lib.sdpa_status_string.argtypes = [ctypes.c_int]
            lib.sdpa_status_string.restype = ctypes.c_char_p
            lib.sdpa_device_status.argtypes = [ctypes.c_void_p]
            lib.sdpa_device_status.restype = ctypes.c_int
            lib.sdpa_debug_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
            lib.sdpa_debug_set_wait_limit_ns.restype = ctypes.c_uint64
            lib.sdpa_abi_version.restype = ctypes.c_int
            lib.sdpa_debug_set_option.argtypes = [ctypes.c_int, ctypes.c_int]
            lib.sdpa_debug_set_option.restype = ctypes.c_int
            lib.sdpa_last_launch_count.restype = ctypes.c_int
            lib.sdpa_host_staging_size.argtypes = [P, ctypes.c_int]
            lib.sdpa_host_staging_size.restype = ctypes.c_size_t
            lib.sdpa_forward_host.argtypes = [P] + [ctypes.c_void_p] * 6 + [
                ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p]
            lib.sdpa_forward_host.restype = ctypes.c_int
            lib.sdpa_forward_decode_noalloc.argtypes = [P] + [ctypes.c_void_p] * 6
            lib.sdpa_forward_decode_noalloc.restype = ctypes.c_int
            lib.sdpa_backward_workspace_size.argtypes = [P]
            lib.sdpa_backward_workspace_size.restype = ctypes.c_size_t
            lib.sdpa_backward.argtypes = [P] + [ctypes.c_void_p] * 10 + [ctypes.c_size_t,
                                                                         ctypes.c_void_p]
            lib.sdpa_backward.restype = ctypes.c_int
            PP, vp = ctypes.POINTER(SdpaPagedParams), ctypes.c_void_p
            lib.sdpa_paged_write.argtypes = [PP] + [vp] * 7
            lib.sdpa_paged_write.restype = ctypes.c_int
            lib.sdpa_paged_workspace_size.argtypes = [PP]
            lib.sdpa_paged_workspace_size.restype = ctypes.c_size_t
            lib.sdpa_paged_forward.argtypes = [PP] + [vp] * 6 + [ctypes.c_size_t, vp]
            lib.sdpa_paged_forward.restype = ctypes.c_int
            lib.sdpa_paged_scores.argtypes = [PP] + [vp] * 5 + [ctypes.c_int32, vp,
                                                                ctypes.c_size_t, vp]
            lib.sdpa_paged_scores.restype = ctypes.c_int
            lib.sdpa_paged_evict.argtypes = [PP, ctypes.c_int32, ctypes.c_int32] + [vp] * 5 + [
                ctypes.c_int32] + [vp] * 3
            lib.sdpa_paged_evict.restype = ctypes.c_int
            lib.sdpa_rope_table.argtypes = [vp, ctypes.c_int64, ctypes.c_int32, vp,
                                            ctypes.c_double, vp]
            lib.sdpa_rope_table.restype = ctypes.c_int
            lib.sdpa_rope.argtypes = [ctypes.POINTER(SdpaRopeParams)] + [vp] * 5
            lib.sdpa_rope.restype = ctypes.c_int
            lib.sdpa_paged_append.argtypes = [PP, ctypes.POINTER(SdpaRotation)] + [vp] * 9
            lib.sdpa_paged_append.restype = ctypes.c_int
            FP = ctypes.POINTER(SdpaFp4Cache)
            lib.sdpa_paged_append_fp4.argtypes = [PP, ctypes.POINTER(SdpaRotation), FP] + [vp] * 10
            lib.sdpa_paged_append_fp4.restype = ctypes.c_int
            lib.sdpa_paged_forward_fp4.argtypes = [PP, FP] + [vp] * 4 + [ctypes.c_size_t, vp]
            lib.sdpa_paged_forward_fp4.restype = ctypes.c_int
            _lib = lib
    return _lib


def make_params(B, Hq, Hkv, Lq, Lk, D, dtype, scale, causal=False, mask_ptr=None,
                mask_stride=(0, 0, 0, 1), sinks_ptr=None, kv_capacity=0, seq_lens_q_ptr=None,
                seq_lens_kv_ptr=None, flags=0, strides=None) -> SdpaParams:
    """strides: None, or element strides (batch, head, row) of q, k, v and o
    as four 3-tuples; sets SDPA_FLAG_STRIDES."""
    p = SdpaParams()
    p.batch, p.num_q_heads, p.num_kv_heads = int(B), int(Hq), int(Hkv)
    p.seq_len_q, p.seq_len_kv, p.head_dim = int(Lq), int(Lk), int(D)
    p.dtype = int(dtype)
    p.scale = float(scale)
    p.causal = 1 if causal else 0
    p.reserved0 = 0
    p.mask = mask_ptr
    for i in range(4):
        p.mask_stride[i] = int(mask_stride[i])
    p.sinks = sinks_ptr
    p.kv_capacity = int(kv_capacity)
    p.flags = int(flags)
    if strides is not None:
        p.flags |= SDPA_FLAG_STRIDES
        for field, st in zip(("q_stride", "k_stride", "v_stride", "o_stride"), strides):
            arr = getattr(p, field)
            for i in range(3):
                arr[i] = int(st[i])
    p.seq_lens_q = seq_lens_q_ptr
    p.seq_lens_kv = seq_lens_kv_ptr
    return p


def sdpa_status_string(status: int) -> str:
    return load_library().sdpa_status_string(int(status)).decode()


def sdpa_select_kernel(params: SdpaParams):
    """Returns (kernel name, status code) for a params struct."""
    st = ctypes.c_int(0)
    k = load_library().sdpa_select_kernel(ctypes.byref(params), ctypes.byref(st))
    return KERNELS.get(k, str(k)), st.value


def sdpa_workspace_size(params: SdpaParams) -> int:
    return int(load_library().sdpa_workspace_size(ctypes.byref(params)))


def sdpa_forward_raw(params: SdpaParams, q, k, v, o, lse, workspace, workspace_bytes, stream) -> int:
    """Direct call of the C entry point with integer device addresses."""
    pp = ctypes.byref(params) if params is not None else None
    return int(load_library().sdpa_forward(pp, q, k, v, o, lse, workspace,
                                           int(workspace_bytes), stream))


def sdpa_forward_decode_noalloc_raw(params: SdpaParams, q, k, v, o, lse, stream) -> int:
    """Direct call of the allocation-free decode entry point (integer device
    addresses; partial results in the library's static device scratch)."""
    pp = ctypes.byref(params) if params is not None else None
    return int(load_library().sdpa_forward_decode_noalloc(pp, q, k, v, o, lse, stream))


def sdpa_backward_raw(params: SdpaParams, q, k, v, o, d_o, lse, dq, dk, dv, workspace,
                      workspace_bytes, stream) -> int:
    """Direct call of the backward entry point with integer device addresses."""
    pp = ctypes.byref(params) if params is not None else None
    return int(load_library().sdpa_backward(pp, q, k, v, o, d_o, lse, dq, dk, dv, workspace,
                                            int(workspace_bytes), stream))


def sdpa_backward_workspace_size(params: SdpaParams) -> int:
    return int(load_library().sdpa_backward_workspace_size(ctypes.byref(params)))


def sdpa_backward(q, k, v, o, lse, d_o, scale=None, causal=False, mask=None, sinks=None,
                  dq=None, dk=None, dv=None, workspace=None, stream=None, seq_lens_q=None,
                  seq_lens_kv=None):
    """dQ, dK, dV of sdpa_forward on the GPU (fp32/fp16/bf16, head_dim 64 or
    128).

    q, k, v, mask, sinks, scale, causal and the per-batch lengths
    (seq_lens_q, seq_lens_kv: int32 CUDA tensors of B elements) as given to
    sdpa_forward; o and lse its outputs; d_o the gradient of the loss with
    respect to o (o's shape and dtype).  Tensors need a contiguous last
    dimension; dq, dk, dv default to the layouts of q, k, v.  dk and dv sum
    over the query heads of each kv head; rows past a batch's lengths get
    zero gradients.  Returns (dq, dk, dv).
    """
    torch = _torch()
    for t in (q, k, v, o, d_o):
        if t.dim() != 4 or not t.is_cuda or t.stride(-1) != 1:
            raise ValueError("q, k, v, o, d_o must be 4-D CUDA tensors with a contiguous last "
                             "dimension")
    if not (q.dtype == k.dtype == v.dtype == o.dtype == d_o.dtype):
        raise TypeError("q, k, v, o, d_o must share a dtype")
    B, Hq, Lq, D = q.shape
    _, Hkv, Lk, _ = k.shape
    if v.shape != k.shape or o.shape != q.shape or d_o.shape != q.shape:
        raise ValueError("shape mismatch")
    if lse is None or lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Lq) \
            or not lse.is_contiguous():
        raise ValueError("lse must be the forward's contiguous float32 [B, Hq, Lq] output")
    if d_o.stride() != o.stride():
        raise ValueError("d_o must have o's layout (strides)")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    flags = 0
    mask_ptr, mstride = None, (0, 0, 0, 1)
    if mask is not None:
        if (mask.dtype != q.dtype and mask.dtype != torch.bool) or mask.device != q.device:
            raise TypeError("mask must have q's dtype (or bool) and q's device")
        if mask.dtype == torch.bool:
            flags |= SDPA_FLAG_BOOL_MASK
        mexp = mask.expand(B, Hq, Lq, Lk)
        mstride = tuple(int(s) for s in mexp.stride())
        if Lk == 1:
            mstride = mstride[:3] + (1,)
        mask_ptr = mexp.data_ptr()
    sinks_ptr = None
    if sinks is not None:
        if sinks.dtype != torch.float32 or not sinks.is_cuda or sinks.numel() != Hq:
            raise TypeError("sinks must be a float32 CUDA tensor with Hq elements")
        sinks = sinks.contiguous()
        sinks_ptr = sinks.data_ptr()
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for g, t in ((dq, q), (dk, k), (dv, v)):
        if g.shape != t.shape or g.dtype != t.dtype or g.stride() != t.stride():
            raise ValueError("dq, dk, dv must have the shapes, dtype and layouts of q, k, v")
    lens = []
    for t in (seq_lens_q, seq_lens_kv):
        if t is not None:
            if t.dtype != torch.int32 or not t.is_cuda or t.numel() != B:
                raise TypeError("seq_lens_q / seq_lens_kv must be int32 CUDA tensors of B elements")
            t = t.contiguous()
        lens.append(t)
    strides = tuple(tuple(int(s) for s in t.stride()[:3]) for t in (q, k, v, o))
    params = make_params(B, Hq, Hkv, Lq, Lk, D, dtype_code(q.dtype), scale, causal, mask_ptr,
                         mstride, sinks_ptr, flags=flags, strides=strides,
                         seq_lens_q_ptr=None if lens[0] is None else lens[0].data_ptr(),
                         seq_lens_kv_ptr=None if lens[1] is None else lens[1].data_ptr())
    nbytes = sdpa_backward_workspace_size(params)
    if workspace is None and nbytes > 0:
        workspace = _workspace(nbytes, q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    st = sdpa_backward_raw(params, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                           d_o.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                           dv.data_ptr(), ws_ptr, ws_bytes, stream)
    if st != 0:
        raise SdpaError(st, sdpa_status_string(st))
    return dq, dk, dv


def sdpa_device_status(stream=None) -> int:
    return int(load_library().sdpa_device_status(stream))


def sdpa_debug_set_wait_limit_ns(ns: int) -> int:
    return int(load_library().sdpa_debug_set_wait_limit_ns(int(ns)))


def sdpa_debug_set_option(option, value: int) -> int:
    """Set a test hook of the library (a DEBUG_OPTIONS name or its number);
    returns the previous value."""
    code = DEBUG_OPTIONS[option] if isinstance(option, str) else int(option)
    prev = int(load_library().sdpa_debug_set_option(code, int(value)))
    if prev == -1 and not 0 <= code < len(DEBUG_OPTIONS):
        raise ValueError("unknown debug option %r" % (option,))
    return prev


def sdpa_abi_version() -> int:
    return int(load_library().sdpa_abi_version())


def sdpa_last_launch_count() -> int:
    """Kernels enqueued by this thread's last sdpa_forward call (C ABI)."""
    return int(load_library().sdpa_last_launch_count())


# ----------------------------------------------------------------- torch layer
_ws_cache = {}


_torch_module = None
_dtype_codes = {}


def _torch():
    """torch, imported on first use (the C ABI needs none of it)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _dtype_codes.update({torch.float32: SDPA_F32, torch.float16: SDPA_F16,
                             torch.bfloat16: SDPA_BF16})
        _torch_module = torch
    return _torch_module


def dtype_code(t) -> int:
    code = _dtype_codes.get(t)
    if code is None:
        _torch()
        if t not in _dtype_codes:
            raise TypeError("unsupported dtype %s" % t)
        code = _dtype_codes[t]
    return code


def _workspace(nbytes: int, device):
    torch = _torch()
    key = (device.index, threading.get_ident())
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def sdpa_forward(q, k, v, scale=None, causal=False, mask=None, sinks=None, out=None,
                 lse=None, return_lse=True, workspace=None, stream=None, kv_len=None,
                 seq_lens_q=None, seq_lens_kv=None, shared_gpu=False):
    """O (and LSE) of softmax(scale * q k^T + mask [+ sinks]) v on the GPU.

    q [B, Hq, Lq, D], k/v [B, Hkv, C, D]: CUDA tensors of one dtype (float32,
    float16 or bfloat16) whose last dimension is contiguous; any strides of
    the other dimensions (multiples of 16 bytes), e.g. a [B, L, H, D] tensor
    seen through .transpose(1, 2).  The keys are rows [0, Lk) of k and v, Lk
    = kv_len (default C: with kv_len < C, k and v are a fixed-capacity KV
    cache).  out defaults to q's layout.  mask: None, a tensor of q's dtype
    broadcastable to [B, Hq, Lq, Lk] (additive), or a bool tensor of that
    shape (True = the key is visible).  sinks: None or float32 [Hq].  seq_lens_q,
    seq_lens_kv: None or int32 CUDA tensors [B] of per-batch lengths (padding
    masks; rows past a batch's query length see no key).  scale defaults to
    1/sqrt(D).  shared_gpu: the call runs beside other kernels (sets
    SDPA_FLAG_SHARED_GPU: launch shapes not fitted to an idle GPU).  Returns
    (o, lse) or o.
    """
    torch = _torch()
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, H, L, D]")
    for t in (q, k, v):
        if not t.is_cuda:
            raise ValueError("q, k, v must be CUDA tensors")
        if t.stride(-1) != 1:
            raise ValueError("the last dimension of q, k, v must be contiguous")
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise TypeError("q, k, v must share a dtype")
    B, Hq, Lq, D = q.shape
    _, Hkv, cap, _ = k.shape
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape")
    Lk = cap if kv_len is None else int(kv_len)
    if Lk < 0 or Lk > cap:
        raise ValueError("kv_len must be within [0, k.shape[2]]")
    lens = []
    for t in (seq_lens_q, seq_lens_kv):
        if t is not None:
            if t.dtype != torch.int32 or not t.is_cuda or t.numel() != B or not t.is_contiguous():
                raise TypeError("seq_lens_q / seq_lens_kv must be contiguous int32 CUDA "
                                "tensors with B elements")
            lens.append(t.data_ptr())
        else:
            lens.append(None)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dt = dtype_code(q.dtype)
    mask_ptr, mstride = None, (0, 0, 0, 1)
    flags = SDPA_FLAG_SHARED_GPU if shared_gpu else 0
    if mask is not None:
        if (mask.dtype != q.dtype and mask.dtype != torch.bool) or mask.device != q.device:
            raise TypeError("mask must have q's dtype (or bool) and q's device")
        if mask.dtype == torch.bool:
            flags |= SDPA_FLAG_BOOL_MASK
        mexp = mask.expand(B, Hq, Lq, Lk)
        mstride = tuple(int(s) for s in mexp.stride())
        if Lk == 1:
            mstride = mstride[:3] + (1,)
        mask_ptr = mexp.data_ptr()
    sinks_ptr = None
    if sinks is not None:
        if sinks.dtype != torch.float32 or not sinks.is_cuda or sinks.numel() != Hq:
            raise TypeError("sinks must be a float32 CUDA tensor with Hq elements")
        sinks = sinks.contiguous()
        sinks_ptr = sinks.data_ptr()
    if out is None:
        out = torch.empty_like(q)  # q's layout (a dense permutation stays one)
    elif (tuple(out.shape) != (B, Hq, Lq, D) or out.dtype != q.dtype or not out.is_cuda
          or out.stride(-1) != 1):
        raise ValueError("out must be a CUDA tensor like q with a contiguous last dimension")
    dense = all(t.is_contiguous() for t in (q, k, v, out))
    strides = None if dense else tuple(tuple(int(s) for s in t.stride()[:3])
                                       for t in (q, k, v, out))
    params = make_params(B, Hq, Hkv, Lq, Lk, D, dt, scale, causal, mask_ptr, mstride, sinks_ptr,
                         kv_capacity=cap if (dense and cap != Lk) else 0, seq_lens_q_ptr=lens[0],
                         seq_lens_kv_ptr=lens[1], flags=flags, strides=strides)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    nbytes = sdpa_workspace_size(params)
    if workspace is None and nbytes > 0:
        workspace = _workspace(nbytes, q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    st = sdpa_forward_raw(params, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                          lse.data_ptr() if lse is not None else None, ws_ptr, ws_bytes, stream)
    if st != 0:
        raise SdpaError(st, sdpa_status_string(st))
    return (out, lse) if return_lse else out


# --------------------------------------------------- host-buffer entry point
_host_cache = {}


def sdpa_host_staging_size(params, pieces: int) -> int:
    return int(load_library().sdpa_host_staging_size(ctypes.byref(params), int(pieces)))


def sdpa_forward_host(q, k, v, scale=None, causal=False, mask=None, sinks=None, out=None,
                      lse=None, chunks=8, device=None):
    """sdpa_forward on host tensors through the C call sdpa_forward_host.

    q [B, Hq, Lq, D] and k/v [B, Hkv, Lk, D] are contiguous CPU tensors of one
    dtype (pinned, so that the copies overlap the kernels); mask and sinks,
    if given, are CUDA tensors as for sdpa_forward.  The library cuts the
    (batch, kv-head) pairs into about `chunks` pieces and overlaps each
    piece's copies with the others' kernels on its own streams, forked from
    and joined back to the current stream of `device`; the results (`out`,
    `lse` or new pinned tensors, returned) are complete once that stream
    reaches the end of the call, e.g. after torch.cuda.synchronize().  This
    function only allocates the device staging area (cached per device,
    size and stream: calls on different streams never share one).
    """
    torch = _torch()
    for t in (q, k, v):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous host tensors")
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise TypeError("q, k, v must share a dtype")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, H, L, D]")
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    B, Hq, Lq, D = q.shape
    _, Hkv, Lk, _ = k.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, pin_memory=True)
    for t in (out, lse):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("out and lse must be contiguous host tensors")
    mask_ptr, mstride, flags = None, (0, 0, 0, 1), 0
    if mask is not None:
        if (mask.dtype != q.dtype and mask.dtype != torch.bool) or not mask.is_cuda:
            raise TypeError("mask must have q's dtype (or bool) and live on the GPU")
        if mask.dtype == torch.bool:
            flags |= SDPA_FLAG_BOOL_MASK
        mexp = mask.expand(B, Hq, Lq, Lk)
        if mexp.stride(3) != 1:
            raise ValueError("mask must be contiguous along the key dimension")
        mask_ptr, mstride = mexp.data_ptr(), tuple(mexp.stride())
    sinks_ptr = None
    if sinks is not None:
        if sinks.dtype != torch.float32 or not sinks.is_cuda or sinks.numel() != Hq:
            raise TypeError("sinks must be a float32 CUDA tensor of Hq values")
        sinks_ptr = sinks.data_ptr()
    params = make_params(B, Hq, Hkv, Lq, Lk, D, dtype_code(q.dtype), scale, causal, mask_ptr,
                         mstride, sinks_ptr)
    params.flags |= flags
    pieces = max(1, int(chunks))
    nbytes = sdpa_host_staging_size(params, pieces)
    if nbytes == 0:
        raise SdpaError(2, "problem not supported by sdpa_forward_host")
    stream = torch.cuda.current_stream(device)
    key = (device.index, nbytes, stream.cuda_stream)
    buf = _host_cache.get(key)
    if buf is None:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _host_cache[key] = buf
    st = load_library().sdpa_forward_host(ctypes.byref(params), q.data_ptr(), k.data_ptr(),
                                          v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                          buf.data_ptr(), nbytes, pieces, stream.cuda_stream)
    if st != 0:
        raise SdpaError(st, sdpa_status_string(st))
    return out, lse


# ------------------------------------------------------------ paged KV cache
# SdpaPagedParams as one struct.pack call: filling the ctypes fields one by one
# costs several times as much, and single-token calls are bound by the host.
_PAGED = struct.Struct("<6ifi3iIQqQQQ10q")
_STRIDE2 = struct.Struct("<2q").pack  # two strides as a C array
_paged_fn = {}
_PAGED_KEPT = 4  # workspaces (some 20 or 40 MB each) that a thread keeps at most


class _PagedLocal(threading.local):
    """A thread's workspaces by (device, stream, D), oldest first; they go with
    the thread."""

    def __init__(self):
        self.ws = {}


_paged_local = _PagedLocal()


def _paged_call(name, structs=1):
    """The C entry point taking its parameter structs (the first arguments) as
    bytes."""
    fn = _paged_fn.get(name)
    if fn is None:
        lib = load_library()
        typed = getattr(lib, name)
        fn = type(typed)((name, lib))
        fn.argtypes = [ctypes.c_char_p] * structs + typed.argtypes[structs:]
        fn.restype = typed.restype
        _paged_fn[name] = fn
    return fn


def _paged_cache(dev, k_pages, v_pages, page_table, seq_lens_kv, cu_seqlens_q, code=None):
    """Checks of what the paged calls share (code: the dtype code of q and o
    where it is not the cache's).  Returns the fields of
    SdpaPagedParams that describe the cache: (kv heads, D, dtype code, pages,
    page size), the batch's fields, and the strides of k and v."""
    int32 = _torch().int32
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    shape, ks, dtype = k_pages.shape, k_pages.stride(), k_pages.dtype
    if len(shape) != 4 or ks[3] != 1 or k_pages.get_device() != dev:
        raise ValueError("k_pages must be [pages, kv heads, page_size, D] on the same device "
                         "with a contiguous last dimension")
    vs = ks
    if v_pages is not None:
        vs = v_pages.stride()
        if v_pages.shape != shape or vs[3] != 1 or v_pages.get_device() != dev:
            raise ValueError("v_pages must have k_pages' shape and device and a contiguous last "
                             "dimension")
        if v_pages.dtype is not dtype:
            raise TypeError("k_pages and v_pages must share a dtype")
    B = seq_lens_kv.numel()
    if (seq_lens_kv.dtype is not int32 or seq_lens_kv.get_device() != dev
            or not seq_lens_kv.is_contiguous()):
        raise TypeError("seq_lens_kv must be a contiguous int32 CUDA tensor")
    if page_table.dtype is not int32 or page_table.get_device() != dev:
        raise TypeError("page_table must be an int32 CUDA tensor")
    ts, tst = page_table.shape, page_table.stride()
    if len(ts) != 2 or ts[0] != B or (tst[1] != 1 and ts[1] > 1):
        raise ValueError("page_table must be [sequences, pages] with contiguous rows")
    cu = 0
    if cu_seqlens_q is not None:
        if (cu_seqlens_q.dtype is not int32 or cu_seqlens_q.get_device() != dev
                or cu_seqlens_q.numel() != B + 1 or not cu_seqlens_q.is_contiguous()):
            raise TypeError("cu_seqlens_q must be a contiguous int32 CUDA tensor of sequences + "
                            "1 elements")
        cu = cu_seqlens_q.data_ptr()
    pages, heads, page, D = shape
    return (heads, D, dtype_code(dtype) if code is None else code, pages, page, B, ts[1], page_table.data_ptr(), tst[0], cu,
            seq_lens_kv.data_ptr(), ks, vs)


def _paged_pack(c, T, hq, scale, causal, sinks, qs, os):
    heads, D, dt, pages, page, B, cols, table, tstride, cu, lens, ks, vs = c
    return _PAGED.pack(B, T, hq, heads, D, dt, scale, causal, pages, page, cols, 0, table,
                       tstride, cu, lens, sinks, qs[0], qs[1], os[0], os[1], ks[0], ks[1], ks[2],
                       vs[0], vs[1], vs[2])


def _paged_queries(q, c):
    """q's shape and strides, checked against the cache's."""
    shape, st = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != c[1] or st[2] != 1:
        raise ValueError("q must be [tokens, heads, D] with a contiguous last dimension")
    if dtype_code(q.dtype) != c[2]:
        raise TypeError("q and the cache must share a dtype")
    return shape, st


def _check_lse(lse, shape, dev):
    if (lse.dtype is not _torch().float32 or lse.get_device() != dev
            or lse.shape != shape[:2] or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [tokens, Hq] CUDA tensor")


def _paged_results(q, sinks, out, lse, return_lse, dev):
    """The attention calls' sinks checked, and out, its strides and lse, made
    where they are not given."""
    torch = _torch()
    shape = q.shape
    if sinks is not None and (sinks.dtype is not torch.float32 or sinks.get_device() != dev
                              or sinks.numel() != shape[1] or not sinks.is_contiguous()):
        raise TypeError("sinks must be a contiguous float32 CUDA tensor with Hq elements")
    if out is None:
        out = torch.empty_like(q)
        os = out.stride()
    else:
        os = out.stride()
        if (out.shape != shape or os[2] != 1 or out.dtype is not q.dtype
                or out.get_device() != dev):
            raise ValueError("out must be like q with a contiguous last dimension")
    if lse is not None:
        _check_lse(lse, shape, dev)
    elif return_lse:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device)
    return out, os, lse


def _check_scores(scores, c, dev, what="scores"):
    """The strides of a scores tensor."""
    s, st = scores.shape, scores.stride()
    if (len(s) != 3 or s[0] != c[5] or s[1] != c[0] or (st[2] != 1 and s[2] > 1)
            or scores.dtype is not _torch().float32 or scores.get_device() != dev):
        raise ValueError("%s must be a float32 CUDA tensor [sequences, kv heads, positions] with "
                         "contiguous rows" % what)
    return st


def _check_int32(t, n, dev, what):
    if (t.dtype is not _torch().int32 or t.get_device() != dev or t.numel() != n
            or not t.is_contiguous()):
        raise ValueError("%s must be a contiguous int32 CUDA tensor of %d elements" % (what, n))


def _new_workspace(device, D):
    p = SdpaPagedParams()
    p.num_seqs = p.num_tokens = p.num_q_heads = p.num_kv_heads = p.page_size = 1
    p.head_dim, p.scale = D, 1.0
    torch = _torch()
    return torch.empty(max(sdpa_paged_workspace_size(p), 16), dtype=torch.uint8, device=device)


def _paged_workspace(workspace, dev, device, D, stream):
    """(tensor, address, bytes) of the given workspace, or of one that the
    binding keeps for this thread and the current torch stream, whose calls
    follow one another (those of two threads may interleave their kernels).  It
    comes from that stream's memory, so that one that is dropped (the thread's
    end, or its oldest where it uses more than _PAGED_KEPT) serves nothing else
    before the calls in flight are done.  A call under graph capture gets one of
    its own, which belongs to the graph's pool, so that graphs share none."""
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the same device")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    keep = not _torch()._C._cuda_isCurrentStreamCapturing()
    if keep:
        mine, key = _paged_local.ws, (dev, stream, D)
        kept = mine.get(key)
        if kept is not None:
            return kept
    ws = _new_workspace(device, D)
    made = (ws, ws.data_ptr(), ws.numel())
    if keep:
        if len(mine) >= _PAGED_KEPT:
            del mine[next(iter(mine))]
        mine[key] = made
    return made


def _elsewhere(dev, stream, call):
    """call() with `dev` current and, where a raw stream handle is given, that
    stream current: what the call allocates then belongs to it."""
    torch = _torch()
    with torch.cuda.device(dev):
        if stream is None:
            return call()
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev)):
            return call()


def _paged_status(st):
    if st != 0:
        raise SdpaError(st, sdpa_status_string(st))


def sdpa_paged_workspace_size(params) -> int:
    """Bytes of workspace that sdpa_paged_forward and sdpa_paged_scores need
    for a SdpaPagedParams."""
    return int(load_library().sdpa_paged_workspace_size(ctypes.byref(params)))


def sdpa_paged_write(k, v, k_pages, v_pages, page_table, seq_lens_kv, cu_seqlens_q=None,
                     stream=None):
    """Copy the new tokens' keys and values into a paged KV cache.

    k, v: [T, Hkv, D] packed new tokens.  k_pages, v_pages: [pages, Hkv,
    page_size, D] by shape, any strides with a contiguous last dimension (a
    [pages, page_size, Hkv, D] tensor through .transpose(1, 2), for instance).
    page_table: int32 [B, columns], position p of sequence b in page
    page_table[b, p // page_size].  seq_lens_kv: int32 [B], keys of each
    sequence with its new tokens, which are its last ones.  cu_seqlens_q:
    int32 [B + 1], sequence b's tokens are rows cu[b] .. cu[b + 1]; None: one
    token a sequence.  Rows past the last sequence are not written, nor are
    tokens whose position is negative or past the table's columns.
    """
    dev = k.get_device()
    c = _paged_cache(dev, k_pages, v_pages, page_table, seq_lens_kv, cu_seqlens_q)
    cuda = _torch()._C
    if stream is not None or cuda._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, lambda: sdpa_paged_write(
            k, v, k_pages, v_pages, page_table, seq_lens_kv, cu_seqlens_q))
    shape, kn, vn, dtype = k.shape, k.stride(), v.stride(), k_pages.dtype
    if (len(shape) != 3 or shape[1] != c[0] or shape[2] != c[1] or v.shape != shape
            or kn[2] != 1 or vn[2] != 1 or v.get_device() != dev):
        raise ValueError("k and v must be [tokens, kv heads, D] on the same device with a "
                         "contiguous last dimension")
    if k.dtype is not dtype or v.dtype is not dtype:
        raise TypeError("k, v and the cache must share a dtype")
    p = _paged_pack(c, shape[0], 0, 1.0, 1, 0, (0, 0), (0, 0))
    _paged_status(_paged_call("sdpa_paged_write")(
        p, k.data_ptr(), v.data_ptr(), _STRIDE2(kn[0], kn[1]), _STRIDE2(vn[0], vn[1]),
        k_pages.data_ptr(), v_pages.data_ptr(), cuda._cuda_getCurrentRawStream(dev)))


def sdpa_paged_forward(q, k_pages, v_pages, page_table, seq_lens_kv, cu_seqlens_q=None,
                       scale=None, causal=True, sinks=None, out=None, lse=None, return_lse=True,
                       workspace=None, stream=None):
    """O (and LSE) of the new tokens' attention over a paged KV cache.

    q: [T, Hq, D] packed new tokens (already in the cache: see
    sdpa_paged_write); the cache arguments as for sdpa_paged_write.  causal:
    a token sees the keys up to its own position (else all of its
    sequence's).  sinks: None or float32 [Hq].  scale defaults to 1/sqrt(D).
    out: [T, Hq, D] and lse: float32 [T, Hq]; rows past the last sequence are
    left as they are.  workspace: a uint8 tensor of
    sdpa_paged_workspace_size bytes (one is allocated otherwise).  float32,
    float16, bfloat16; D 64 or 128.  Returns (out, lse) or out.
    """
    torch = _torch()
    dev = q.get_device()
    c = _paged_cache(dev, k_pages, v_pages, page_table, seq_lens_kv, cu_seqlens_q)
    shape, qs = _paged_queries(q, c)
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, lambda: sdpa_paged_forward(
            q, k_pages, v_pages, page_table, seq_lens_kv, cu_seqlens_q, scale, causal, sinks, out,
            lse, return_lse, _new_workspace(q.device, c[1]) if workspace is None else workspace))
    out, os, lse = _paged_results(q, sinks, out, lse, return_lse, dev)
    s = torch._C._cuda_getCurrentRawStream(dev)
    _, wp, wn = _paged_workspace(workspace, dev, q.device, c[1], s)
    p = _paged_pack(c, shape[0], shape[1], 1.0 / math.sqrt(c[1]) if scale is None else scale,
                    1 if causal else 0, 0 if sinks is None else sinks.data_ptr(), qs, os)
    _paged_status(_paged_call("sdpa_paged_forward")(
        p, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), wp, wn, s))
    return (out, lse) if return_lse else out


def sdpa_paged_scores(q, k_pages, lse, scores, page_table, seq_lens_kv, cu_seqlens_q=None,
                      scale=None, causal=True, workspace=None, stream=None):
    """Add the attention weight that each cached key receives from the new
    tokens to `scores` (float32 [B, Hkv, positions], in place, returned): the
    sum over the tokens that see the key and the query heads of its kv head of
    exp(scale * q . k - lse).

    q and the cache arguments as given to sdpa_paged_forward, lse its second
    result.
    """
    cuda = _torch()._C
    dev = q.get_device()
    c = _paged_cache(dev, k_pages, None, page_table, seq_lens_kv, cu_seqlens_q)
    shape, qs = _paged_queries(q, c)
    if stream is not None or cuda._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, lambda: sdpa_paged_scores(
            q, k_pages, lse, scores, page_table, seq_lens_kv, cu_seqlens_q, scale, causal,
            _new_workspace(q.device, c[1]) if workspace is None else workspace))
    ss = _check_scores(scores, c, dev)
    _check_lse(lse, shape, dev)
    s = cuda._cuda_getCurrentRawStream(dev)
    _, wp, wn = _paged_workspace(workspace, dev, q.device, c[1], s)
    p = _paged_pack(c, shape[0], shape[1], 1.0 / math.sqrt(c[1]) if scale is None else scale,
                    1 if causal else 0, 0, qs, (0, 0))
    _paged_status(_paged_call("sdpa_paged_scores")(
        p, q.data_ptr(), k_pages.data_ptr(), lse.data_ptr(), scores.data_ptr(),
        _STRIDE2(ss[0], ss[1]), scores.shape[2], wp, wn, s))
    return scores


def sdpa_paged_evict(k_pages, v_pages, scores, page_table, seq_lens_kv, keep, recent=0,
                     scores_out=None, seq_lens_out=None, kept=None, stream=None):
    """Cut every sequence longer than `keep` back to `keep` keys per kv head:
    its newest min(recent, keep) keys stay, and of the others those of largest
    score (ties to the lower position).  The kept rows of the cache move to
    positions 0, 1, ... of the sequence's own pages, in place; those pages
    must not be shared with another sequence.

    scores: float32 [B, Hkv, positions] as from sdpa_paged_scores.  Returns
    (kept, seq_lens, scores): the old positions int32 [B, Hkv, keep] (-1
    behind the last), the new lengths int32 [B], and the kept keys' scores in
    their new places (0 behind them).  scores_out and seq_lens_out may be
    `scores` and `seq_lens_kv` themselves.
    """
    torch = _torch()
    dev = k_pages.get_device()
    c = _paged_cache(dev, k_pages, v_pages, page_table, seq_lens_kv, None)
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, lambda: sdpa_paged_evict(
            k_pages, v_pages, scores, page_table, seq_lens_kv, keep, recent, scores_out,
            seq_lens_out, kept))
    ss = _check_scores(scores, c, dev)
    keep, recent, B, heads = int(keep), int(recent), c[5], c[0]
    if keep < 1 or recent < 0:
        raise ValueError("keep must be at least 1 and recent at least 0")
    device = scores.device
    if scores_out is None:
        scores_out = (torch.empty_like(scores) if scores.is_contiguous() else
                      torch.empty_strided(scores.shape, ss, dtype=torch.float32, device=device))
    elif scores_out.shape != scores.shape or _check_scores(scores_out, c, dev, "scores_out") != ss:
        raise ValueError("scores_out must have the shape and strides of scores")
    if seq_lens_out is None:
        seq_lens_out = torch.empty_like(seq_lens_kv)
    else:
        _check_int32(seq_lens_out, B, dev, "seq_lens_out")
    if kept is None:
        kept = torch.empty((B, heads, keep), dtype=torch.int32, device=device)
    else:
        _check_int32(kept, B * heads * keep, dev, "kept")
    p = _paged_pack(c, 0, 0, 1.0, 1, 0, (0, 0), (0, 0))
    _paged_status(_paged_call("sdpa_paged_evict")(
        p, keep, recent, k_pages.data_ptr(), v_pages.data_ptr(), scores.data_ptr(),
        scores_out.data_ptr(), _STRIDE2(ss[0], ss[1]), scores.shape[2], kept.data_ptr(),
        seq_lens_out.data_ptr(), torch._C._cuda_getCurrentRawStream(dev)))
    return kept, seq_lens_out, scores_out


# ------------------------------------------------------------ rotary positions
# SdpaRotation, SdpaRopeParams and SdpaFp4Cache as pack calls
_ROTATION = struct.Struct("<QqiiQ")
_ROPE = struct.Struct("<7iIQqiiQq12q")
_FP4 = struct.Struct("<4Q6qQQ")


def rope_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_length=None,
                     beta_fast=32.0, beta_slow=1.0):
    """Angles per position of a head's rotary_dim / 2 pairs, and the gain of the
    rotation: (list of floats, float).

    Pair i turns by base^(-2 i / rotary_dim) a position.  For contexts longer
    than those a model was trained on, `factor` times as long:
      scaling="linear"  positions count 1 / factor (Chen et al., 2023);
      scaling="ntk"     the base grows by factor^(R / (R - 2)), so that the
                        slowest pair counts 1 / factor and the fastest stays;
      scaling="yarn"    pairs that turn more than beta_fast times within
                        original_length positions stay, those that turn less
                        than beta_slow times count 1 / factor, those between
                        are blended, and the gain is 0.1 ln(factor) + 1 (Peng
                        et al., 2023).
    """
    R = int(rotary_dim)
    if R < 2 or R % 2 or not base > 0.0 or not factor > 0.0:
        raise ValueError("rotary_dim must be even and positive, base and factor positive")
    half = R // 2
    if scaling == "ntk":
        if R == 2:
            raise ValueError("scaling='ntk' needs more than one pair")
        base = base * factor ** (R / (R - 2))
    freq = [base ** (-2.0 * i / R) for i in range(half)]
    if scaling is None or scaling == "ntk":
        return freq, 1.0
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling != "yarn":
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    if original_length is None or original_length < 1 or not beta_fast > beta_slow > 0.0 \
            or base <= 1.0:
        raise ValueError("scaling='yarn' needs original_length >= 1, beta_fast > beta_slow > 0 "
                         "and a base above 1")

    def pair_of(turns):  # the (fractional) pair that turns so often in original_length
        return R * math.log(original_length / (2.0 * math.pi * turns)) / (2.0 * math.log(base))

    lo = max(math.floor(pair_of(beta_fast)), 0)
    hi = min(math.ceil(pair_of(beta_slow)), R - 1)
    span = max(hi - lo, 0.001)
    ramp = [min(max((i - lo) / span, 0.0), 1.0) for i in range(half)]
    return ([f * (1.0 - r) + f / factor * r for f, r in zip(freq, ramp)],
            0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0)


def sdpa_rope_table(length, rotary_dim, base=10000.0, scaling=None, factor=1.0,
                    original_length=None, beta_fast=32.0, beta_slow=1.0, inv_freq=None, gain=None,
                    device=None, stream=None):
    """The rotation table float32 [length, rotary_dim / 2, 2] on the GPU: cosine
    and sine of position * frequency, from angles in 64 bits, times the gain.

    Frequencies and gain are those of rope_frequencies(rotary_dim, base,
    scaling, factor, ...), unless inv_freq (rotary_dim / 2 numbers) or gain are
    given.  rotary_dim: a multiple of 16 (the rotary calls' rule).
    """
    torch = _torch()
    length, R = int(length), int(rotary_dim)
    freq, own = rope_frequencies(R, base, scaling, factor, original_length, beta_fast, beta_slow)
    if inv_freq is not None:
        freq = [float(f) for f in inv_freq]
        if len(freq) != R // 2:
            raise ValueError("inv_freq must have rotary_dim / 2 numbers")
    if length < 0:
        raise ValueError("length must not be negative")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else \
        torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device")
    dev = torch.cuda.current_device() if device.index is None else device.index
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, lambda: sdpa_rope_table(
            length, R, inv_freq=freq, gain=own if gain is None else gain))
    table = torch.empty((length, R // 2, 2), dtype=torch.float32, device=device)
    _paged_status(load_library().sdpa_rope_table(
        table.data_ptr(), length, R, (ctypes.c_double * len(freq))(*freq),
        float(own if gain is None else gain), torch._C._cuda_getCurrentRawStream(dev)))
    return table


def _check_table(table, dev):
    """Positions and rotated elements of a rotation table."""
    s = table.shape
    if (len(s) != 3 or s[2] != 2 or table.dtype is not _torch().float32
            or table.get_device() != dev or not table.is_contiguous()):
        raise ValueError("the rotation table must be a contiguous float32 CUDA tensor [positions, "
                         "rotary_dim / 2, 2] on the same device")
    return s[0], 2 * s[1]


def _rope_out(out, x, shape, dtype, dev):
    """The strides of a given output."""
    st = out.stride()
    if out.shape != shape or out.dtype is not dtype or out.get_device() != dev or st[3] != 1:
        raise ValueError("q_out and k_out must be like their inputs with a contiguous last "
                         "dimension")
    return st


def _rope(q, k, table, positions, interleaved, q_out, k_out, stream, transpose):
    torch = _torch()
    dev = q.get_device()
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    shape, dtype, qs = q.shape, q.dtype, q.stride()
    if len(shape) != 4 or qs[3] != 1:
        raise ValueError("q must be [batch, heads, length, D] with a contiguous last dimension")
    B, H, L, D = shape
    heads, kp, kop, ks, ko = 0, None, None, (0, 0, 0), (0, 0, 0)
    if k is not None:
        kshape, ks = k.shape, k.stride()
        if (len(kshape) != 4 or kshape[0] != B or kshape[2] != L or kshape[3] != D or ks[3] != 1
                or k.get_device() != dev):
            raise ValueError("k must be [batch, kv heads, length, D] like q")
        if k.dtype is not dtype:
            raise TypeError("q and k must share a dtype")
        heads, kp = kshape[1], k.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    P, R = _check_table(table, dev)
    pos, pstride = 0, 0
    if positions is not None:
        if positions.dtype is not torch.int32 or positions.get_device() != dev:
            raise TypeError("positions must be an int32 CUDA tensor on the same device")
        ps, pst = positions.shape, positions.stride()
        n = len(ps)
        if (n not in (1, 2) or ps[-1] != L or (n == 2 and ps[0] != B and ps[0] != 1)
                or (L > 1 and pst[-1] != 1)):
            raise ValueError("positions must be [length] or [batch, length] with contiguous rows")
        pos = positions.data_ptr()
        pstride = pst[0] if n == 2 and ps[0] > 1 else 0
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, lambda: _rope(q, k, table, positions, interleaved, q_out,
                                                     k_out, None, transpose))
    if q_out is None:
        q_out = torch.empty_like(q)
        qo = q_out.stride()
    else:
        qo = _rope_out(q_out, q, shape, dtype, dev)
    if k is not None:
        if k_out is None:
            k_out = torch.empty_like(k)
            ko = k_out.stride()
        else:
            ko = _rope_out(k_out, k, kshape, dtype, dev)
        kop = k_out.data_ptr()
    p = _ROPE.pack(B, H, heads, L, D, dtype_code(dtype), transpose, 0, table.data_ptr(), P, R,
                   1 if interleaved else 0, pos, pstride, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2],
                   qo[0], qo[1], qo[2], ko[0], ko[1], ko[2])
    _paged_status(_paged_call("sdpa_rope")(p, q.data_ptr(), kp, q_out.data_ptr(), kop,
                                           torch._C._cuda_getCurrentRawStream(dev)))
    return q_out, k_out


def sdpa_rope(q, k, table, positions=None, interleaved=False, q_out=None, k_out=None,
              stream=None):
    """Rotary positions of q [B, Hq, L, D] and k [B, Hkv, L, D] (k may be None).

    table: float32 [positions, R / 2, 2] as sdpa_rope_table makes it, R <= D a
    multiple of 16: the first R elements of a head turn in pairs (i, i + R / 2),
    or (2 i, 2 i + 1) where interleaved; the others pass.  positions: int32
    [L] or [B, L]; None: 0 .. L - 1.  Any strides with a contiguous last
    dimension (multiples of 16 bytes); D 64, 128 or 512; float32, float16,
    bfloat16.  q_out and k_out may be q and k themselves.  A position outside
    the table leaves its row unrotated and sets the device status word.
    Returns (q_out, k_out).
    """
    return _rope(q, k, table, positions, interleaved, q_out, k_out, stream, 0)


def sdpa_rope_backward(dq_out, dk_out, table, positions=None, interleaved=False, dq=None,
                       dk=None, stream=None):
    """Gradients of q and k from those of sdpa_rope's results (the transposed
    rotation): arguments as for sdpa_rope, which may be given dq_out and dk_out
    themselves as dq and dk.  Returns (dq, dk)."""
    return _rope(dq_out, dk_out, table, positions, interleaved, dq, dk, stream, 1)


def _rotation(table, positions, interleaved, T, dev):
    """SdpaRotation of a step's packed tokens, packed (None: no table)."""
    if table is None:
        if positions is not None:
            raise ValueError("positions without a rotation table")
        return None
    P, R = _check_table(table, dev)
    pos = 0
    if positions is not None:
        _check_int32(positions, T, dev, "positions")
        pos = positions.data_ptr()
    return _ROTATION.pack(table.data_ptr(), P, R, 1 if interleaved else 0, pos)


def _new_tokens(q, k, v, q_out, c, dev):
    """Checks of an append's tokens.  Returns (tokens, heads of q, strides of q,
    q_out and its strides)."""
    shape, dtype = k.shape, k.dtype
    if (len(shape) != 3 or shape[1] != c[0] or shape[2] != c[1] or v.shape != shape
            or k.stride(2) != 1 or v.stride(2) != 1 or v.get_device() != dev):
        raise ValueError("k and v must be [tokens, kv heads, D] on the same device with a "
                         "contiguous last dimension")
    if v.dtype is not dtype:
        raise TypeError("k and v must share a dtype")
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        return shape[0], 0, (0, 0), None, (0, 0)
    qsh, qs = q.shape, q.stride()
    if (len(qsh) != 3 or qsh[0] != shape[0] or qsh[2] != shape[2] or qs[2] != 1
            or q.get_device() != dev):
        raise ValueError("q must be [tokens, heads, D] on the same device with a contiguous last "
                         "dimension")
    if q.dtype is not dtype:
        raise TypeError("q, k and v must share a dtype")
    if q_out is None:
        q_out = _torch().empty_like(q)
    elif (q_out.shape != qsh or q_out.dtype is not dtype or q_out.get_device() != dev
          or q_out.stride(2) != 1):
        raise ValueError("q_out must be like q with a contiguous last dimension")
    return shape[0], qsh[1], qs, q_out, q_out.stride()


def sdpa_paged_append(q, k, v, k_pages, v_pages, page_table, seq_lens_kv, rope_table,
                      cu_seqlens_q=None, positions=None, interleaved=False, q_out=None,
                      stream=None):
    """Rotate a step's new tokens and write them to the paged cache: q rotated to
    q_out, k rotated to its page row, v to its page row (sdpa_rope and
    sdpa_paged_write in one pass).

    q: [T, Hq, D] or None, k and v: [T, Hkv, D] packed new tokens; the cache
    arguments as for sdpa_paged_write; rope_table and interleaved as for
    sdpa_rope.  positions: int32 [T]; None: a token's place in its sequence
    (give them where keys were evicted).  q_out may be q; rows past the last
    sequence are left as they are.  Returns q_out (None without q).
    """
    dev = k.get_device()
    c = _paged_cache(dev, k_pages, v_pages, page_table, seq_lens_kv, cu_seqlens_q)
    cuda = _torch()._C
    if rope_table is None:
        raise ValueError("rope_table is needed (sdpa_paged_write writes rows as they are)")
    if stream is not None or cuda._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, lambda: sdpa_paged_append(
            q, k, v, k_pages, v_pages, page_table, seq_lens_kv, rope_table, cu_seqlens_q,
            positions, interleaved, q_out))
    T, hq, qs, q_out, os = _new_tokens(q, k, v, q_out, c, dev)
    if k.dtype is not k_pages.dtype:
        raise TypeError("k, v and the cache must share a dtype")
    kn, vn = k.stride(), v.stride()
    p = _paged_pack(c, T, hq, 1.0, 1, 0, qs, os)
    _paged_status(_paged_call("sdpa_paged_append", 2)(
        p, _rotation(rope_table, positions, interleaved, T, dev),
        None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
        None if q is None else q_out.data_ptr(), _STRIDE2(kn[0], kn[1]), _STRIDE2(vn[0], vn[1]),
        k_pages.data_ptr(), v_pages.data_ptr(), cuda._cuda_getCurrentRawStream(dev)))
    return q_out


# ---------------------------------------------------------- 4-bit paged KV cache
def _fp4_scales(t, want, dev):
    """The strides of k_scales or v_scales."""
    torch = _torch()
    dtype, st = t.dtype, t.stride()
    if dtype is not torch.uint8 and dtype is not torch.float8_e4m3fn:
        raise TypeError("k_scales and v_scales must be uint8 or float8_e4m3fn")
    if t.shape != want or t.get_device() != dev or st[3] != 1:
        raise ValueError("k_scales and v_scales must be [pages, kv heads, page_size, D / 16] "
                         "on the same device with a contiguous last dimension")
    return st


def _fp4_gain(g, heads, dev):
    """The address of a gain tensor."""
    if (g.dtype is not _torch().float32 or g.get_device() != dev or g.numel() != heads
            or not g.is_contiguous()):
        raise ValueError("k_gain and v_gain must be contiguous float32 CUDA tensors of one "
                         "number a kv head")
    return g.data_ptr()


def _fp4_cache(dev, dtype, k_pages, v_pages, k_scales, v_scales, page_table, seq_lens_kv,
               cu_seqlens_q, k_gain, v_gain):
    """Checks of a 4-bit cache: the fields of _paged_cache for rows of `dtype`,
    and SdpaFp4Cache packed."""
    if k_pages.dtype is not _torch().uint8:
        raise TypeError("k_pages and v_pages must be uint8 (two codes a byte)")
    heads, half, code, pages, page, B, cols, table, tst, cu, lens, ks, vs = _paged_cache(
        dev, k_pages, v_pages, page_table, seq_lens_kv, cu_seqlens_q, dtype_code(dtype))
    want = (pages, heads, page, half // 8)
    kss, vss = _fp4_scales(k_scales, want, dev), _fp4_scales(v_scales, want, dev)
    return (heads, 2 * half, code, pages, page, B, cols, table, tst, cu, lens, ks, vs), _FP4.pack(
        k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), kss[0],
        kss[1], kss[2], vss[0], vss[1], vss[2],
        0 if k_gain is None else _fp4_gain(k_gain, heads, dev),
        0 if v_gain is None else _fp4_gain(v_gain, heads, dev))


def sdpa_paged_append_fp4(q, k, v, k_pages, v_pages, k_scales, v_scales, page_table, seq_lens_kv,
                          rope_table=None, cu_seqlens_q=None, positions=None, interleaved=False,
                          k_gain=None, v_gain=None, q_out=None, k_out=None, v_out=None,
                          stream=None):
    """sdpa_paged_append into a 4-bit cache: the rows of k (rotated, rounded to
    their type) and v as 4-bit floats with an 8-bit scale for 16 elements.

    k_pages, v_pages: uint8 [pages, Hkv, page_size, D / 2] (two codes a byte, the
    even element's in the low half); k_scales, v_scales: uint8 or float8_e4m3fn
    [pages, Hkv, page_size, D / 16]; any strides with a contiguous last
    dimension (the pages' multiples of 16 bytes, the scales' of D / 16).
    k_gain, v_gain: float32 [Hkv] or None (1): an element stands for code *
    scale * gain, so that a head's magnitudes fit 2^-10 .. 2688.  rope_table
    None: no rotation (q is copied).  k_out, v_out: None, or [T, Hkv, D] tensors
    of one layout that receive what the written rows stand for, in k's dtype.
    Everything else as for sdpa_paged_append.  Returns q_out (None without q).
    """
    torch = _torch()
    dev = k.get_device()
    c, cache = _fp4_cache(dev, k.dtype, k_pages, v_pages, k_scales, v_scales, page_table,
                          seq_lens_kv, cu_seqlens_q, k_gain, v_gain)
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, lambda: sdpa_paged_append_fp4(
            q, k, v, k_pages, v_pages, k_scales, v_scales, page_table, seq_lens_kv, rope_table,
            cu_seqlens_q, positions, interleaved, k_gain, v_gain, q_out, k_out, v_out))
    T, hq, qs, q_out, os = _new_tokens(q, k, v, q_out, c, dev)
    ostr = None
    for out in (k_out, v_out):
        if out is not None:
            st = out.stride()
            if (out.shape != k.shape or out.dtype is not k.dtype or out.get_device() != dev
                    or st[2] != 1 or (ostr is not None and st != ostr)):
                raise ValueError("k_out and v_out must be like k, of one layout, with a contiguous "
                                 "last dimension")
            ostr = st
    kn, vn = k.stride(), v.stride()
    p = _paged_pack(c, T, hq, 1.0, 1, 0, qs, os)
    _paged_status(_paged_call("sdpa_paged_append_fp4", 3)(
        p, _rotation(rope_table, positions, interleaved, T, dev), cache,
        None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
        None if q is None else q_out.data_ptr(), _STRIDE2(kn[0], kn[1]), _STRIDE2(vn[0], vn[1]),
        None if k_out is None else k_out.data_ptr(), None if v_out is None else v_out.data_ptr(),
        None if ostr is None else _STRIDE2(ostr[0], ostr[1]),
        torch._C._cuda_getCurrentRawStream(dev)))
    return q_out


def sdpa_paged_forward_fp4(q, k_pages, v_pages, k_scales, v_scales, page_table, seq_lens_kv,
                           cu_seqlens_q=None, scale=None, causal=True, sinks=None, k_gain=None,
                           v_gain=None, out=None, lse=None, return_lse=True, workspace=None,
                           stream=None):
    """O (and LSE) of the new tokens' attention over a 4-bit paged cache.

    The cache as for sdpa_paged_append_fp4; everything else as for
    sdpa_paged_forward (q and out float32, float16 or bfloat16; D 64 or 128).
    Returns (out, lse) or out.
    """
    torch = _torch()
    dev = q.get_device()
    c, cache = _fp4_cache(dev, q.dtype, k_pages, v_pages, k_scales, v_scales, page_table,
                          seq_lens_kv, cu_seqlens_q, k_gain, v_gain)
    shape, qs = _paged_queries(q, c)
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, lambda: sdpa_paged_forward_fp4(
            q, k_pages, v_pages, k_scales, v_scales, page_table, seq_lens_kv, cu_seqlens_q, scale,
            causal, sinks, k_gain, v_gain, out, lse, return_lse,
            _new_workspace(q.device, c[1]) if workspace is None else workspace))
    out, os, lse = _paged_results(q, sinks, out, lse, return_lse, dev)
    s = torch._C._cuda_getCurrentRawStream(dev)
    _, wp, wn = _paged_workspace(workspace, dev, q.device, c[1], s)
    p = _paged_pack(c, shape[0], shape[1], 1.0 / math.sqrt(c[1]) if scale is None else scale,
                    1 if causal else 0, 0 if sinks is None else sinks.data_ptr(), qs, os)
    _paged_status(_paged_call("sdpa_paged_forward_fp4", 2)(
        p, cache, q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), wp, wn,
        s))
    return (out, lse) if return_lse else out
