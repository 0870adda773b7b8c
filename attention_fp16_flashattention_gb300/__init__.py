"""Fused FP16 attention for one GB300 (sm_103a): Python binding of libgbattn.

The CUDA library (``libgbattn.so``, built in-tree from ``csrc/`` by
``build.py``) does all the work; this module only marshals arguments.  PyTorch
supplies device memory and the current CUDA stream.  Every function has the
name of the C entry point it calls (see ``include/gbattn.h``) and raises
``GbattnError`` when that call returns a non-zero status.  There is no CPU
path: if the library is missing, the first call raises.

The library is loaded lazily, so the seeded input generators in ``inputs``
can be imported on a machine without a GPU.
"""

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgbattn.so")

_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t

_SIGNATURES = {
    "gbattn_version": (_i, []),
    "gbattn_status_string": (ctypes.c_char_p, [_i]),
    "gbattn_device_status": (_i, [_vp, ctypes.POINTER(ctypes.c_uint32)]),
    "gbattn_set_wait_limit_ns": (_i, [ctypes.c_uint64]),
    "gbattn_launch_count": (ctypes.c_uint64, []),
    "gbattn_test_inject_fault": (_i, [_i]),
    "attn_dense_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _f, _vp]),
    "attn_dense_mask_fwd": (_i, [_vp, _vp, _vp, _vp, ctypes.c_longlong, ctypes.c_longlong, _vp, _vp,
                                 _i, _i, _i, _i, _i, _f, _vp]),
    "attn_causal_prefill_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "attn_causal_prefill_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                     _vp, _f, _i, _vp, _sz, _vp]),
    "e4m3_paged_to_fp16": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _vp, _vp, _vp]),
    "attn_causal_prefill_paged_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                           _i, _i, _i, _i, _f, _f, _f, _i, _vp, _sz, _vp]),
    "attn_paged_decode_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "attn_paged_decode_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                   _i, _i, _f, _f, _f, _vp, _sz, _vp]),
    "kv_paged_append_f16": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i,
                                 _i, _i, _vp]),
    "attn_paged_decode_f16_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "attn_paged_decode_f16_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                       _i, _i, _i, _i, _f, _vp, _sz, _vp]),
    "attn_paged_decode_shared_f16_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "attn_paged_decode_shared_f16_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i,
                                              _i, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]),
    "kv_paged_evict": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                            _i, _i, _i, _i, _vp]),
    "attn_diff_paged_decode_f16_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "attn_diff_paged_decode_f16_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _f, _vp, _f, _vp, _vp,
                                            _i, _i, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]),
    "attn_diff_prefill_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "attn_diff_prefill_fwd": (_i, [_vp, _vp, _vp, _vp, _i, _f, _vp, _f, _vp, _vp, _vp, _vp, _i, _i,
                                   _i, _i, _i, _i, _vp, _vp, _vp, _f, _i, _vp, _sz, _vp]),
    "kv_paged_extend": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                             _i, _vp]),
    "kv_paged_release": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "qk_norm_rope_f16": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                              _vp, _vp, _vp, _vp, _vp, _f, _f, _vp]),
    "kv_paged_rope_append": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i,
                                  _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _f, _f, _f,
                                  _f, _vp]),
    "vsa_select_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "vsa_select_blocks": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "vsa_sparse_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                            _i, _i, _f, _vp, _sz, _vp]),
    "vsa_sparse_workspace_size": (_sz, []),
    "vsa_select_coarse_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "vsa_select_blocks_coarse": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp,
                                      _vp, _sz, _vp]),
    "vsa_pair_workspace_size": (_sz, [_i, _i, _i]),
    "vsa_pair_query_cubes": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp]),
}

PROB_SPLIT = 1          # flags of the causal prefill calls (GBATTN_PROB_SPLIT)

DEV_WAIT_TIMEOUT = 1
DEV_BAD_PAGE = 2
DEV_BAD_INDEX = 4
DEV_BAD_LENGTH = 8
DEV_NO_PAGES = 16

_Strides3 = ctypes.c_int64 * 3


class GbattnError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def load():
    """Load libgbattn.so (once) and declare its C signatures."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_string(status):
    return load().gbattn_status_string(int(status)).decode()


def _check(fn, rc):
    if rc != 0:
        raise GbattnError(fn, rc)


def _stream(stream):
    """The CUDA stream handle of `stream`, or of the current device's current stream."""
    import torch
    if stream is not None:
        return stream.cuda_stream
    # torch.cuda.current_stream().cuda_stream without building a Stream object (3 us a call)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, ndim=None):
    try:   # the usual case in one line: a call's argument checks cost as much as its launch
        if t.is_cuda and t.dtype is dtype and t.is_contiguous() and ndim in (None, t.dim()):
            return
    except AttributeError:
        pass
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _need_view(t, name, dtype):
    """A [B, H, S, D] CUDA view whose last dimension is contiguous (any other strides)."""
    try:
        if t.is_cuda and t.dtype is dtype and t.dim() == 4 and t.stride(3) == 1:
            return
    except AttributeError:
        pass
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be a 4-D view with a contiguous last dimension")


def _strides(t):
    """{batch, head, row} element strides of a [B, H, S, D] view, or None when dense."""
    if t.is_contiguous():
        return None
    b, h, s, _ = t.stride()
    return _Strides3(b, h, s)


def _same_layout(a, b):
    """Whether two tensors of one shape have the same strides where a stride means anything: along a
    dimension of one entry it may be any number."""
    sa, sb = a.stride(), b.stride()
    return sa == sb or all(x == y or n == 1 for n, x, y in zip(a.shape, sa, sb))


def _scale(scale, D):
    return float(1.0 / D ** 0.5) if scale is None else float(scale)


def version():
    return load().gbattn_version()


def launch_count():
    """Kernels launched by the library since it was loaded."""
    return int(load().gbattn_launch_count())


def set_wait_limit_ns(ns):
    _check("gbattn_set_wait_limit_ns", load().gbattn_set_wait_limit_ns(int(ns)))


def test_inject_fault(mode):
    """Test hook: 1 makes attention launches skip their query load, 2 stops their K/V loads
    after two rounds of the ring, or after one tile in the FP16 decodes' form for short caches
    (timeout paths, mid-stream for 2); 0 restores."""
    _check("gbattn_test_inject_fault", load().gbattn_test_inject_fault(int(mode)))


def device_status(stream=None):
    """Read and clear the device status word (gbattn_device_flag bits)."""
    out = ctypes.c_uint32(0)
    _check("gbattn_device_status", load().gbattn_device_status(_stream(stream), ctypes.byref(out)))
    return out.value


def attn_dense_fwd(q, k, v, o=None, lse=None, scale=None, stream=None):
    """Dense non-causal attention. q [B,H,Sq,D], k/v [B,H,Skv,D] FP16 -> o [B,H,Sq,D].

    q, k, v and o may be strided views with a contiguous last dimension (e.g. the
    slices of a packed [B,S,3,H,D] QKV tensor, permuted to [B,H,S,D]); k and v
    must share their strides."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need_view(t, n, torch.float16)
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    if tuple(k.shape) != (B, H, Skv, D) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, H, Skv, D] matching q")
    if not _same_layout(k, v):
        raise ValueError("k and v must have the same strides")
    o = torch.empty((B, H, Sq, D), dtype=torch.float16, device=q.device) if o is None else o
    _need_view(o, "o", torch.float16)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    rc = load().attn_dense_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Sq, Skv, D,
                               _strides(q), _strides(k), _strides(o), _scale(scale, D),
                               _stream(stream))
    _check("attn_dense_fwd", rc)
    return o


def attn_dense_mask_fwd(q, k, v, mask, o=None, lse=None, scale=None, stream=None):
    """Dense attention with an additive FP16 mask broadcastable to [B,H,Sq,Skv]
    (rows of Skv contiguous; a size-1 batch or head dimension is shared)."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.float16, 4)
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    if tuple(k.shape) != (B, H, Skv, D) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, H, Skv, D] matching q")
    if not isinstance(mask, torch.Tensor) or not mask.is_cuda or mask.dtype != torch.float16:
        raise ValueError("mask must be a CUDA float16 tensor")
    m4 = mask.reshape((1, 1) + tuple(mask.shape)) if mask.dim() == 2 else mask
    if m4.dim() != 4 or tuple(m4.shape[2:]) != (Sq, Skv) or m4.shape[0] not in (1, B) \
            or m4.shape[1] not in (1, H):
        raise ValueError("mask must broadcast to [B, H, Sq, Skv]")
    if m4.stride(3) != 1 or m4.stride(2) != Skv:
        raise ValueError("mask rows must be contiguous [Sq][Skv]")
    sb = m4.stride(0) if m4.shape[0] > 1 else 0
    sh = m4.stride(1) if m4.shape[1] > 1 else 0
    o = torch.empty_like(q) if o is None else o
    _need(o, "o", torch.float16, 4)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    rc = load().attn_dense_mask_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(m4), sb, sh, _ptr(o), _ptr(lse),
                                    B, H, Sq, Skv, D, _scale(scale, D), _stream(stream))
    _check("attn_dense_mask_fwd", rc)
    return o


def attn_causal_prefill_workspace_size(B, Hq, Q_pad, KV, D):
    return int(load().attn_causal_prefill_workspace_size(B, Hq, Q_pad, KV, D))


def attn_causal_prefill_fwd(q, k, v, q_real=None, o=None, lse=None, scale=None, workspace=None,
                            prob_split=False, stream=None):
    """Causal prefill with shared-KV heads. q [B,Hq,Q_pad,D], k/v [B,Hkv,KV,D] FP16.

    Strided views with a contiguous last dimension are accepted as for
    attn_dense_fwd.  prob_split=True carries the probabilities into the PV
    product as FP16 hi + lo (GBATTN_PROB_SPLIT)."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need_view(t, n, torch.float16)
    B, Hq, Qp, D = q.shape
    Hkv, KV = k.shape[1], k.shape[2]
    if tuple(v.shape) != tuple(k.shape) or k.shape[0] != B or k.shape[3] != D:
        raise ValueError("k and v must be [B, Hkv, KV, D] matching q")
    if not _same_layout(k, v):
        raise ValueError("k and v must have the same strides")
    q_real = Qp if q_real is None else int(q_real)
    o = torch.empty((B, Hq, Qp, D), dtype=torch.float16, device=q.device) if o is None else o
    _need_view(o, "o", torch.float16)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    if workspace is None:
        nbytes = attn_causal_prefill_workspace_size(B, Hq, Qp, KV, D)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    rc = load().attn_causal_prefill_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv,
                                        Qp, q_real, KV, D, _strides(q), _strides(k), _strides(o),
                                        _scale(scale, D), PROB_SPLIT if prob_split else 0,
                                        _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream))
    _check("attn_causal_prefill_fwd", rc)
    return o


def attn_causal_prefill_paged_fwd(q, k_pages, v_pages, page_table, kv_len, k_scale, v_scale,
                                  q_real=None, o=None, lse=None, scale=None, workspace=None,
                                  prob_split=False, stream=None):
    """Causal prefill over paged E4M3 K/V (the bridge fused in).  q [B,Hq,Q_pad,D] FP16;
    pages [P,page,Hkv,D] uint8; page_table int32 [B,max_pages] (or [max_pages] for B=1)."""
    import torch
    _need(q, "q", torch.float16, 4)
    _need(k_pages, "k_pages", torch.uint8, 4)
    _need(v_pages, "v_pages", torch.uint8, 4)
    B, Hq, Qp, D = q.shape
    table = page_table.reshape(1, -1) if page_table.dim() == 1 else page_table
    _need(table, "page_table", torch.int32, 2)
    if table.shape[0] != B:
        raise ValueError("page_table needs one row per batch entry")
    P, ps, Hkv, Dk = k_pages.shape
    if tuple(v_pages.shape) != tuple(k_pages.shape) or Dk != D:
        raise ValueError("k_pages and v_pages must be [P, page, Hkv, D] matching q")
    q_real = Qp if q_real is None else int(q_real)
    o = torch.empty_like(q) if o is None else o
    _need(o, "o", torch.float16, 4)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    if workspace is None:
        nbytes = attn_causal_prefill_workspace_size(B, Hq, Qp, int(kv_len), D)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    rc = load().attn_causal_prefill_paged_fwd(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(table), _ptr(o), _ptr(lse), B, Hq, Hkv, Qp,
        q_real, int(kv_len), D, P, ps, table.shape[1], float(k_scale), float(v_scale),
        _scale(scale, D), PROB_SPLIT if prob_split else 0, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check("attn_causal_prefill_paged_fwd", rc)
    return o


def e4m3_paged_to_fp16(k_pages, v_pages, page_table, kv_len, k_scale, v_scale, k_out=None,
                       v_out=None, stream=None):
    """Paged E4M3 bytes [P, page, Hkv, D] -> FP16 [Hkv, kv_len, D] for K and V."""
    import torch
    _need(k_pages, "k_pages", torch.uint8, 4)
    _need(v_pages, "v_pages", torch.uint8, 4)
    _need(page_table, "page_table", torch.int32, 1)
    P, ps, Hkv, D = k_pages.shape
    if tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages and v_pages must have the same shape")
    if k_out is None:
        k_out = torch.empty((Hkv, kv_len, D), dtype=torch.float16, device=k_pages.device)
    if v_out is None:
        v_out = torch.empty((Hkv, kv_len, D), dtype=torch.float16, device=k_pages.device)
    _need(k_out, "k_out", torch.float16)
    _need(v_out, "v_out", torch.float16)
    rc = load().e4m3_paged_to_fp16(_ptr(k_pages), _ptr(v_pages), _ptr(page_table), P, ps,
                                   int(kv_len), Hkv, D, float(k_scale), float(v_scale),
                                   _ptr(k_out), _ptr(v_out), _stream(stream))
    _check("e4m3_paged_to_fp16", rc)
    return k_out, v_out


def attn_paged_decode_workspace_size(B, Hq, Hkv, nq, max_kv_len, D):
    return int(load().attn_paged_decode_workspace_size(B, Hq, Hkv, nq, max_kv_len, D))


def attn_paged_decode_fwd(q, k_pages, v_pages, page_table, kv_lens, k_scale, v_scale,
                          max_kv_len=None, o=None, lse=None, scale=None, workspace=None,
                          stream=None):
    """Decode over paged E4M3 caches. q [B,Hq,nq,D] FP16; pages [P,page,Hkv,D] uint8;
    page_table int32 [B,max_pages]; kv_lens int32 [B] (device).  max_kv_len defaults to
    max_pages * page_size (no device read)."""
    import torch
    _need(q, "q", torch.float16, 4)
    _need(k_pages, "k_pages", torch.uint8, 4)
    _need(v_pages, "v_pages", torch.uint8, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(kv_lens, "kv_lens", torch.int32, 1)
    B, Hq, nq, D = q.shape
    P, ps, Hkv, Dk = k_pages.shape
    if tuple(v_pages.shape) != tuple(k_pages.shape) or Dk != D:
        raise ValueError("k_pages and v_pages must be [P, page, Hkv, D] matching q")
    if page_table.shape[0] != B or kv_lens.shape[0] != B:
        raise ValueError("page_table and kv_lens need one row per sequence")
    max_pages = page_table.shape[1]
    max_kv_len = max_pages * ps if max_kv_len is None else int(max_kv_len)
    o = torch.empty_like(q) if o is None else o
    _need(o, "o", torch.float16, 4)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    if workspace is None:
        nbytes = attn_paged_decode_workspace_size(B, Hq, Hkv, nq, max_kv_len, D)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    rc = load().attn_paged_decode_fwd(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                      _ptr(kv_lens), _ptr(o), _ptr(lse), B, Hq, Hkv, nq, D, P,
                                      ps, max_pages, max_kv_len, float(k_scale), float(v_scale),
                                      _scale(scale, D), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(stream))
    _check("attn_paged_decode_fwd", rc)
    return o


def _need_shape(t, name, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _same_device(*tensors):
    """Every tensor given on the current device: the call's stream and kernels run there."""
    import torch
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")


def _current_device(t, name):
    """The current device, for a call whose first tensor is t (on a GPU, so CUDA is initialised)."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return torch._C._cuda_getDevice()


def _need_on(t, name, dtype, ndim, dev):
    """_need, and on the current device `dev`.  Calls on one token's work are bound by the host, so
    the usual case is one line."""
    try:
        if (t.dtype is dtype and t.dim() == ndim and t.get_device() == dev
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    _need(t, name, dtype, ndim)
    _same_device(t)


def _need_is(t, name, dtype, shape, dev):
    """_need_on and _need_shape (a tuple) in one."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    _need_on(t, name, dtype, len(shape), dev)
    _need_shape(t, name, shape)


def _need_view_on(t, name, dtype, dev):
    """_need_view, and on the current device `dev`."""
    try:
        if t.dtype is dtype and t.dim() == 4 and t.get_device() == dev and t.stride(3) == 1:
            return
    except AttributeError:
        pass
    _need_view(t, name, dtype)
    _same_device(t)


def _raw_stream(stream, dev):
    """The handle of `stream`, or of device dev's current stream (_stream, the device known)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _new_tensor(shape, dtype, device, stream):
    """A tensor this module allocates for a call on `stream` (None: the current stream), taken
    from that stream's memory so that nothing queued on another stream still uses it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _maker(stream):
    """_new_tensor for `stream`, called as torch.empty, which it is without one."""
    import torch
    if stream is None:
        return torch.empty
    return lambda shape, dtype, device: _new_tensor(shape, dtype, device, stream)


def _new_like(t, stream):
    """_new_tensor of a contiguous tensor's shape and type."""
    import torch
    return torch.empty_like(t) if stream is None else _new_tensor(t.shape, t.dtype, t.device, stream)


def _scratch(nbytes, device, stream):
    """Workspace bytes for one call on `stream`."""
    import torch
    return _new_tensor(max(int(nbytes), 16), torch.uint8, device, stream)


def _int32(x, name):
    """x as the 32-bit integer that the library takes (ctypes would cut it to 32 bits in silence)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} does not fit 32 bits: {x}")
    return x


def _need_workspace(workspace, dev):
    """A caller's workspace: as many bytes as it counts, on the current device `dev`.  A view with
    gaps or a repeated (expanded) dimension covers other memory than its byte count says."""
    import torch
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.get_device() != dev:
        _same_device(workspace)


def _need_paged_f16(k_pages, v_pages, page_table, kv_lens, B, Hkv, D, dev):
    """Checks an FP16 page pool with its table; returns (pages, page size, KV heads, max pages)."""
    import torch
    _need_on(k_pages, "k_pages", torch.float16, 4, dev)
    _need_on(v_pages, "v_pages", torch.float16, 4, dev)
    _need_on(page_table, "page_table", torch.int32, 2, dev)
    _need_on(kv_lens, "kv_lens", torch.int32, 1, dev)
    shape = k_pages.shape
    P, ps, h, d = shape
    if v_pages.shape != shape or d != D or (Hkv is not None and h != Hkv):
        raise ValueError("k_pages and v_pages must be [P, page, Hkv, D] matching the tokens")
    rows, max_pages = page_table.shape
    if rows != B or kv_lens.shape[0] != B:
        raise ValueError("page_table and kv_lens need one row per sequence")
    return P, ps, h, max_pages


def kv_paged_append_f16(k_new, v_new, k_pages, v_pages, page_table, kv_lens, new_lens=None,
                        weights=None, stream=None):
    """Append new tokens to paged FP16 caches, in place.  k_new, v_new [B,Hkv,n,D] FP16 (views
    with a contiguous last dimension and equal strides); pages [P,page,Hkv,D] FP16; page_table
    int32 [B,max_pages]; kv_lens int32 [B] (device): lengths after the call.  new_lens int32 [B]
    (device) appends only the first rows of each sequence; weights FP32 [P,Hkv,page] gets zeros
    at the new slots."""
    import torch
    dev = _current_device(k_new, "k_new")
    _need_view_on(k_new, "k_new", torch.float16, dev)
    _need_view_on(v_new, "v_new", torch.float16, dev)
    B, Hkv, n, D = k_new.shape
    if v_new.shape != k_new.shape or not _same_layout(k_new, v_new):
        raise ValueError("k_new and v_new must have the same shape and strides")
    P, ps, _, max_pages = _need_paged_f16(k_pages, v_pages, page_table, kv_lens, B, Hkv, D, dev)
    if new_lens is not None:
        _need_on(new_lens, "new_lens", torch.int32, 1, dev)
        _need_shape(new_lens, "new_lens", (B,))
    if weights is not None:
        _need_on(weights, "weights", torch.float32, 3, dev)
        _need_shape(weights, "weights", (P, Hkv, ps))
    rc = load().kv_paged_append_f16(k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(),
                                    v_pages.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(),
                                    _ptr(new_lens), _ptr(weights), B, Hkv, n, D, _strides(k_new), P,
                                    ps, max_pages, _raw_stream(stream, dev))
    _check("kv_paged_append_f16", rc)
    return k_pages, v_pages


def attn_paged_decode_f16_workspace_size(B, Hq, Hkv, nq, max_kv_len, D, weights=False):
    return int(load().attn_paged_decode_f16_workspace_size(B, Hq, Hkv, nq, max_kv_len, D,
                                                           1 if weights else 0))


def attn_paged_decode_f16_fwd(q, k_pages, v_pages, page_table, kv_lens, max_kv_len=None, o=None,
                              lse=None, weights=None, scale=None, workspace=None, stream=None):
    """Decode over paged FP16 caches. q [B,Hq,nq,D] FP16; pages [P,page,Hkv,D] FP16; page_table
    int32 [B,max_pages]; kv_lens int32 [B] (device).  weights FP32 [P,Hkv,page] grows by the
    attention every cached token receives (what kv_paged_evict ranks by).  max_kv_len defaults to
    max_pages * page_size (no device read); a bound near the longest cache makes short caches faster,
    and with weights the workspace (allocated here without one) holds a score for every query row and
    token up to it."""
    import torch
    dev = _current_device(q, "q")
    _need_on(q, "q", torch.float16, 4, dev)
    B, Hq, nq, D = q.shape
    P, ps, Hkv, max_pages = _need_paged_f16(k_pages, v_pages, page_table, kv_lens, B, None, D, dev)
    max_kv_len = _int32(max_pages * ps if max_kv_len is None else max_kv_len, "max_kv_len")
    if o is None:
        o = _new_like(q, stream)
    else:
        _need_on(o, "o", torch.float16, 4, dev)
        _need_shape(o, "o", q.shape)
    if lse is not None:
        _need_on(lse, "lse", torch.float32, 3, dev)
        _need_shape(lse, "lse", (B, Hq, nq))
    if weights is not None:
        _need_on(weights, "weights", torch.float32, 3, dev)
        _need_shape(weights, "weights", (P, Hkv, ps))
    if workspace is None:
        workspace = _scratch(attn_paged_decode_f16_workspace_size(B, Hq, Hkv, nq, max_kv_len, D,
                                                                  weights is not None),
                             q.device, stream)
    else:
        _need_workspace(workspace, dev)
    rc = load().attn_paged_decode_f16_fwd(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                          page_table.data_ptr(), kv_lens.data_ptr(), o.data_ptr(),
                                          _ptr(lse), _ptr(weights), B, Hq, Hkv, nq, D, P, ps,
                                          max_pages, max_kv_len, _scale(scale, D),
                                          workspace.data_ptr(), workspace.nbytes,
                                          _raw_stream(stream, dev))
    _check("attn_paged_decode_f16_fwd", rc)
    return o


def attn_paged_decode_shared_f16_workspace_size(B, Hq, Hkv, nq, groups, max_prefix_len, max_own_len, D):
    return int(load().attn_paged_decode_shared_f16_workspace_size(B, Hq, Hkv, nq, groups,
                                                                  max_prefix_len, max_own_len, D))


def attn_paged_decode_shared_f16_fwd(q, k_pages, v_pages, page_table, kv_lens, group_starts,
                                     prefix_lens, max_prefix_len=None, max_own_len=None, o=None,
                                     lse=None, scale=None, workspace=None, stream=None):
    """attn_paged_decode_f16_fwd for requests that share prefixes: sequences group_starts[g] ..
    group_starts[g+1]-1 (int32 [groups+1], from 0 to B) have their first prefix_lens[g] tokens (int32
    [groups], multiples of the page size) in the pages of the first of them, and those are read once.
    kv_lens counts prefix and own tokens.  max_prefix_len and max_own_len (what is behind the
    prefix) default to max_pages * page_size each; near the longest ones they let short caches run in
    one kernel and keep the workspace small.  Prefixes of a few hundred tokens, or of few sequences, are
    as quick with attn_paged_decode_f16_fwd."""
    import torch
    dev = _current_device(q, "q")
    _need_on(q, "q", torch.float16, 4, dev)
    B, Hq, nq, D = q.shape
    P, ps, Hkv, max_pages = _need_paged_f16(k_pages, v_pages, page_table, kv_lens, B, None, D, dev)
    _need_on(prefix_lens, "prefix_lens", torch.int32, 1, dev)
    groups = prefix_lens.shape[0]
    _need_is(group_starts, "group_starts", torch.int32, (groups + 1,), dev)
    max_prefix_len = _int32(max_pages * ps if max_prefix_len is None else max_prefix_len, "max_prefix_len")
    max_own_len = _int32(max_pages * ps if max_own_len is None else max_own_len, "max_own_len")
    if o is None:
        o = _new_like(q, stream)
    else:
        _need_is(o, "o", torch.float16, q.shape, dev)
    if lse is not None:
        _need_is(lse, "lse", torch.float32, (B, Hq, nq), dev)
    if workspace is None:
        workspace = _scratch(attn_paged_decode_shared_f16_workspace_size(
            B, Hq, Hkv, nq, groups, max_prefix_len, max_own_len, D), q.device, stream)
    else:
        _need_workspace(workspace, dev)
    rc = load().attn_paged_decode_shared_f16_fwd(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(),
        group_starts.data_ptr(), prefix_lens.data_ptr(), o.data_ptr(), _ptr(lse), B, Hq, Hkv, nq, D,
        groups, P, ps, max_pages, max_prefix_len, max_own_len, _scale(scale, D), workspace.data_ptr(),
        workspace.nbytes, _raw_stream(stream, dev))
    _check("attn_paged_decode_shared_f16_fwd", rc)
    return o


def kv_paged_evict(k_pages, v_pages, weights, page_table, kv_lens, budget, sink=0, recent=0,
                   dst_table=None, max_kv_len=None, new_lens=None, kept=None, stream=None):
    """Evict the tokens of paged caches (FP16 or uint8 E4M3 pages) that received the least
    attention: every KV head keeps its first `sink` tokens, its last `recent` and the heaviest of
    the rest, `budget` in all, in slots 0.. of dst_table's pages (None: in place).  Rotated keys keep
    their rotation, so positions of later tokens go on from the text, not from new_lens.  Returns
    (new_lens int32 [B], kept int32 [B,Hkv,budget]: old slots, -1 past the new length)."""
    import torch
    if not isinstance(k_pages, torch.Tensor) or k_pages.dtype not in (torch.float16, torch.uint8):
        raise ValueError("k_pages must be a float16 or uint8 tensor")
    cur = _current_device(k_pages, "k_pages")
    _need_on(k_pages, "k_pages", k_pages.dtype, 4, cur)
    _need_on(v_pages, "v_pages", k_pages.dtype, 4, cur)
    _need_on(weights, "weights", torch.float32, 3, cur)
    _need_on(page_table, "page_table", torch.int32, 2, cur)
    _need_on(kv_lens, "kv_lens", torch.int32, 1, cur)
    P, ps, Hkv, D = k_pages.shape
    B, max_pages = page_table.shape
    _need_shape(v_pages, "v_pages", k_pages.shape)
    _need_shape(weights, "weights", (P, Hkv, ps))
    _need_shape(kv_lens, "kv_lens", (B,))
    dst = page_table if dst_table is None else dst_table
    _need_on(dst, "dst_table", torch.int32, 2, cur)
    if dst.shape[0] != B:
        raise ValueError("dst_table needs one row per sequence")
    max_kv_len = _int32(max_pages * ps if max_kv_len is None else max_kv_len, "max_kv_len")
    budget, sink, recent = _int32(budget, "budget"), _int32(sink, "sink"), _int32(recent, "recent")
    if budget <= 0:
        raise ValueError("budget must be positive")
    dev = k_pages.device
    if new_lens is None:
        new_lens = _new_tensor((B,), torch.int32, dev, stream)
    if kept is None:
        kept = _new_tensor((B, Hkv, budget), torch.int32, dev, stream)
    _need_on(new_lens, "new_lens", torch.int32, 1, cur)
    _need_shape(new_lens, "new_lens", (B,))
    _need_on(kept, "kept", torch.int32, 3, cur)
    _need_shape(kept, "kept", (B, Hkv, budget))
    rc = load().kv_paged_evict(k_pages.data_ptr(), v_pages.data_ptr(), weights.data_ptr(),
                               page_table.data_ptr(), dst.data_ptr(), kv_lens.data_ptr(),
                               new_lens.data_ptr(), kept.data_ptr(), B, Hkv, D,
                               k_pages.element_size(), P, ps, max_pages, dst.shape[1], max_kv_len,
                               budget, sink, recent, _raw_stream(stream, cur))
    _check("kv_paged_evict", rc)
    return new_lens, kept


def _need_diff(lambda_vecs, norm_weight, Hq, D, dev):
    """Checks the learned tensors of differential heads; returns lambda_heads (1 or Hq)."""
    import torch
    _need(lambda_vecs, "lambda_vecs", torch.float32)
    if lambda_vecs.get_device() != dev:
        _same_device(lambda_vecs)
    shape = tuple(lambda_vecs.shape)
    heads = shape[1] if len(shape) == 3 else 1
    if shape != (4, Hq, D // 2) and shape not in ((4, D // 2), (4, 1, D // 2)):
        raise ValueError("lambda_vecs must be [4, D/2], [4, 1, D/2] or [4, Hq, D/2]")
    if norm_weight is not None:
        _need_on(norm_weight, "norm_weight", torch.float32, 1, dev)
        _need_shape(norm_weight, "norm_weight", (D,))
    return heads


def attn_diff_paged_decode_f16_workspace_size(B, Hq, Hkv, nq, max_kv_len, D):
    return int(load().attn_diff_paged_decode_f16_workspace_size(B, Hq, Hkv, nq, max_kv_len, D))


def attn_diff_paged_decode_f16_fwd(q, k_pages, v_pages, page_table, kv_lens, lambda_vecs,
                                   lambda_init, norm_weight=None, eps=1e-5, max_kv_len=None,
                                   o=None, lse=None, scale=None, workspace=None, stream=None):
    """Differential attention of the newest tokens over paged FP16 caches: q [B,Hq,nq,128] and
    the cached keys hold two halves of 64, one per softmax map.  lambda_vecs FP32 [4,Hq or 1,64]
    (lq1, lk1, lq2, lk2); norm_weight FP32 [128] or None; lse FP32 [B,Hq,2,nq].  scale defaults to
    1/sqrt(64)."""
    import torch
    dev = _current_device(q, "q")
    _need_on(q, "q", torch.float16, 4, dev)
    B, Hq, nq, D = q.shape
    P, ps, Hkv, max_pages = _need_paged_f16(k_pages, v_pages, page_table, kv_lens, B, None, D, dev)
    heads = _need_diff(lambda_vecs, norm_weight, Hq, D, dev)
    max_kv_len = _int32(max_pages * ps if max_kv_len is None else max_kv_len, "max_kv_len")
    if o is None:
        o = _new_like(q, stream)
    else:
        _need_on(o, "o", torch.float16, 4, dev)
        _need_shape(o, "o", q.shape)
    if lse is not None:
        _need_on(lse, "lse", torch.float32, 4, dev)
        _need_shape(lse, "lse", (B, Hq, 2, nq))
    if workspace is None:
        workspace = _scratch(attn_diff_paged_decode_f16_workspace_size(B, Hq, Hkv, nq, max_kv_len,
                                                                       D), q.device, stream)
    else:
        _need_workspace(workspace, dev)
    rc = load().attn_diff_paged_decode_f16_fwd(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
        kv_lens.data_ptr(), lambda_vecs.data_ptr(), heads, float(lambda_init), _ptr(norm_weight),
        float(eps), o.data_ptr(), _ptr(lse), B, Hq, Hkv, nq, D, P, ps, max_pages, max_kv_len,
        _scale(scale, D // 2), workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, dev))
    _check("attn_diff_paged_decode_f16_fwd", rc)
    return o


def attn_diff_prefill_workspace_size(B, Hq, Sq, Skv, D):
    return int(load().attn_diff_prefill_workspace_size(B, Hq, Sq, Skv, D))


def attn_diff_prefill_fwd(q, k, v, lambda_vecs, lambda_init, norm_weight=None, eps=1e-5,
                          causal=True, q_lens=None, kv_lens=None, o=None, lse=None, scale=None,
                          workspace=None, stream=None):
    """Differential attention of prompts: q [B,Hq,Sq,128], k/v [B,Hkv,Skv,128] FP16, q and k two
    halves of 64, one per softmax map.  Strided views with a contiguous last dimension as for
    attn_dense_fwd.  lambda_vecs FP32 [4,Hq or 1,64] (lq1, lk1, lq2, lk2); norm_weight FP32 [128]
    or None; q_lens, kv_lens int32 [B] (device) or None: padded batches; lse FP32 [B,Hq,2,Sq].
    scale defaults to 1/sqrt(64)."""
    import torch
    dev = _current_device(q, "q")
    _need_view_on(q, "q", torch.float16, dev)
    _need_view_on(k, "k", torch.float16, dev)
    _need_view_on(v, "v", torch.float16, dev)
    B, Hq, Sq, D = q.shape
    Bk, Hkv, Skv, Dk = k.shape
    if v.shape != k.shape or Bk != B or Dk != D:
        raise ValueError("k and v must be [B, Hkv, Skv, D] matching q")
    if not _same_layout(k, v):
        raise ValueError("k and v must have the same strides")
    heads = _need_diff(lambda_vecs, norm_weight, Hq, D, dev)
    for t, n in ((q_lens, "q_lens"), (kv_lens, "kv_lens")):
        if t is not None:
            _need_on(t, n, torch.int32, 1, dev)
            _need_shape(t, n, (B,))
    if o is None:
        o = _new_tensor((B, Hq, Sq, D), torch.float16, q.device, stream)
    else:
        _need_view_on(o, "o", torch.float16, dev)
        _need_shape(o, "o", (B, Hq, Sq, D))
    if lse is not None:
        _need_on(lse, "lse", torch.float32, 4, dev)
        _need_shape(lse, "lse", (B, Hq, 2, Sq))
    if workspace is None:
        workspace = _scratch(attn_diff_prefill_workspace_size(B, Hq, Sq, Skv, D), q.device, stream)
    else:
        _need_workspace(workspace, dev)
    rc = load().attn_diff_prefill_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), lambda_vecs.data_ptr(), heads, float(lambda_init),
        _ptr(norm_weight), float(eps), _ptr(q_lens), _ptr(kv_lens), o.data_ptr(), _ptr(lse), B, Hq,
        Hkv, Sq, Skv, D, _strides(q), _strides(k), _strides(o), _scale(scale, D // 2),
        1 if causal else 0, workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, dev))
    _check("attn_diff_prefill_fwd", rc)
    return o


def _need_tables(page_table, kv_lens, free_pages, free_count, cur):
    """Checks what the page-table calls share; returns (B, max_pages, capacity)."""
    import torch
    _need_on(page_table, "page_table", torch.int32, 2, cur)
    _need_on(free_pages, "free_pages", torch.int32, 1, cur)
    B, max_pages = page_table.shape
    _need_is(kv_lens, "kv_lens", torch.int32, (B,), cur)
    _need_is(free_count, "free_count", torch.int32, (1,), cur)
    return B, max_pages, free_pages.shape[0]


def kv_paged_extend(page_table, kv_lens, new_lens, free_pages, free_count, page_size,
                    num_phys_pages, max_tokens=None, row_tokens=None, kv_lens_out=None,
                    free_count_out=None, token_starts=None, positions=None, slots=None,
                    stream=None):
    """Pages and slots for the new tokens of a batch, from the stack of free pages: page_table int32
    [B,max_pages] is extended in place, kv_lens and new_lens int32 [B], free_pages int32 [capacity]
    with its first free_count[0] entries on the stack (free_count int32 [1]), all on the device.
    max_tokens (the sequences' new tokens end to end) or row_tokens (every sequence's in a row of
    its own) asks for the tokens' positions and slots, int32 [max_tokens] or [B,row_tokens], -1
    where there is no token or its sequence is rejected or gets no pages (end to end, such a sequence
    keeps its places between the others').  Tokens past max_tokens have no slot, and kv_lens_out does not
    count them.  A position is the token's place in the cache: after kv_paged_evict, what the sequence
    has lost is to be added before queries and keys are rotated by it.  Returns (kv_lens_out [B], free_count_out [1], token_starts [B+1],
    positions, slots); each may be given, the first two as kv_lens and free_count themselves; the
    last three are None where neither max_tokens nor row_tokens asks for them."""
    import torch
    cur = _current_device(page_table, "page_table")
    B, max_pages, capacity = _need_tables(page_table, kv_lens, free_pages, free_count, cur)
    _need_is(new_lens, "new_lens", torch.int32, (B,), cur)
    page_size, num_phys_pages = _int32(page_size, "page_size"), _int32(num_phys_pages, "num_phys_pages")
    if max_tokens is not None and row_tokens is not None:
        raise ValueError("max_tokens and row_tokens exclude each other")
    rows = 0 if row_tokens is None else _int32(row_tokens, "row_tokens")
    if row_tokens is not None and rows <= 0:
        raise ValueError("row_tokens must be positive")
    n = B * rows if row_tokens is not None else 0 if max_tokens is None else max_tokens
    n = _int32(n, "max_tokens")
    if max_tokens is not None and n <= 0:
        raise ValueError("max_tokens must be positive")
    if n == 0 and not (token_starts is None and positions is None and slots is None):
        raise ValueError("token_starts, positions and slots need max_tokens or row_tokens")
    # Five tensors are quicker to make than five views of one (20 and 25 us a call).
    dev, shape, new = page_table.device, (B, rows) if rows else (n,), _maker(stream)
    if kv_lens_out is None:
        kv_lens_out = new((B,), dtype=torch.int32, device=dev)
    else:
        _need_is(kv_lens_out, "kv_lens_out", torch.int32, (B,), cur)
    if free_count_out is None:
        free_count_out = new((1,), dtype=torch.int32, device=dev)
    else:
        _need_is(free_count_out, "free_count_out", torch.int32, (1,), cur)
    if n:
        if token_starts is None:
            token_starts = new((B + 1,), dtype=torch.int32, device=dev)
        else:
            _need_is(token_starts, "token_starts", torch.int32, (B + 1,), cur)
        if positions is None:
            positions = new(shape, dtype=torch.int32, device=dev)
        else:
            _need_is(positions, "positions", torch.int32, shape, cur)
        if slots is None:
            slots = new(shape, dtype=torch.int32, device=dev)
        else:
            _need_is(slots, "slots", torch.int32, shape, cur)
    rc = load().kv_paged_extend(page_table.data_ptr(), kv_lens.data_ptr(), new_lens.data_ptr(),
                                free_pages.data_ptr(), free_count.data_ptr(), kv_lens_out.data_ptr(),
                                free_count_out.data_ptr(), _ptr(token_starts), _ptr(positions),
                                _ptr(slots), B, max_pages, page_size, num_phys_pages, capacity, rows,
                                n, _raw_stream(stream, cur))
    _check("kv_paged_extend", rc)
    return kv_lens_out, free_count_out, token_starts, positions, slots


def kv_paged_release(page_table, kv_lens, free_pages, free_count, page_size, num_phys_pages,
                     keep_lens=None, free_count_out=None, stream=None):
    """Give pages back to the stack of free pages (kv_paged_extend): those of every sequence's tokens
    from keep_lens int32 [B] (None: 0) to kv_lens, as far as they hold none that stay.  free_pages is
    written in place; returns free_count_out int32 [1] (may be free_count itself)."""
    import torch
    cur = _current_device(page_table, "page_table")
    B, max_pages, capacity = _need_tables(page_table, kv_lens, free_pages, free_count, cur)
    if keep_lens is not None:
        _need_is(keep_lens, "keep_lens", torch.int32, (B,), cur)
    if free_count_out is None:
        free_count_out = _maker(stream)((1,), dtype=torch.int32, device=page_table.device)
    else:
        _need_is(free_count_out, "free_count_out", torch.int32, (1,), cur)
    rc = load().kv_paged_release(page_table.data_ptr(), kv_lens.data_ptr(), _ptr(keep_lens),
                                 free_pages.data_ptr(), free_count.data_ptr(),
                                 free_count_out.data_ptr(), B, max_pages,
                                 _int32(page_size, "page_size"),
                                 _int32(num_phys_pages, "num_phys_pages"), capacity,
                                 _raw_stream(stream, cur))
    _check("kv_paged_release", rc)
    return free_count_out


def rope_frequencies(rot, base=10000.0, factor=1.0, trained_len=None, method="linear",
                     low_turns=1.0, high_turns=32.0, device="cuda"):
    """Frequencies FP32 [rot/2] for the rotary calls: base^(-2p/rot) radians per position for pair p,
    scaled for contexts `factor` times as long as those a model was trained on.
      "linear": every frequency divided by factor
      "base":   base * factor^(rot/(rot-2)) in place of base: the slowest pair is divided by factor,
                the fastest stays
      "turns":  with r = trained_len * frequency / (2 pi), the turns of a pair within the trained length,
                pairs with r >= high_turns stay, those with r <= low_turns are divided by factor, the
                ones between weighted by (r - low_turns) / (high_turns - low_turns)
      "pairs":  the same ends, the weight falling with the pair's number instead, from the (whole)
                number of the pair that makes high_turns to that of the one that makes low_turns
    Computed in 64 bits on the host, once for a model."""
    import numpy as np
    import torch
    rot = int(rot)
    if rot <= 0 or rot % 2 or not base > 1 or not factor > 0:
        raise ValueError("rot must be even and positive, base above 1, factor positive")
    pair = np.arange(rot // 2, dtype=np.float64)
    if method == "base":
        if rot < 4:
            raise ValueError('"base" needs rot >= 4')
        f = (base * factor ** (rot / (rot - 2.0))) ** (-2 * pair / rot)
    else:
        f = base ** (-2 * pair / rot)
        if method == "linear":
            f = f / factor
        elif method in ("turns", "pairs"):
            if trained_len is None or not 0 < low_turns < high_turns:
                raise ValueError("trained_len and 0 < low_turns < high_turns are needed")
            turns = trained_len * f / (2 * np.pi)
            if method == "turns":
                keep = (turns - low_turns) / (high_turns - low_turns)
            else:
                # the pair (not whole) that makes r turns: trained_len base^(-2p/rot) = 2 pi r
                at = [rot / 2 * np.log(trained_len / (2 * np.pi * r)) / np.log(base)
                      for r in (high_turns, low_turns)]
                first, last = max(np.floor(at[0]), 0.0), min(np.ceil(at[1]), rot - 1.0)
                keep = 1 - (pair - first) / max(last - first, 1e-3)
            keep = np.clip(keep, 0.0, 1.0)
            f = f * (keep + (1 - keep) / factor)
        else:
            raise ValueError(f"unknown method {method!r}")
    return torch.from_numpy(f.astype(np.float32)).to(device)


def _need_rope(positions, freqs, q_weight, k_weight, sections, B, S, D, dev):
    """Checks what the rotary calls share; returns (rot, axes, sections for C)."""
    import torch
    if freqs is None:
        rot = 0
    else:
        _need_on(freqs, "freqs", torch.float32, 1, dev)
        rot = 2 * freqs.shape[0]
    axes = 1
    if positions is not None:
        shape = (B, S)
        if isinstance(positions, torch.Tensor) and positions.dim() == 3:
            axes = positions.shape[0]
            shape = (axes, B, S)
        _need_is(positions, "positions", torch.int32, shape, dev)
    if q_weight is not None:
        _need_is(q_weight, "q_weight", torch.float32, (D,), dev)
    if k_weight is not None:
        _need_is(k_weight, "k_weight", torch.float32, (D,), dev)
    c_sections = None
    if sections is not None:
        sections = [_int32(n, "sections") for n in sections]
        if len(sections) != axes:
            raise ValueError("sections needs one entry per axis of positions")
        c_sections = (ctypes.c_int32 * axes)(*sections)
    return rot, axes, c_sections


def qk_norm_rope_f16(q, k, positions, freqs, q_weight=None, k_weight=None, eps=1e-6,
                     interleaved=False, sections=None, rope_scale=1.0, q_out=None, k_out=None,
                     stream=None):
    """Per-head RMS norms (q_weight, k_weight FP32 [D] or None) and rotation by position of queries
    q [B,Hq,S,D] and keys k [B,Hk,S,D] (or None), FP16 views with a contiguous last dimension.
    positions int32 [B,S] or [axes,B,S] (with sections: pairs per axis); freqs FP32 [rot/2]
    (rope_frequencies), the first rot elements of a head are rotated; None: no rotation.
    interleaved pairs elements (2p, 2p+1), else (p, p + rot/2).  A negative position is padding: its
    rows are not written.  q_out and k_out may be q and k themselves.  Returns (q_out, k_out)."""
    import torch
    dev = _current_device(q, "q")
    _need_view_on(q, "q", torch.float16, dev)
    B, Hq, S, D = q.shape
    rot, axes, c_sections = _need_rope(positions, freqs, q_weight, k_weight, sections, B, S, D, dev)
    Hk = 0
    if k is not None:
        _need_view_on(k, "k", torch.float16, dev)
        Hk = k.shape[1]
        _need_shape(k, "k", (B, Hk, S, D))
        if k_out is None:
            k_out = _maker(stream)((B, Hk, S, D), dtype=torch.float16, device=q.device)
        else:
            _need_view_on(k_out, "k_out", torch.float16, dev)
            _need_shape(k_out, "k_out", (B, Hk, S, D))
    elif k_out is not None:
        raise ValueError("k_out without k")
    if q_out is None:
        q_out = _maker(stream)((B, Hq, S, D), dtype=torch.float16, device=q.device)
    else:
        _need_view_on(q_out, "q_out", torch.float16, dev)
        _need_shape(q_out, "q_out", (B, Hq, S, D))
    rc = load().qk_norm_rope_f16(
        q.data_ptr(), _ptr(k), _ptr(positions), _ptr(freqs), _ptr(q_weight), _ptr(k_weight),
        q_out.data_ptr(), _ptr(k_out), B, Hq, Hk, S, D, rot, 1 if interleaved else 0, axes,
        c_sections, _strides(q), None if k is None else _strides(k), _strides(q_out),
        None if k is None else _strides(k_out), float(eps), float(rope_scale),
        _raw_stream(stream, dev))
    _check("qk_norm_rope_f16", rc)
    return q_out, k_out


def kv_paged_rope_append(q, k_new, v_new, slots, k_pages, v_pages, positions, freqs, q_weight=None,
                         k_weight=None, eps=1e-6, interleaved=False, sections=None, rope_scale=1.0,
                         k_scale=1.0, v_scale=1.0, weights=None, q_out=None, stream=None):
    """qk_norm_rope_f16 on the way into a paged cache: q [B,Hq,S,D] goes to q_out, k_new [B,Hkv,S,D]
    to its slots int32 [B,S] (kv_paged_extend; negative: padding) of k_pages [P,page,Hkv,D], by its
    position in the text (kv_paged_extend's, and what kv_paged_evict has taken from the sequence), and
    v_new, not rotated, to those of v_pages.  Pages are FP16, or uint8 E4M3 codes of value / scale
    (k_scale, v_scale).  weights FP32 [P,Hkv,page] gets zeros at the new slots.  Tokens packed end to
    end are B = 1 and S tokens.  Returns q_out."""
    import torch
    dev = _current_device(q, "q")
    _need_view_on(q, "q", torch.float16, dev)
    _need_view_on(k_new, "k_new", torch.float16, dev)
    _need_view_on(v_new, "v_new", torch.float16, dev)
    B, Hq, S, D = q.shape
    Hkv = k_new.shape[1]
    _need_shape(k_new, "k_new", (B, Hkv, S, D))
    if v_new.shape != k_new.shape or not _same_layout(k_new, v_new):
        raise ValueError("k_new and v_new must have the same shape and strides")
    rot, axes, c_sections = _need_rope(positions, freqs, q_weight, k_weight, sections, B, S, D, dev)
    _need_is(slots, "slots", torch.int32, (B, S), dev)
    if not isinstance(k_pages, torch.Tensor) or k_pages.dtype not in (torch.float16, torch.uint8):
        raise ValueError("k_pages must be a float16 or uint8 tensor")
    dtype = k_pages.dtype
    _need_on(k_pages, "k_pages", dtype, 4, dev)
    P, ps = k_pages.shape[:2]
    _need_shape(k_pages, "k_pages", (P, ps, Hkv, D))
    _need_is(v_pages, "v_pages", dtype, (P, ps, Hkv, D), dev)
    if weights is not None:
        _need_is(weights, "weights", torch.float32, (P, Hkv, ps), dev)
    if q_out is None:
        q_out = _maker(stream)((B, Hq, S, D), dtype=torch.float16, device=q.device)
    else:
        _need_view_on(q_out, "q_out", torch.float16, dev)
        _need_shape(q_out, "q_out", (B, Hq, S, D))
    rc = load().kv_paged_rope_append(
        q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), slots.data_ptr(), _ptr(positions),
        _ptr(freqs), _ptr(q_weight), _ptr(k_weight), q_out.data_ptr(), k_pages.data_ptr(),
        v_pages.data_ptr(), _ptr(weights), B, Hq, Hkv, S, D, rot, 1 if interleaved else 0, axes,
        c_sections, _strides(q), _strides(k_new), _strides(q_out), 2 if dtype is torch.float16 else 1, P, ps,
        float(eps), float(rope_scale), float(k_scale), float(v_scale), _raw_stream(stream, dev))
    _check("kv_paged_rope_append", rc)
    return q_out


def vsa_select_workspace_size(B, H, S, D, block):
    return int(load().vsa_select_workspace_size(B, H, S, D, block))


def vsa_select_blocks(q, k, topk, block=64, prefix=0, cube_valid=None, idx=None, workspace=None,
                      stream=None):
    """Top-k key cubes per query cube.  q, k [B,H,S,D] FP16: `prefix` prefix tokens, then
    cube-major video tokens; cube_valid int32 [cubes] real tokens per cube (None: full).
    Returns idx int32 [B,H,(S-prefix)/block,topk]."""
    import torch
    _need(q, "q", torch.float16, 4)
    _need(k, "k", torch.float16, 4)
    B, H, S, D = q.shape
    if tuple(k.shape) != tuple(q.shape):
        raise ValueError("q and k must have the same shape")
    nc = (S - int(prefix)) // block
    if cube_valid is not None:
        _need(cube_valid, "cube_valid", torch.int32, 1)
    if idx is None:
        idx = torch.empty((B, H, nc, topk), dtype=torch.int32, device=q.device)
    _need(idx, "idx", torch.int32)
    if workspace is None:
        workspace = torch.empty(max(vsa_select_workspace_size(B, H, S, D, block), 16),
                                dtype=torch.uint8, device=q.device)
    rc = load().vsa_select_blocks(_ptr(q), _ptr(k), B, H, S, D, block, int(topk), int(prefix),
                                  _ptr(cube_valid), _ptr(idx), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream))
    _check("vsa_select_blocks", rc)
    return idx


def vsa_select_coarse_workspace_size(B, H, S, D, block=64):
    return int(load().vsa_select_coarse_workspace_size(B, H, S, D, block))


def vsa_select_blocks_coarse(q, k, v, topk, block=64, prefix=0, cube_valid=None, scale=None,
                             idx=None, coarse=None, workspace=None, stream=None):
    """The selection plus the coarse branch: returns (idx int32 [B,H,cubes,topk], coarse FP32
    [B,H,cubes,D]), coarse[i] = softmax over all key cubes of scale * pooled q_i . pooled k_j,
    times the pooled values."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.float16, 4)
    B, H, S, D = q.shape
    if tuple(k.shape) != tuple(q.shape) or tuple(v.shape) != tuple(q.shape):
        raise ValueError("q, k and v must have the same shape")
    nc = (S - int(prefix)) // block
    if cube_valid is not None:
        _need(cube_valid, "cube_valid", torch.int32, 1)
    if idx is None:
        idx = torch.empty((B, H, nc, topk), dtype=torch.int32, device=q.device)
    if coarse is None:
        coarse = torch.empty((B, H, nc, D), dtype=torch.float32, device=q.device)
    _need(idx, "idx", torch.int32)
    _need(coarse, "coarse", torch.float32)
    if workspace is None:
        workspace = torch.empty(max(vsa_select_coarse_workspace_size(B, H, S, D, block), 16),
                                dtype=torch.uint8, device=q.device)
    rc = load().vsa_select_blocks_coarse(_ptr(q), _ptr(k), _ptr(v), B, H, S, D, block, int(topk),
                                         int(prefix), _ptr(cube_valid), _scale(scale, D), _ptr(idx),
                                         _ptr(coarse), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         _stream(stream))
    _check("vsa_select_blocks_coarse", rc)
    return idx, coarse


def vsa_pair_query_cubes(idx, pairs=None, workspace=None, stream=None):
    """Query-cube pairs for vsa_sparse_fwd.  idx int32 [B,H,cubes,topk] ->
    pairs int32 [B,H,ceil(cubes/2),2] (second entry -1 for a lone cube), greedy by selection
    overlap, longest union first.  workspace: vsa_pair_workspace_size bytes (allocated here
    when None)."""
    import torch
    _need(idx, "idx", torch.int32, 4)
    B, H, nc, topk = idx.shape
    if pairs is None:
        pairs = torch.empty((B, H, (nc + 1) // 2, 2), dtype=torch.int32, device=idx.device)
    _need(pairs, "pairs", torch.int32)
    if workspace is None:
        workspace = torch.empty(int(load().vsa_pair_workspace_size(B, H, nc)), dtype=torch.uint8,
                                device=idx.device)
    rc = load().vsa_pair_query_cubes(_ptr(idx), B, H, nc, topk, _ptr(pairs), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream))
    _check("vsa_pair_query_cubes", rc)
    return pairs


_SPARSE_COUNTERS = {}


def sparse_counter(stream=None):
    """The item counter vsa_sparse_fwd uses on `stream` (default: the current stream) when
    it is given no workspace: zeroed device bytes, one buffer per stream, which every call
    leaves at zero.  Calls on one stream run one after another, so they can share it; a
    caller that replays a captured graph on another stream while that stream is busy
    passes its own workspace instead."""
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    key = (s.device.index if s.device.index is not None else torch.cuda.current_device(),
           s.cuda_stream)
    buf = _SPARSE_COUNTERS.get(key)
    if buf is None:
        n = int(load().vsa_sparse_workspace_size())
        buf = torch.zeros(n, dtype=torch.uint8, device=s.device)
        torch.cuda.synchronize(s.device)
        _SPARSE_COUNTERS[key] = buf
    return buf


def vsa_sparse_fwd(q, k, v, idx, block=64, prefix=0, cube_valid=None, pairs=None, o=None,
                   lse=None, scale=None, coarse=None, gate=None, workspace=None, stream=None):
    """Block-sparse attention over the cubes in idx.  q/k/v [B,H,S,D] FP16: `prefix` dense
    prefix tokens, then cube-major video tokens; cube_valid int32 [cubes] or None; pairs from
    vsa_pair_query_cubes or None (adjacent cubes).  coarse (FP32 [B,H,cubes,D] from
    vsa_select_blocks_coarse) and gate (FP16 [B,H,S,D]) add gate * coarse[cube] to every real
    video token's output.  workspace: the item counter (zeroed, left zero by every call);
    None takes this stream's (sparse_counter), False splits the items statically."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.float16, 4)
    _need(idx, "idx", torch.int32, 4)
    if cube_valid is not None:
        _need(cube_valid, "cube_valid", torch.int32, 1)
    if pairs is not None:
        _need(pairs, "pairs", torch.int32, 4)
    B, H, S, D = q.shape
    topk = idx.shape[3]
    if (coarse is None) != (gate is None):
        raise ValueError("coarse and gate go together")
    if coarse is not None:
        _need(coarse, "coarse", torch.float32, 4)
        _need(gate, "gate", torch.float16, 4)
    o = torch.empty_like(q) if o is None else o
    _need(o, "o", torch.float16, 4)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    if workspace is None:
        workspace = sparse_counter(stream)
    ws = None if workspace is False else workspace
    rc = load().vsa_sparse_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(pairs), int(prefix),
                               _ptr(cube_valid), _ptr(coarse), _ptr(gate),
                               _ptr(o), _ptr(lse), B, H, S, D, block, topk, _scale(scale, D),
                               _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                               _stream(stream))
    _check("vsa_sparse_fwd", rc)
    return o
