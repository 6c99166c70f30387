"""ctypes binding of libgdn.so (declared in include/gdn.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream.  There is no
fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

GDN_BF16, GDN_FP32 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "misaligned pointer",
          4: "workspace missing or too small", 5: "CUDA runtime error",
          6: "device-side wait timed out"}
EXPORTS = ("gdn_version", "gdn_chunk_size", "gdn_fwd_workspace_size", "gdn_bwd_workspace_size",
           "gdn_fwd", "gdn_fwd_noalloc", "gdn_fwd_noalloc_status", "gdn_bwd", "gdn_decode",
           "gdn_device_status", "gdn_status_string", "gdn_trace_install", "gdn_kernel_name",
           "gdn_set_wait_limit", "gdn_set_test_hook", "gdn_linrec_states_size", "gdn_linrec_fwd", "gdn_linrec_status",
           "gdn_linrec_bwd", "gdn_linrec_decode", "gdn_qk_norm_rope_fwd",
           "gdn_qk_norm_rope_bwd_workspace_size", "gdn_qk_norm_rope_bwd")
GDN_TEST_STALL_COPY, GDN_TEST_FAIL_LAUNCH = 1, 2


class GdnError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__("%s: %s (status %d)" % (what, STATUS.get(code, "?"), code))
        self.code = code


class GdnDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("n_seqs", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("flags", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]

GDN_FLAG_PIECE_SCAN = 1
GDN_FLAG_QK_L2NORM = 2
GDN_FLAG_VALUE_SLICES = 4
GDN_LINREC_COMPLEMENT = 1
GDN_NORM_NONE, GDN_NORM_L2, GDN_NORM_RMS = 0, 1, 2
GDN_QK_INTERLEAVED = 1


class GdnLinrecDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "D", "n_seqs", "x_stride", "g_stride",
                                              "o_stride", "dx_stride", "dg_stride")] + \
               [(n, ctypes.c_int32) for n in ("dtype", "g_dtype", "flags", "reserved")]


class GdnQkDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "Hq", "Hk", "d", "rot", "q_stride",
                                              "k_stride", "qo_stride", "ko_stride", "dq_stride",
                                              "dk_stride")] + \
               [(n, ctypes.c_int32) for n in ("dtype", "norm", "flags")] + [("eps", ctypes.c_float)]


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load libgdn.so (raises if it was not built: there is no other path)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError("libgdn.so not built (run gated_delta_rule_99_b200.build)")
            L = ctypes.CDLL(LIB_PATH)
            vp, sz, i32p, fp = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p
            dp = ctypes.POINTER(GdnDesc)
            L.gdn_version.restype = ctypes.c_int
            L.gdn_chunk_size.restype = ctypes.c_int
            for n in ("gdn_fwd_workspace_size", "gdn_bwd_workspace_size"):
                getattr(L, n).restype = sz
                getattr(L, n).argtypes = [dp]
            L.gdn_fwd.restype = ctypes.c_int
            L.gdn_fwd.argtypes = [dp, vp, vp, vp, fp, fp, i32p, i32p, fp, vp, fp, vp, sz, vp]
            L.gdn_fwd_noalloc.restype = ctypes.c_int
            L.gdn_fwd_noalloc.argtypes = [dp, vp, vp, vp, fp, fp, i32p, i32p, fp, vp, fp, vp]
            L.gdn_fwd_noalloc_status.restype = ctypes.c_int
            L.gdn_fwd_noalloc_status.argtypes = [vp]
            L.gdn_set_wait_limit.restype = None
            L.gdn_set_wait_limit.argtypes = [ctypes.c_uint32]
            L.gdn_set_test_hook.restype = None
            L.gdn_set_test_hook.argtypes = [ctypes.c_int32]
            L.gdn_bwd.restype = ctypes.c_int
            L.gdn_bwd.argtypes = [dp, vp, vp, vp, fp, fp, i32p, i32p, fp, vp, fp, vp, vp, vp, fp,
                                  fp, fp, vp, sz, vp]
            L.gdn_decode.restype = ctypes.c_int
            L.gdn_decode.argtypes = [dp, vp, vp, vp, fp, fp, fp, vp, vp]
            lp = ctypes.POINTER(GdnLinrecDesc)
            L.gdn_linrec_states_size.restype = sz
            L.gdn_linrec_states_size.argtypes = [lp]
            L.gdn_linrec_fwd.restype = ctypes.c_int
            L.gdn_linrec_fwd.argtypes = [lp, vp, vp, i32p, i32p, fp, vp, fp, fp, vp]
            L.gdn_linrec_bwd.restype = ctypes.c_int
            L.gdn_linrec_bwd.argtypes = [lp, vp, vp, i32p, i32p, fp, vp, fp, vp, vp, fp, fp, vp,
                                         sz, vp]
            L.gdn_linrec_status.restype = ctypes.c_int
            L.gdn_linrec_status.argtypes = [vp]
            L.gdn_linrec_decode.restype = ctypes.c_int
            L.gdn_linrec_decode.argtypes = [lp, vp, vp, fp, vp, vp]
            qp = ctypes.POINTER(GdnQkDesc)
            L.gdn_qk_norm_rope_fwd.restype = ctypes.c_int
            L.gdn_qk_norm_rope_fwd.argtypes = [qp, vp, vp, i32p, fp, fp, fp, vp, vp, vp]
            L.gdn_qk_norm_rope_bwd_workspace_size.restype = sz
            L.gdn_qk_norm_rope_bwd_workspace_size.argtypes = [qp]
            L.gdn_qk_norm_rope_bwd.restype = ctypes.c_int
            L.gdn_qk_norm_rope_bwd.argtypes = [qp, vp, vp, i32p, fp, fp, fp, vp, vp, vp, vp, fp, fp,
                                               vp, sz, vp]
            L.gdn_device_status.restype = ctypes.c_int
            L.gdn_device_status.argtypes = [vp, vp]
            L.gdn_status_string.restype = ctypes.c_char_p
            L.gdn_status_string.argtypes = [ctypes.c_int]
            L.gdn_trace_install.restype = None
            L.gdn_trace_install.argtypes = [ctypes.c_void_p]
            L.gdn_kernel_name.restype = ctypes.c_char_p
            L.gdn_kernel_name.argtypes = [ctypes.c_int32]
            _lib = L
    return _lib


def make_desc(B, T, H, dk, dv, n_seqs=0, dtype=GDN_BF16, scale=1.0, flags=0) -> GdnDesc:
    return GdnDesc(int(B), int(T), int(H), int(dk), int(dv), int(n_seqs), int(dtype), float(scale),
                   int(flags), 0)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, dtype=None, shape=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _desc_from(q, v, cu_host, scale, flags=0):
    B, T, H, K = q.shape
    V = v.shape[-1]
    n_seqs = 0 if cu_host is None else cu_host.numel() - 1
    dt = {torch.bfloat16: GDN_BF16, torch.float32: GDN_FP32}.get(q.dtype)
    if dt is None:
        raise ValueError("q must be bf16 or fp32")
    return make_desc(B, T, H, K, V, n_seqs, dt, scale, flags), (B, T, H, K, V, n_seqs)


def _check_mirror(cu_seqlens_host):
    """The library reads the mirror on the host: an address on a device would end the process."""
    if cu_seqlens_host is not None and cu_seqlens_host.device.type != "cpu":
        raise ValueError("cu_seqlens_host must be a CPU tensor, got one on %s" % cu_seqlens_host.device)


def _seqlens(cu_seqlens, cu_seqlens_host, device):
    if cu_seqlens is None and cu_seqlens_host is None:
        return None, None
    _check_mirror(cu_seqlens_host)
    host = cu_seqlens_host if cu_seqlens_host is not None else cu_seqlens.cpu()
    host = host.to(torch.int32).contiguous()
    dev = cu_seqlens if cu_seqlens is not None and cu_seqlens.is_cuda else host.to(device)
    if dev.numel() < host.numel():  # the kernels read as many offsets as the mirror has
        raise ValueError("cu_seqlens has %d values, its host mirror %d" % (dev.numel(), host.numel()))
    return dev.to(torch.int32).contiguous(), host


def fwd_workspace_size(desc: GdnDesc) -> int:
    return int(lib().gdn_fwd_workspace_size(ctypes.byref(desc)))


def bwd_workspace_size(desc: GdnDesc) -> int:
    return int(lib().gdn_bwd_workspace_size(ctypes.byref(desc)))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def gdn_fwd(q, k, v, g, beta, cu_seqlens=None, h0=None, scale=1.0, output_final_state=True,
            o=None, hT=None, workspace=None, cu_seqlens_host=None, stream=None, piece_scan=False,
            qk_l2norm=False, value_slices=False):
    """Forward of the gated delta rule through the C ABI.  Returns (o, hT);
    hT is None when output_final_state is False.  piece_scan sets
    GDN_FLAG_PIECE_SCAN (parallel pieces of long dense rows, joined exactly);
    qk_l2norm sets GDN_FLAG_QK_L2NORM (q and k rows divided by their norms);
    value_slices sets GDN_FLAG_VALUE_SLICES (chains split by value columns)."""
    L = lib()
    cu_dev, cu_host = _seqlens(cu_seqlens, cu_seqlens_host, q.device)
    flags = ((GDN_FLAG_PIECE_SCAN if piece_scan else 0) | (GDN_FLAG_QK_L2NORM if qk_l2norm else 0)
             | (GDN_FLAG_VALUE_SLICES if value_slices else 0))
    desc, (B, T, H, K, V, n_seqs) = _desc_from(q, v, cu_host, scale, flags)
    N = n_seqs if n_seqs else B
    _check(q, "q", q.dtype, (B, T, H, K)); _check(k, "k", q.dtype, (B, T, H, K))
    _check(v, "v", q.dtype, (B, T, H, V))
    _check(g, "g", torch.float32, (B, T, H)); _check(beta, "beta", torch.float32, (B, T, H))
    _check(h0, "h0", torch.float32, (N, H, K, V))
    if o is None:
        o = torch.empty(B, T, H, V, dtype=q.dtype, device=q.device)
    if hT is None and output_final_state:
        hT = torch.empty(N, H, K, V, dtype=torch.float32, device=q.device)
    _check(o, "o", q.dtype, (B, T, H, V)); _check(hT, "hT", torch.float32, (N, H, K, V))
    need = L.gdn_fwd_workspace_size(ctypes.byref(desc))
    if need == 0:
        raise GdnError(2, "gdn_fwd_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    rc = L.gdn_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                   _ptr(cu_dev), None if cu_host is None else ctypes.c_void_p(cu_host.data_ptr()),
                   _ptr(h0), _ptr(o), _ptr(hT), _ptr(workspace), workspace.numel(),
                   _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_fwd")
    return o, hT


def gdn_bwd(q, k, v, g, beta, do, cu_seqlens=None, h0=None, dhT=None, scale=1.0, grads=None,
            workspace=None, cu_seqlens_host=None, stream=None, want_dh0=True, qk_l2norm=False,
            piece_scan=False):
    """Backward through the C ABI.  Returns (dq, dk, dv, dg, dbeta, dh0); with
    qk_l2norm, dq and dk are the gradients w.r.t. the raw (unnormalised) q and k;
    piece_scan sets GDN_FLAG_PIECE_SCAN (both chains of long dense rows in
    parallel pieces, joined exactly)."""
    L = lib()
    cu_dev, cu_host = _seqlens(cu_seqlens, cu_seqlens_host, q.device)
    flags = (GDN_FLAG_QK_L2NORM if qk_l2norm else 0) | (GDN_FLAG_PIECE_SCAN if piece_scan else 0)
    desc, (B, T, H, K, V, n_seqs) = _desc_from(q, v, cu_host, scale, flags)
    N = n_seqs if n_seqs else B
    _check(q, "q", q.dtype, (B, T, H, K)); _check(k, "k", q.dtype, (B, T, H, K))
    _check(v, "v", q.dtype, (B, T, H, V)); _check(do, "do", q.dtype, (B, T, H, V))
    _check(g, "g", torch.float32, (B, T, H)); _check(beta, "beta", torch.float32, (B, T, H))
    _check(h0, "h0", torch.float32, (N, H, K, V)); _check(dhT, "dhT", torch.float32, (N, H, K, V))
    if grads is None:
        e = lambda *s, dt=q.dtype: torch.empty(*s, dtype=dt, device=q.device)
        grads = (e(B, T, H, K), e(B, T, H, K), e(B, T, H, V), e(B, T, H, dt=torch.float32),
                 e(B, T, H, dt=torch.float32),
                 e(N, H, K, V, dt=torch.float32) if want_dh0 else None)
    dq, dk, dv, dg, dbeta, dh0 = grads
    need = L.gdn_bwd_workspace_size(ctypes.byref(desc))
    if need == 0:
        raise GdnError(2, "gdn_bwd_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    rc = L.gdn_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                   _ptr(cu_dev), None if cu_host is None else ctypes.c_void_p(cu_host.data_ptr()),
                   _ptr(h0), _ptr(do), _ptr(dhT), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg),
                   _ptr(dbeta), _ptr(dh0), _ptr(workspace), workspace.numel(), _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_bwd")
    return dq, dk, dv, dg, dbeta, dh0


def gdn_decode(q, k, v, g, beta, state, scale=1.0, o=None, stream=None, qk_l2norm=False):
    """Recurrent decode through the C ABI: advances ``state`` ([B][H][dk][dv]
    fp32, updated in place) through the T tokens of q, k, v ([B][T][H][D]) and
    returns o."""
    L = lib()
    desc, (B, T, H, K, V, _) = _desc_from(q, v, None, scale,
                                         GDN_FLAG_QK_L2NORM if qk_l2norm else 0)
    _check(q, "q", q.dtype, (B, T, H, K)); _check(k, "k", q.dtype, (B, T, H, K))
    _check(v, "v", q.dtype, (B, T, H, V))
    _check(g, "g", torch.float32, (B, T, H)); _check(beta, "beta", torch.float32, (B, T, H))
    _check(state, "state", torch.float32, (B, H, K, V))
    if o is None:
        o = torch.empty(B, T, H, V, dtype=q.dtype, device=q.device)
    _check(o, "o", q.dtype, (B, T, H, V))
    rc = L.gdn_decode(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                      _ptr(state), _ptr(o), _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_decode")
    return o


# ------------------------------------------------------- gated linear recurrence
_DT = {torch.bfloat16: GDN_BF16, torch.float32: GDN_FP32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


class _Here:
    """The context of a call on the current device and stream: nothing to change."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_here = _Here()


def _scope(first, stream, used):
    """(context, device index, stream handle) of a call whose tensors live on the first one's
    device: allocations and launches go to ``stream`` (None: that device's current stream),
    whatever the current device is; tensors used on another stream than the current one are
    recorded on it."""
    index = first.get_device()
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        if torch.cuda.current_device() == index:
            return _here, index, _raw_stream(index)
        stream = torch.cuda.current_stream(index)
    elif stream.device.index != index:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, first.device))
    elif stream != torch.cuda.current_stream(index):
        for t in used:
            if t is not None and t.is_cuda:
                t.record_stream(stream)
    return torch.cuda.stream(stream), index, stream.cuda_stream


def _like(t):
    """An empty contiguous tensor of this shape and type (the format given costs a microsecond)."""
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _pointer(t, name, index, dtype, shape):
    """Address of a contiguous tensor of this type and shape (None: any) on the call's device;
    None for None."""
    if t is None:
        return None
    if (t.get_device() != index or t.dtype is not dtype or not t.is_contiguous() or
            (shape is not None and t.shape != shape)):
        _check(t, name, dtype, shape)
        raise ValueError("%s is on %s, the call's tensors on cuda:%d" % (name, t.device, index))
    return t.data_ptr()


def _row_stride(t, name, dtype, shape):
    """Elements from one token to the next of a (B, T, ...) tensor whose values of one token
    are adjacent and whose tokens are evenly spaced over all rows (a column slice of a wider
    contiguous tensor is; a transposed or expanded one is not)."""
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.is_contiguous():
        return 0
    width = 1
    for n, s in zip(reversed(shape[2:]), reversed(t.stride()[2:])):
        if n > 1 and s != width:
            raise ValueError("%s: the values of one token must be adjacent" % name)
        width *= n
    B, T = shape[:2]
    s = t.stride(1) if T > 1 else t.stride(0) if B > 1 else width
    if s < width or (B > 1 and T > 1 and t.stride(0) != T * s):
        raise ValueError("%s: tokens must be evenly spaced over all rows, without overlap" % name)
    return s


def _rows(t, name, index):
    """What a descriptor depends on of a tensor of rows, after the check of its device."""
    if t is None:
        return None
    if t.get_device() != index:
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        raise ValueError("%s is on %s, the call's tensors on cuda:%d" % (name, t.device, index))
    return t.dtype, t.shape, t.stride()


class _Plans(dict):
    """Descriptors of earlier calls by what they are made of (types, shapes, strides, options)."""
    limit = 1024

    def keep(self, key, plan):
        if len(self) >= self.limit:
            self.clear()
        self[key] = plan
        return plan


_linrec_plans, _qk_plans = _Plans(), _Plans()


def _linrec_plan(x, g, index, n_seqs, complement, do=None, o=None, dx=None, dg=None):
    """(descriptor, reference to it, bytes of states)."""
    key = (_rows(x, "x", index), _rows(g, "g", index), n_seqs, bool(complement),
           _rows(do, "do", index), _rows(o, "o", index), _rows(dx, "dx", index),
           _rows(dg, "dg", index))
    plan = _linrec_plans.get(key)
    if plan is not None:
        return plan
    if x.dim() != 3:
        raise ValueError("x must have shape (B, T, D), got %s" % (tuple(x.shape),))
    if x.dtype not in _DT:
        raise ValueError("x must be bf16 or fp32")
    if g.dtype not in (x.dtype, torch.float32):
        raise ValueError("g must be %s or torch.float32, got %s" % (x.dtype, g.dtype))
    shape = tuple(x.shape)
    row = lambda t, name, dt: 0 if t is None else _row_stride(t, name, dt, shape)
    desc = GdnLinrecDesc(*shape, n_seqs, row(x, "x", x.dtype), row(g, "g", g.dtype),
                         row(do, "do", x.dtype) if do is not None else row(o, "o", x.dtype),
                         row(dx, "dx", x.dtype), row(dg, "dg", g.dtype), _DT[x.dtype],
                         _DT[g.dtype], GDN_LINREC_COMPLEMENT if complement else 0, 0)
    ref = ctypes.byref(desc)
    return _linrec_plans.keep(key, (desc, ref, int(lib().gdn_linrec_states_size(ref))))


def _offsets(cu_seqlens, cu_seqlens_host, index):
    """(device offsets, their address, the host mirror's address, number of documents)."""
    if cu_seqlens is None and cu_seqlens_host is None:
        return None, None, None, 0
    if (cu_seqlens is None or cu_seqlens_host is None or cu_seqlens.get_device() != index or
            cu_seqlens.dtype is not torch.int32 or cu_seqlens_host.dtype is not torch.int32 or
            not cu_seqlens.is_contiguous() or not cu_seqlens_host.is_contiguous()):
        if cu_seqlens is not None and cu_seqlens.is_cuda and cu_seqlens.get_device() != index:
            raise ValueError("cu_seqlens is on %s, the call's tensors on cuda:%d"
                             % (cu_seqlens.device, index))
        cu_seqlens, cu_seqlens_host = _seqlens(cu_seqlens, cu_seqlens_host,
                                               torch.device("cuda", index))
    else:
        _check_mirror(cu_seqlens_host)
    if cu_seqlens.shape != cu_seqlens_host.shape or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must have one dimension and 2 values or more, and its host "
                         "mirror the same number")
    return (cu_seqlens, cu_seqlens_host), cu_seqlens.data_ptr(), cu_seqlens_host.data_ptr(), \
        cu_seqlens_host.numel() - 1


def gdn_linrec_fwd(x, g, cu_seqlens=None, h0=None, complement=False, output_final_state=True,
                   save_states=False, o=None, hT=None, states=None, cu_seqlens_host=None,
                   stream=None):
    """Gated linear recurrence h_t = exp(g_t) h_{t-1} + w_t x_t per channel, o = h (w = 1, or
    1 - exp(g_t) with ``complement``), through the C ABI.  x, g: (B, T, D), which may be column
    slices of a wider tensor; h0: (N, D) fp32.  Returns (o, hT), or (o, hT, states) with
    ``save_states``: a buffer that spares gdn_linrec_bwd recomputing the states."""
    L = lib()
    scope, index, handle = _scope(x, stream, (x, g, h0, cu_seqlens, o, hT, states))
    with scope:
        _kept, cu, cu_host, n_seqs = _offsets(cu_seqlens, cu_seqlens_host, index)
        _, ref, need = _linrec_plan(x, g, index, n_seqs, complement, o=o)
        N = (n_seqs or x.shape[0], x.shape[2])
        if o is None:
            o = _like(x)
        if hT is None and output_final_state:
            hT = x.new_empty(N, dtype=torch.float32)
        if save_states or states is not None:
            if need == 0:
                raise GdnError(1, "gdn_linrec_states_size")
            if states is None:
                states = x.new_empty(need, dtype=torch.uint8)
            elif states.numel() < need:
                raise GdnError(4, "gdn_linrec_fwd")
        rc = L.gdn_linrec_fwd(ref, x.data_ptr(), g.data_ptr(), cu, cu_host,
                              _pointer(h0, "h0", index, torch.float32, N), o.data_ptr(),
                              _pointer(hT, "hT", index, torch.float32, N),
                              _pointer(states, "states", index, torch.uint8, None), handle)
    if rc:
        raise GdnError(rc, "gdn_linrec_fwd")
    return (o, hT, states) if states is not None else (o, hT)


def gdn_linrec_bwd(x, g, do, cu_seqlens=None, h0=None, dhT=None, complement=False, states=None,
                   grads=None, workspace=None, cu_seqlens_host=None, stream=None, want_dh0=True):
    """Gradients (dx, dg, dh0) of gdn_linrec_fwd for upstream ``do`` and ``dhT``, through the C
    ABI.  ``states``: what gdn_linrec_fwd returned for the same x, g, cu_seqlens and h0; without
    it the states are recomputed into the workspace."""
    L = lib()
    dx, dg, dh0 = grads if grads is not None else (None, None, None)
    scope, index, handle = _scope(x, stream, (x, g, do, h0, dhT, cu_seqlens, dx, dg, dh0, states,
                                              workspace))
    with scope:
        _kept, cu, cu_host, n_seqs = _offsets(cu_seqlens, cu_seqlens_host, index)
        _, ref, need = _linrec_plan(x, g, index, n_seqs, complement, do=do, dx=dx, dg=dg)
        N = (n_seqs or x.shape[0], x.shape[2])
        if grads is None:
            dx = _like(x)
            dg = _like(g)
            dh0 = x.new_empty(N, dtype=torch.float32) if want_dh0 else None
        if need == 0:
            raise GdnError(1, "gdn_linrec_states_size")
        if states is not None:
            if states.numel() < need:
                raise GdnError(4, "gdn_linrec_bwd")
        elif workspace is None:
            workspace = x.new_empty(need, dtype=torch.uint8)
        rc = L.gdn_linrec_bwd(ref, x.data_ptr(), g.data_ptr(), cu, cu_host,
                              _pointer(h0, "h0", index, torch.float32, N), do.data_ptr(),
                              _pointer(dhT, "dhT", index, torch.float32, N), _ptr(dx), _ptr(dg),
                              _pointer(dh0, "dh0", index, torch.float32, N),
                              _pointer(states, "states", index, torch.uint8, None),
                              _pointer(workspace, "workspace", index, torch.uint8, None),
                              0 if workspace is None else workspace.numel(), handle)
    if rc:
        raise GdnError(rc, "gdn_linrec_bwd")
    return dx, dg, dh0


def linrec_status(stream=None, device=None) -> int:
    """Status code (0: ok) of the gdn_linrec_fwd and gdn_linrec_bwd calls on the stream, and of
    captured ones replayed on its device, after waiting for the stream.  Each timeout is told once to
    every host thread that asks.  Without a stream the current stream of ``device`` is taken (a
    device, its index or a tensor on it; None: the current one)."""
    if stream is None:
        stream = torch.cuda.current_stream(device.device if isinstance(device, torch.Tensor) else device)
    with torch.cuda.device(stream.device):
        return int(lib().gdn_linrec_status(ctypes.c_void_p(stream.cuda_stream)))


def gdn_linrec_decode(x, g, state, complement=False, o=None, stream=None):
    """One-token form through the C ABI: advances ``state`` ((B, D) fp32, in place) through the
    T tokens of x and g ((B, T, D)) and returns o."""
    scope, index, handle = _scope(x, stream, (x, g, state, o))
    with scope:
        _, ref, _ = _linrec_plan(x, g, index, 0, complement, o=o)
        if o is None:
            o = _like(x)
        rc = lib().gdn_linrec_decode(ref, x.data_ptr(), g.data_ptr(),
                                     _pointer(state, "state", index, torch.float32,
                                              (x.shape[0], x.shape[2])), o.data_ptr(), handle)
    if rc:
        raise GdnError(rc, "gdn_linrec_decode")
    return o


# ------------------------------------------- q/k normalisation with the position rotation
_NORMS = {None: (GDN_NORM_NONE, 0.0), "l2": (GDN_NORM_L2, 0.0), "rms": (GDN_NORM_RMS, 1e-6)}


def _qk_plan(q, k, inv_freq, norm, eps, interleaved, index, outs, raws):
    """(descriptor, reference to it, bytes of the backward's workspace).  outs: the rotated q and
    k or their gradients, raws: the gradients of the raw q and k (None where not given)."""
    turned = None if inv_freq is None else inv_freq.shape
    key = (_rows(q, "q", index), _rows(k, "k", index), turned, norm, eps, bool(interleaved),
           _rows(outs[0], "qo", index), _rows(outs[1], "ko", index), _rows(raws[0], "dq", index),
           _rows(raws[1], "dk", index))
    plan = _qk_plans.get(key)
    if plan is not None:
        return plan
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must have shape (B, T, heads, d)")
    if q.dtype not in _DT:
        raise ValueError("q must be bf16 or fp32")
    if norm not in _NORMS:
        raise ValueError("norm must be None, 'l2' or 'rms', got %r" % (norm,))
    if inv_freq is not None and inv_freq.dim() != 1:
        raise ValueError("inv_freq must have one dimension")
    B, T, Hq, d = q.shape
    Hk = k.shape[2]
    shapes = ((B, T, Hq, d), (B, T, Hk, d))
    row = lambda t, name, i: 0 if t is None else _row_stride(t, name, q.dtype, shapes[i])
    code, default = _NORMS[norm]
    desc = GdnQkDesc(B, T, Hq, Hk, d, 2 * turned.numel() if turned else 0, row(q, "q", 0), row(k, "k", 1),
                     row(outs[0], "qo", 0), row(outs[1], "ko", 1), row(raws[0], "dq", 0),
                     row(raws[1], "dk", 1), _DT[q.dtype], code,
                     GDN_QK_INTERLEAVED if interleaved else 0, default if eps is None else eps)
    ref = ctypes.byref(desc)
    return _qk_plans.keep(key, (desc, ref, int(lib().gdn_qk_norm_rope_bwd_workspace_size(ref))))


def _qk_inputs(q, positions, inv_freq, q_weight, k_weight, index):
    """Addresses of the inputs beside the rows."""
    d = q.shape[3:]
    return (_pointer(positions, "positions", index, torch.int32, q.shape[:2]),
            _pointer(inv_freq, "inv_freq", index, torch.float32, None),
            _pointer(q_weight, "q_weight", index, torch.float32, d),
            _pointer(k_weight, "k_weight", index, torch.float32, d))


def gdn_qk_norm_rope_fwd(q, k, inv_freq=None, positions=None, norm="rms", q_weight=None,
                         k_weight=None, eps=None, interleaved=False, qo=None, ko=None,
                         stream=None):
    """Rows of q (B, T, Hq, d) and k (B, T, Hk, d) normalised (``norm``: "rms", "l2" or None),
    multiplied by the weights (d,) fp32, and turned by the angles positions x inv_freq
    (positions: (B, T) int32, or None to count along each row; inv_freq: (rot/2,) fp32, or None
    for no rotation), through the C ABI.  q and k may be column slices of one projection.  eps
    defaults to 1e-6 for "rms" and 0 for "l2".  Returns (qo, ko)."""
    scope, index, handle = _scope(q, stream, (q, k, inv_freq, positions, q_weight, k_weight, qo, ko))
    with scope:
        _, ref, _ = _qk_plan(q, k, inv_freq, norm, eps, interleaved, index, (qo, ko), (None, None))
        if qo is None:
            qo = _like(q)
        if ko is None:
            ko = _like(k)
        rc = lib().gdn_qk_norm_rope_fwd(ref, q.data_ptr(), k.data_ptr(),
                                        *_qk_inputs(q, positions, inv_freq, q_weight, k_weight, index),
                                        qo.data_ptr(), ko.data_ptr(), handle)
    if rc:
        raise GdnError(rc, "gdn_qk_norm_rope_fwd")
    return qo, ko


def gdn_qk_norm_rope_bwd(q, k, dqo, dko, inv_freq=None, positions=None, norm="rms",
                         q_weight=None, k_weight=None, eps=None, interleaved=False, grads=None,
                         workspace=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of gdn_qk_norm_rope_fwd for upstream dqo, dko,
    through the C ABI; a weight that is None has no gradient (None)."""
    dq, dk, dqw, dkw = grads if grads is not None else (None, None, None, None)
    scope, index, handle = _scope(q, stream, (q, k, dqo, dko, inv_freq, positions, q_weight,
                                              k_weight, dq, dk, dqw, dkw, workspace))
    with scope:
        _, ref, need = _qk_plan(q, k, inv_freq, norm, eps, interleaved, index, (dqo, dko), (dq, dk))
        d = q.shape[3:]
        if grads is None:
            dq = _like(q)
            dk = _like(k)
            dqw = None if q_weight is None else q.new_empty(d, dtype=torch.float32)
            dkw = None if k_weight is None else q.new_empty(d, dtype=torch.float32)
        if workspace is None and need and (dqw is not None or dkw is not None):
            workspace = q.new_empty(need, dtype=torch.uint8)
        rc = lib().gdn_qk_norm_rope_bwd(ref, q.data_ptr(), k.data_ptr(),
                                        *_qk_inputs(q, positions, inv_freq, q_weight, k_weight, index),
                                        dqo.data_ptr(), dko.data_ptr(), _ptr(dq), _ptr(dk),
                                        _pointer(dqw, "dq_weight", index, torch.float32, d),
                                        _pointer(dkw, "dk_weight", index, torch.float32, d),
                                        _pointer(workspace, "workspace", index, torch.uint8, None),
                                        0 if workspace is None else workspace.numel(), handle)
    if rc:
        raise GdnError(rc, "gdn_qk_norm_rope_bwd")
    return dq, dk, dqw, dkw


def device_status(workspace, stream=None) -> int:
    return int(lib().gdn_device_status(_ptr(workspace), _stream(stream)))


def set_wait_limit(polls: int) -> None:
    """Testing hook: device-side waits of later calls from this thread give up
    after ``polls`` polls (0 restores the built-in limit)."""
    lib().gdn_set_wait_limit(int(polls))


def set_test_hook(hook: int) -> None:
    """Testing hook: plant GDN_TEST_STALL_COPY or GDN_TEST_FAIL_LAUNCH in later
    calls from this thread (0 removes it)."""
    lib().gdn_set_test_hook(int(hook))


class GdnTrace(ctypes.Structure):
    _fields_ = [("capacity", ctypes.c_int32), ("count", ctypes.c_int32),
                ("dropped", ctypes.c_int32), ("pad", ctypes.c_int32),
                ("events", ctypes.POINTER(ctypes.c_void_p)),
                ("kernel_ids", ctypes.POINTER(ctypes.c_int32))]


class LaunchTrace:
    """Records a pair of CUDA events around every library kernel launch made
    from this thread while active (``with LaunchTrace(n) as t: ...``).
    ``per_kernel()`` returns {name: (launches, total_ms)} after a sync."""

    def __init__(self, capacity: int):
        self.capacity = int(capacity)
        self.torch_events = [torch.cuda.Event(enable_timing=True)
                             for _ in range(2 * self.capacity)]
        for e in self.torch_events:  # torch creates the CUDA event on first record
            e.record()
        torch.cuda.current_stream().synchronize()
        self._ev = (ctypes.c_void_p * (2 * self.capacity))(
            *[e.cuda_event for e in self.torch_events])
        self._ids = (ctypes.c_int32 * self.capacity)()
        self.trace = GdnTrace(self.capacity, 0, 0, 0, self._ev, self._ids)

    def __enter__(self):
        lib().gdn_trace_install(ctypes.byref(self.trace))
        return self

    def __exit__(self, *exc):
        lib().gdn_trace_install(None)
        return False

    def reset(self):
        self.trace.count = 0
        self.trace.dropped = 0

    @property
    def count(self):
        return int(self.trace.count)

    def per_kernel(self):
        out = {}
        for i in range(self.trace.count):
            name = lib().gdn_kernel_name(self._ids[i]).decode()
            ms = self.torch_events[2 * i].elapsed_time(self.torch_events[2 * i + 1])
            n, t = out.get(name, (0, 0.0))
            out[name] = (n + 1, t + ms)
        return out
