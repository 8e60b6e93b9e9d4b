"""ctypes binding of libw4a4 (include/w4a4.h, tq.h, decode.h) for torch tensors.

Argument marshalling only: every step of the computation runs in the CUDA
library.  Importing this module raises ImportError when libw4a4.so has not
been built (``python -m w4a4_post_quantized_b200.build``); there is no
fallback.

The functions carry the C names.  Tensors must be contiguous CUDA tensors;
bf16 data is passed as torch.bfloat16, packed int4 codes as torch.uint8.
Calls are asynchronous on the given stream (default: torch's current stream).
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a4.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m w4a4_post_quantized_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)

W4A4_OK, W4A4_ERR_ARG, W4A4_ERR_SHAPE, W4A4_ERR_ALIGN, W4A4_ERR_UNSUPPORTED, W4A4_ERR_CUDA, \
    W4A4_ERR_TIMEOUT = range(7)
W4A4_DEV_TIMEOUT = 0x1
W4A4_DEV_RANGE = 0x2
W4A4_FLAG_GELU = 0x1
W4A4_FLAG_PLAIN = 0x2
W4A4_FLAG_INT8 = 0x4
W4A4_FLAG_UNPACKED = 0x8
W4A4_FLAG_GELU_OUT = 0x10
W4A4_FLAG_X_DEVICE = 0x20
W4A4_FLAG_FWHT = 0x100
W4A4_FLAG_FP16 = 0x200
W4A4_FLAG_ROPE_PAIRS = 0x400
W4A4_FLAG_Y_DEVICE = 0x40
W4A4_DEBUG_STALL = 0x80000000

_vp, _i32, _i64, _u32, _f32, _sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                    ctypes.c_float, ctypes.c_size_t)


class W4A4WeightsT(ctypes.Structure):
    _fields_ = [("N", _i32), ("K", _i32), ("qw", _vp), ("scale_ch", _vp), ("bias", _vp),
                ("smooth", _vp), ("inv_smooth", _vp), ("qw8", _vp), ("colsum", _vp), ("flags", _u32)]


class GroupWeightsT(ctypes.Structure):
    _fields_ = [("N", _i32), ("K", _i32), ("group", _i32), ("flags", _u32), ("data", _vp)]


class KVCacheT(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("n_pages", _i64), ("page_size", _i32), ("n_heads", _i32),
                ("head_dim", _i32), ("flags", _u32), ("stride_page", _i64), ("stride_token", _i64),
                ("stride_head", _i64)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_workspace_bytes = _sig("w4a4_workspace_bytes", _sz, [_i64, _i32])
_workspace_bytes_min = _sig("w4a4_workspace_bytes_min", _sz, [_i64, _i32, _u32])
_prepare = _sig("w4a4_prepare_weights", ctypes.c_int,
                [_vp, _vp, _i32, _i32, _vp, _i64, _f32, _u32, ctypes.POINTER(W4A4WeightsT), _vp])
_quantize = _sig("w4a4_quantize_act", ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp, _u32, _vp])
_linear = _sig("w4a4_linear", ctypes.c_int, [_vp, _vp, _i64, ctypes.POINTER(W4A4WeightsT), _vp, _vp])
_linear_ex = _sig("w4a4_linear_ex", ctypes.c_int,
                  [_vp, _vp, _i64, ctypes.POINTER(W4A4WeightsT), _vp, _u32, _vp])
_fused = _sig("w4a4_linear_fused", ctypes.c_int,
              [_vp, _i64, ctypes.POINTER(W4A4WeightsT), _vp, _vp, _sz, _u32, _vp])
_fused_noalloc = _sig("w4a4_linear_fused_noalloc", ctypes.c_int,
                      [_vp, _i64, ctypes.POINTER(W4A4WeightsT), _vp, _u32, _vp])
_gemm_s32 = _sig("w4a4_gemm_s32", ctypes.c_int, [_vp, _i64, ctypes.POINTER(W4A4WeightsT), _vp, _vp])
_gemm_s32_ex = _sig("w4a4_gemm_s32_ex", ctypes.c_int,
                    [_vp, _i64, ctypes.POINTER(W4A4WeightsT), _vp, _u32, _vp])
_weights_bytes = _sig("w4a4_weights_bytes", _sz, [_i32, _i32, _u32])
_weights_bind = _sig("w4a4_weights_bind", ctypes.c_int,
                     [_vp, _sz, _i32, _i32, _u32, ctypes.POINTER(W4A4WeightsT)])
_pipe_create = _sig("w4a4_host_pipe_create", ctypes.c_int, [ctypes.POINTER(_vp)])
_pipe_destroy = _sig("w4a4_host_pipe_destroy", ctypes.c_int, [_vp])
_host_ws_bytes = _sig("w4a4_host_workspace_bytes", _sz, [_i64, _i32, _i32])
_fused_host = _sig("w4a4_linear_fused_host", ctypes.c_int,
                   [_vp, _i64, ctypes.POINTER(W4A4WeightsT), _vp, _i64, _vp, _sz, _vp, _u32, _vp])
_expand = _sig("w4a4_expand_weights", ctypes.c_int, [ctypes.POINTER(W4A4WeightsT), _vp])
_get_status = _sig("w4a4_get_device_status", ctypes.c_int, [_vp, ctypes.POINTER(_u32)])
_clear_status = _sig("w4a4_clear_device_status", ctypes.c_int, [_vp])
_tq_codebook = _sig("tq_codebook", ctypes.c_int, [_i32, _i32, _vp, _vp])
_tq_encode = _sig("tq_encode", ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp])
_tq_decode = _sig("tq_decode", ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp, _vp, _vp])
_tq_rotation_qr = _sig("tq_rotation_qr", ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp])
_tq_encode_dense = _sig("tq_encode_dense", ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp])
_tq_decode_dense = _sig("tq_decode_dense", ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp])
_group_bytes = _sig("w4a4_group_weights_bytes", _sz, [_i32, _i32, _i32])
_group_bind = _sig("w4a4_group_bind", ctypes.c_int,
                   [_vp, _sz, _i32, _i32, _i32, _u32, ctypes.POINTER(GroupWeightsT)])
_group_quantize = _sig("w4a4_group_quantize", ctypes.c_int, [_vp, ctypes.POINTER(GroupWeightsT), _vp])
_group_pack = _sig("w4a4_group_pack", ctypes.c_int, [_vp, _vp, ctypes.POINTER(GroupWeightsT), _vp])
_group_dequantize = _sig("w4a4_group_dequantize", ctypes.c_int, [ctypes.POINTER(GroupWeightsT), _vp, _vp])
_group_gemv = _sig("w4a4_group_gemv", ctypes.c_int,
                   [_vp, _i64, ctypes.POINTER(GroupWeightsT), _vp, _vp, _u32, _vp])
_rope_table = _sig("w4a4_rope_table", ctypes.c_int, [_i32, _i32, ctypes.c_double, _vp])
_kv_append = _sig("w4a4_kv_append", ctypes.c_int, [ctypes.POINTER(KVCacheT), ctypes.c_char_p, _vp])
_kv_attend_ws = _sig("w4a4_kv_attend_workspace_bytes", _sz, [_i32, _i32, _i32, _i32])
_kv_attend = _sig("w4a4_kv_attend", ctypes.c_int, [ctypes.POINTER(KVCacheT), ctypes.c_char_p, _vp])
# w4a4_kv_append_t and w4a4_kv_attend_t, field by field (packing them costs a third of what
# ctypes takes to convert as many arguments)
_append_t = struct.Struct("PPPPqqqqPPPPPiiiiiI")
_attend_t = struct.Struct("PPPPPPqNiiiif4x")
_status_string = _sig("w4a4_status_string", ctypes.c_char_p, [ctypes.c_int])
_version = _sig("w4a4_version", ctypes.c_char_p, [])


class W4A4Error(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {_status_string(code).decode()} (status {code})")


def _check(rc: int, where: str) -> None:
    if rc != W4A4_OK:
        raise W4A4Error(rc, where)


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    if not t.is_contiguous():
        raise ValueError("tensors passed to libw4a4 must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def version() -> str:
    return _version().decode()


def w4a4_workspace_bytes(M: int, K: int) -> int:
    return int(_workspace_bytes(M, K))


def w4a4_workspace_bytes_min(M: int, K: int, flags: int) -> int:
    return int(_workspace_bytes_min(M, K, flags))


def w4a4_weights_bytes(N: int, K: int, flags: int = 0) -> int:
    return int(_weights_bytes(N, K, flags))


class PreparedWeights:
    """Device arrays of one prepared layer and the C struct that points at
    them: one torch-owned allocation of w4a4_weights_bytes(N, K, layout) bytes,
    laid out by w4a4_weights_bind; the attributes (qw, scale_ch, ...) are typed
    views into it.  expanded=True also holds the widened int8 copy of the codes
    (qw8, N*K bytes) and the per-row code sums the fast GEMM path uses;
    expanded=False keeps only the packed int4 codes.  int8=True (the W8A8
    setting) holds qw8 with the 8-bit codes and no packed codes."""

    def __init__(self, N: int, K: int, device="cuda", expanded: bool = True, int8: bool = False):
        self.N, self.K = N, K
        self.device = torch.device(device)
        layout = W4A4_FLAG_INT8 if int8 else (W4A4_FLAG_UNPACKED if expanded else 0)
        nbytes = w4a4_weights_bytes(N, K, layout)
        if nbytes == 0:
            raise W4A4Error(W4A4_ERR_SHAPE, "w4a4_weights_bytes")
        self.storage = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.struct = W4A4WeightsT()
        _check(_weights_bind(_ptr(self.storage), nbytes, N, K, layout, ctypes.byref(self.struct)),
               "w4a4_weights_bind")
        base = self.storage.data_ptr()

        def view(addr, count, dtype, shape):
            if not addr:
                return None
            off = addr - base
            nb = count * torch.empty((), dtype=dtype).element_size()
            return self.storage[off:off + nb].view(dtype).view(shape)
        st = self.struct
        self.qw = view(st.qw, N * K // 2, torch.uint8, (N, K // 2))
        self.scale_ch = view(st.scale_ch, N, torch.float32, (N,))
        self.bias = view(st.bias, N, torch.float32, (N,))
        self.smooth = view(st.smooth, K, torch.float32, (K,))
        self.inv_smooth = view(st.inv_smooth, K, torch.float32, (K,))
        self.qw8 = view(st.qw8, N * K, torch.int8, (N, K))
        self.colsum = view(st.colsum, N, torch.int32, (N,))

    @property
    def flags(self) -> int:
        return int(self.struct.flags)


def w4a4_prepare_weights(W: torch.Tensor, bias, X_calib, alpha: float = 0.5, flags: int = 0,
                         out: PreparedWeights | None = None, expanded: bool = True,
                         stream=None) -> PreparedWeights:
    N, K = W.shape
    out = out or PreparedWeights(N, K, W.device, expanded=expanded, int8=bool(flags & W4A4_FLAG_INT8))
    mc = 0 if X_calib is None else X_calib.shape[0]
    _check(_prepare(_ptr(W), _ptr(bias), N, K, _ptr(X_calib), mc, alpha, flags,
                    ctypes.byref(out.struct), _stream(stream)), "w4a4_prepare_weights")
    return out


def w4a4_quantize_act(X: torch.Tensor, inv_smooth, flags: int = 0, qx=None, scale_tok=None,
                      stream=None):
    M, K = X.shape
    width = K if flags & (W4A4_FLAG_INT8 | W4A4_FLAG_UNPACKED) else K // 2
    qx = qx if qx is not None else torch.empty((M, width), dtype=torch.uint8, device=X.device)
    scale_tok = scale_tok if scale_tok is not None else torch.empty(M, dtype=torch.float32, device=X.device)
    _check(_quantize(_ptr(X), M, K, _ptr(inv_smooth), _ptr(qx), _ptr(scale_tok), flags,
                     _stream(stream)), "w4a4_quantize_act")
    return qx, scale_tok


def w4a4_linear(qx: torch.Tensor, scale_tok: torch.Tensor, w: PreparedWeights, Y=None, stream=None):
    M = qx.shape[0]
    Y = Y if Y is not None else torch.empty((M, w.N), dtype=torch.bfloat16, device=qx.device)
    _check(_linear(_ptr(qx), _ptr(scale_tok), M, ctypes.byref(w.struct), _ptr(Y), _stream(stream)),
           "w4a4_linear")
    return Y


def w4a4_linear_ex(qx: torch.Tensor, scale_tok: torch.Tensor, w: PreparedWeights, flags: int = 0, Y=None,
                   stream=None):
    M = qx.shape[0]
    Y = Y if Y is not None else torch.empty((M, w.N), dtype=torch.bfloat16, device=qx.device)
    _check(_linear_ex(_ptr(qx), _ptr(scale_tok), M, ctypes.byref(w.struct), _ptr(Y), flags,
                      _stream(stream)), "w4a4_linear_ex")
    return Y


def w4a4_linear_fused(X: torch.Tensor, w: PreparedWeights, Y=None, workspace=None, flags: int = 0,
                      stream=None):
    M = X.shape[0]
    Y = Y if Y is not None else torch.empty((M, w.N), dtype=torch.bfloat16, device=X.device)
    need = w4a4_workspace_bytes(M, w.K)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=X.device)
    _check(_fused(_ptr(X), M, ctypes.byref(w.struct), _ptr(Y), _ptr(workspace),
                  workspace.numel() * workspace.element_size(), flags, _stream(stream)),
           "w4a4_linear_fused")
    return Y


W4A4_NOALLOC_SCRATCH_BYTES = 8 << 20


def w4a4_linear_fused_noalloc(X: torch.Tensor, w: PreparedWeights, Y=None, flags: int = 0,
                              stream=None):
    """w4a4_linear_fused without a workspace argument, for callers that may
    not allocate device memory where they run: the library's built-in scratch
    array (W4A4_NOALLOC_SCRATCH_BYTES per GPU) holds the intermediate codes.
    Calls that overlap on the GPU share that array and must not be issued."""
    M = X.shape[0]
    if Y is None:  # allocating the output here is a convenience of this binding only
        Y = torch.empty((M, w.N), dtype=torch.bfloat16, device=X.device)
    _check(_fused_noalloc(_ptr(X), M, ctypes.byref(w.struct), _ptr(Y), flags, _stream(stream)),
           "w4a4_linear_fused_noalloc")
    return Y


class HostPipe:
    """The copy streams and events of w4a4_linear_fused_host (created on the
    current device by the library; freed with the object)."""

    def __init__(self):
        h = _vp()
        _check(_pipe_create(ctypes.byref(h)), "w4a4_host_pipe_create")
        self.handle = h

    def close(self):
        if self.handle:
            _check(_pipe_destroy(self.handle), "w4a4_host_pipe_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def w4a4_host_workspace_bytes(chunk_rows: int, K: int, N: int) -> int:
    return _host_ws_bytes(chunk_rows, K, N)


def w4a4_linear_fused_host(X_host: torch.Tensor, w: PreparedWeights, Y_host=None, chunk_rows: int = 2816,
                           workspace=None, pipe: HostPipe | None = None, flags: int = 0, stream=None):
    """Y_host = w4a4_linear_fused(X_host) with X_host / Y_host in (pinned) host
    memory; row chunks of chunk_rows are copied in, computed and copied out
    concurrently.  Returns Y_host (enqueued: synchronize `stream` before reading)."""
    M = X_host.shape[0]
    if Y_host is None:  # a convenience of this binding only
        Y_host = (torch.empty((M, w.N), dtype=torch.bfloat16, device=w.device)
                  if flags & W4A4_FLAG_Y_DEVICE else
                  torch.empty((M, w.N), dtype=torch.bfloat16, pin_memory=True))
    if workspace is None:
        workspace = torch.empty(w4a4_host_workspace_bytes(chunk_rows, w.K, w.N), dtype=torch.uint8,
                                device=w.device)
    if pipe is None:
        raise ValueError("w4a4_linear_fused_host needs a HostPipe")
    _check(_fused_host(_ptr(X_host), M, ctypes.byref(w.struct), _ptr(Y_host), chunk_rows, _ptr(workspace),
                       workspace.numel(), pipe.handle, flags, _stream(stream)), "w4a4_linear_fused_host")
    return Y_host


def w4a4_expand_weights(w: PreparedWeights, stream=None) -> PreparedWeights:
    _check(_expand(ctypes.byref(w.struct), _stream(stream)), "w4a4_expand_weights")
    return w


def w4a4_gemm_s32(qx: torch.Tensor, w: PreparedWeights, acc=None, stream=None):
    M = qx.shape[0]
    acc = acc if acc is not None else torch.empty((M, w.N), dtype=torch.int32, device=qx.device)
    _check(_gemm_s32(_ptr(qx), M, ctypes.byref(w.struct), _ptr(acc), _stream(stream)), "w4a4_gemm_s32")
    return acc


def w4a4_gemm_s32_ex(qx: torch.Tensor, w: PreparedWeights, flags: int = 0, acc=None, stream=None):
    M = qx.shape[0]
    acc = acc if acc is not None else torch.empty((M, w.N), dtype=torch.int32, device=qx.device)
    _check(_gemm_s32_ex(_ptr(qx), M, ctypes.byref(w.struct), _ptr(acc), flags, _stream(stream)),
           "w4a4_gemm_s32_ex")
    return acc


def w4a4_get_device_status(stream=None) -> int:
    v = _u32(0)
    rc = _get_status(_stream(stream), ctypes.byref(v))
    if not (rc in (W4A4_OK, W4A4_ERR_TIMEOUT) or (rc == W4A4_ERR_ARG and v.value)):
        _check(rc, "w4a4_get_device_status")
    return int(v.value)


def w4a4_clear_device_status(stream=None) -> None:
    _check(_clear_status(_stream(stream)), "w4a4_clear_device_status")


# ------------------------------------------------- 3DTurboQuant codec (include/tq.h)
def tq_codebook(d: int = 1024, b: int = 4):
    """Host Lloyd-Max codebook: (centroids [2^b], boundaries [2^b - 1]) as fp32 numpy arrays."""
    import numpy as np
    c = np.empty(1 << b, np.float32)
    t = np.empty((1 << b) - 1, np.float32)
    _check(_tq_codebook(d, b, c.ctypes.data_as(_vp), t.ctypes.data_as(_vp)), "tq_codebook")
    return c, t


def tq_encode(X: torch.Tensor, signs: torch.Tensor, boundaries: torch.Tensor, codes=None, norms=None,
              stream=None):
    """X [n, d] fp32 -> (codes uint8 [n, d/2], norms fp32 [n])."""
    n, d = X.shape
    codes = codes if codes is not None else torch.empty((n, d // 2), dtype=torch.uint8, device=X.device)
    norms = norms if norms is not None else torch.empty(n, dtype=torch.float32, device=X.device)
    _check(_tq_encode(_ptr(X), n, d, _ptr(signs), _ptr(boundaries), _ptr(codes), _ptr(norms),
                      _stream(stream)), "tq_encode")
    return codes, norms


def tq_decode(codes: torch.Tensor, norms: torch.Tensor, signs: torch.Tensor, centroids: torch.Tensor,
              Y=None, stream=None):
    """(codes [n, d/2], norms [n]) -> Y [n, d] fp32."""
    n, d = codes.shape[0], codes.shape[1] * 2
    Y = Y if Y is not None else torch.empty((n, d), dtype=torch.float32, device=codes.device)
    _check(_tq_decode(_ptr(codes), _ptr(norms), n, d, _ptr(signs), _ptr(centroids), _ptr(Y),
                      _stream(stream)), "tq_decode")
    return Y


# ---------------------------------- the page's dense rotation (QR of a Gaussian)
def tq_rotation_qr(G):
    """Host: Pi = the sign-fixed Q factor of the d x d Gaussian matrix G (numpy
    float64), as tf32 hi / lo terms of Pi and of Pi^T: returns
    (pi_hi, pi_lo, pit_hi, pit_lo), numpy float32 [d, d] each."""
    import numpy as np
    G = np.ascontiguousarray(G, dtype=np.float64)
    d = G.shape[0]
    out = [np.empty((d, d), np.float32) for _ in range(4)]
    _check(_tq_rotation_qr(G.ctypes.data_as(_vp), d, *[o.ctypes.data_as(_vp) for o in out]),
           "tq_rotation_qr")
    return tuple(out)


def tq_encode_dense(X: torch.Tensor, pi_hi: torch.Tensor, pi_lo: torch.Tensor, boundaries: torch.Tensor,
                    codes=None, norms=None, stream=None):
    """X [n, d] fp32 -> (codes uint8 [n, d/2], norms fp32 [n]) with the dense Pi."""
    n, d = X.shape
    codes = codes if codes is not None else torch.empty((n, d // 2), dtype=torch.uint8, device=X.device)
    norms = norms if norms is not None else torch.empty(n, dtype=torch.float32, device=X.device)
    _check(_tq_encode_dense(_ptr(X), n, d, _ptr(pi_hi), _ptr(pi_lo), _ptr(boundaries), _ptr(codes),
                            _ptr(norms), _stream(stream)), "tq_encode_dense")
    return codes, norms


def tq_decode_dense(codes: torch.Tensor, norms: torch.Tensor, pit_hi: torch.Tensor, pit_lo: torch.Tensor,
                    centroids: torch.Tensor, Y=None, stream=None):
    """(codes [n, d/2], norms [n]) -> Y [n, d] fp32 with the dense Pi."""
    n, d = codes.shape[0], codes.shape[1] * 2
    Y = Y if Y is not None else torch.empty((n, d), dtype=torch.float32, device=codes.device)
    _check(_tq_decode_dense(_ptr(codes), _ptr(norms), n, d, _ptr(pit_hi), _ptr(pit_lo), _ptr(centroids),
                            _ptr(Y), _stream(stream)), "tq_decode_dense")
    return Y


# ------------------------------------------- single-token operators (include/decode.h)
def _here(dev: torch.device, stream):
    """The raw current stream when the call can run as things stand: on the
    current device, on torch's current stream.  Otherwise None, and the call is made
    again inside _elsewhere.  (torch.cuda.current_stream() builds an object, 3 us of a
    call whose kernel takes 2; the raw handle and the raw device number cost 0.1 each.)"""
    if stream is None and dev.index == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(dev.index)
    return None


def _elsewhere(dev: torch.device, stream):
    """A context in which `dev` is current and `stream` (where given) torch's
    stream, so that what a call allocates belongs to the stream it is used on."""
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
    return torch.cuda.stream(stream)


def _need(t: torch.Tensor, name: str, dtype, dev, shape) -> int:
    """The address of a contiguous tensor of that type, device and shape."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dtype, dev, shape) -> tuple[int, int]:
    """Address and row stride of a tensor [T, heads, head_dim] whose rows are dense."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev:
        raise ValueError(f"{name}: need {dtype} of shape {tuple(shape)} on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    T, H, D = shape
    row, head, one = t.stride()
    if one != 1 or (head != D and H > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous, strides are {t.stride()}")
    return t.data_ptr(), row if T > 1 else H * D


def _half_flag(dtype) -> int:
    if dtype == torch.bfloat16:
        return 0
    if dtype == torch.float16:
        return W4A4_FLAG_FP16
    raise ValueError(f"need torch.bfloat16 or torch.float16, got {dtype}")


def _cuda_device(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def w4a4_group_weights_bytes(N: int, K: int, group: int) -> int:
    return int(_group_bytes(N, K, group))


class GroupWeights:
    """4-bit weights [N, K] with one step per `group` inputs: one torch-owned
    allocation of w4a4_group_weights_bytes(N, K, group) bytes, laid out by
    w4a4_group_bind, to be filled by w4a4_group_quantize or w4a4_group_pack.
    dtype: of the steps and of the tokens they multiply."""

    def __init__(self, N: int, K: int, group: int = 128, dtype=torch.bfloat16, device="cuda"):
        self.N, self.K, self.group, self.dtype = N, K, group, dtype
        flags = _half_flag(dtype)
        nbytes = w4a4_group_weights_bytes(N, K, group)
        if nbytes == 0:
            raise W4A4Error(W4A4_ERR_UNSUPPORTED if group not in (32, 64, 128) else W4A4_ERR_SHAPE,
                            "w4a4_group_weights_bytes")
        self.storage = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.device = self.storage.device
        self.struct = GroupWeightsT()
        self.ref = ctypes.byref(self.struct)
        _check(_group_bind(_ptr(self.storage), nbytes, N, K, group, flags, self.ref), "w4a4_group_bind")


def w4a4_group_quantize(W: torch.Tensor, group: int = 128, out: GroupWeights | None = None,
                        stream=None) -> GroupWeights:
    """W [N, K] bf16 or fp16 -> 4-bit codes with one step per `group` inputs."""
    dev = _cuda_device(W, "W")
    st = _here(dev, stream)
    if st is None:
        with _elsewhere(dev, stream):
            return w4a4_group_quantize(W, group, out)
    if out is None:
        out = GroupWeights(W.shape[0], W.shape[1], group, W.dtype, dev)
    if out.group != group:
        raise ValueError(f"out has groups of {out.group}, asked for {group}")
    _check(_group_quantize(_need(W, "W", out.dtype, out.device, (out.N, out.K)), out.ref, st),
           "w4a4_group_quantize")
    return out


def w4a4_group_pack(codes: torch.Tensor, scales: torch.Tensor, out: GroupWeights | None = None,
                    stream=None) -> GroupWeights:
    """codes [N, K/2] uint8 (element 2i in the low nibble) and scales [N,
    K/group] made elsewhere -> GroupWeights."""
    dev = _cuda_device(codes, "codes")
    st = _here(dev, stream)
    if st is None:
        with _elsewhere(dev, stream):
            return w4a4_group_pack(codes, scales, out)
    if out is None:
        N, K = codes.shape[0], 2 * codes.shape[1]
        if scales.dim() != 2 or scales.shape[1] == 0 or K % scales.shape[1]:
            raise ValueError(f"scales {tuple(scales.shape)} do not divide {K} inputs into groups")
        out = GroupWeights(N, K, K // scales.shape[1], scales.dtype, dev)
    c = _need(codes, "codes", torch.uint8, out.device, (out.N, out.K // 2))
    s = _need(scales, "scales", out.dtype, out.device, (out.N, out.K // out.group))
    _check(_group_pack(c, s, out.ref, st), "w4a4_group_pack")
    return out


def w4a4_group_dequantize(w: GroupWeights, W=None, stream=None) -> torch.Tensor:
    """The weights [N, K] that the codes and steps stand for."""
    st = _here(w.device, stream)
    if st is None:
        with _elsewhere(w.device, stream):
            return w4a4_group_dequantize(w, W)
    if W is None:
        W = torch.empty(w.N, w.K, dtype=w.dtype, device=w.device)
    _check(_group_dequantize(w.ref, _need(W, "W", w.dtype, w.device, (w.N, w.K)), st), "w4a4_group_dequantize")
    return W


def w4a4_group_gemv(X: torch.Tensor, w: GroupWeights, bias=None, Y=None, flags: int = 0,
                    stream=None) -> torch.Tensor:
    """Y [M, N] = X [M, K] W^T + bias for up to 16 tokens."""
    dev, dt = w.device, w.dtype
    st = _here(dev, stream)
    if st is None:
        with _elsewhere(dev, stream):
            return w4a4_group_gemv(X, w, bias, Y, flags)
    M = X.shape[0]
    x = _need(X, "X", dt, dev, (M, w.K))
    if Y is None:
        Y = X.new_empty(M, w.N)  # 1.4 us; a tuple of sizes takes 1.9, torch.empty 2.5
        y = Y.data_ptr()
    else:
        y = _need(Y, "Y", dt, dev, (M, w.N))
    _check(_group_gemv(x, M, w.ref, None if bias is None else _need(bias, "bias", dt, dev, (w.N,)), y, flags, st),
           "w4a4_group_gemv")
    return Y


def w4a4_rope_table(n_pos: int, rot_dim: int, base: float = 10000.0):
    """Host: the rotation table [n_pos, rot_dim] (numpy fp32), cos then sin per row."""
    import numpy as np
    table = np.empty((n_pos, rot_dim), np.float32)
    _check(_rope_table(n_pos, rot_dim, base, table.ctypes.data_as(_vp)), "w4a4_rope_table")
    return table


class KVCache:
    """Keys and values in pages: two tensors [n_pages, page_size, heads,
    head_dim] of the same strides, the last dimension contiguous.  A pool kept
    as [n_pages, heads, page_size, head_dim] is passed transposed(1, 2)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        dev = _cuda_device(k, "k")
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or v.device != dev or k.stride() != v.stride():
            raise ValueError("k and v must be 4-dimensional and agree in shape, strides, type and device")
        if k.stride(3) != 1:
            raise ValueError(f"head_dim must be contiguous, strides are {k.stride()}")
        self.k, self.v, self.device, self.dtype = k, v, dev, k.dtype
        P, S, H, D = k.shape
        self.n_heads, self.head_dim, self.page_size, self.n_pages = H, D, S, P
        # a dimension of one element has no stride of its own
        sp, ss, sh = (k.stride(i) if k.shape[i] > 1 else 0 for i in range(3))
        self.struct = KVCacheT(k.data_ptr(), v.data_ptr(), P, S, H, D, _half_flag(k.dtype), sp, ss, sh)
        self.ref = ctypes.byref(self.struct)


def w4a4_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, pages: torch.Tensor, pos: torch.Tensor,
                   q=None, q_out=None, table=None, table_pos=None, seq=None, flags: int = 0, stream=None):
    """k, v [T, heads, head_dim] enter the cache at position pos [T] (int32; negative: left out) of sequence
    seq [T] (default: token t is sequence t), whose pages are the row of pages [n_seqs, max_pages].  Keys, and
    q [T, q_heads, head_dim], are rotated by row table_pos[t] (default pos[t]) of table [n, rot_dim] fp32.
    Returns the rotated q (None without q)."""
    dev, dt = cache.device, cache.dtype
    st = _here(dev, stream)
    if st is None:
        with _elsewhere(dev, stream):
            return w4a4_kv_append(cache, k, v, pages, pos, q, q_out, table, table_pos, seq, flags)
    T = k.shape[0]
    kp, ks = _rows(k, "k", dt, dev, (T, cache.n_heads, cache.head_dim))
    vp, vs = _rows(v, "v", dt, dev, (T, cache.n_heads, cache.head_dim))
    qp = qs = op = hq = tp = n_table = rot = 0
    if q is not None:
        hq = q.shape[1]
        shape = (T, hq, cache.head_dim)
        qp, qs = _rows(q, "q", dt, dev, shape)
        if q_out is None:
            q_out = q.new_empty(T, hq, cache.head_dim)
            op = q_out.data_ptr()
        else:
            op = _need(q_out, "q_out", dt, dev, shape)
    n_seqs, max_pages = pages.shape
    if table is not None:
        n_table, rot = table.shape
        tp = _need(table, "table", torch.float32, dev, (n_table, rot))
    if seq is None and T > n_seqs:
        raise ValueError(f"{T} tokens for {n_seqs} sequences need seq")
    _check(_kv_append(cache.ref, _append_t.pack(
        kp, vp, qp, op, ks, vs, qs, T, _need(pages, "pages", torch.int32, dev, (n_seqs, max_pages)),
        0 if seq is None else _need(seq, "seq", torch.int32, dev, (T,)), _need(pos, "pos", torch.int32, dev, (T,)),
        0 if table_pos is None else _need(table_pos, "table_pos", torch.int32, dev, (T,)), tp,
        n_seqs, max_pages, hq, n_table, rot, flags), st), "w4a4_kv_append")
    return None if q is None else q_out


def w4a4_kv_attend_workspace_bytes(n_seqs: int, n_q_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(_kv_attend_ws(n_seqs, n_q_heads, n_kv_heads, head_dim))


def w4a4_kv_attend(q: torch.Tensor, cache: KVCache, pages: torch.Tensor, lens: torch.Tensor, scale=None,
                   window: int = 0, out=None, lse=None, workspace=None, stream=None) -> torch.Tensor:
    """One new token per sequence: q [n_seqs, q_heads, head_dim] against the lens [n_seqs] (int32) cached
    tokens of its sequence, the last `window` of them where window > 0.  scale: 1 / sqrt(head_dim) by
    default.  lse [n_seqs, q_heads] fp32 receives the logarithm of the sum of exponentials."""
    dev, dt = cache.device, cache.dtype
    st = _here(dev, stream)
    if st is None:
        with _elsewhere(dev, stream):
            return w4a4_kv_attend(q, cache, pages, lens, scale, window, out, lse, workspace)
    B, Hq, D = q.shape
    qp, qs = _rows(q, "q", dt, dev, (B, Hq, cache.head_dim))
    max_pages = pages.shape[1]
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty(B, Hq, D)
        op = out.data_ptr()
    else:
        op = _need(out, "out", dt, dev, (B, Hq, D))
    if workspace is None:
        need = _kv_attend_ws(B, Hq, cache.n_heads, D)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: need a contiguous tensor on {dev}")
    _check(_kv_attend(cache.ref, _attend_t.pack(
        qp, op, 0 if lse is None else _need(lse, "lse", torch.float32, dev, (B, Hq)), workspace.data_ptr(),
        _need(pages, "pages", torch.int32, dev, (B, max_pages)), _need(lens, "lens", torch.int32, dev, (B,)),
        qs, workspace.nbytes, B, max_pages, Hq, window, D ** -0.5 if scale is None else scale), st),
        "w4a4_kv_attend")
    return out
