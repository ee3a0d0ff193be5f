"""Thin Python binding of libsketch (include/sketch.h).

Argument marshalling only: every step of the method runs in the library's CUDA
kernels.  PyTorch supplies device memory (including the workspace each call
needs) and the stream.  There is no CPU fallback: if the compiled library is
missing, every call raises.
"""
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libsketch.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_WORKSPACE = 3
ERR_CUDA = 4

PROJ_RADEMACHER = 0
PROJ_GAUSSIAN_QR = 1

OP_SAMPLE_PROJECTION = 0
OP_PROJECT_INPUTS = 1
OP_ACCUMULATE = 2
OP_UPDATE_NORMSGD = 3
OP_UPDATE_SGD = 4
OP_LAYER_NORM_BACKWARD = 5
OP_CROSS_ENTROPY_FORWARD = 6
OP_CROSS_ENTROPY_BACKWARD = 7
OP_RMS_NORM_BACKWARD = 8
OP_GRAD_NORM = 9

DTYPE_BF16 = 0
DTYPE_FP32 = 1

DEV_H_ZERO = 1
DEV_H_NONFINITE = 2
DEV_W_NONFINITE = 4
DEV_QR_BREAKDOWN = 8
DEV_BAD_TARGET = 16

EXPORTS = ("sketch_workspace_bytes", "sketch_sample_projection", "sketch_project_inputs",
           "sketch_accumulate", "sketch_apply_update_normsgd", "sketch_apply_update_sgd",
           "sketch_workspace_bytes_batched", "sketch_sample_projection_batched",
           "sketch_project_inputs_batched", "sketch_accumulate_batched",
           "sketch_apply_update_normsgd_batched", "sketch_apply_update_sgd_batched",
           "sketch_apply_update_normsgd_noalloc", "sketch_noalloc_scratch_bytes",
           "sketch_read_device_errors", "sketch_read_exact_count", "sketch_kernel_launches",
           "sketch_projection_split_elems",
           "sketch_split_projection_batched", "sketch_project_inputs_fp32xp_batched",
           "sketch_accumulate_fp32xp_batched", "sketch_split_projection_grouped",
           "sketch_layer_norm_forward", "sketch_layer_norm_backward", "sketch_cross_entropy_forward",
           "sketch_cross_entropy_backward", "sketch_adamw_batched", "sketch_rms_norm_forward",
           "sketch_rms_norm_backward", "sketch_quantize_blocks", "sketch_matmul_blocks",
           "sketch_grad_norm_batched", "sketch_grad_scale_batched", "sketch_status_string",
           "sketch_last_error")


class ProjectionProblem(ctypes.Structure):
    _fields_ = [("P", ctypes.c_void_p), ("k", ctypes.c_int64), ("layer", ctypes.c_uint32)]


class ProjectProblem(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("T", ctypes.c_int64), ("k", ctypes.c_int64),
                ("ld_x", ctypes.c_int64), ("P", ctypes.c_void_p), ("XP", ctypes.c_void_p),
                ("ld_xp", ctypes.c_int64), ("P_split", ctypes.c_void_p)]


class SplitProblem(ctypes.Structure):
    _fields_ = [("P", ctypes.c_void_p), ("k", ctypes.c_int64), ("P_split", ctypes.c_void_p)]


class AccumulateProblem(ctypes.Structure):
    _fields_ = [("D", ctypes.c_void_p), ("T", ctypes.c_int64), ("d", ctypes.c_int64),
                ("ld_d", ctypes.c_int64), ("XP", ctypes.c_void_p), ("ld_xp", ctypes.c_int64),
                ("C", ctypes.c_void_p)]


class UpdateProblem(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("d", ctypes.c_int64), ("k", ctypes.c_int64),
                ("ld_w", ctypes.c_int64), ("C", ctypes.c_void_p), ("P", ctypes.c_void_p),
                ("layer", ctypes.c_uint32), ("wnorm2_in", ctypes.c_void_p),
                ("wnorm2_out", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


class AdamWProblem(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("G", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("layer", ctypes.c_uint32), ("w_type", ctypes.c_int), ("g_type", ctypes.c_int)]


class GradProblem(ctypes.Structure):
    _fields_ = [("G", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_int64), ("type", ctypes.c_int)]


class SketchError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s (status %d)" % (message, status))
        self.status = status


_lib = None
_c = ctypes
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_u32 = ctypes.c_uint32
_u64 = ctypes.c_uint64
_SIGS = {
    "sketch_workspace_bytes": (ctypes.c_size_t, [_c.c_int, _i64, _i64, _i64, _i64]),
    "sketch_sample_projection": (_c.c_int, [_c.c_int, _u64, _u32, _u32, _i64, _i64, _vp, _vp, _vp,
                                            _c.c_size_t, _vp]),
    "sketch_project_inputs": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp,
                                         _c.c_size_t, _vp]),
    "sketch_accumulate": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _c.c_int, _vp,
                                     _c.c_size_t, _vp]),
    "sketch_apply_update_normsgd": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _c.c_float,
                                               _u64, _u32, _u32, _vp, _vp, _vp, _vp, _c.c_size_t,
                                               _vp]),
    "sketch_apply_update_sgd": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _c.c_float, _u64,
                                           _u32, _u32, _vp, _vp, _c.c_size_t, _vp]),
    "sketch_read_device_errors": (_c.c_int, [_c.POINTER(_c.c_int32), _vp]),
    "sketch_read_exact_count": (_c.c_int, [_c.POINTER(_c.c_uint64), _vp]),
    "sketch_kernel_launches": (_c.c_uint64, []),
    "sketch_projection_split_elems": (_c.c_size_t, [_i64, _i64]),
    "sketch_split_projection_batched": (_c.c_int, [_c.c_int, _vp, _i64, _vp]),
    "sketch_split_projection_grouped": (_c.c_int, [_c.c_int, _vp, _i64, _vp]),
    "sketch_project_inputs_fp32xp_batched": (_c.c_int, [_c.c_int, _vp, _i64, _vp, _c.c_size_t, _vp]),
    "sketch_accumulate_fp32xp_batched": (_c.c_int, [_c.c_int, _vp, _i64, _c.c_int, _vp, _c.c_size_t, _vp]),
    "sketch_workspace_bytes_batched": (ctypes.c_size_t, [_c.c_int, _c.c_int, _vp, _vp, _vp, _i64]),
    "sketch_sample_projection_batched": (_c.c_int, [_c.c_int, _u64, _u32, _c.c_int, _vp, _i64, _vp, _vp,
                                                    _c.c_size_t, _vp]),
    "sketch_project_inputs_batched": (_c.c_int, [_c.c_int, _vp, _i64, _vp, _c.c_size_t, _vp]),
    "sketch_accumulate_batched": (_c.c_int, [_c.c_int, _vp, _i64, _c.c_int, _vp, _c.c_size_t, _vp]),
    "sketch_apply_update_normsgd_batched": (_c.c_int, [_c.c_int, _vp, _i64, _c.c_float, _u64, _u32, _vp,
                                                       _c.c_size_t, _vp]),
    "sketch_apply_update_sgd_batched": (_c.c_int, [_c.c_int, _vp, _i64, _c.c_float, _u64, _u32, _vp,
                                                   _c.c_size_t, _vp]),
    "sketch_apply_update_normsgd_noalloc": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _c.c_float,
                                                       _u64, _u32, _u32, _vp, _vp, _vp, _vp]),
    "sketch_noalloc_scratch_bytes": (ctypes.c_size_t, []),
    "sketch_layer_norm_forward": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _vp, _vp, _c.c_int, _c.c_float,
                                             _vp, _i64, _vp, _vp, _vp]),
    "sketch_layer_norm_backward": (_c.c_int, [_vp, _i64, _vp, _c.c_int, _i64, _i64, _i64, _vp, _c.c_int, _vp,
                                              _vp, _vp, _i64, _vp, _vp, _c.c_int, _vp, _c.c_size_t, _vp]),
    "sketch_cross_entropy_forward": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _c.c_float, _vp,
                                                _vp, _vp, _vp, _c.c_size_t, _vp]),
    "sketch_cross_entropy_backward": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _c.c_float, _vp,
                                                 _vp, _vp, _i64, _vp, _c.c_int, _i64, _vp, _i64, _i64, _vp,
                                                 _c.c_int, _vp, _vp, _c.c_size_t, _vp]),
    "sketch_adamw_batched": (_c.c_int, [_c.c_int, _vp] + [_c.c_double] * 5 + [_vp, _u64, _u32, _vp]),
    "sketch_rms_norm_forward": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _c.c_int,
                                           _c.c_float, _vp, _i64, _vp, _i64, _vp, _vp, _vp]),
    "sketch_rms_norm_backward": (_c.c_int, [_vp, _i64, _vp, _c.c_int, _i64, _i64, _i64, _vp, _c.c_int, _vp, _vp, _i64,
                                            _vp, _i64, _vp, _c.c_int, _vp, _c.c_size_t, _vp]),
    "sketch_quantize_blocks": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _c.c_int, _vp, _i64, _vp, _vp, _i64, _vp]),
    "sketch_matmul_blocks": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp,
                                        _c.c_int, _i64, _c.c_int, _vp]),
    "sketch_grad_norm_batched": (_c.c_int, [_c.c_int, _vp, _c.c_float, _vp, _vp, _vp, _c.c_size_t, _vp]),
    "sketch_grad_scale_batched": (_c.c_int, [_c.c_int, _vp, _vp, _vp]),
    "sketch_status_string": (_c.c_char_p, [_c.c_int]),
    "sketch_last_error": (_c.c_char_p, []),
}


def lib():
    """Load libsketch.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libsketch.so is not built (expected at %s); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`" % LIB_PATH)
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _check(status):
    if status != OK:
        l = lib()
        raise SketchError(status, "%s: %s" % (l.sketch_status_string(status).decode(),
                                              l.sketch_last_error().decode()))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream), s


def _rows(t, dtype, name):
    """Row-major 2-D CUDA tensor of ``dtype`` with unit column stride; returns ld."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s must be 2-D with unit column stride" % name)
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], ((t.shape[1] + 7) // 8) * 8)


def _contig(t, dtype, name):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA %s tensor" % (name, dtype))


def _workspace(nbytes, device, stream, given=None):
    """The caller's workspace tensor if given (checked), else a fresh one."""
    if nbytes == 0:
        return None
    if given is not None:
        if not given.is_cuda or given.numel() * given.element_size() < nbytes:
            raise ValueError("workspace needs %d bytes" % nbytes)
        return given
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def read_device_errors(stream=None, device=None):
    """Read and clear the device error word (bits of timed-out waits); syncs the stream."""
    dev = device if device is not None else torch.cuda.current_device()
    h, _ = _stream_handle(stream, dev)
    flags = ctypes.c_int32(0)
    _check(lib().sketch_read_device_errors(ctypes.byref(flags), h))
    return int(flags.value)


def read_exact_count(stream=None, device=None):
    """Read and clear the count of weights the update calls recomputed on their
    exact path (instrumentation); syncs the stream."""
    dev = device if device is not None else torch.cuda.current_device()
    h, _ = _stream_handle(stream, dev)
    n = ctypes.c_uint64(0)
    _check(lib().sketch_read_exact_count(ctypes.byref(n), h))
    return int(n.value)


def kernel_launches():
    """Kernels this library has launched in this process (counted on the host)."""
    return int(lib().sketch_kernel_launches())


def workspace_bytes(op, T=0, d=0, k=0, r=1):
    return int(lib().sketch_workspace_bytes(op, T, d, k, r))


def sample_projection(kind, seed, layer, step, P, dev_status=None, stream=None):
    """Fill P (k x r fp32) with the projection for (seed, layer, step)."""
    _contig(P, torch.float32, "P")
    k, r = P.shape
    h, s = _stream_handle(stream, P.device)
    nbytes = workspace_bytes(OP_SAMPLE_PROJECTION, 0, 0, k, r) if kind == PROJ_GAUSSIAN_QR else 0
    ws = _workspace(nbytes, P.device, s)
    _check(lib().sketch_sample_projection(kind, seed & 0xFFFFFFFFFFFFFFFF, layer, step, k, r,
                                          _ptr(P), _ptr(dev_status), _ptr(ws), nbytes, h))
    return P


def project_inputs(X, P, XP, stream=None):
    """XP[:, :r] = bf16(X P)."""
    ld_x = _rows(X, torch.bfloat16, "X")
    ld_xp = _rows(XP, torch.bfloat16, "XP")
    _contig(P, torch.float32, "P")
    T, k = X.shape
    r = P.shape[1]
    if P.shape[0] != k or XP.shape[0] != T or XP.shape[1] < r:
        raise ValueError("shape mismatch: X %s, P %s, XP %s" % (tuple(X.shape), tuple(P.shape),
                                                                tuple(XP.shape)))
    h, s = _stream_handle(stream, X.device)
    nbytes = workspace_bytes(OP_PROJECT_INPUTS, T, 0, k, r)
    ws = _workspace(nbytes, X.device, s)
    _check(lib().sketch_project_inputs(_ptr(X), T, k, ld_x, _ptr(P), r, _ptr(XP), ld_xp, _ptr(ws),
                                       nbytes, h))
    return XP


def accumulate(D, XP, C, overwrite=False, r=None, stream=None):
    """C = (0 if overwrite else C) + D^T XP[:, :r]."""
    ld_d = _rows(D, torch.bfloat16, "D")
    ld_xp = _rows(XP, torch.bfloat16, "XP")
    _contig(C, torch.float32, "C")
    T, d = D.shape
    r = C.shape[1] if r is None else r
    if C.shape[0] != d or XP.shape[0] != T or XP.shape[1] < r or C.shape[1] != r:
        raise ValueError("shape mismatch: D %s, XP %s, C %s" % (tuple(D.shape), tuple(XP.shape),
                                                                tuple(C.shape)))
    h, s = _stream_handle(stream, D.device)
    nbytes = workspace_bytes(OP_ACCUMULATE, T, d, 0, r)
    ws = _workspace(nbytes, D.device, s)
    _check(lib().sketch_accumulate(_ptr(D), T, d, ld_d, _ptr(XP), ld_xp, r, _ptr(C),
                                   1 if overwrite else 0, _ptr(ws), nbytes, h))
    return C


def apply_update_normsgd(W, C, P, tau, seed, layer, step, wnorm2_in=None, wnorm2_out=None,
                         dev_status=None, stream=None):
    """W <- SR_bf16(W - tau ||W|| H / ||H||), H = C P^T, in place."""
    ld_w = _rows(W, torch.bfloat16, "W")
    _contig(C, torch.float32, "C")
    _contig(P, torch.float32, "P")
    d, k = W.shape
    r = C.shape[1]
    if C.shape[0] != d or P.shape != (k, r):
        raise ValueError("shape mismatch: W %s, C %s, P %s" % (tuple(W.shape), tuple(C.shape),
                                                               tuple(P.shape)))
    h, s = _stream_handle(stream, W.device)
    nbytes = workspace_bytes(OP_UPDATE_NORMSGD, 0, d, k, r)
    ws = _workspace(nbytes, W.device, s)
    _check(lib().sketch_apply_update_normsgd(_ptr(W), d, k, ld_w, _ptr(C), _ptr(P), r, float(tau),
                                             seed & 0xFFFFFFFFFFFFFFFF, layer, step,
                                             _ptr(wnorm2_in), _ptr(wnorm2_out), _ptr(dev_status),
                                             _ptr(ws), nbytes, h))
    return W


def apply_update_normsgd_noalloc(W, C, P, tau, seed, layer, step, wnorm2_in=None, wnorm2_out=None,
                                 dev_status=None, stream=None):
    """apply_update_normsgd without a workspace: the library's fixed device
    scratch array is used instead (for callers that cannot allocate)."""
    ld_w = _rows(W, torch.bfloat16, "W")
    _contig(C, torch.float32, "C")
    _contig(P, torch.float32, "P")
    d, k = W.shape
    r = C.shape[1]
    if C.shape[0] != d or P.shape != (k, r):
        raise ValueError("shape mismatch: W %s, C %s, P %s" % (tuple(W.shape), tuple(C.shape),
                                                               tuple(P.shape)))
    h, _ = _stream_handle(stream, W.device)
    _check(lib().sketch_apply_update_normsgd_noalloc(_ptr(W), d, k, ld_w, _ptr(C), _ptr(P), r,
                                                     float(tau), seed & 0xFFFFFFFFFFFFFFFF, layer,
                                                     step, _ptr(wnorm2_in), _ptr(wnorm2_out),
                                                     _ptr(dev_status), h))
    return W


def apply_update_sgd(W, C, P, alpha_eta, seed, layer, step, dev_status=None, stream=None):
    """W <- SR_bf16(W - alpha_eta C P^T), in place."""
    ld_w = _rows(W, torch.bfloat16, "W")
    _contig(C, torch.float32, "C")
    _contig(P, torch.float32, "P")
    d, k = W.shape
    r = C.shape[1]
    if C.shape[0] != d or P.shape != (k, r):
        raise ValueError("shape mismatch: W %s, C %s, P %s" % (tuple(W.shape), tuple(C.shape),
                                                               tuple(P.shape)))
    h, s = _stream_handle(stream, W.device)
    nbytes = workspace_bytes(OP_UPDATE_SGD, 0, d, k, r)
    ws = _workspace(nbytes, W.device, s)
    _check(lib().sketch_apply_update_sgd(_ptr(W), d, k, ld_w, _ptr(C), _ptr(P), r,
                                         float(alpha_eta), seed & 0xFFFFFFFFFFFFFFFF, layer, step,
                                         _ptr(dev_status), _ptr(ws), nbytes, h))
    return W


# --------------------------------------------------------------------------
# Batched forms: one call per phase for a whole stack of layers
# --------------------------------------------------------------------------

def _i64_array(vals):
    return (ctypes.c_int64 * len(vals))(*vals)


def workspace_bytes_batched(op, T=None, d=None, k=None, r=1):
    n = len(next(x for x in (T, d, k) if x is not None))
    arr = [None if x is None else _i64_array(x) for x in (T, d, k)]
    return int(lib().sketch_workspace_bytes_batched(
        op, n, *[None if a is None else ctypes.cast(a, ctypes.c_void_p) for a in arr], r))


def sample_projection_batched(kind, seed, step, Ps, layers, dev_status=None, ws=None, stream=None):
    """Fill every P (k_i x r fp32) for (seed, layers[i], step)."""
    n = len(Ps)
    r = Ps[0].shape[1]
    probs = (ProjectionProblem * n)()
    for i, (P, layer) in enumerate(zip(Ps, layers)):
        _contig(P, torch.float32, "P")
        if P.shape[1] != r:
            raise ValueError("all projections of a batch share r")
        probs[i] = ProjectionProblem(P.data_ptr(), P.shape[0], layer)
    h, s = _stream_handle(stream, Ps[0].device)
    nbytes = (workspace_bytes_batched(OP_SAMPLE_PROJECTION, k=[P.shape[0] for P in Ps], r=r)
              if kind == PROJ_GAUSSIAN_QR else 0)
    wsb = _workspace(nbytes, Ps[0].device, s, ws)
    _check(lib().sketch_sample_projection_batched(kind, seed & 0xFFFFFFFFFFFFFFFF, step, n, probs, r,
                                                  _ptr(dev_status), _ptr(wsb), nbytes, h))
    return Ps


def projection_split_elems(k, r):
    return int(lib().sketch_projection_split_elems(k, r))


def split_projection_batched(Ps, splits=None, stream=None):
    """BF16 splits of the projections Ps (k x r fp32) for project_inputs_batched;
    returns the list of split buffers (uint16, allocated when not given)."""
    n = len(Ps)
    r = Ps[0].shape[1]
    if splits is None:
        splits = [torch.empty(projection_split_elems(P.shape[0], r), dtype=torch.int16, device=P.device)
                  for P in Ps]
    probs = (SplitProblem * n)()
    for i, (P, S) in enumerate(zip(Ps, splits)):
        _contig(P, torch.float32, "P")
        if P.shape[1] != r or S.numel() * S.element_size() < 2 * projection_split_elems(P.shape[0], r):
            raise ValueError("shape mismatch in problem %d" % i)
        probs[i] = SplitProblem(P.data_ptr(), P.shape[0], S.data_ptr())
    h, _ = _stream_handle(stream, Ps[0].device)
    _check(lib().sketch_split_projection_batched(n, probs, r, h))
    return splits


class SplitGroup(ctypes.Structure):
    _fields_ = [("P", ctypes.c_void_p), ("m", ctypes.c_int), ("k", ctypes.c_int64), ("P_split", ctypes.c_void_p)]


def split_projection_grouped(groups, splits=None, stream=None):
    """Splits of concatenated projections: groups is a list of lists of P
    (k x r fp32, one k per group); group g's split is that of [P_0 | ... |
    P_{m-1}] (k x m r), for project_inputs_grouped_batched.  Returns the split
    buffers (uint16, allocated when not given)."""
    n = len(groups)
    r = groups[0][0].shape[1]
    if splits is None:
        splits = [torch.empty(projection_split_elems(g[0].shape[0], len(g) * r), dtype=torch.int16,
                              device=g[0].device) for g in groups]
    probs = (SplitGroup * n)()
    keep = []
    for i, (g, S) in enumerate(zip(groups, splits)):
        k = g[0].shape[0]
        for P in g:
            _contig(P, torch.float32, "P")
            if P.shape != (k, r):
                raise ValueError("shape mismatch in group %d" % i)
        if S.numel() * S.element_size() < 2 * projection_split_elems(k, len(g) * r):
            raise ValueError("split buffer of group %d too small" % i)
        ptrs = (ctypes.c_void_p * len(g))(*[P.data_ptr() for P in g])
        keep.append(ptrs)
        probs[i] = SplitGroup(ctypes.cast(ptrs, ctypes.c_void_p), len(g), k, S.data_ptr())
    h, _ = _stream_handle(stream, groups[0][0].device)
    _check(lib().sketch_split_projection_grouped(n, probs, r, h))
    return splits


def project_inputs_grouped_batched(Xs, splits, r_total, XPs, ws=None, stream=None):
    """XP = bf16(X [P_0 | ... | P_{m-1}]) (T x r_total, r_total = m r) for each
    problem, from the splits of split_projection_grouped; member q's XP is
    XP[:, q r:(q + 1) r]."""
    n = len(Xs)
    probs = (ProjectProblem * n)()
    for i, (X, S, XP) in enumerate(zip(Xs, splits, XPs)):
        ld_x = _rows(X, torch.bfloat16, "X")
        ld_xp = _rows(XP, torch.bfloat16, "XP")
        if XP.shape[0] != X.shape[0] or XP.shape[1] < r_total:
            raise ValueError("shape mismatch in problem %d" % i)
        if S.numel() * S.element_size() < 2 * projection_split_elems(X.shape[1], r_total):
            raise ValueError("split buffer of problem %d too small" % i)
        probs[i] = ProjectProblem(X.data_ptr(), X.shape[0], X.shape[1], ld_x, None, XP.data_ptr(), ld_xp,
                                  S.data_ptr())
    h, s = _stream_handle(stream, Xs[0].device)
    nbytes = workspace_bytes_batched(OP_PROJECT_INPUTS, T=[X.shape[0] for X in Xs],
                                     k=[X.shape[1] for X in Xs], r=r_total)
    wsb = _workspace(nbytes, Xs[0].device, s, ws)
    _check(lib().sketch_project_inputs_batched(n, probs, r_total, _ptr(wsb), nbytes, h))
    return XPs


def _project_batched(Xs, Ps, XPs, ws, stream, splits, fn, xp_cols):
    n = len(Xs)
    r = Ps[0].shape[1]
    probs = (ProjectProblem * n)()
    for i, (X, P, XP) in enumerate(zip(Xs, Ps, XPs)):
        ld_x = _rows(X, torch.bfloat16, "X")
        ld_xp = _rows(XP, torch.bfloat16, "XP")
        _contig(P, torch.float32, "P")
        if P.shape != (X.shape[1], r) or XP.shape[0] != X.shape[0] or XP.shape[1] < xp_cols:
            raise ValueError("shape mismatch in problem %d" % i)
        probs[i] = ProjectProblem(X.data_ptr(), X.shape[0], X.shape[1], ld_x, P.data_ptr(),
                                  XP.data_ptr(), ld_xp, splits[i].data_ptr() if splits is not None else None)
    h, s = _stream_handle(stream, Xs[0].device)
    nbytes = workspace_bytes_batched(OP_PROJECT_INPUTS, T=[X.shape[0] for X in Xs],
                                     k=[X.shape[1] for X in Xs], r=r)
    wsb = _workspace(nbytes, Xs[0].device, s, ws)
    _check(getattr(lib(), fn)(n, probs, r, _ptr(wsb), nbytes, h))
    return XPs


def project_inputs_batched(Xs, Ps, XPs, ws=None, stream=None, splits=None):
    """XP = bf16(X P) for each problem; `splits` (from split_projection_batched
    for these Ps) skips splitting P again."""
    return _project_batched(Xs, Ps, XPs, ws, stream, splits, "sketch_project_inputs_batched", Ps[0].shape[1])


def _accumulate_batched(Ds, XPs, Cs, overwrite, ws, stream, fn, xp_cols):
    n = len(Ds)
    r = Cs[0].shape[1]
    probs = (AccumulateProblem * n)()
    for i, (D, XP, C) in enumerate(zip(Ds, XPs, Cs)):
        ld_d = _rows(D, torch.bfloat16, "D")
        ld_xp = _rows(XP, torch.bfloat16, "XP")
        _contig(C, torch.float32, "C")
        if C.shape != (D.shape[1], r) or XP.shape[0] != D.shape[0] or XP.shape[1] < xp_cols:
            raise ValueError("shape mismatch in problem %d" % i)
        probs[i] = AccumulateProblem(D.data_ptr(), D.shape[0], D.shape[1], ld_d, XP.data_ptr(), ld_xp,
                                     C.data_ptr())
    h, s = _stream_handle(stream, Ds[0].device)
    nbytes = workspace_bytes_batched(OP_ACCUMULATE, T=[D.shape[0] for D in Ds],
                                     d=[D.shape[1] for D in Ds], r=r)
    wsb = _workspace(nbytes, Ds[0].device, s, ws)
    _check(getattr(lib(), fn)(n, probs, r, 1 if overwrite else 0, _ptr(wsb), nbytes, h))
    return Cs


def accumulate_batched(Ds, XPs, Cs, overwrite=False, ws=None, stream=None):
    return _accumulate_batched(Ds, XPs, Cs, overwrite, ws, stream, "sketch_accumulate_batched", Cs[0].shape[1])


def xp_split_cols(r):
    """Columns of the fp32-accurate XP form: a BF16 pair, 2 * round16(r)."""
    return 2 * ((r + 15) // 16 * 16)


def project_inputs_fp32xp_batched(Xs, Ps, XPs, ws=None, stream=None, splits=None):
    """XP kept to ~2^-17 relative as a BF16 pair (hi in columns [0, r), lo at
    [round16(r), round16(r) + r)); each XP is T x >= xp_split_cols(r) BF16."""
    return _project_batched(Xs, Ps, XPs, ws, stream, splits, "sketch_project_inputs_fp32xp_batched",
                            xp_split_cols(Ps[0].shape[1]))


def accumulate_fp32xp_batched(Ds, XPs, Cs, overwrite=False, ws=None, stream=None):
    """C = (0 or C) + D^T (XP_hi + XP_lo) from the fp32-accurate XP form."""
    return _accumulate_batched(Ds, XPs, Cs, overwrite, ws, stream, "sketch_accumulate_fp32xp_batched",
                               xp_split_cols(Cs[0].shape[1]))


def _update_batched(normsgd, Ws, Cs, Ps, step_size, seed, layers, step, wnorm2_in, wnorm2_out,
                    dev_status, ws, stream):
    n = len(Ws)
    r = Cs[0].shape[1]
    probs = (UpdateProblem * n)()
    for i in range(n):
        W, C, P = Ws[i], Cs[i], Ps[i]
        ld_w = _rows(W, torch.bfloat16, "W")
        _contig(C, torch.float32, "C")
        _contig(P, torch.float32, "P")
        if C.shape != (W.shape[0], r) or P.shape != (W.shape[1], r):
            raise ValueError("shape mismatch in problem %d" % i)
        pick = (lambda lst: None if lst is None else lst[i])
        probs[i] = UpdateProblem(W.data_ptr(), W.shape[0], W.shape[1], ld_w, C.data_ptr(), P.data_ptr(),
                                 layers[i], _ptr(pick(wnorm2_in)), _ptr(pick(wnorm2_out)),
                                 _ptr(pick(dev_status)))
    h, s = _stream_handle(stream, Ws[0].device)
    op = OP_UPDATE_NORMSGD if normsgd else OP_UPDATE_SGD
    nbytes = workspace_bytes_batched(op, d=[W.shape[0] for W in Ws], k=[W.shape[1] for W in Ws], r=r)
    wsb = _workspace(nbytes, Ws[0].device, s, ws)
    fn = lib().sketch_apply_update_normsgd_batched if normsgd else lib().sketch_apply_update_sgd_batched
    _check(fn(n, probs, r, float(step_size), seed & 0xFFFFFFFFFFFFFFFF, step, _ptr(wsb), nbytes, h))
    return Ws


def apply_update_normsgd_batched(Ws, Cs, Ps, tau, seed, layers, step, wnorm2_in=None, wnorm2_out=None,
                                 dev_status=None, ws=None, stream=None):
    """Normalized-SGD update of every W_i (lists of per-layer tensors; the
    optional lists hold one-element device tensors or None entries)."""
    return _update_batched(True, Ws, Cs, Ps, tau, seed, layers, step, wnorm2_in, wnorm2_out,
                           dev_status, ws, stream)


def apply_update_sgd_batched(Ws, Cs, Ps, alpha_eta, seed, layers, step, dev_status=None, ws=None,
                             stream=None):
    return _update_batched(False, Ws, Cs, Ps, alpha_eta, seed, layers, step, None, None, dev_status,
                           ws, stream)


# --------------------------------------------------------------------------
# Training operators around the sketched layers
# --------------------------------------------------------------------------

_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}

# These calls are short enough for Python's share to show, so their checks and
# marshalling are lean: addresses and the stream's handle as plain numbers, each
# property of a tensor asked once.


def _dtype(t, name):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError("%s must be bfloat16 or float32, got %s" % (name, t.dtype)) from None


def _addr(t):
    return None if t is None else t.data_ptr()


def _stream_of(stream, device):
    """Handle of the given stream, or of the device's current one."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _scratch(op, T, d, k, r, device, stream, given):
    """(workspace of a call, its address, its size): the caller's, or one that belongs to the call's stream."""
    nbytes = lib().sketch_workspace_bytes(op, T, d, k, r)
    if given is not None:
        if given.device != device or not given.is_contiguous() or given.numel() * given.element_size() < nbytes:
            raise ValueError("workspace needs %d contiguous bytes on %s" % (nbytes, device))
    elif nbytes == 0:
        return None, None, 0
    elif stream is None:
        given = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        given = _workspace(nbytes, device, stream)
    return given, given.data_ptr(), nbytes


def _norm_rows(t, shape, dtype, device, name):
    """Row stride of a 2-D CUDA activation tensor with X's shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError("%s must have X's shape, type and device" % name)
    ld, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        raise ValueError("%s must have unit column stride" % name)
    return ld if shape[0] > 1 else shape[1]


def _norm_x(X):
    if not X.is_cuda or X.dim() != 2:
        raise ValueError("X must be a 2-D CUDA tensor")
    return X.shape, X.dtype, X.device


def _vector(t, n, dtype, device, name):
    """Check a contiguous vector of n values on ``device``, of ``dtype`` (any when that is None)."""
    if not t.is_contiguous() or t.numel() != n or t.device != device or (dtype is not None and t.dtype != dtype):
        raise ValueError("%s must be a contiguous %s vector of %d on %s" % (name, dtype or "", n, device))


def _norm_weights(gamma, beta, k, device):
    for t, name in ((gamma, "gamma"), (beta, "beta")):
        if t is not None:
            _vector(t, k, None, device, name)
    if gamma is not None and beta is not None and gamma.dtype != beta.dtype:
        raise ValueError("gamma and beta must have one type")
    t = gamma if gamma is not None else beta
    return DTYPE_FP32 if t is None else _dtype(t, "gamma and beta")


def layer_norm_forward(X, gamma, beta, Y, mean, rstd, eps=1e-5, stream=None):
    """Y = (X - mean) rstd gamma + beta over the rows of X (T x k, BF16 or fp32);
    mean and rstd (T fp32) are written for the backward pass.  gamma and beta
    (k, BF16 or fp32) may be None.  Y may be X."""
    x_type = _dtype(X, "X")
    shape, dtype, dev = _norm_x(X)
    T, k = shape
    ld_x, ld_y = _norm_rows(X, shape, dtype, dev, "X"), _norm_rows(Y, shape, dtype, dev, "Y")
    w_type = _norm_weights(gamma, beta, k, dev)
    _vector(mean, T, torch.float32, dev, "mean")
    _vector(rstd, T, torch.float32, dev, "rstd")
    st = lib().sketch_layer_norm_forward(X.data_ptr(), x_type, T, k, ld_x, _addr(gamma), _addr(beta), w_type, eps,
                                         Y.data_ptr(), ld_y, mean.data_ptr(), rstd.data_ptr(),
                                         _stream_of(stream, dev))
    if st:
        _check(st)
    return Y


def layer_norm_backward(dY, X, gamma, mean, rstd, dX=None, dgamma=None, dbeta=None, overwrite=False, ws=None,
                        stream=None):
    """dX (X's type, may be dY), and dgamma, dbeta (k fp32; replaced with
    overwrite, else added to) of layer_norm_forward; each may be None."""
    x_type = _dtype(X, "X")
    shape, dtype, dev = _norm_x(X)
    T, k = shape
    ld_x, ld_dy = _norm_rows(X, shape, dtype, dev, "X"), _norm_rows(dY, shape, dtype, dev, "dY")
    ld_dx = 0 if dX is None else _norm_rows(dX, shape, dtype, dev, "dX")
    w_type = _norm_weights(gamma, None, k, dev)
    _vector(mean, T, torch.float32, dev, "mean")
    _vector(rstd, T, torch.float32, dev, "rstd")
    for t, name in ((dgamma, "dgamma"), (dbeta, "dbeta")):
        if t is not None:
            _vector(t, k, torch.float32, dev, name)
    keep, ws_at, nbytes = _scratch(OP_LAYER_NORM_BACKWARD, T, 0, k, 0, dev, stream, ws)
    st = lib().sketch_layer_norm_backward(dY.data_ptr(), ld_dy, X.data_ptr(), x_type, T, k, ld_x, _addr(gamma),
                                          w_type, mean.data_ptr(), rstd.data_ptr(), _addr(dX), ld_dx,
                                          _addr(dgamma), _addr(dbeta), 1 if overwrite else 0, ws_at, nbytes,
                                          _stream_of(stream, dev))
    if st:
        _check(st)
    return dX


def _head(X, W, targets):
    ld_x, ld_w = _rows(X, torch.bfloat16, "X"), _rows(W, torch.bfloat16, "W")
    if W.shape[1] != X.shape[1] or W.device != X.device:
        raise ValueError("shape or device mismatch: X %s, W %s" % (tuple(X.shape), tuple(W.shape)))
    _vector(targets, X.shape[0], torch.int64, X.device, "targets")
    return ld_x, ld_w


def _status_word(t, device):
    if t is not None:
        _vector(t, 1, torch.int32, device, "dev_status")


def cross_entropy_forward(X, W, targets, loss, lse, scale=1.0, dev_status=None, ws=None, stream=None):
    """Per-token loss = lse - l[target] and lse = log sum exp(l) (T fp32 each) of
    the logits l = scale X W^T, which are not stored; X (T x k) and W (V x k)
    BF16, targets T int64.  A negative target: loss 0."""
    ld_x, ld_w = _head(X, W, targets)
    T, k = X.shape
    V = W.shape[0]
    dev = X.device
    _vector(loss, T, torch.float32, dev, "loss")
    _vector(lse, T, torch.float32, dev, "lse")
    _status_word(dev_status, dev)
    keep, ws_at, nbytes = _scratch(OP_CROSS_ENTROPY_FORWARD, T, V, k, 0, dev, stream, ws)
    st = lib().sketch_cross_entropy_forward(X.data_ptr(), T, k, ld_x, W.data_ptr(), V, ld_w, targets.data_ptr(), scale,
                                            loss.data_ptr(), lse.data_ptr(), _addr(dev_status), ws_at, nbytes,
                                            _stream_of(stream, dev))
    if st:
        _check(st)
    return loss


def cross_entropy_backward(X, W, targets, lse, g, dX=None, dW=None, XP=None, C=None, overwrite=False, scale=1.0,
                           dev_status=None, ws=None, stream=None):
    """Gradients of cross_entropy_forward for the per-token upstream gradient g
    (T fp32): dX (T x k BF16), dW (V x k; BF16, or fp32) and the head's gradient
    sketch C (+)= D^T XP (V x r fp32, with XP = X P, T x r BF16); each may be
    None.  An fp32 dW and C are replaced with overwrite, else added to."""
    ld_x, ld_w = _head(X, W, targets)
    T, k = X.shape
    V = W.shape[0]
    dev = X.device
    _vector(lse, T, torch.float32, dev, "lse")
    _vector(g, T, torch.float32, dev, "g")
    _status_word(dev_status, dev)
    ld_dx = ld_dw = ld_xp = r = dw_type = 0
    if dX is not None:
        ld_dx = _rows(dX, torch.bfloat16, "dX")
    if dW is not None:
        dw_type = _dtype(dW, "dW")
        ld_dw = _rows(dW, dW.dtype, "dW")
    if (dX is not None and (dX.shape != X.shape or dX.device != dev)) or (
            dW is not None and (dW.shape != W.shape or dW.device != dev)):
        raise ValueError("dX and dW must have the shapes and the device of X and W")
    if (C is None) != (XP is None):
        raise ValueError("C and XP are given together")
    if C is not None:
        _contig(C, torch.float32, "C")
        ld_xp = _rows(XP, torch.bfloat16, "XP")
        r = C.shape[1]
        if C.dim() != 2 or C.shape[0] != V or XP.shape[0] != T or XP.shape[1] < r or C.device != dev or XP.device != dev:
            raise ValueError("shape or device mismatch: XP %s, C %s" % (tuple(XP.shape), tuple(C.shape)))
    keep, ws_at, nbytes = _scratch(OP_CROSS_ENTROPY_BACKWARD, T, V, k, r, dev, stream, ws)
    st = lib().sketch_cross_entropy_backward(X.data_ptr(), T, k, ld_x, W.data_ptr(), V, ld_w, targets.data_ptr(),
                                             scale, lse.data_ptr(), g.data_ptr(), _addr(dX), ld_dx, _addr(dW),
                                             dw_type, ld_dw, _addr(XP), ld_xp, r, _addr(C), 1 if overwrite else 0,
                                             _addr(dev_status), ws_at, nbytes, _stream_of(stream, dev))
    if st:
        _check(st)
    return dX


def adamw_problems(Ws, Gs, ms, vs, m_scales=None, v_scales=None, layers=None):
    """The problem table of adamw_batched: lists of contiguous, 16-byte aligned
    tensors of one size per problem.  States: fp32 m and v, or float8_e4m3fn codes of m and
    sqrt(v) with an fp32 scale per 256 values each."""
    n = len(Ws)
    eight = m_scales is not None
    if not (len(Gs) == len(ms) == len(vs) == n > 0) or (v_scales is not None) != eight or (
            eight and not (len(m_scales) == len(v_scales) == n)) or (layers is not None and len(layers) != n):
        raise ValueError("the lists of a batch have one length, and at least one tensor")
    probs = (AdamWProblem * n)()
    state = torch.float8_e4m3fn if eight else torch.float32
    for i in range(n):
        W, G, dev = Ws[i], Gs[i], Ws[i].device
        if dev.type != "cuda" or dev != Ws[0].device:
            raise ValueError("tensor %d must be a CUDA tensor on one device with the others" % i)
        size = W.numel()
        _vector(W, size, None, dev, "W")
        _vector(G, size, None, dev, "G")
        _vector(ms[i], size, state, dev, "m")
        _vector(vs[i], size, state, dev, "v")
        for t, name in ((W, "W"), (G, "G"), (ms[i], "m"), (vs[i], "v")):
            if size and t.data_ptr() % 16:
                raise ValueError("%s of tensor %d must be 16-byte aligned" % (name, i))
        scales = (None, None)
        if eight:
            for t in (m_scales[i], v_scales[i]):
                _vector(t, (size + 255) // 256, torch.float32, dev, "a state's scales")
            scales = (m_scales[i].data_ptr(), v_scales[i].data_ptr())
            if size == 0:  # an empty tensor has no address; any non-NULL one keeps the call's form
                scales = (W.element_size(), W.element_size())
        probs[i] = AdamWProblem(W.data_ptr(), G.data_ptr(), ms[i].data_ptr(), vs[i].data_ptr(), scales[0], scales[1],
                                size, i if layers is None else layers[i], _dtype(W, "W"), _dtype(G, "G"))
    return probs


def adamw_batched(probs, lr, betas, eps, weight_decay, seed, step, grad_scale=None, device=None, stream=None):
    """One AdamW step (counted from 0) of the tensors of adamw_problems.  grad_scale:
    a one-element fp32 tensor on their device that multiplies the gradients."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    if grad_scale is not None:
        _vector(grad_scale, 1, torch.float32, dev, "grad_scale")
    st = lib().sketch_adamw_batched(len(probs), probs, lr, betas[0], betas[1], eps, weight_decay, _addr(grad_scale),
                                    seed & 0xFFFFFFFFFFFFFFFF, step, _stream_of(stream, dev))
    if st:
        _check(st)


# --------------------------------------------------------------------------
# The residual stream's norm, 8-bit products, clipping
# --------------------------------------------------------------------------

SCALE_BLOCK = 128  # columns, or rows and columns of a weight, that share a scale


def _set_device(index):
    """Make device ``index`` current; returns the one before.  (Looked up here, as below: a
    PyTorch without CUDA has none of these functions, and imports this module all the same.)"""
    return torch._C._cuda_exchangeDevice(index)


def _launch(index, name, *args):
    """Call the library with device ``index`` current, whatever device was."""
    fn = getattr(_lib or lib(), name)
    before = _set_device(index)
    try:
        st = fn(*args)
    finally:
        if before != index:
            _set_device(before)
    if st:
        _check(st)


def _stream_on(stream, index):
    """Handle of the given stream, or of the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device.index != index:
        raise ValueError("the stream is not one of cuda:%d" % index)
    return stream.cuda_stream


def _take_back(at):
    torch._C._cuda_cudaCachingAllocator_raw_delete(at)


def _borrow(op, T, k, index, handle, given):
    """(address, size, what _take_back gets after the call) of a call's workspace: the
    caller's, or one that PyTorch's allocator lends to the call's stream, where its next
    user comes after the call.  Not a tensor, whose making takes as long as two launches."""
    nbytes = lib().sketch_workspace_bytes(op, T, 0, k, 0)
    if given is not None:
        if given.get_device() != index or not given.is_contiguous() or given.numel() * given.element_size() < nbytes:
            raise ValueError("workspace needs %d contiguous bytes on cuda:%d" % (nbytes, index))
        return given.data_ptr(), nbytes, None
    if nbytes == 0:
        return None, 0, None
    before = _set_device(index)
    try:
        at = torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, handle)  # of the current device
    finally:
        if before != index:
            _set_device(before)
    return at, nbytes, at


def code_rows(T, k, device="cuda"):
    """An uninitialised T x k matrix of E4M3 codes whose rows start on 16 bytes, as
    the 8-bit calls want them."""
    return torch.empty(T, (k + 15) // 16 * 16, dtype=torch.float8_e4m3fn, device=device)[:, :k]


def _matrix(t, name):
    if not t.is_cuda or t.dim() != 2:
        raise ValueError("%s must be a 2-D CUDA tensor" % name)
    return t.shape, t.dtype, t.get_device()


def _like(t, shape, dtype, index, name):
    """Row stride of an activation matrix of this shape and type, on device ``index``."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError("%s must be a %d x %d %s matrix on cuda:%d" % (name, *shape, dtype, index))
    ld, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        raise ValueError("%s must have unit column stride" % name)
    return ld if shape[0] > 1 else shape[1]


def _flat(t, n, dtype, index, name):
    """Check n contiguous values of ``dtype`` on device ``index``."""
    if t.numel() != n or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of %d values on cuda:%d" % (name, dtype, n, index))


def _gamma(t, k, index):
    if t is None:
        return DTYPE_FP32
    _flat(t, k, t.dtype, index, "gamma")
    return _dtype(t, "gamma")


def _codes(t, T, k, index, name):
    """Row stride of a T x k matrix of codes."""
    if t.dtype is not torch.float8_e4m3fn or t.get_device() != index or t.shape != (T, k):
        raise ValueError("%s must be a %d x %d float8_e4m3fn matrix on cuda:%d" % (name, T, k, index))
    ld, unit = t.stride()
    if unit != 1 and k > 1:
        raise ValueError("%s must have unit column stride" % name)
    return ld if T > 1 else (k + 15) // 16 * 16


def _scales(t, rows, cols, index, name):
    if t.dtype is not torch.float32 or t.get_device() != index or t.shape != (rows, cols):
        raise ValueError("%s must be a %d x %d float32 matrix on cuda:%d" % (name, rows, cols, index))
    return t.stride()


def _groups(n):
    return (n + SCALE_BLOCK - 1) // SCALE_BLOCK


def rms_norm_forward(X, gamma, rstd=None, R=None, S=None, Y=None, Q=None, scale=None, eps=1e-6, stream=None):
    """Root-mean-square norm of the rows of s = X + R (T x k, BF16 or fp32; R may be
    None): y = s rstd gamma.  S (only with R; may be X or R) receives s, Y (may be X or R) receives
    y, and Q with scale (T x ceil(k / 128) fp32) y as E4M3 codes with a scale for each
    row's 128 columns; Y or Q is given.  rstd (T fp32) is for the backward pass.  gamma
    (k, BF16 or fp32) may be None."""
    shape, dtype, dev = _matrix(X, "X")
    x_type = _dtype(X, "X")
    T, k = shape
    ld_x = _like(X, shape, dtype, dev, "X")
    ld_r = 0 if R is None else _like(R, shape, dtype, dev, "R")
    ld_s = 0 if S is None else _like(S, shape, dtype, dev, "S")
    ld_y = 0 if Y is None else _like(Y, shape, dtype, dev, "Y")
    ld_q = 0 if Q is None else _codes(Q, T, k, dev, "Q")
    if scale is not None:
        _flat(scale, T * _groups(k), torch.float32, dev, "scale")
    w_type = _gamma(gamma, k, dev)
    if rstd is not None:
        _flat(rstd, T, torch.float32, dev, "rstd")
    _launch(dev, "sketch_rms_norm_forward", X.data_ptr(), x_type, T, k, ld_x, _addr(R), ld_r, _addr(S),
            ld_s, _addr(gamma), w_type, eps, _addr(Y), ld_y, _addr(Q), ld_q, _addr(scale), _addr(rstd),
            _stream_on(stream, dev))
    return Y if Y is not None else Q


def rms_norm_backward(dY, S, gamma, rstd, dS=None, dX=None, dgamma=None, overwrite=False, ws=None, stream=None):
    """dX (may be dY or dS) and dgamma (k fp32; replaced with overwrite, else added
    to) of rms_norm_forward; each may be None.  dS: the gradient that reaches S
    from the rest of the stream, added to dX, which is the gradient of X and of R."""
    shape, dtype, dev = _matrix(S, "S")
    x_type = _dtype(S, "S")
    T, k = shape
    ld_s, ld_dy = _like(S, shape, dtype, dev, "S"), _like(dY, shape, dtype, dev, "dY")
    ld_ds = 0 if dS is None else _like(dS, shape, dtype, dev, "dS")
    ld_dx = 0 if dX is None else _like(dX, shape, dtype, dev, "dX")
    w_type = _gamma(gamma, k, dev)
    _flat(rstd, T, torch.float32, dev, "rstd")
    if dgamma is not None:
        _flat(dgamma, k, torch.float32, dev, "dgamma")
    handle = _stream_on(stream, dev)
    ws_at, nbytes, lent = (None, 0, None) if dgamma is None else _borrow(OP_RMS_NORM_BACKWARD, T, k, dev, handle, ws)
    try:
        _launch(dev, "sketch_rms_norm_backward", dY.data_ptr(), ld_dy, S.data_ptr(), x_type, T, k, ld_s,
                _addr(gamma), w_type, rstd.data_ptr(), _addr(dS), ld_ds, _addr(dX), ld_dx, _addr(dgamma),
                1 if overwrite else 0, ws_at, nbytes, handle)
    finally:
        if lent is not None:
            _take_back(lent)
    return dX


def quantize_blocks(X, Q, scale, rows=1, Qt=None, stream=None):
    """E4M3 codes of X (T x k, BF16 or fp32) with a scale for each row's 128 columns,
    or with rows=128 (weights) for each 128 rows and 128 columns; scale:
    ceil(T / rows) x ceil(k / 128) fp32.  Qt (k x T, rows=128 only): the same codes transposed,
    with scales scale.t(); Q may then be None."""
    shape, dtype, dev = _matrix(X, "X")
    x_type = _dtype(X, "X")
    T, k = shape
    ld_x = _like(X, shape, dtype, dev, "X")
    ld_q = 0 if Q is None else _codes(Q, T, k, dev, "Q")
    ld_qt = 0 if Qt is None else _codes(Qt, k, T, dev, "Qt")
    _flat(scale, (T + rows - 1) // rows * _groups(k) if rows > 0 else 0, torch.float32, dev, "scale")
    _launch(dev, "sketch_quantize_blocks", X.data_ptr(), x_type, T, k, ld_x, rows, _addr(Q), ld_q,
            scale.data_ptr(), _addr(Qt), ld_qt, _stream_on(stream, dev))
    return Q


def matmul_blocks(A, a_scale, B, b_scale, Y, overwrite=True, stream=None):
    """Y = A B^T of codes with block scales: A (T x k) with a_scale (T x ceil(k /
    128)), B (N x k) with b_scale (ceil(N / 128) x ceil(k / 128), any strides).  A layer's output
    takes B = Q of its weight W and b_scale = scale, its input's gradient B = Qt
    and b_scale = scale.t().  Y (T x N) BF16, or fp32, which overwrite=False adds to
    (a BF16 Y is refused then: its earlier terms would be lost).  A block's two scales are
    multiplied by each other first: their product stays in fp32's normal range, 2^-126 to 2^128."""
    (T, k), _, dev = _matrix(A, "A")
    N = _matrix(B, "B")[0][0]
    ld_a, ld_b = _codes(A, T, k, dev, "A"), _codes(B, N, k, dev, "B")
    ld_as, unit = _scales(a_scale, T, _groups(k), dev, "a_scale")
    if unit != 1 and _groups(k) > 1:
        raise ValueError("a_scale must have unit column stride")
    if T == 1:
        ld_as = _groups(k)
    bs_row, bs_col = _scales(b_scale, _groups(N), _groups(k), dev, "b_scale")
    y_type = _dtype(Y, "Y")
    if not overwrite and y_type == DTYPE_BF16:
        raise ValueError("overwrite=False needs a float32 Y")
    ld_y = _like(Y, (T, N), Y.dtype, dev, "Y")
    if T == 1:
        ld_y = (N + 7) // 8 * 8
    _launch(dev, "sketch_matmul_blocks", A.data_ptr(), T, k, ld_a, a_scale.data_ptr(), ld_as, B.data_ptr(),
            N, ld_b, b_scale.data_ptr(), bs_row, bs_col, Y.data_ptr(), y_type, ld_y, 1 if overwrite else 0,
            _stream_on(stream, dev))
    return Y


def _written_twice(spans):
    """Whether one of the (address, bytes, written) that is written overlaps another one."""
    end = end_written = 0
    for start, size, written in sorted(s for s in spans if s[1]):
        if start < (end if written else end_written):
            return True
        end = max(end, start + size)
        if written:
            end_written = max(end_written, start + size)
    return False


def grad_problems(Gs, outs=None):
    """The problem table of grad_norm_batched and grad_scale_batched: contiguous
    tensors of any shapes, and those that receive the scaled ones (the same by default).
    The norm counts a tensor as often as it is listed; the scaling refuses a table in
    which what it writes overlaps another tensor."""
    Gs = list(Gs)
    outs = Gs if outs is None else list(outs)
    if not Gs or len(outs) != len(Gs):
        raise ValueError("the lists of a batch have one length, and at least one tensor")
    probs = (GradProblem * len(Gs))()
    spans = []
    for i, (G, out) in enumerate(zip(Gs, outs)):
        dev = G.device
        if dev.type != "cuda" or dev != Gs[0].device:
            raise ValueError("tensor %d must be a CUDA tensor on one device with the others" % i)
        _vector(G, G.numel(), None, dev, "G")
        _vector(out, G.numel(), G.dtype, dev, "out")
        probs[i] = GradProblem(G.data_ptr(), out.data_ptr(), G.numel(), _dtype(G, "G"))
        size = G.numel() * G.element_size()
        spans.append((out.data_ptr(), size, True))
        if out.data_ptr() != G.data_ptr():
            spans.append((G.data_ptr(), size, False))
    probs.tensors = Gs, outs  # kept as long as the table
    probs.written_twice = _written_twice(spans)
    return probs


def _problems_on(probs, index):
    """Number of a table's tensors, which lie on device ``index``."""
    tensors = getattr(probs, "tensors", None)
    if tensors is not None and tensors[0][0].get_device() != index:
        raise ValueError("the tensors of the table are not on cuda:%d" % index)
    return len(probs)


def grad_norm_batched(probs, norm, scale=None, max_norm=1.0, ws=None, stream=None):
    """norm = sqrt(sum of squares over the tensors of grad_problems), and scale = 1
    where norm <= max_norm, else max_norm / norm (one-element fp32 tensors)."""
    if not norm.is_cuda:
        raise ValueError("norm must be a CUDA tensor")
    dev = norm.get_device()
    _flat(norm, 1, torch.float32, dev, "norm")
    if scale is not None:
        _flat(scale, 1, torch.float32, dev, "scale")
    n = _problems_on(probs, dev)
    handle = _stream_on(stream, dev)
    ws_at, nbytes, lent = _borrow(OP_GRAD_NORM, n, 0, dev, handle, ws)
    try:
        _launch(dev, "sketch_grad_norm_batched", n, probs, max_norm, norm.data_ptr(), _addr(scale), ws_at, nbytes, handle)
    finally:
        if lent is not None:
            _take_back(lent)
    return norm


def grad_scale_batched(probs, scale, stream=None):
    """out = G * scale for the tensors of grad_problems; scale: a one-element fp32 tensor."""
    if not scale.is_cuda:
        raise ValueError("scale must be a CUDA tensor")
    if getattr(probs, "written_twice", False):
        raise ValueError("a tensor that is written overlaps another one of the table")
    dev = scale.get_device()
    _flat(scale, 1, torch.float32, dev, "scale")
    _launch(dev, "sketch_grad_scale_batched", _problems_on(probs, dev), probs, scale.data_ptr(), _stream_on(stream, dev))
