"""Python binding of libgdn_gb300.so, the sm_103a gated delta-rule library.

Argument marshalling only: each function checks that the torch tensors it is
given are contiguous fp32 CUDA tensors of the sizes the C call will touch,
derives the shape, and calls the C entry point of the same name on the
current (or given) CUDA stream.  Every step of the computation runs in the
library's CUDA kernels; there is no other implementation behind these
functions, and importing them fails loudly when the library is not built.

Layouts (see include/gdn.h):
    S [B][vh][kd][vd];  q, k [B][T][kh][kd];  v, o [B][T][vh][vd];
    g, beta [B][T][vh];  ckpt [M][B][vh][kd][vd].
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import _build

__all__ = [
    "GDNError", "gdn_step", "gdn_step_m", "gdn_mark", "gdn_rollback",
    "gdn_rollback_seq", "gdn_prefill_workspace", "gdn_prefill",
    "gdn_strerror", "gdn_version", "library_path", "load",
    "GDN_PREC_FP32", "GDN_PREC_BF16X3", "GDN_PREC_BF16", "GDN_MAX_TOKENS",
    "gdn_prefill_timeouts", "gdn_layer_prologue_m", "gdn_layer_workspace",
    "gdn_layer_step_m", "gdn_layer_hist_rollback",
    "gdn_layer_step_m_noalloc", "GDN_NOALLOC_SCRATCH_BYTES",
    "gdn_gated_rmsnorm_m", "gdn_linattn_step", "gdn_linattn_step_m",
    "gdn_linattn_prefill_workspace", "gdn_linattn_prefill",
    "gdn_quant_linear", "KVCache", "Rope", "gdn_rope_freqs", "gdn_rope_m",
    "gdn_kv_write_m", "gdn_kv_read", "gdn_attn_workspace", "gdn_attn_step_m",
]

GDN_OK, GDN_EINVAL, GDN_ESHAPE, GDN_EALIGN = 0, -1, -2, -3
GDN_ECUDA, GDN_ERANGE, GDN_EPTR, GDN_EALIAS = -4, -5, -6, -7
GDN_ESCRATCH = -8
GDN_PREC_FP32, GDN_PREC_BF16X3, GDN_PREC_BF16 = 0, 1, 2
GDN_MAX_TOKENS = 1 << 20
GDN_NOALLOC_SCRATCH_BYTES = 16 << 20
GDN_F32, GDN_BF16 = 0, 1
GDN_DECAY_TOKEN, GDN_DECAY_HEAD = 0, 1
GDN_QUANT_MAX_DIM = 1 << 20
GDN_KV_BF16, GDN_KV_INT8, GDN_KV_E4M3 = 0, 1, 2
GDN_KV_MAX_HEADS, GDN_KV_MAX_POSITIONS = 4096, 1 << 30
GDN_ATTN_MAX_TOKENS, GDN_ATTN_MAX_SCALE = 64, 2.3e38
GDN_ROPE_HALF, GDN_ROPE_PAIRS = 0, 1
GDN_ROPE_PLAIN, GDN_ROPE_LINEAR, GDN_ROPE_NTK, GDN_ROPE_BAND = 0, 1, 2, 3
_KINDS = {torch.bfloat16: GDN_KV_BF16, torch.int8: GDN_KV_INT8,
          torch.float8_e4m3fn: GDN_KV_E4M3}
_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}

# Every symbol include/gdn.h declares.
EXPORTS = ("gdn_step", "gdn_step_m", "gdn_mark", "gdn_rollback",
           "gdn_rollback_seq", "gdn_prefill_workspace", "gdn_prefill",
           "gdn_prefill_timeouts", "gdn_wait_timeouts", "gdn_layer_prologue_m",
           "gdn_layer_workspace", "gdn_layer_step_m",
           "gdn_layer_hist_rollback", "gdn_gated_rmsnorm_m",
           "gdn_layer_step_m_noalloc", "gdn_linattn_step",
           "gdn_linattn_step_m", "gdn_linattn_prefill_workspace",
           "gdn_linattn_prefill", "gdn_quant_linear", "gdn_rope_freqs",
           "gdn_rope_m", "gdn_kv_write_m", "gdn_kv_read",
           "gdn_attn_workspace", "gdn_attn_step_m", "gdn_strerror",
           "gdn_version")


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gdn_strerror(status)} (status {status})")


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("kh", ctypes.c_int),
                ("vh", ctypes.c_int), ("kd", ctypes.c_int),
                ("vd", ctypes.c_int)]


class _Cache(ctypes.Structure):
    _fields_ = [(x, ctypes.c_void_p) for x in ("k", "v", "k_scale", "v_scale")] + \
        [(x, ctypes.c_int) for x in ("kind", "pages", "kvh", "page", "hd")]


class _Rope(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("rot", ctypes.c_int),
                ("layout", ctypes.c_int), ("amp", ctypes.c_float)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load():
    """Load libgdn_gb300.so (built by ``_build.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        raise ImportError(
            f"{_build.LIB} is not built; run __graft_entry__.build() "
            "(or python -m gated_deltanet_linear_gb300._build)")
    lib = ctypes.CDLL(_build.LIB)
    vp, ip, cp = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(Shape)
    sig = {
        "gdn_step": [cp] + [vp] * 7 + [vp],
        "gdn_step_m": [cp, ip] + [vp] * 9 + [vp],
        "gdn_mark": [cp, vp, vp, vp],
        "gdn_rollback": [cp, ip, ip, vp, vp, vp, vp],
        "gdn_rollback_seq": [cp, ip, vp, vp, vp, vp, vp, vp],
        "gdn_prefill": [cp, ip] + [vp] * 7 + [ip, ip, vp, ctypes.c_size_t, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.gdn_prefill_workspace.argtypes = [cp, ip, ip, ip]
    lib.gdn_prefill_workspace.restype = ctypes.c_size_t
    lib.gdn_layer_prologue_m.argtypes = [cp, ip, ip, ctypes.c_float] + [vp] * 14
    lib.gdn_layer_prologue_m.restype = ctypes.c_int
    lib.gdn_layer_workspace.argtypes = [cp, ip]
    lib.gdn_layer_workspace.restype = ctypes.c_size_t
    lib.gdn_layer_step_m.argtypes = [cp, ip, ip, ctypes.c_float] + [vp] * 13 + \
        [ctypes.c_size_t, vp]
    lib.gdn_layer_step_m.restype = ctypes.c_int
    lib.gdn_gated_rmsnorm_m.argtypes = [cp, ip, ctypes.c_float] + [vp] * 5
    lib.gdn_gated_rmsnorm_m.restype = ctypes.c_int
    lib.gdn_layer_step_m_noalloc.argtypes = [cp, ip, ip, ctypes.c_float] + \
        [vp] * 12 + [vp]
    lib.gdn_layer_step_m_noalloc.restype = ctypes.c_int
    lib.gdn_layer_hist_rollback.argtypes = [cp, ip, ip] + [vp] * 6
    lib.gdn_layer_hist_rollback.restype = ctypes.c_int
    fp, sz = ctypes.c_float, ctypes.c_size_t
    lib.gdn_linattn_step.argtypes = [cp, ip, ip, fp] + [vp] * 7
    lib.gdn_linattn_step.restype = ctypes.c_int
    lib.gdn_linattn_step_m.argtypes = [cp, ip, ip, ip, fp] + [vp] * 9
    lib.gdn_linattn_step_m.restype = ctypes.c_int
    lib.gdn_linattn_prefill_workspace.argtypes = [cp, ip, ip]
    lib.gdn_linattn_prefill_workspace.restype = sz
    lib.gdn_linattn_prefill.argtypes = [cp, ip, ip, ip, fp] + [vp] * 9 + [sz, vp]
    lib.gdn_linattn_prefill.restype = ctypes.c_int
    lib.gdn_quant_linear.argtypes = [ip] * 5 + [vp] * 5
    lib.gdn_quant_linear.restype = ctypes.c_int
    dp, kv = ctypes.c_double, ctypes.POINTER(_Cache)
    rp, ll = ctypes.POINTER(_Rope), ctypes.c_longlong
    lib.gdn_rope_freqs.argtypes = [ip, dp, ip, dp, dp, dp, dp,
                                   ctypes.POINTER(ctypes.c_double), ctypes.POINTER(fp)]
    lib.gdn_rope_freqs.restype = ctypes.c_int
    lib.gdn_rope_m.argtypes = [ip, ip, ip, ip, rp, vp, ll, vp, vp, vp]
    lib.gdn_rope_m.restype = ctypes.c_int
    lib.gdn_kv_write_m.argtypes = [kv, ip, ip, ip, ip, rp, vp, ll, vp, ll, vp,
                                   ll, vp, vp, ip, vp, vp, vp, vp]
    lib.gdn_kv_write_m.restype = ctypes.c_int
    lib.gdn_kv_read.argtypes = [kv, ip, ip, ip, vp, ip, vp, vp, vp, vp, vp, vp]
    lib.gdn_kv_read.restype = ctypes.c_int
    lib.gdn_attn_workspace.argtypes = [kv, ip, ip]
    lib.gdn_attn_workspace.restype = sz
    lib.gdn_attn_step_m.argtypes = [kv, ip, ip, ip, ip, fp, vp, vp, ip, vp, vp,
                                    vp, vp, vp, vp, sz, vp]
    lib.gdn_attn_step_m.restype = ctypes.c_int
    lib.gdn_prefill_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.gdn_prefill_timeouts.restype = ctypes.c_int
    lib.gdn_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.gdn_wait_timeouts.restype = ctypes.c_int
    lib.gdn_strerror.argtypes = [ctypes.c_int]
    lib.gdn_strerror.restype = ctypes.c_char_p
    lib.gdn_version.restype = ctypes.c_int
    _lib = lib
    return lib


def gdn_strerror(status: int) -> str:
    return load().gdn_strerror(int(status)).decode()


def gdn_version() -> int:
    return load().gdn_version()


# The current stream's handle without the Stream object around it (0.3 us a
# call instead of 2.9 us on a GB300 host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _t(x, name, numel):
    """Pointer of a contiguous fp32 CUDA tensor with exactly numel elements."""
    if x is None:
        return None
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    if x.numel() != numel:
        raise ValueError(f"{name} has {x.numel()} elements, expected {numel}")
    return x.data_ptr()


def _io(x, name, numel):
    """Pointer of a token input or output: a contiguous fp32 CUDA tensor, or a
    page-locked (pinned) CPU tensor, which the kernels read or write over the
    host link."""
    if isinstance(x, torch.Tensor) and not x.is_cuda:
        if not x.is_pinned():
            raise ValueError(f"{name}: a CPU tensor must be pinned "
                             "(tensor.pin_memory())")
        if x.dtype != torch.float32 or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor")
        if x.numel() != numel:
            raise ValueError(f"{name} has {x.numel()} elements, expected {numel}")
        return x.data_ptr()
    return _t(x, name, numel)


def _shape(S, q):
    if S.dim() != 4:
        raise ValueError("S must be [B][vh][kd][vd]")
    B, vh, kd, vd = S.shape
    kh = q.shape[-2]
    return Shape(B, kh, vh, kd, vd)


def _check(status, where):
    if status != GDN_OK:
        raise GDNError(status, where)


def gdn_step(S, q, k, v, g, beta, o, stream=None):
    """One token for all heads; S is updated in place, o written.  The token
    tensors (q, k, v, g, beta, o) may be CUDA tensors or pinned CPU tensors."""
    sh = _shape(S, q)
    B, kh, vh, kd, vd = sh.B, sh.kh, sh.vh, sh.kd, sh.vd
    args = (_t(S, "S", B * vh * kd * vd), _io(q, "q", B * kh * kd),
            _io(k, "k", B * kh * kd), _io(v, "v", B * vh * vd),
            _io(g, "g", B * vh), _io(beta, "beta", B * vh),
            _io(o, "o", B * vh * vd))
    _check(load().gdn_step(ctypes.byref(sh), *args, _stream(stream)),
           "gdn_step")


def gdn_step_m(S_in, S_out, ckpt, q, k, v, g, beta, o, M=None, stream=None):
    """M tokens in one launch (M defaults to q.shape[1]).  The token tensors
    may be CUDA tensors or pinned CPU tensors, as for gdn_step."""
    sh = _shape(S_in, q)
    B, kh, vh, kd, vd = sh.B, sh.kh, sh.vh, sh.kd, sh.vd
    M = int(q.shape[1] if M is None else M)
    n = B * vh * kd * vd
    args = (_t(S_in, "S_in", n), _t(S_out, "S_out", n),
            _t(ckpt, "ckpt", M * n), _io(q, "q", B * M * kh * kd),
            _io(k, "k", B * M * kh * kd), _io(v, "v", B * M * vh * vd),
            _io(g, "g", B * M * vh), _io(beta, "beta", B * M * vh),
            _io(o, "o", B * M * vh * vd))
    _check(load().gdn_step_m(ctypes.byref(sh), M, *args, _stream(stream)),
           "gdn_step_m")


def gdn_mark(S, snap, kh, stream=None):
    """snap = S (device copy on the stream)."""
    B, vh, kd, vd = S.shape
    sh = Shape(B, kh, vh, kd, vd)
    n = B * vh * kd * vd
    _check(load().gdn_mark(ctypes.byref(sh), _t(S, "S", n),
                           _t(snap, "snap", n), _stream(stream)), "gdn_mark")


def gdn_rollback(S, M, m, snap, ckpt, kh, stream=None):
    """S = snap (m == 0) or ckpt[m-1] (1 <= m <= M)."""
    B, vh, kd, vd = S.shape
    sh = Shape(B, kh, vh, kd, vd)
    n = B * vh * kd * vd
    _check(load().gdn_rollback(ctypes.byref(sh), int(M), int(m),
                               _t(snap, "snap", n),
                               _t(ckpt, "ckpt", int(M) * n),
                               _t(S, "S", n), _stream(stream)), "gdn_rollback")


def gdn_rollback_seq(S, M, m_dev, snap, ckpt, kh, err_dev=None, stream=None):
    """Per-sequence rollback; m_dev is an int32 CUDA tensor [B]."""
    B, vh, kd, vd = S.shape
    sh = Shape(B, kh, vh, kd, vd)
    n = B * vh * kd * vd
    for x, name, cnt in ((m_dev, "m_dev", B), (err_dev, "err_dev", 1)):
        if x is not None and (not x.is_cuda or x.dtype != torch.int32 or
                              not x.is_contiguous() or x.numel() != cnt):
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor "
                             f"of {cnt} elements")
    _check(load().gdn_rollback_seq(
        ctypes.byref(sh), int(M), m_dev.data_ptr(), _t(snap, "snap", n),
        _t(ckpt, "ckpt", int(M) * n), _t(S, "S", n),
        None if err_dev is None else err_dev.data_ptr(), _stream(stream)),
        "gdn_rollback_seq")


def gdn_prefill_workspace(B, kh, vh, T, chunk=64, precision=GDN_PREC_FP32,
                          kd=128, vd=128):
    sh = Shape(B, kh, vh, kd, vd)
    return int(load().gdn_prefill_workspace(ctypes.byref(sh), int(T),
                                            int(chunk), int(precision)))


def gdn_prefill_timeouts():
    """Chunked-prefill CTAs that gave up waiting on the tensor cores (0)."""
    c = ctypes.c_uint(0)
    _check(load().gdn_prefill_timeouts(ctypes.byref(c)), "gdn_prefill_timeouts")
    return int(c.value)


def gdn_wait_timeouts():
    """Bounded waits that ran out in any kernel since the library was loaded
    on the current device (synchronises the device)."""
    n = ctypes.c_uint(0)
    _check(load().gdn_wait_timeouts(ctypes.byref(n)), "gdn_wait_timeouts")
    return int(n.value)


def gdn_prefill(S, q, k, v, g, beta, o, precision=GDN_PREC_FP32, chunk=64,
                workspace=None, stream=None):
    """T = q.shape[1] tokens; S updated in place (S_0 -> S_T).

    precision: GDN_PREC_FP32 (token-serial, exact to the single-step path),
    GDN_PREC_BF16X3 or GDN_PREC_BF16 (chunk-parallel on tensor cores)."""
    sh = _shape(S, q)
    B, kh, vh, kd, vd = sh.B, sh.kh, sh.vh, sh.kd, sh.vd
    T = int(q.shape[1])
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_ptr = workspace.data_ptr()
        ws_bytes = workspace.numel() * workspace.element_size()
    args = (_t(S, "S", B * vh * kd * vd), _t(q, "q", B * T * kh * kd),
            _t(k, "k", B * T * kh * kd), _t(v, "v", B * T * vh * vd),
            _t(g, "g", B * T * vh), _t(beta, "beta", B * T * vh),
            _t(o, "o", B * T * vh * vd))
    _check(load().gdn_prefill(ctypes.byref(sh), T, *args, int(chunk),
                              int(precision), ws_ptr, ws_bytes,
                              _stream(stream)), "gdn_prefill")


def _layer_shape(hist, x, kh, vh=None, kd=128, vd=128):
    B, ck1, conv_dim = hist.shape
    vh = (conv_dim - 2 * int(kh) * kd) // vd if vh is None else vh
    return Shape(B, int(kh), vh, kd, vd), int(x.shape[1]), ck1 + 1, conv_dim


def gdn_layer_prologue_m(hist_in, hist_out, x, conv_w, a, b, A_log, dt_bias,
                         q, k, v, g, beta, kh, eps=1e-6, stream=None):
    """conv1d + SiLU with history, q/k norm and gates for M = x.shape[1]
    tokens, writing q, k, v, g, beta (the inputs of gdn_step_m)."""
    sh, M, ck, conv_dim = _layer_shape(hist_in, x, kh)
    B, vh = sh.B, sh.vh
    nh = B * (ck - 1) * conv_dim
    args = (_t(hist_in, "hist_in", nh), _t(hist_out, "hist_out", nh),
            _t(x, "x", B * M * conv_dim), _t(conv_w, "conv_w", conv_dim * ck),
            _t(a, "a", B * M * vh), _t(b, "b", B * M * vh),
            _t(A_log, "A_log", vh), _t(dt_bias, "dt_bias", vh),
            _t(q, "q", B * M * sh.kh * 128), _t(k, "k", B * M * sh.kh * 128),
            _t(v, "v", B * M * vh * 128), _t(g, "g", B * M * vh),
            _t(beta, "beta", B * M * vh))
    _check(load().gdn_layer_prologue_m(ctypes.byref(sh), M, ck, float(eps),
                                       *args, _stream(stream)),
           "gdn_layer_prologue_m")


def gdn_layer_workspace(B, kh, vh, M, kd=128, vd=128):
    sh = Shape(B, kh, vh, kd, vd)
    return int(load().gdn_layer_workspace(ctypes.byref(sh), int(M)))


def gdn_layer_step_m(S_in, S_out, ckpt, hist_in, hist_out, x, conv_w, a, b,
                     A_log, dt_bias, o, kh, workspace, eps=1e-6, stream=None):
    """Layer prologue + update over M = x.shape[1] tokens; the intermediate
    q, k, v, g, beta live in `workspace` (gdn_layer_workspace bytes)."""
    if S_in.dim() != 4:
        raise ValueError("S must be [B][vh][kd][vd]")
    B, vh, kd, vd = S_in.shape
    sh = Shape(B, int(kh), vh, kd, vd)
    M = int(x.shape[1])
    ck = int(conv_w.shape[1])
    conv_dim = 2 * int(kh) * kd + vh * vd
    n = B * vh * kd * vd
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    args = (_t(S_in, "S_in", n), _t(S_out, "S_out", n),
            _t(ckpt, "ckpt", M * n),
            _t(hist_in, "hist_in", B * (ck - 1) * conv_dim),
            _t(hist_out, "hist_out", B * (ck - 1) * conv_dim),
            _t(x, "x", B * M * conv_dim), _t(conv_w, "conv_w", conv_dim * ck),
            _t(a, "a", B * M * vh), _t(b, "b", B * M * vh),
            _t(A_log, "A_log", vh), _t(dt_bias, "dt_bias", vh),
            _t(o, "o", B * M * vh * vd))
    _check(load().gdn_layer_step_m(
        ctypes.byref(sh), M, ck, float(eps), *args, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "gdn_layer_step_m")


def gdn_gated_rmsnorm_m(o, z, w, y, eps=1e-6, stream=None):
    """Gated RMSNorm of o [B][M][vh][vd] with gate z (same shape) and
    per-channel weight w [vd] into y (y may be o)."""
    if o.dim() != 4:
        raise ValueError("o must be [B][M][vh][vd]")
    B, M, vh, vd = o.shape
    sh = Shape(B, 1, vh, 128, vd)
    n = o.numel()
    _check(load().gdn_gated_rmsnorm_m(
        ctypes.byref(sh), M, float(eps), _t(o, "o", n), _t(z, "z", n),
        _t(w, "w", vd), _t(y, "y", n), _stream(stream)),
        "gdn_gated_rmsnorm_m")


def gdn_layer_step_m_noalloc(S_in, S_out, ckpt, hist_in, hist_out, x, conv_w,
                             a, b, A_log, dt_bias, o, kh, eps=1e-6,
                             stream=None):
    """gdn_layer_step_m for callers that cannot allocate device memory: the
    intermediate q, k, v, g, beta go to the library's own static scratch of
    GDN_NOALLOC_SCRATCH_BYTES (shared by every call on the device; calls that
    overlap on the GPU race).  Larger requests raise GDNError with
    GDN_ESCRATCH."""
    if S_in.dim() != 4:
        raise ValueError("S must be [B][vh][kd][vd]")
    B, vh, kd, vd = S_in.shape
    sh = Shape(B, int(kh), vh, kd, vd)
    M = int(x.shape[1])
    ck = int(conv_w.shape[1])
    conv_dim = 2 * int(kh) * kd + vh * vd
    n = B * vh * kd * vd
    args = (_t(S_in, "S_in", n), _t(S_out, "S_out", n),
            _t(ckpt, "ckpt", M * n),
            _t(hist_in, "hist_in", B * (ck - 1) * conv_dim),
            _t(hist_out, "hist_out", B * (ck - 1) * conv_dim),
            _t(x, "x", B * M * conv_dim), _t(conv_w, "conv_w", conv_dim * ck),
            _t(a, "a", B * M * vh), _t(b, "b", B * M * vh),
            _t(A_log, "A_log", vh), _t(dt_bias, "dt_bias", vh),
            _t(o, "o", B * M * vh * vd))
    _check(load().gdn_layer_step_m_noalloc(
        ctypes.byref(sh), M, ck, float(eps), *args, _stream(stream)),
        "gdn_layer_step_m_noalloc")


def gdn_layer_hist_rollback(hist, M, m_dev, hist_snap, x, kh, kd=128, vd=128,
                            err_dev=None, stream=None):
    """Conv history after m_dev[b] of the M tokens of a layer launch."""
    B, ck1, conv_dim = hist.shape
    vh = (conv_dim - 2 * int(kh) * kd) // vd
    sh = Shape(B, int(kh), vh, kd, vd)
    for t_, name, cnt in ((m_dev, "m_dev", B), (err_dev, "err_dev", 1)):
        if t_ is not None and (not t_.is_cuda or t_.dtype != torch.int32 or
                               not t_.is_contiguous() or t_.numel() != cnt):
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor "
                             f"of {cnt} elements")
    _check(load().gdn_layer_hist_rollback(
        ctypes.byref(sh), int(M), ck1 + 1, m_dev.data_ptr(),
        _t(hist_snap, "hist_snap", hist.numel()),
        _t(x, "x", B * int(M) * conv_dim), _t(hist, "hist", hist.numel()),
        None if err_dev is None else err_dev.data_ptr(), _stream(stream)),
        "gdn_layer_hist_rollback")


# The C structure of a shape, made once for each (0.3 us).
_shape5 = functools.lru_cache(maxsize=64)(Shape)


def _tok(x, name, shape, dtype):
    """Pointer of a contiguous CUDA tensor of this shape and type.  (On the path
    of every call below: one comparison each, the messages out of the way.)"""
    try:
        if x.is_cuda and x.dtype is dtype and x.shape == shape and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        pass
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype != dtype or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {tuple(shape)}")


def _linattn(S, q, k, v, g, o, M):
    """Shape, element type, decay mode and pointers (q, k, v, g, o) of a
    linear-attention call; M None: one token without a token dimension."""
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("S must be [B][vh][kd][vd]")
    B, vh, kd, vd = S.shape
    qs = q.shape
    dtype = q.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("q, k, v, o must be float32 or bfloat16")
    if len(qs) < 2:
        raise ValueError("q must be [B][T][kh][kd]")
    kh = qs[-2]
    if M is None:
        lead = tuple(qs[:-2])
        if lead != (B,) and lead != (B, 1):
            raise ValueError(f"q has shape {tuple(qs)}: one token for each of "
                             f"{B} sequences expected")
    else:
        lead = (B, M)
    qk, vo = lead + (kh, kd), lead + (vh, vd)
    head = g.dim() == 1
    return (_shape5(B, kh, vh, kd, vd), code,
            GDN_DECAY_HEAD if head else GDN_DECAY_TOKEN,
            _tok(q, "q", qk, dtype), _tok(k, "k", qk, dtype),
            _tok(v, "v", vo, dtype),
            _tok(g, "g", (vh,) if head else lead + (vh,), torch.float32),
            _tok(o, "o", vo, dtype))


def gdn_linattn_step(S, q, k, v, g, o, scale=1.0, stream=None):
    """One token of linear attention with a decay for each head: S = exp(g) S
    + k v^T in place, o = scale S^T q.  q, k [B][kh][kd] (or [B][1][kh][kd]),
    v, o likewise with vh, all float32 or all bfloat16; g per token [B][vh]
    (or [B][1][vh]) or per head [vh]."""
    sh, dtype, decay, *ptrs = _linattn(S, q, k, v, g, o, None)
    r = (_lib or load()).gdn_linattn_step(
        ctypes.byref(sh), dtype, decay, scale,
        _tok(S, "S", S.shape, torch.float32), *ptrs, _stream(stream))
    if r:
        raise GDNError(r, "gdn_linattn_step")


def gdn_linattn_step_m(S_in, S_out, ckpt, q, k, v, g, o, scale=1.0,
                       stream=None):
    """M = q.shape[1] tokens of gdn_linattn_step in one launch; S_out may be
    S_in; ckpt [M][B][vh][kd][vd] or None receives the state after each
    token."""
    if q.dim() != 4:
        raise ValueError("q must be [B][M][kh][kd]")
    M = q.shape[1]
    sh, dtype, decay, *ptrs = _linattn(S_in, q, k, v, g, o, M)
    f32, ss = torch.float32, S_in.shape
    sp = _tok(S_in, "S_in", ss, f32)
    r = (_lib or load()).gdn_linattn_step_m(
        ctypes.byref(sh), M, dtype, decay, scale, sp,
        sp if S_out is S_in else _tok(S_out, "S_out", ss, f32),
        None if ckpt is None else _tok(ckpt, "ckpt", (M, *ss), f32), *ptrs,
        _stream(stream))
    if r:
        raise GDNError(r, "gdn_linattn_step_m")


def gdn_linattn_prefill_workspace(B, kh, vh, T, dtype=torch.float32, kd=128,
                                  vd=128):
    """Bytes of workspace gdn_linattn_prefill needs for this shape."""
    sh = Shape(B, kh, vh, kd, vd)
    return int(load().gdn_linattn_prefill_workspace(ctypes.byref(sh), int(T),
                                                    _DTYPES[dtype]))


def gdn_linattn_prefill(S, q, k, v, g, o, scale=1.0, lens=None, err_dev=None,
                        workspace=None, stream=None):
    """Prompts of T = q.shape[1] tokens, S updated in place.  lens (int32 CUDA
    tensor [B]): the first lens[b] rows of sequence b count; its other rows
    of o keep what they held.  A length outside 0..T leaves the sequence as it
    was and sets err_dev (int32 CUDA tensor of one element)."""
    if q.dim() != 4:
        raise ValueError("q must be [B][T][kh][kd]")
    T = q.shape[1]
    sh, dtype, decay, *ptrs = _linattn(S, q, k, v, g, o, T)
    lens_ptr = None if lens is None else _tok(lens, "lens", (sh.B,), torch.int32)
    err_ptr = None if err_dev is None else _tok(err_dev, "err_dev", (1,), torch.int32)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.nbytes
    r = (_lib or load()).gdn_linattn_prefill(
        ctypes.byref(sh), T, dtype, decay, scale,
        _tok(S, "S", S.shape, torch.float32), *ptrs, lens_ptr, err_ptr, ws_ptr,
        ws_bytes, _stream(stream))
    if r:
        raise GDNError(r, "gdn_linattn_prefill")


def gdn_quant_linear(x, qw, scales, y, stream=None):
    """y = x W^T with 4-bit weights: x [rows][K] and y [rows][N] float32 or
    bfloat16, qw uint8 [N][K/2] (element 2j in the low half of byte j, two's
    complement), scales float16 [N][K/group], group 32, 64 or 128."""
    xs, ss, dtype = x.shape, scales.shape, x.dtype
    if len(xs) != 2 or len(ss) != 2:
        raise ValueError("x and scales must have two dimensions")
    rows, K = xs
    N, groups = ss
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("x and y must be float32 or bfloat16")
    if groups < 1 or K % groups:
        raise ValueError(f"{groups} scales for a row of {K} elements")
    r = (_lib or load()).gdn_quant_linear(
        rows, N, K, K // groups, code, _tok(x, "x", xs, dtype),
        _tok(qw, "qw", (N, K // 2), torch.uint8),
        _tok(scales, "scales", ss, torch.float16),
        _tok(y, "y", (rows, N), dtype), _stream(stream))
    if r:
        raise GDNError(r, "gdn_quant_linear")


class KVCache:
    """A paged key-value cache: k, v [pages][kvh][page][hd] bfloat16, int8 or
    float8_e4m3fn; the 8-bit types with k_scale, v_scale float32
    [pages][kvh][page].  It refers to the tensors, which stay the caller's."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "kind", "shape", "c", "ref")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be [pages][kvh][page][hd]")
        self.kind = _KINDS.get(k.dtype)
        if self.kind is None:
            raise ValueError("k and v must be bfloat16, int8 or float8_e4m3fn")
        if (self.kind == GDN_KV_BF16) != (k_scale is None) or \
                (self.kind == GDN_KV_BF16) != (v_scale is None):
            raise ValueError("8-bit caches have scales, bfloat16 caches none")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.shape = pages, kvh, page, hd = tuple(k.shape)
        ptrs = [_tok(k, "k", k.shape, k.dtype), _tok(v, "v", k.shape, k.dtype), None, None]
        if k_scale is not None:
            ptrs[2] = _tok(k_scale, "k_scale", k.shape[:3], torch.float32)
            ptrs[3] = _tok(v_scale, "v_scale", k.shape[:3], torch.float32)
        self.c = _Cache(*ptrs, self.kind, pages, kvh, page, hd)
        self.ref = ctypes.byref(self.c)


class Rope:
    """Rotary positions: freq float64 [rot / 2] radians a position (CUDA), the
    layout of the pairs, the amplitude (see gdn_rope_freqs)."""

    __slots__ = ("freq", "rot", "layout", "amp", "c", "ref")

    def __init__(self, freq, layout=GDN_ROPE_HALF, amp=1.0):
        if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
            raise ValueError("freq must be [rot / 2]")
        ptr = _tok(freq, "freq", freq.shape, torch.float64)
        self.freq, self.rot, self.layout, self.amp = freq, 2 * freq.numel(), layout, amp
        self.c = _Rope(ptr, self.rot, layout, amp)
        self.ref = ctypes.byref(self.c)


def gdn_rope_freqs(rot, base=10000.0, scaling=GDN_ROPE_PLAIN, factor=1.0,
                   context=0.0, low=1.0, high=32.0, device="cuda"):
    """(freq, amp) for Rope: float64 [rot / 2] on the device, computed on the
    host, and the amplitude."""
    freq = torch.empty(max(0, int(rot) // 2), dtype=torch.float64)
    amp = ctypes.c_float(1.0)
    r = (_lib or load()).gdn_rope_freqs(
        rot, base, scaling, factor, context, low, high,
        ctypes.cast(freq.data_ptr(), ctypes.POINTER(ctypes.c_double)), ctypes.byref(amp))
    if r:
        raise GDNError(r, "gdn_rope_freqs")
    return freq.to(device), amp.value


def _rows(x, name, shape):
    """Stride from token to token of x, of this shape [B][M][heads][hd] or
    [rows][heads][hd]: heads and channels contiguous, tokens evenly spaced (the
    rows of a projection).  (On the path of every call; that x is device memory
    the library checks.)"""
    st = x.stride()
    heads, hd = shape[-2:]
    if st[-1] == 1 and (st[-2] == hd or heads == 1):
        if len(shape) == 3:
            return st[0] if shape[0] > 1 else heads * hd
        B, M = shape[:2]
        if M == 1:
            return st[0] if B > 1 else heads * hd
        if B <= 1 or st[0] == M * st[1]:
            return st[1]
    if not x.numel():
        return heads * hd
    raise ValueError(f"{name}: heads and channels must be contiguous, tokens evenly spaced")


def _same(x, name, shape, dtype):
    """Pointer of a contiguous tensor of this shape and type (device memory or
    not is the library's to say)."""
    try:
        if x.dtype is dtype and x.shape == shape and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        pass
    return _tok(x, name, shape, dtype)


def _code(dtype):
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("tokens must be float32 or bfloat16")
    return code


def _ints(x, name, shape):
    return None if x is None else _same(x, name, shape, torch.int32)


def gdn_rope_m(x, pos, rope, y, stream=None):
    """y = x turned to positions pos: x, y [rows][heads][hd] float32 or
    bfloat16 (x may have a stride from row to row; y may be x), pos int32
    [rows]."""
    shape, dtype = x.shape, x.dtype
    if len(shape) != 3:
        raise ValueError("x must be [rows][heads][hd]")
    rows, heads, hd = shape
    r = (_lib or load()).gdn_rope_m(
        rows, heads, hd, _code(dtype), rope.ref, x.data_ptr(), _rows(x, "x", shape),
        _ints(pos, "pos", (rows,)), _same(y, "y", shape, dtype), _stream(stream))
    if r:
        raise GDNError(r, "gdn_rope_m")


def _paged(cache, B, table, start, counts, err_dev):
    """Pointers of table, start, counts, err_dev and the table's columns."""
    ts = table.shape
    if len(ts) != 2 or ts[0] != B or table.dtype is not torch.int32 or \
            not table.is_contiguous():
        raise ValueError(f"table must be a contiguous int32 tensor [{B}][columns]")
    one = (B,)
    return (table.data_ptr(), ts[1],
            None if start is None else _same(start, "start", one, torch.int32),
            None if counts is None else _same(counts, "counts", one, torch.int32),
            None if err_dev is None else _same(err_dev, "err_dev", (1,), torch.int32))


def gdn_kv_write_m(cache, k, v, table, start, rope=None, q=None, q_out=None,
                   counts=None, err_dev=None, stream=None):
    """The keys and values k, v [B][M][kvh][hd] of M tokens of every sequence
    to positions start[b] + m of their pages; rope turns k on the way, and q
    [B][M][qh][hd] into q_out.  q, k, v may be slices of one projection."""
    _, kvh, _, hd = cache.shape
    shape, dtype = k.shape, k.dtype
    if len(shape) != 4 or shape[2] != kvh or shape[3] != hd or v.shape != shape or \
            v.dtype is not dtype:
        raise ValueError(f"k and v must be [B][M][{kvh}][{hd}] of one type")
    B, M = shape[:2]
    qp = qo = None
    qs = qh = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        qshape = q.shape
        qh = qshape[2] if len(qshape) == 4 else 0
        if qshape != (B, M, qh, hd) or q.dtype is not dtype:
            raise ValueError(f"q must be [B][M][qh][{hd}] of the type of k")
        qp, qs = q.data_ptr(), _rows(q, "q", qshape)
        qo = _same(q_out, "q_out", qshape, dtype)
    tp, cols, sp, cp, ep = _paged(cache, B, table, start, counts, err_dev)
    r = (_lib or load()).gdn_kv_write_m(
        cache.ref, B, M, qh, _code(dtype),
        None if rope is None else rope.ref, qp, qs, k.data_ptr(), _rows(k, "k", shape),
        v.data_ptr(), _rows(v, "v", shape), qo,
        tp, cols, sp, cp, ep, _stream(stream))
    if r:
        raise GDNError(r, "gdn_kv_write_m")


def gdn_kv_read(cache, table, start, k, v, counts=None, err_dev=None,
                stream=None):
    """Positions start[b] .. start[b] + T - 1 (start None: from 0) of every
    sequence into k, v [B][T][kvh][hd], float32 or bfloat16."""
    shape, dtype = k.shape, k.dtype
    if len(shape) != 4 or shape[2] != cache.shape[1] or shape[3] != cache.shape[3]:
        raise ValueError("k must be [B][T][kvh][hd]")
    B, T = shape[:2]
    tp, cols, sp, cp, ep = _paged(cache, B, table, start, counts, err_dev)
    r = (_lib or load()).gdn_kv_read(
        cache.ref, B, T, _code(dtype), tp, cols, sp, cp,
        _same(k, "k", shape, dtype), _same(v, "v", shape, dtype), ep,
        _stream(stream))
    if r:
        raise GDNError(r, "gdn_kv_read")


def gdn_attn_workspace(cache, M, qh):
    """Bytes of workspace gdn_attn_step_m needs."""
    return int((_lib or load()).gdn_attn_workspace(cache.ref, M, qh))


def gdn_attn_step_m(cache, q, table, start, o, scale=None, counts=None,
                    lse=None, err_dev=None, workspace=None, stream=None):
    """M = q.shape[1] tokens of every sequence against positions 0 ..
    start[b] + m of the cache, their own among them: q, o [B][M][qh][hd]
    float32 or bfloat16, lse float32 [B][M][qh] or None; scale defaults to
    hd^-0.5."""
    qs, dtype = q.shape, q.dtype
    if len(qs) != 4 or qs[3] != cache.shape[3]:
        raise ValueError("q must be [B][M][qh][hd]")
    B, M, qh, hd = qs
    tp, cols, sp, cp, ep = _paged(cache, B, table, start, counts, err_dev)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.nbytes
    r = (_lib or load()).gdn_attn_step_m(
        cache.ref, B, M, qh, _code(dtype),
        hd ** -0.5 if scale is None else scale, _same(q, "q", qs, dtype), tp, cols,
        sp, cp, _same(o, "o", qs, dtype),
        None if lse is None else _same(lse, "lse", qs[:3], torch.float32), ep,
        ws_ptr, ws_bytes, _stream(stream))
    if r:
        raise GDNError(r, "gdn_attn_step_m")
