"""Python binding of ``libsdm.so``, the MI355X (gfx950) Sparse Delta Memory layer forward.

Argument marshalling only: every step of the computation runs in the library's HIP
kernels. Tensors are ``torch`` device tensors (contiguous); the call is enqueued on
``torch.cuda.current_stream()`` unless a stream is given. The names follow the C ABI in
``include/sdm.h`` (``sdm_init_from_M0`` -> :func:`init_from_M0`, ...).

If ``libsdm.so`` has not been built (``python -m sparse_memory_linear_amd.build``), every
call raises :class:`SdmLibraryMissing`; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "SDM_F32", "SDM_BF16", "SdmError", "SdmLibraryMissing", "Shape", "lib", "lib_path",
    "make_shape", "check_shape", "workspace_bytes", "init_from_M0", "address", "recurrent",
    "forward", "forward_static", "STATIC_SCRATCH_BYTES", "forward_uses_chunkwise", "decode_step", "workspace_error", "status_string", "abi_version",
    "decay_state_init", "workspace_bytes_decay", "recurrent_decay", "forward_decay", "decode_step_decay",
    "materialize", "gates", "output_gate", "head_mix", "output_project", "recurrent_log", "recurrent_backward",
    "backward_workspace_bytes", "address_backward", "workspace_bytes_chunked", "recurrent_chunked",
    "SDM_ACT_NONE", "SDM_ACT_SILU", "SDM_ACT_SIGMOID", "ConvShape", "ScanShape", "NormShape",
    "make_conv_shape", "check_conv_shape", "short_conv", "short_conv_step", "short_conv_backward",
    "short_conv_backward_workspace_bytes", "make_scan_shape", "check_scan_shape", "selective_scan",
    "selective_scan_workspace_bytes", "selective_scan_step", "selective_scan_backward",
    "selective_scan_backward_workspace_bytes", "make_norm_shape", "check_norm_shape", "block_norm",
    "block_norm_backward", "block_norm_backward_workspace_bytes",
]

SDM_F32 = 0
SDM_BF16 = 1
SDM_ACT_NONE = 0
SDM_ACT_SILU = 1
SDM_ACT_SIGMOID = 2
STATIC_SCRATCH_BYTES = 64 << 20  # SDM_STATIC_SCRATCH_BYTES of the header

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libsdm.so")


class SdmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


class SdmLibraryMissing(RuntimeError):
    pass


class Shape(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
        ("N", ctypes.c_int64),
        ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
        ("kappa", ctypes.c_int32), ("W", ctypes.c_int32), ("R", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32), ("mem_dtype", ctypes.c_int32),
    ]

    def __repr__(self):
        return type(self).__name__ + "(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class ConvShape(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("C", ctypes.c_int32), ("K", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64),
    ]
    __repr__ = Shape.__repr__


class ScanShape(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("G", ctypes.c_int32),
        ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
        ("ld_x", ctypes.c_int64), ("ld_b", ctypes.c_int64), ("ld_c", ctypes.c_int64), ("ld_dt", ctypes.c_int64),
    ]
    __repr__ = Shape.__repr__


class NormShape(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("D", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("r_dtype", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("gate_act", ctypes.c_int32),
        ("gate_rows", ctypes.c_int64), ("eps", ctypes.c_float), ("scale", ctypes.c_float),
    ]
    __repr__ = Shape.__repr__


_lib = None
_P = ctypes.c_void_p
_SP = ctypes.POINTER(Shape)
_SIGS = {
    "sdm_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sdm_abi_version": (ctypes.c_int, []),
    "sdm_check_shape": (ctypes.c_int, [_SP]),
    "sdm_workspace_bytes": (ctypes.c_size_t, [_SP]),
    "sdm_init_from_M0": (ctypes.c_int, [_SP, _P, _P, _P]),
    "sdm_address": (ctypes.c_int, [_SP, _P, _P, ctypes.c_int32, _P, _P, _P, _P]),
    "sdm_address_init": (ctypes.c_int, [_SP, _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_int32,
                                        ctypes.c_int32, _P]),
    "sdm_recurrent": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "sdm_forward": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "sdm_forward_static": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "sdm_forward_uses_chunkwise": (ctypes.c_int, [_SP]),
    "sdm_decode_step": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "sdm_workspace_error": (ctypes.c_int, [_P, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int64), _P]),
    "sdm_decay_state_init": (ctypes.c_int, [_SP, _P, _P, _P]),
    "sdm_workspace_bytes_decay": (ctypes.c_size_t, [_SP]),
    "sdm_recurrent_decay": (ctypes.c_int, [_SP] + [_P] * 12 + [ctypes.c_size_t, _P]),
    "sdm_forward_decay": (ctypes.c_int, [_SP] + [_P] * 13 + [ctypes.c_size_t, _P]),
    "sdm_decode_step_decay": (ctypes.c_int, [_SP] + [_P] * 11),
    "sdm_materialize": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P]),
    "sdm_gates": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, _P]),
    "sdm_output_gate": (ctypes.c_int, [_SP, _P, _P, _P, ctypes.c_float, _P, _P]),
    "sdm_head_mix": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P]),
    "sdm_output_project": (ctypes.c_int, [_SP, _P, _P, _P, ctypes.c_float, _P, ctypes.c_int32, _P, _P]),
    "sdm_recurrent_log": (ctypes.c_int, [_SP] + [_P] * 11 + [ctypes.c_size_t, _P]),
    "sdm_backward_workspace_bytes": (ctypes.c_size_t, [_SP]),
    "sdm_workspace_bytes_chunked": (ctypes.c_size_t, [_SP]),
    "sdm_recurrent_chunked": (ctypes.c_int, [_SP] + [_P] * 10 + [ctypes.c_size_t, _P]),
    "sdm_address_backward": (ctypes.c_int, [_SP, _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P]),
    "sdm_recurrent_backward": (ctypes.c_int, [_SP] + [_P] * 17 + [ctypes.c_size_t, _P]),
    "sdm_check_conv_shape": (ctypes.c_int, [_P]),
    "sdm_short_conv": (ctypes.c_int, [_P] * 9),
    "sdm_short_conv_step": (ctypes.c_int, [_P] * 7),
    "sdm_short_conv_backward_workspace_bytes": (ctypes.c_size_t, [_P]),
    "sdm_short_conv_backward": (ctypes.c_int, [_P] * 13 + [ctypes.c_size_t, _P]),
    "sdm_check_scan_shape": (ctypes.c_int, [_P]),
    "sdm_selective_scan_workspace_bytes": (ctypes.c_size_t, [_P]),
    "sdm_selective_scan": (ctypes.c_int, [_P] * 13 + [ctypes.c_size_t, _P]),
    "sdm_selective_scan_step": (ctypes.c_int, [_P] * 11),
    "sdm_selective_scan_backward_workspace_bytes": (ctypes.c_size_t, [_P]),
    "sdm_selective_scan_backward": (ctypes.c_int, [_P] * 21 + [ctypes.c_size_t, _P]),
    "sdm_check_norm_shape": (ctypes.c_int, [_P]),
    "sdm_block_norm": (ctypes.c_int, [_P] * 9),
    "sdm_block_norm_backward_workspace_bytes": (ctypes.c_size_t, [_P]),
    "sdm_block_norm_backward": (ctypes.c_int, [_P] * 14 + [ctypes.c_size_t, _P]),
}


def lib():
    """The loaded ``libsdm.so`` (ctypes CDLL). Raises if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise SdmLibraryMissing(
                f"{lib_path} is not built; run `python -m sparse_memory_linear_amd.build` "
                "(no fallback implementation exists)")
        L = ctypes.CDLL(lib_path)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(code: int) -> str:
    try:
        return lib().sdm_status_string(int(code)).decode()
    except SdmLibraryMissing:
        return str(code)


def abi_version() -> int:
    return lib().sdm_abi_version()


def make_shape(B, H, T, N, d_k, d_v, kappa, W, R, in_dtype=SDM_BF16, mem_dtype=SDM_BF16) -> Shape:
    return Shape(int(B), int(H), int(T), int(N), int(d_k), int(d_v), int(kappa), int(W), int(R), _dt(in_dtype),
                 _dt(mem_dtype))


def _dt(x) -> int:
    if isinstance(x, str):
        return {"f32": SDM_F32, "bf16": SDM_BF16}[x]
    return int(x)


def _act(x) -> int:
    if isinstance(x, str):
        return {"none": SDM_ACT_NONE, "silu": SDM_ACT_SILU, "sigmoid": SDM_ACT_SIGMOID}[x]
    return int(x)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to libsdm must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _check(code: int, where: str):
    if code != 0:
        raise SdmError(code, where)


def check_shape(shape: Shape) -> int:
    return lib().sdm_check_shape(ctypes.byref(shape))


def workspace_bytes(shape: Shape) -> int:
    return lib().sdm_workspace_bytes(ctypes.byref(shape))


def init_from_M0(shape: Shape, M0, M, stream=None):
    _check(lib().sdm_init_from_M0(ctypes.byref(shape), _ptr(M0), _ptr(M), _stream(stream)), "sdm_init_from_M0")


def address(shape: Shape, x, subkeys, n_sel: int, idx, weight, score=None, stream=None):
    _check(lib().sdm_address(ctypes.byref(shape), _ptr(x), _ptr(subkeys), int(n_sel), _ptr(idx), _ptr(weight),
                             _ptr(score), _stream(stream)), "sdm_address")


def address_init(shape: Shape, x, subkeys, n_sel: int, idx, weight, M0, M, part: int, nparts: int, score=None,
                 stream=None):
    _check(lib().sdm_address_init(ctypes.byref(shape), _ptr(x), _ptr(subkeys), int(n_sel), _ptr(idx),
                                  _ptr(weight), _ptr(score), _ptr(M0), _ptr(M), int(part), int(nparts),
                                  _stream(stream)), "sdm_address_init")


def recurrent(shape: Shape, widx, wgt, ridx, rgt, v, alpha, beta, M, o, ws, stream=None):
    _check(lib().sdm_recurrent(ctypes.byref(shape), _ptr(widx), _ptr(wgt), _ptr(ridx), _ptr(rgt), _ptr(v),
                               _ptr(alpha), _ptr(beta), _ptr(M), _ptr(o), _ptr(ws), ws.numel() * ws.element_size(),
                               _stream(stream)), "sdm_recurrent")


def forward(shape: Shape, q, k, v, alpha, beta, subkeys, M, o, ws, widx_out=None, ridx_out=None, stream=None):
    _check(lib().sdm_forward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                             _ptr(subkeys), _ptr(M), _ptr(o), _ptr(widx_out), _ptr(ridx_out), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "sdm_forward")


def forward_uses_chunkwise(shape: Shape) -> bool:
    """True where sdm_forward runs the chunkwise form of the recurrence for this shape."""
    r = lib().sdm_forward_uses_chunkwise(ctypes.byref(shape))
    if r < 0:
        raise SdmError(-1, "sdm_forward_uses_chunkwise")
    return bool(r)


def forward_static(shape: Shape, q, k, v, alpha, beta, subkeys, M, o, widx_out=None, ridx_out=None, stream=None):
    _check(lib().sdm_forward_static(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                    _ptr(subkeys), _ptr(M), _ptr(o), _ptr(widx_out), _ptr(ridx_out),
                                    _stream(stream)), "sdm_forward_static")


def decode_step(shape: Shape, q, k, v, alpha, beta, subkeys, M, o, stream=None):
    _check(lib().sdm_decode_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                 _ptr(subkeys), _ptr(M), _ptr(o), _stream(stream)), "sdm_decode_step")


def workspace_error(ws, stream=None) -> int:
    out = ctypes.c_int64(0)
    _check(lib().sdm_workspace_error(_ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(out), _stream(stream)),
           "sdm_workspace_error")
    return out.value


# ----------------------------------------------------------------------------- whole-table decay
def decay_state_init(shape: Shape, lam, lrun, stream=None):
    _check(lib().sdm_decay_state_init(ctypes.byref(shape), _ptr(lam), _ptr(lrun), _stream(stream)),
           "sdm_decay_state_init")


def workspace_bytes_decay(shape: Shape) -> int:
    return lib().sdm_workspace_bytes_decay(ctypes.byref(shape))


def recurrent_decay(shape: Shape, widx, wgt, ridx, rgt, v, alpha, beta, M, lam, lrun, o, ws, stream=None):
    _check(lib().sdm_recurrent_decay(ctypes.byref(shape), _ptr(widx), _ptr(wgt), _ptr(ridx), _ptr(rgt), _ptr(v),
                                     _ptr(alpha), _ptr(beta), _ptr(M), _ptr(lam), _ptr(lrun), _ptr(o), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)), "sdm_recurrent_decay")


def forward_decay(shape: Shape, q, k, v, alpha, beta, subkeys, M, lam, lrun, o, ws, widx_out=None, ridx_out=None,
                  stream=None):
    _check(lib().sdm_forward_decay(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                   _ptr(subkeys), _ptr(M), _ptr(lam), _ptr(lrun), _ptr(o), _ptr(widx_out),
                                   _ptr(ridx_out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "sdm_forward_decay")


def decode_step_decay(shape: Shape, q, k, v, alpha, beta, subkeys, M, lam, lrun, o, stream=None):
    _check(lib().sdm_decode_step_decay(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                       _ptr(subkeys), _ptr(M), _ptr(lam), _ptr(lrun), _ptr(o), _stream(stream)),
           "sdm_decode_step_decay")


def materialize(shape: Shape, M, lam, lrun, out, stream=None):
    _check(lib().sdm_materialize(ctypes.byref(shape), _ptr(M), _ptr(lam), _ptr(lrun), _ptr(out), _stream(stream)),
           "sdm_materialize")


# ----------------------------------------------------------------------------- gates and output
def gates(shape: Shape, a, b, A_log, dt_bias, alpha, beta, stream=None):
    _check(lib().sdm_gates(ctypes.byref(shape), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(alpha), _ptr(beta),
                           _stream(stream)), "sdm_gates")


def output_gate(shape: Shape, o, z, w, eps: float, x, stream=None):
    _check(lib().sdm_output_gate(ctypes.byref(shape), _ptr(o), _ptr(z), _ptr(w), float(eps), _ptr(x),
                                 _stream(stream)), "sdm_output_gate")


def head_mix(x, Wo, y, M: int, K: int, N: int, stream=None):
    _check(lib().sdm_head_mix(_ptr(x), _ptr(Wo), _ptr(y), int(M), int(K), int(N), _stream(stream)), "sdm_head_mix")


# ----------------------------------------------------------------------------- backward
def output_project(shape: Shape, o, z, w, eps: float, Wo, d_model: int, y, stream=None):
    _check(lib().sdm_output_project(ctypes.byref(shape), _ptr(o), _ptr(z), _ptr(w), float(eps), _ptr(Wo),
                                    int(d_model), _ptr(y), _stream(stream)), "sdm_output_project")


def recurrent_log(shape: Shape, widx, wgt, ridx, rgt, v, alpha, beta, M, o, xlog, ws, stream=None):
    _check(lib().sdm_recurrent_log(ctypes.byref(shape), _ptr(widx), _ptr(wgt), _ptr(ridx), _ptr(rgt), _ptr(v),
                                   _ptr(alpha), _ptr(beta), _ptr(M), _ptr(o), _ptr(xlog), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)), "sdm_recurrent_log")


def backward_workspace_bytes(shape: Shape) -> int:
    return lib().sdm_backward_workspace_bytes(ctypes.byref(shape))


def recurrent_backward(shape: Shape, widx, wgt, ridx, rgt, v, alpha, beta, M, xlog, go, G, dv, dalpha, dbeta, dwgt,
                       drgt, ws, stream=None):
    _check(lib().sdm_recurrent_backward(ctypes.byref(shape), _ptr(widx), _ptr(wgt), _ptr(ridx), _ptr(rgt), _ptr(v),
                                        _ptr(alpha), _ptr(beta), _ptr(M), _ptr(xlog), _ptr(go), _ptr(G), _ptr(dv),
                                        _ptr(dalpha), _ptr(dbeta), _ptr(dwgt), _ptr(drgt), _ptr(ws), ws.numel() * ws.element_size(),
                                        _stream(stream)), "sdm_recurrent_backward")


def address_backward(shape: Shape, x, subkeys, n_sel: int, idx, weight, dweight, dx, dsub, stream=None):
    _check(lib().sdm_address_backward(ctypes.byref(shape), _ptr(x), _ptr(subkeys), int(n_sel), _ptr(idx),
                                      _ptr(weight), _ptr(dweight), _ptr(dx), _ptr(dsub), _stream(stream)),
           "sdm_address_backward")


def workspace_bytes_chunked(shape: Shape) -> int:
    return lib().sdm_workspace_bytes_chunked(ctypes.byref(shape))


def recurrent_chunked(shape: Shape, widx, wgt, ridx, rgt, v, alpha, beta, M, o, ws, stream=None):
    _check(lib().sdm_recurrent_chunked(ctypes.byref(shape), _ptr(widx), _ptr(wgt), _ptr(ridx), _ptr(rgt), _ptr(v),
                                       _ptr(alpha), _ptr(beta), _ptr(M), _ptr(o), _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream(stream)), "sdm_recurrent_chunked")


# ----------------------------------------------------------------------------- convolution, scan, norm
_torch = None  # torch, and the types of the tensors by the sdm_dtype: looked up once, on the first call
_TYPES = {}


def _load_torch():
    global _torch, _TYPES
    import torch
    _TYPES = dict(enumerate((torch.float32, torch.bfloat16, torch.int32)))
    _torch = torch


_I32 = 2  # index of int32 among the types


class _Args:
    """Pointers of one call's tensors: each checked for type, shape and strides, and for lying on the one
    GPU of the call, before the library sees an address."""
    __slots__ = ("where", "device")

    def __init__(self, where: str):
        if _torch is None:
            _load_torch()
        self.where, self.device = where, -1

    def _take(self, name, t, dtype):
        if t is None:
            raise ValueError(f"{self.where}: {name} is missing")
        if t.dtype is not _TYPES.get(dtype):
            raise ValueError(f"{self.where}: {name} is {t.dtype}, not {_TYPES.get(dtype, f'of sdm_dtype {dtype}')}")
        d = t.get_device()
        if d != self.device or d < 0:
            if d < 0:
                raise ValueError(f"{self.where}: {name} is not on a GPU")
            if self.device >= 0:
                raise ValueError(f"{self.where}: {name} is on GPU {d}, another tensor on GPU {self.device}")
            self.device = d
        return t.data_ptr()

    def flat(self, name, t, dtype, *shape):
        """A contiguous tensor of `shape`."""
        p = self._take(name, t, dtype)
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{self.where}: {name} has shape {tuple(t.shape)} and strides {t.stride()}, not a "
                             f"contiguous {shape}")
        return p

    def maybe(self, name, t, dtype, *shape):
        """The same, or None."""
        return None if t is None else self.flat(name, t, dtype, *shape)

    def rows(self, name, t, dtype, B, T, width, ld):
        """[B, T, width], or [B, T, ...] with the last dimensions flattened to `width`: rows `ld` apart."""
        p = self._take(name, t, dtype)
        shape, stride = t.shape, t.stride()
        if shape == (B, T, width) and stride == (T * ld, ld, 1):
            return p
        ok = len(shape) >= 3 and shape[0] == B and shape[1] == T
        inner = 1
        for d in range(len(shape) - 1, 1, -1):
            ok = ok and (shape[d] == 1 or stride[d] == inner)
            inner *= shape[d]
        ok = ok and inner == width and (T <= 1 or stride[1] == ld) and (B == 1 or T == 0 or stride[0] == T * ld)
        if not ok:
            raise ValueError(f"{self.where}: {name} has shape {tuple(shape)} and strides {stride}, not rows of "
                             f"{width} values with token stride {ld} for B={B}, T={T}")
        return p

    def workspace(self, ws):
        """(pointer, bytes) of the workspace; its size is checked by the library."""
        if ws is None:
            return None, 0
        d = ws.get_device()
        if d < 0 or (self.device >= 0 and d != self.device) or not ws.is_contiguous():
            raise ValueError(f"{self.where}: ws is not a contiguous tensor on the GPU of the call")
        return ws.data_ptr(), ws.numel() * ws.element_size()

    def call(self, shape, stream, *args):
        """Runs the entry point on `stream`, or on the current stream of the tensors' GPU."""
        f, dev, C = getattr(_lib or lib(), self.where), self.device, _torch._C
        here = C._cuda_getDevice() if dev >= 0 else _torch.cuda.current_device()  # (tensors there: initialised)
        if dev < 0:
            dev = here
        if stream is None:
            stream = C._cuda_getCurrentRawStream(dev)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        if dev == here:
            code = f(ctypes.byref(shape), *args, stream)
        else:
            with _torch.cuda.device(dev):
                code = f(ctypes.byref(shape), *args, stream)
        if code != 0:
            raise SdmError(code, self.where)


def make_conv_shape(B, T, C, K, in_dtype=SDM_BF16, act=SDM_ACT_SILU, ld_x=None, ld_y=None) -> ConvShape:
    return ConvShape(int(B), int(T), int(C), int(K), _dt(in_dtype), _act(act), int(C if ld_x is None else ld_x),
                     int(C if ld_y is None else ld_y))


def check_conv_shape(shape: ConvShape) -> int:
    return lib().sdm_check_conv_shape(ctypes.byref(shape))


def short_conv(shape: ConvShape, x, w, y, bias=None, lengths=None, s_in=None, s_out=None, stream=None):
    s, a = shape, _Args("sdm_short_conv")
    a.call(s, stream, a.rows("x", x, s.in_dtype, s.B, s.T, s.C, s.ld_x), a.flat("w", w, SDM_F32, s.C, s.K),
           a.maybe("bias", bias, SDM_F32, s.C), a.maybe("lengths", lengths, _I32, s.B),
           a.maybe("s_in", s_in, s.in_dtype, s.B, s.K - 1, s.C),
           a.maybe("s_out", s_out, s.in_dtype, s.B, s.K - 1, s.C),
           a.rows("y", y, s.in_dtype, s.B, s.T, s.C, s.ld_y))


def short_conv_step(shape: ConvShape, x, w, state, y, bias=None, stream=None):
    s, a = shape, _Args("sdm_short_conv_step")
    a.call(s, stream, a.rows("x", x, s.in_dtype, s.B, s.T, s.C, s.ld_x), a.flat("w", w, SDM_F32, s.C, s.K),
           a.maybe("bias", bias, SDM_F32, s.C),
           a.flat("state", state, s.in_dtype, s.B, s.K - 1, s.C), a.rows("y", y, s.in_dtype, s.B, s.T, s.C, s.ld_y))


def short_conv_backward_workspace_bytes(shape: ConvShape) -> int:
    return lib().sdm_short_conv_backward_workspace_bytes(ctypes.byref(shape))


def short_conv_backward(shape: ConvShape, x, w, dy, dx, dw, ws, bias=None, dbias=None, lengths=None, s_in=None,
                        ds_out=None, ds_in=None, stream=None):
    s, a = shape, _Args("sdm_short_conv_backward")
    a.call(s, stream, a.rows("x", x, s.in_dtype, s.B, s.T, s.C, s.ld_x), a.flat("w", w, SDM_F32, s.C, s.K),
           a.maybe("bias", bias, SDM_F32, s.C), a.maybe("lengths", lengths, _I32, s.B),
           a.maybe("s_in", s_in, s.in_dtype, s.B, s.K - 1, s.C),
           a.rows("dy", dy, SDM_F32, s.B, s.T, s.C, s.ld_y),
           a.maybe("ds_out", ds_out, SDM_F32, s.B, s.K - 1, s.C),
           a.rows("dx", dx, SDM_F32, s.B, s.T, s.C, s.ld_x), a.flat("dw", dw, SDM_F32, s.C, s.K),
           a.maybe("dbias", dbias, SDM_F32, s.C),
           a.maybe("ds_in", ds_in, SDM_F32, s.B, s.K - 1, s.C), *a.workspace(ws))


def make_scan_shape(B, T, H, G, d_k, d_v, in_dtype=SDM_BF16, ld_x=None, ld_b=None, ld_c=None, ld_dt=None) -> ScanShape:
    return ScanShape(int(B), int(T), int(H), int(G), int(d_k), int(d_v), _dt(in_dtype),
                     int(H * d_v if ld_x is None else ld_x), int(G * d_k if ld_b is None else ld_b),
                     int(G * d_k if ld_c is None else ld_c), int(H if ld_dt is None else ld_dt))


def check_scan_shape(shape: ScanShape) -> int:
    return lib().sdm_check_scan_shape(ctypes.byref(shape))


def _scan_inputs(a: _Args, s: ScanShape, x, Bm, Cm, dt, A_log, dt_bias, D):
    return (a.rows("x", x, s.in_dtype, s.B, s.T, s.H * s.d_v, s.ld_x),
            a.rows("Bm", Bm, s.in_dtype, s.B, s.T, s.G * s.d_k, s.ld_b),
            a.rows("Cm", Cm, s.in_dtype, s.B, s.T, s.G * s.d_k, s.ld_c), a.rows("dt", dt, SDM_F32, s.B, s.T, s.H, s.ld_dt),
            a.flat("A_log", A_log, SDM_F32, s.H), a.flat("dt_bias", dt_bias, SDM_F32, s.H),
            a.maybe("D", D, SDM_F32, s.H))


def selective_scan_workspace_bytes(shape: ScanShape) -> int:
    return lib().sdm_selective_scan_workspace_bytes(ctypes.byref(shape))


def selective_scan(shape: ScanShape, x, Bm, Cm, dt, A_log, dt_bias, o, ws, D=None, lengths=None, s_in=None,
                   s_out=None, stream=None):
    s, a = shape, _Args("sdm_selective_scan")
    state = (s.B, s.H, s.d_v, s.d_k)
    a.call(s, stream, *_scan_inputs(a, s, x, Bm, Cm, dt, A_log, dt_bias, D),
           a.maybe("lengths", lengths, _I32, s.B),
           a.maybe("s_in", s_in, SDM_F32, *state), a.maybe("s_out", s_out, SDM_F32, *state),
           a.flat("o", o, SDM_F32, s.B, s.H, s.T, s.d_v), *a.workspace(ws))


def selective_scan_step(shape: ScanShape, x, Bm, Cm, dt, A_log, dt_bias, state, o, D=None, stream=None):
    s, a = shape, _Args("sdm_selective_scan_step")
    a.call(s, stream, *_scan_inputs(a, s, x, Bm, Cm, dt, A_log, dt_bias, D),
           a.flat("state", state, SDM_F32, s.B, s.H, s.d_v, s.d_k), a.flat("o", o, SDM_F32, s.B, s.H, s.T, s.d_v))


def selective_scan_backward_workspace_bytes(shape: ScanShape) -> int:
    return lib().sdm_selective_scan_backward_workspace_bytes(ctypes.byref(shape))


def selective_scan_backward(shape: ScanShape, x, Bm, Cm, dt, A_log, dt_bias, go, dx, dBm, dCm, ddt, dA_log, ddt_bias,
                            ws, D=None, dD=None, lengths=None, s_in=None, ds_out=None, ds_in=None, stream=None):
    s, a = shape, _Args("sdm_selective_scan_backward")
    state = (s.B, s.H, s.d_v, s.d_k)
    a.call(s, stream, *_scan_inputs(a, s, x, Bm, Cm, dt, A_log, dt_bias, D),
           a.maybe("lengths", lengths, _I32, s.B),
           a.maybe("s_in", s_in, SDM_F32, *state), a.flat("go", go, SDM_F32, s.B, s.H, s.T, s.d_v),
           a.maybe("ds_out", ds_out, SDM_F32, *state),
           a.rows("dx", dx, SDM_F32, s.B, s.T, s.H * s.d_v, s.ld_x),
           a.rows("dBm", dBm, SDM_F32, s.B, s.T, s.G * s.d_k, s.ld_b),
           a.rows("dCm", dCm, SDM_F32, s.B, s.T, s.G * s.d_k, s.ld_c),
           a.rows("ddt", ddt, SDM_F32, s.B, s.T, s.H, s.ld_dt), a.flat("dA_log", dA_log, SDM_F32, s.H),
           a.flat("ddt_bias", ddt_bias, SDM_F32, s.H), a.maybe("dD", dD, SDM_F32, s.H),
           a.maybe("ds_in", ds_in, SDM_F32, *state), *a.workspace(ws))


def make_norm_shape(M, D, y_dtype=SDM_F32, r_dtype=SDM_F32, x_dtype=SDM_BF16, gate_dtype=SDM_F32, gate_rows=0,
                    gate_act=SDM_ACT_NONE, eps=1e-5, scale=1.0) -> NormShape:
    return NormShape(int(M), int(D), _dt(y_dtype), _dt(r_dtype), _dt(x_dtype), _dt(gate_dtype), _act(gate_act),
                     int(gate_rows), float(eps), float(scale))


def check_norm_shape(shape: NormShape) -> int:
    return lib().sdm_check_norm_shape(ctypes.byref(shape))


def block_norm(shape: NormShape, y, r, r_out, gate=None, w_post=None, w_pre=None, x=None, stream=None):
    s, a = shape, _Args("sdm_block_norm")
    a.call(s, stream, a.flat("y", y, s.y_dtype, s.M, s.D), a.flat("r", r, s.r_dtype, s.M, s.D),
           a.maybe("gate", gate, s.gate_dtype, s.gate_rows, s.D),
           a.maybe("w_post", w_post, SDM_F32, s.D), a.maybe("w_pre", w_pre, SDM_F32, s.D),
           a.flat("r_out", r_out, s.r_dtype, s.M, s.D), a.maybe("x", x, s.x_dtype, s.M, s.D))


def block_norm_backward_workspace_bytes(shape: NormShape) -> int:
    return lib().sdm_block_norm_backward_workspace_bytes(ctypes.byref(shape))


def block_norm_backward(shape: NormShape, y, r, dy, dr, ws, gate=None, w_post=None, w_pre=None, dr_out=None, dx=None,
                        dgate=None, dw_post=None, dw_pre=None, stream=None):
    s, a = shape, _Args("sdm_block_norm_backward")
    a.call(s, stream, a.flat("y", y, s.y_dtype, s.M, s.D), a.flat("r", r, s.r_dtype, s.M, s.D),
           a.maybe("gate", gate, s.gate_dtype, s.gate_rows, s.D),
           a.maybe("w_post", w_post, SDM_F32, s.D), a.maybe("w_pre", w_pre, SDM_F32, s.D),
           a.maybe("dr_out", dr_out, SDM_F32, s.M, s.D), a.maybe("dx", dx, SDM_F32, s.M, s.D),
           a.flat("dy", dy, SDM_F32, s.M, s.D), a.flat("dr", dr, SDM_F32, s.M, s.D),
           a.maybe("dgate", dgate, SDM_F32, s.gate_rows, s.D),
           a.maybe("dw_post", dw_post, SDM_F32, s.D), a.maybe("dw_pre", dw_pre, SDM_F32, s.D),
           *a.workspace(ws))
