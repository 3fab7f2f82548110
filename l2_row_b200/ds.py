"""Thin ctypes binding of libds (include/ds.h): argument marshalling only.

Every step of the computation runs in the CUDA kernels of libds.so.  If the
library has not been built (``python -m l2_row_b200.build``) importing this
module raises: there is no CPU fallback.

The five calls keep their C names and take lists of segments:

    ds_wn_forward(segs, out_dtype, eps, stream=None)
    ds_wn_backward(segs, gy_dtype, eps, stream=None)
    ds_row_renorm(segs, eps, stream=None)
    ds_grad_project(segs, eps, stream=None)       (grad_w = the gradient, in place)
    ds_renorm_momentum(segs, eps, stream=None)    (grad_w = the momentum, in place)
    ds_l2_rows(segs, eps, stream=None)
    ds_slerp_rows(segs, eps, stream=None)
    ds_gate_l2_rows(segs, eps, stream=None)       (Dory's gated rows)
    ds_swiglu_l2_rows(segs, eps, stream=None)     (Dory's SwiGLU rows)
    ds_l2_rows_backward(segs, eps, stream=None)
    ds_slerp_rows_backward(segs, eps, dalpha=None, workspace=None, stream=None)

and the language-model rows, each with its gradient:

    ds_embed_rows(segs, w_dtype, out_dtype, eps, stream=None)            (ESeg)
    ds_embed_rows_backward(segs, w_dtype, dy_dtype, eps, workspace=None, stream=None)
    ds_qk_norm_rows(segs, dtype, eps, stream=None)                       (QNSeg)
    ds_qk_norm_rows_backward(segs, dtype, grad_dtype, eps, dwq=None, dwk=None,
                             workspace=None, stream=None)                (QNGSeg)
    ds_logp_rows(segs, dtype, stream=None)                               (LSeg)
    ds_logp_rows_backward(segs, dtype, grad_dtype=None, stream=None)

which also check that their tensors have the types the call names and lie on
the current device (``ValueError``).  A tensor of one row may have any row
stride and width.

A segment is a ``WSeg`` / ``ASeg`` of CUDA tensors (2-D, unit column stride,
row stride = leading dimension) or a raw ``ds_wseg`` / ``ds_aseg`` structure.
``stream`` defaults to torch's current CUDA stream.  A failing call raises
``DSError`` carrying the status code and the library's message.
"""
from __future__ import annotations

import ctypes as ct
import os
import struct
from dataclasses import dataclass
from typing import Any, Sequence

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libds.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libds.so is not built ({LIB_PATH}); run `python -m l2_row_b200.build`")
if os.path.isdir(_build.CSRC) and (_build.library_keys(LIB_PATH) or ("",))[0] != _build.sources_key():
    # its structures and kernels may be others than the ones this module packs arguments for
    raise ImportError(f"libds.so ({LIB_PATH}) was not built from the sources beside it; run `python -m l2_row_b200.build`")

_lib = ct.CDLL(LIB_PATH)

DS_OK, DS_ERR_INVALID_ARG, DS_ERR_ALIGNMENT, DS_ERR_UNSUPPORTED_DTYPE = 0, 1, 2, 3
DS_ERR_TOO_MANY_SEGMENTS, DS_ERR_CUDA, DS_ERR_DEVICE_TIMEOUT, DS_ERR_OVERLAP = 4, 5, 6, 7
DS_F32, DS_BF16 = 0, 1
DS_OP_WN_FORWARD, DS_OP_WN_BACKWARD, DS_OP_ROW_RENORM, DS_OP_L2_ROWS, DS_OP_SLERP_ROWS = range(5)
DS_OP_GRAD_PROJECT, DS_OP_RENORM_MOMENTUM = 5, 6
DS_OP_L2_ROWS_BACKWARD, DS_OP_SLERP_ROWS_BACKWARD = 7, 8
DS_OP_GATE_L2_ROWS, DS_OP_SWIGLU_L2_ROWS = 9, 10
DS_PATH_AUTO, DS_PATH_WARP, DS_PATH_CTA, DS_PATH_CLUSTER, DS_PATH_TWO_PASS = range(5)
DS_MAX_SEGMENTS = 65536
PATH_NAMES = {DS_PATH_WARP: "warp", DS_PATH_CTA: "cta", DS_PATH_CLUSTER: "cluster", DS_PATH_TWO_PASS: "two_pass"}


class ds_wseg(ct.Structure):
    _fields_ = [("w", ct.c_void_p), ("gain", ct.c_void_p), ("w_eff", ct.c_void_p), ("gy", ct.c_void_p),
                ("grad_w", ct.c_void_p), ("grad_g", ct.c_void_p), ("rows", ct.c_int64), ("cols", ct.c_int64),
                ("ld", ct.c_int64), ("ld_out", ct.c_int64), ("radius", ct.c_float), ("gain_scalar", ct.c_int32),
                ("rnorm", ct.c_void_p), ("transposed", ct.c_int32), ("tgroup", ct.c_int32)]


class ds_aseg(ct.Structure):
    _fields_ = [("x", ct.c_void_p), ("r", ct.c_void_p), ("y", ct.c_void_p), ("alpha", ct.c_void_p),
                ("rows", ct.c_int64), ("cols", ct.c_int64), ("ld", ct.c_int64)]


class ds_fseg(ct.Structure):
    _fields_ = [("a", ct.c_void_p), ("b", ct.c_void_p), ("y", ct.c_void_p), ("sa", ct.c_void_p),
                ("sb", ct.c_void_p), ("rows", ct.c_int64), ("cols", ct.c_int64), ("ld", ct.c_int64)]


class ds_agseg(ct.Structure):
    _fields_ = [("x", ct.c_void_p), ("r", ct.c_void_p), ("dy", ct.c_void_p), ("dx", ct.c_void_p),
                ("dr", ct.c_void_p), ("alpha", ct.c_void_p), ("rows", ct.c_int64), ("cols", ct.c_int64),
                ("ld", ct.c_int64), ("ld_d", ct.c_int64)]


class ds_qkseg(ct.Structure):
    _fields_ = [("q", ct.c_void_p), ("k", ct.c_void_p), ("v", ct.c_void_p), ("q_out", ct.c_void_p),
                ("k_cache", ct.c_void_p), ("v_cache", ct.c_void_p), ("pos", ct.c_void_p), ("slot", ct.c_void_p),
                ("inv_freq", ct.c_void_p), ("q_scale", ct.c_void_p), ("rows", ct.c_int64),
                ("cache_rows", ct.c_int64), ("ld_q", ct.c_int64), ("ld_kv", ct.c_int64), ("ld_cache", ct.c_int64),
                ("head_dim", ct.c_int32), ("hq", ct.c_int32), ("hk", ct.c_int32)]


class ds_eseg(ct.Structure):
    _fields_ = [("w", ct.c_void_p), ("gain", ct.c_void_p), ("ids", ct.c_void_p), ("y", ct.c_void_p),
                ("dy", ct.c_void_p), ("grad_w", ct.c_void_p), ("grad_g", ct.c_void_p), ("tokens", ct.c_int64),
                ("vocab", ct.c_int64), ("cols", ct.c_int64), ("ld", ct.c_int64), ("ld_y", ct.c_int64),
                ("ld_g", ct.c_int64), ("radius", ct.c_float), ("unit", ct.c_int32), ("gain_scalar", ct.c_int32),
                ("ids_i64", ct.c_int32), ("accumulate", ct.c_int32)]


class ds_qnseg(ct.Structure):
    _fields_ = [(f, ct.c_void_p) for f in ("q", "k", "v", "q_out", "k_cache", "v_cache", "wq", "wk", "pos", "slot",
                                           "inv_freq")] + \
               [(f, ct.c_int64) for f in ("rows", "cache_rows", "ld_q", "ld_kv", "ld_qo", "ld_cache")] + \
               [(f, ct.c_int32) for f in ("head_dim", "rot_dim", "hq", "hk", "interleaved", "mean")]


class ds_qngseg(ct.Structure):
    _fields_ = [(f, ct.c_void_p) for f in ("q", "k", "dq_out", "dk_out", "dq", "dk", "wq", "wk", "pos", "inv_freq")] + \
               [(f, ct.c_int64) for f in ("rows", "ld_q", "ld_kv", "ld_dqo", "ld_dko", "ld_dq", "ld_dk")] + \
               [(f, ct.c_int32) for f in ("head_dim", "rot_dim", "hq", "hk", "interleaved", "mean")]


class ds_lseg(ct.Structure):
    _fields_ = [(f, ct.c_void_p) for f in ("x", "ids", "logp", "lse", "entropy", "top_id", "top_logp", "dlogp",
                                           "dentropy", "dlse", "dx")] + \
               [(f, ct.c_int64) for f in ("rows", "cols", "ld", "ld_d")] + \
               [("scale", ct.c_float), ("top_k", ct.c_int32), ("ids_i64", ct.c_int32)]


# the same structures as bytes
_ESEG = struct.Struct("@7Q6qf4i4x").pack
_QNSEG = struct.Struct("@11Q6q6i").pack
_QNGSEG = struct.Struct("@10Q7q6i").pack
_LSEG = struct.Struct("@11Q4qf2i4x").pack

_st = ct.c_int
_lib.ds_wn_forward.argtypes = [ct.POINTER(ds_wseg), ct.c_int, ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_wn_backward.argtypes = [ct.POINTER(ds_wseg), ct.c_int, ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_row_renorm.argtypes = [ct.POINTER(ds_wseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_grad_project.argtypes = [ct.POINTER(ds_wseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_renorm_momentum.argtypes = [ct.POINTER(ds_wseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_l2_rows.argtypes = [ct.POINTER(ds_aseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_slerp_rows.argtypes = [ct.POINTER(ds_aseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_l2_rows_backward.argtypes = [ct.POINTER(ds_agseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_gate_l2_rows.argtypes = [ct.POINTER(ds_fseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_swiglu_l2_rows.argtypes = [ct.POINTER(ds_fseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_qk_rows_l2.argtypes = [ct.POINTER(ds_qkseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_row_norms.argtypes = [ct.POINTER(ds_wseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_gain_preserve.argtypes = [ct.POINTER(ds_wseg), ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_slerp_rows_backward.argtypes = [ct.POINTER(ds_agseg), ct.c_int, ct.c_float, ct.c_void_p, ct.c_void_p,
                                        ct.c_uint64, ct.c_void_p]
_lib.ds_slerp_rows_backward_noalloc.argtypes = [ct.POINTER(ds_agseg), ct.c_int, ct.c_float, ct.c_void_p,
                                                ct.c_void_p]
_lib.ds_slerp_rows_backward_noalloc.restype = ct.c_int
_lib.ds_slerp_rows_backward_workspace.argtypes = [ct.c_int64]
_lib.ds_slerp_rows_backward_workspace.restype = ct.c_uint64
_lib.ds_embed_rows.argtypes = [ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_embed_rows_backward.argtypes = [ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_float, ct.c_void_p,
                                        ct.c_uint64, ct.c_void_p]
_lib.ds_qk_norm_rows.argtypes = [ct.c_void_p, ct.c_int, ct.c_int, ct.c_float, ct.c_void_p]
_lib.ds_qk_norm_rows_backward.argtypes = [ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_float, ct.c_void_p,
                                          ct.c_void_p, ct.c_void_p, ct.c_uint64, ct.c_void_p]
_lib.ds_qk_norm_rows_backward_workspace.argtypes = [ct.c_int64]
_lib.ds_qk_norm_rows_backward_workspace.restype = ct.c_uint64
_lib.ds_logp_rows.argtypes = [ct.c_void_p, ct.c_int, ct.c_int, ct.c_void_p]
_lib.ds_logp_rows_backward.argtypes = [ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]
_lib.ds_embed_rows_backward_workspace.argtypes = [ct.c_int64, ct.c_int64, ct.c_int64]
_lib.ds_embed_rows_backward_workspace.restype = ct.c_uint64
for _f in ("ds_wn_forward", "ds_wn_backward", "ds_row_renorm", "ds_grad_project", "ds_renorm_momentum",
           "ds_l2_rows", "ds_slerp_rows", "ds_l2_rows_backward", "ds_slerp_rows_backward",
           "ds_gate_l2_rows", "ds_swiglu_l2_rows", "ds_qk_rows_l2", "ds_row_norms", "ds_gain_preserve",
           "ds_embed_rows", "ds_embed_rows_backward", "ds_qk_norm_rows", "ds_qk_norm_rows_backward",
           "ds_logp_rows", "ds_logp_rows_backward", "ds_get_device_status", "ds_row_class", "ds_debug_force_path", "ds_debug_set_wait_limit_ns",
           "ds_debug_wait_timeout_selftest", "ds_debug_division_check"):
    getattr(_lib, _f).restype = _st
_lib.ds_status_string.argtypes = [ct.c_int]
_lib.ds_status_string.restype = ct.c_char_p
_lib.ds_last_error.argtypes = []
_lib.ds_last_error.restype = ct.c_char_p
_lib.ds_get_device_status.argtypes = [ct.c_void_p]
_lib.ds_launch_count.argtypes = []
_lib.ds_launch_count.restype = ct.c_uint64
_lib.ds_version.argtypes = []
_lib.ds_version.restype = ct.c_int
_lib.ds_row_class.argtypes = [ct.c_int, ct.c_int64, ct.POINTER(ct.c_int), ct.POINTER(ct.c_int),
                              ct.POINTER(ct.c_int)]
_lib.ds_debug_force_path.argtypes = [ct.c_int]
_lib.ds_debug_set_wait_limit_ns.argtypes = [ct.c_uint64]
_lib.ds_debug_wait_timeout_selftest.argtypes = [ct.c_uint64, ct.c_void_p]
_lib.ds_debug_division_check.argtypes = [ct.c_void_p, ct.c_void_p]

#: every symbol include/ds.h declares
EXPORTS = ("ds_wn_forward", "ds_wn_backward", "ds_row_renorm", "ds_grad_project", "ds_renorm_momentum",
           "ds_l2_rows", "ds_slerp_rows", "ds_l2_rows_backward", "ds_slerp_rows_backward",
           "ds_gate_l2_rows", "ds_swiglu_l2_rows", "ds_qk_rows_l2", "ds_row_norms", "ds_gain_preserve",
           "ds_embed_rows", "ds_embed_rows_backward", "ds_embed_rows_backward_workspace",
           "ds_qk_norm_rows", "ds_qk_norm_rows_backward", "ds_qk_norm_rows_backward_workspace",
           "ds_logp_rows", "ds_logp_rows_backward",
           "ds_slerp_rows_backward_workspace", "ds_slerp_rows_backward_noalloc", "ds_status_string", "ds_last_error", "ds_get_device_status", "ds_launch_count", "ds_version",
           "ds_row_class", "ds_debug_force_path", "ds_debug_set_wait_limit_ns", "ds_debug_wait_timeout_selftest",
           "ds_debug_division_check")


def lib() -> ct.CDLL:
    """The loaded libds.so (for direct C-ABI calls)."""
    return _lib


class DSError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.ds_status_string(status).decode()
        detail = _lib.ds_last_error().decode()
        super().__init__(f"{where}: {msg}" + (f" ({detail})" if detail else ""))


def _check(status: int, where: str) -> None:
    if status != DS_OK:
        raise DSError(status, where)


def _stream_ptr(stream) -> int | None:
    if stream is None:
        import torch

        if not torch.cuda.is_available():
            return None
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(dt) -> int:
    if isinstance(dt, int):
        return dt
    s = str(dt).replace("torch.", "")
    if s in ("bf16", "bfloat16"):
        return DS_BF16
    if s in ("f32", "float32", "float"):
        return DS_F32
    raise ValueError(f"unsupported dtype {dt!r}")


# ------------------------------------------------------------ tensor views --

def _mat(t, name: str, rows: int, cols: int) -> tuple[int, int]:
    """(data_ptr, leading dimension) of a 2-D row-major view; (0, cols) for None."""
    if t is None:
        return 0, cols
    if t.dim() != 2 or tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name}: expected shape ({rows}, {cols}), got {tuple(t.shape)}")
    if rows == 0:
        return t.data_ptr(), cols
    if t.stride(1) != 1 and cols > 1:
        raise ValueError(f"{name}: columns must be contiguous")
    return t.data_ptr(), (t.stride(0) if rows > 1 else max(t.stride(0), cols))


def _vec(t) -> int:
    if t is None:
        return 0
    if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
        raise ValueError("per-row vectors must be contiguous 1-D tensors")
    return t.data_ptr()


@dataclass
class WSeg:
    """One weight matrix.  w: fp32 [R, C]; gain: fp32 [R] or None; w_eff:
    forward output [R, C]; gy, grad_w, grad_g: backward input/outputs.
    For ds_grad_project grad_w is the gradient and for ds_renorm_momentum
    the momentum buffer (fp32 [R, C], w's leading dimension, in place).
    gain_scalar: gain is fp32 [1] shared by every row and grad_g fp32 [R + 1]
    (per-row parts, then their sum).  rnorm: fp32 [R] output of
    ds_row_norms / ds_gain_preserve.  transposed: the unit rows are the
    columns of w (GPT-2 Conv1D, stored [in, out] = [C, R]); w, w_eff, gy and
    grad_w are then given in that stored layout.  tgroup (with transposed):
    G consecutive stored columns per unit row, for a ConvTranspose weight
    [in, out, k...] viewed as [in, out * G] (G = the kernel's volume): unit
    rows R = out, row length C = in * G."""

    w: Any
    gain: Any = None
    w_eff: Any = None
    gy: Any = None
    grad_w: Any = None
    grad_g: Any = None
    radius: float = 1.0
    gain_scalar: bool = False
    rnorm: Any = None
    transposed: bool = False
    tgroup: int = 1

    def to_c(self) -> ds_wseg:
        SR, SC = (int(self.w.shape[0]), int(self.w.shape[1]))   # the stored shape
        G = int(self.tgroup) if self.transposed else 1
        if G < 1 or SC % G:
            raise ValueError("tgroup must be >= 1 and divide the stored columns")
        R, C = (SC // G, SR * G) if self.transposed else (SR, SC)
        w, ld = _mat(self.w, "w", SR, SC)
        weff, ld_out = _mat(self.w_eff, "w_eff", SR, SC)
        gy, ld_gy = _mat(self.gy, "gy", SR, SC)
        gw, ld_gw = _mat(self.grad_w, "grad_w", SR, SC)
        if self.w_eff is not None and self.gy is not None and ld_out != ld_gy:
            raise ValueError("w_eff and gy must share a leading dimension")
        if self.grad_w is not None and ld_gw != ld:
            raise ValueError("grad_w must share w's leading dimension")
        return ds_wseg(w, _vec(self.gain), weff, gy, gw, _vec(self.grad_g), R, C, ld,
                       ld_out if self.w_eff is not None else ld_gy, float(self.radius), int(bool(self.gain_scalar)),
                       _vec(self.rnorm), int(bool(self.transposed)), G if self.transposed else 0)


@dataclass
class ASeg:
    """One activation matrix: x (slerp: res), r (slerp: out; l2: residual or
    None), y output, alpha fp32 [C] (slerp only).  bf16 [R, C], shared ld."""

    x: Any
    y: Any
    r: Any = None
    alpha: Any = None

    def to_c(self) -> ds_aseg:
        R, C = (int(self.x.shape[0]), int(self.x.shape[1]))
        x, ld = _mat(self.x, "x", R, C)
        y, ldy = _mat(self.y, "y", R, C)
        r, ldr = _mat(self.r, "r", R, C)
        if ldy != ld or (self.r is not None and ldr != ld):
            raise ValueError("x, r and y must share a leading dimension")
        return ds_aseg(x, r, y, _vec(self.alpha), R, C, ld)


@dataclass
class FSeg:
    """One activation matrix for Dory's rows: a, b, y bf16 [R, C] with a
    shared ld; sa (and for SwiGLU sb) fp32 [C].  Gate: a = o, b = g, sa = sg;
    SwiGLU: a = g, b = u, sa = sug, sb = suu."""

    a: Any
    b: Any
    y: Any
    sa: Any
    sb: Any = None

    def to_c(self) -> ds_fseg:
        R, C = (int(self.a.shape[0]), int(self.a.shape[1]))
        a, ld = _mat(self.a, "a", R, C)
        b, ldb = _mat(self.b, "b", R, C)
        y, ldy = _mat(self.y, "y", R, C)
        if ldb != ld or ldy != ld:
            raise ValueError("a, b and y must share a leading dimension")
        return ds_fseg(a, b, y, _vec(self.sa), _vec(self.sb), R, C, ld)


@dataclass
class QKSeg:
    """Dory's attention rows for ds_qk_rows_l2.  q [R, hq*D], k and v
    [R, hk*D] bf16; q_out [R, hq*D]; k_cache, v_cache [cache_rows, hk*D]
    (row slot[t], or t without slot, receives row t); pos, slot int32 [R];
    inv_freq fp32 [D/2]; q_scale fp32 [hq*D] or None.  Any of q/q_out or
    k/k_cache (v/v_cache) may be None when hq (hk) is 0."""

    head_dim: int
    pos: Any
    inv_freq: Any
    q: Any = None
    q_out: Any = None
    k: Any = None
    k_cache: Any = None
    v: Any = None
    v_cache: Any = None
    slot: Any = None
    q_scale: Any = None

    def to_c(self) -> ds_qkseg:
        D = int(self.head_dim)
        R = int(self.pos.shape[0])
        if self.q is not None:
            if self.q.shape[1] % D:
                raise ValueError("q: width is not a whole number of heads")
            hq = int(self.q.shape[1]) // D
        else:
            hq = 0
        if self.k is not None:
            if self.k.shape[1] % D:
                raise ValueError("k: width is not a whole number of heads")
            hk = int(self.k.shape[1]) // D
        else:
            hk = 0
        q, ld_q = _mat(self.q, "q", R, hq * D)
        qo, ld_qo = _mat(self.q_out, "q_out", R, hq * D)
        k, ld_kv = _mat(self.k, "k", R, hk * D)
        v, ld_v = _mat(self.v, "v", R, hk * D)
        C = 0 if self.k_cache is None else int(self.k_cache.shape[0])
        kc, ld_c = _mat(self.k_cache, "k_cache", C, hk * D)
        vc, ld_vc = _mat(self.v_cache, "v_cache", C, hk * D)
        if hq and ld_qo != ld_q:
            raise ValueError("q and q_out must share a leading dimension")
        if self.v is not None and ld_v != ld_kv:
            raise ValueError("k and v must share a leading dimension")
        if self.v_cache is not None and ld_vc != ld_c:
            raise ValueError("k_cache and v_cache must share a leading dimension")
        return ds_qkseg(q, k, v, qo, kc, vc, _vec(self.pos), _vec(self.slot), _vec(self.inv_freq),
                        _vec(self.q_scale), R, C, ld_q, ld_kv, ld_c, D, hq, hk)


@dataclass
class AGSeg:
    """One activation matrix for the backward calls: x (slerp: res), r (l2:
    residual or None; slerp: out), dy the upstream gradient (bf16 [R, C],
    shared ld), dx (and for slerp dr) fp32 [R, C] outputs with a shared ld,
    alpha fp32 [C] (slerp)."""

    x: Any
    dy: Any
    dx: Any
    r: Any = None
    dr: Any = None
    alpha: Any = None

    def to_c(self) -> ds_agseg:
        R, C = (int(self.x.shape[0]), int(self.x.shape[1]))
        x, ld = _mat(self.x, "x", R, C)
        dy, ldy = _mat(self.dy, "dy", R, C)
        r, ldr = _mat(self.r, "r", R, C)
        dx, ldd = _mat(self.dx, "dx", R, C)
        dr, lddr = _mat(self.dr, "dr", R, C)
        if ldy != ld or (self.r is not None and ldr != ld):
            raise ValueError("x, r and dy must share a leading dimension")
        if self.dr is not None and lddr != ldd:
            raise ValueError("dx and dr must share a leading dimension")
        return ds_agseg(x, r, dy, dx, dr, _vec(self.alpha), R, C, ld, ldd)


# The language-model rows check what their tensors hold: the calls take their
# types from arguments, and a tensor of another type would be read or written
# past its end.  Their smallest calls last a few microseconds on the GPU, so a
# segment is checked in one pass over its tensors and packed into bytes.

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


_CODES = {"bf16": DS_BF16, "f32": DS_F32}


def _type_code(dt) -> int:
    code = _CODES.get(dt) if isinstance(dt, str) else None
    return _dtype_code(dt) if code is None else code


def _tensor_type(code: int):
    return _torch().bfloat16 if code == DS_BF16 else _torch().float32


def _device_of(t) -> int:
    """The device of a call's first tensor, which has to be the current one
    (whose stream the call uses)."""
    dev = t.get_device()
    if dev < 0 or _torch()._C._cuda_getDevice() != dev:
        cur = _torch().cuda.current_device() if _torch().cuda.is_available() else None
        raise ValueError(f"a tensor lies on {t.device}, the current device is {'none' if cur is None else f'cuda:{cur}'}")
    return dev


def _stream_of(stream, dev: int) -> int:
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _wrong(t, name: str, dtype, dev) -> None:
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: expected {str(dtype).replace('torch.', '')}, got {t.dtype}")
    raise ValueError(f"{name}: a tensor lies on {t.device}, the others on cuda:{dev}")


def _matrix(t, name: str, rows: int, cols: int, dtype=None, dev=None) -> tuple[int, int]:
    """(data_ptr, leading dimension) of a 2-D row-major view; (0, cols) for
    None.  dtype, dev: what the tensor has to be (None: not checked)."""
    if t is None:
        return 0, cols
    if (dtype is not None and t.dtype is not dtype) or (dev is not None and t.get_device() != dev):
        if rows or t.dtype is not dtype:
            _wrong(t, name, dtype, dev)
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: expected shape ({rows}, {cols}), got {tuple(t.shape)}")
    s0, s1 = t.stride()
    if rows == 0:
        return t.data_ptr(), cols
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name}: columns must be contiguous")
    if rows > 1:
        return t.data_ptr(), s0
    size = t.element_size()  # one row: its stride leads nowhere, and need not be one that the calls take
    return t.data_ptr(), -(-cols * size // 16) * 16 // size


def _vector(t, name: str, n: int, dtype, dev=None) -> int:
    """data_ptr of a contiguous 1-D tensor of n values; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or (dev is not None and n and t.get_device() != dev):
        _wrong(t, name, dtype, dev)
    if t.numel() != n or t.dim() != 1:
        raise ValueError(f"{name}: expected {n} values, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _id_vector(t, name: str, n: int, dev=None) -> tuple[int, int]:
    """(data_ptr, 1 if 64-bit) of a vector of token ids."""
    if t.dtype is _torch().int64:
        return _vector(t, name, n, _torch().int64, dev), 1
    if t.dtype is not _torch().int32:
        raise ValueError(f"{name}: expected int32 or int64, got {t.dtype}")
    return _vector(t, name, n, _torch().int32, dev), 0


def _workspace(workspace, need: int, dev: int, stream):
    """(data_ptr, bytes, tensor) of the caller's workspace, or of one of `need`
    bytes for this call, allocated for the stream that uses it so that it is
    not handed on before the call's work is done."""
    if workspace is None and (not need or dev < 0):
        return 0, 0, None
    torch = _torch()
    if workspace is None:
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if dev >= 0 and workspace.get_device() != dev:
        _wrong(workspace, "workspace", None, dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _packed(segs, raw, *types) -> tuple[bytes, int, int]:
    """The table of a call as bytes, its segments, and the device (-1: every
    segment is a raw structure)."""
    parts, dev = [], -1
    for s in segs:
        if isinstance(s, raw):
            parts.append(bytes(s))
            continue
        if dev < 0:
            try:
                dev = _device_of(s._first())
            except ValueError:
                s._pack(None, *types)  # a wrong type or shape comes first
                raise
        parts.append(s._pack(dev, *types))
    return parts[0] if len(parts) == 1 else b"".join(parts), len(parts), dev


def _raw_stream(stream, dev: int):
    return _stream_ptr(stream) if dev < 0 else _stream_of(stream, dev)


@dataclass
class ESeg:
    """Embedding rows of one table.  w [V, C] fp32 or bf16; ids int32 or int64
    [T] (negative: padding); y [T, C] output of ds_embed_rows; dy [T, C]
    fp32 or bf16 and grad_w fp32 [V, C], grad_g fp32 [V] ([V + 1] with
    gain_scalar) for ds_embed_rows_backward.  unit: rows are brought to
    length radius (times gain, fp32 [V] or [1] with gain_scalar); otherwise
    y = radius * w and the gradient needs no w.  accumulate: add to grad_w and
    grad_g instead of writing every row."""

    w: Any
    ids: Any
    y: Any = None
    gain: Any = None
    dy: Any = None
    grad_w: Any = None
    grad_g: Any = None
    radius: float = 1.0
    unit: bool = False
    gain_scalar: bool = False
    accumulate: bool = False

    def _first(self):
        return self.ids

    def _pack(self, dev=None, w_type=None, y_type=None, call="") -> bytes:
        """call: "forward" or "backward" packs what that call reads and writes."""
        fwd, back = call != "backward", call != "forward"
        table = self.w if self.w is not None else self.grad_w
        if table is None:
            raise ValueError("w or grad_w is needed")
        V, C = table.shape
        T = self.ids.shape[0]
        f32 = _torch().float32
        ids, wide = _id_vector(self.ids, "ids", T, dev)
        w, ld = _matrix(self.w, "w", V, C, w_type, dev)
        y, ld_y = _matrix(self.y if fwd else None, "y", T, C, y_type, dev)
        dy, ld_dy = _matrix(self.dy if back else None, "dy", T, C, y_type, dev)
        gw, ld_g = _matrix(self.grad_w if back else None, "grad_w", V, C, f32, dev)
        if not y:
            ld_y = ld_dy
        elif dy and ld_y != ld_dy:
            raise ValueError("y and dy must share a leading dimension")
        one = 1 if self.gain_scalar else 0
        gain = grad_g = 0
        if self.gain is not None:
            gain = _vector(self.gain, "gain", 1 if one else V, f32, dev)
            grad_g = _vector(self.grad_g if back else None, "grad_g", V + one, f32, dev)
        return _ESEG(w, gain, ids, y, dy, gw, grad_g, T, V, C, ld, ld_y, ld_g, self.radius, 1 if self.unit else 0, one,
                     wide, 1 if self.accumulate else 0)

    def to_c(self) -> ds_eseg:
        return ds_eseg.from_buffer_copy(self._pack())


def _heads(t, D: int, name: str) -> int:
    if t is None:
        return 0
    if D < 1:
        raise ValueError("head_dim must be positive")
    if t.dim() != 2 or t.shape[1] % D:
        raise ValueError(f"{name}: width is not a whole number of heads")
    return t.shape[1] // D


@dataclass
class QNSeg:
    """q and k rows for ds_qk_norm_rows.  q [R, hq*D], k and v [R, hk*D] (they
    may be columns of one matrix); q_out [R, hq*D]; k_cache, v_cache
    [cache_rows, hk*D] (row slot[t], or t without slot, receives row t; a
    negative slot stores nothing); wq, wk fp32 [D] or None; pos, slot int32
    [R]; inv_freq fp32 [rot_dim/2] (rot_dim None: head_dim; 0: no rotation).
    interleaved: pairs (2i, 2i+1) instead of halves.  mean: the norm over the
    mean of squares (RMS) instead of their sum (L2)."""

    head_dim: int
    q: Any = None
    q_out: Any = None
    k: Any = None
    k_cache: Any = None
    v: Any = None
    v_cache: Any = None
    wq: Any = None
    wk: Any = None
    pos: Any = None
    slot: Any = None
    inv_freq: Any = None
    rot_dim: int | None = None
    interleaved: bool = False
    mean: bool = False

    def _first(self):
        if self.q is None and self.k is None:
            raise ValueError("q or k is needed")
        return self.q if self.q is not None else self.k

    def _pack(self, dev=None, dtype=None) -> bytes:
        D = self.head_dim
        rot = D if self.rot_dim is None else self.rot_dim
        hq, hk = _heads(self.q, D, "q"), _heads(self.k, D, "k")
        R = self._first().shape[0]
        wq, wk = hq * D, hk * D
        q, ld_q = _matrix(self.q, "q", R, wq, dtype, dev)
        qo, ld_qo = _matrix(self.q_out, "q_out", R, wq, dtype, dev)
        k, ld_kv = _matrix(self.k, "k", R, wk, dtype, dev)
        v, ld_v = _matrix(self.v, "v", R, wk, dtype, dev)
        C = 0 if self.k_cache is None else self.k_cache.shape[0]
        kc, ld_c = _matrix(self.k_cache, "k_cache", C, wk, dtype, dev)
        vc, ld_vc = _matrix(self.v_cache, "v_cache", C, wk, dtype, dev)
        if v and ld_v != ld_kv and R > 1:
            raise ValueError("k and v must share a leading dimension")
        if vc and ld_vc != ld_c and C > 1:
            raise ValueError("k_cache and v_cache must share a leading dimension")
        torch = _torch()
        f32, i32 = torch.float32, torch.int32
        pos = inv = 0
        if rot > 0:
            pos = _vector(self.pos, "pos", R, i32, dev)
            inv = _vector(self.inv_freq, "inv_freq", rot // 2, f32, dev)
        return _QNSEG(q, k, v, qo, kc, vc, _vector(self.wq, "wq", D, f32, dev), _vector(self.wk, "wk", D, f32, dev), pos,
                      _vector(self.slot, "slot", R, i32, dev), inv, R, C, ld_q, ld_kv, ld_qo, ld_c, D, rot, hq, hk,
                      1 if self.interleaved else 0, 1 if self.mean else 0)

    def to_c(self) -> ds_qnseg:
        return ds_qnseg.from_buffer_copy(self._pack())


@dataclass
class QNGSeg:
    """The gradient of QNSeg's rows for ds_qk_norm_rows_backward: q, k its
    inputs, dq_out, dk_out the gradients of its outputs (row for row), dq, dk
    the gradients written."""

    head_dim: int
    q: Any = None
    dq_out: Any = None
    dq: Any = None
    k: Any = None
    dk_out: Any = None
    dk: Any = None
    wq: Any = None
    wk: Any = None
    pos: Any = None
    inv_freq: Any = None
    rot_dim: int | None = None
    interleaved: bool = False
    mean: bool = False

    _first = QNSeg._first

    def _pack(self, dev=None, dtype=None, grad_type=None) -> bytes:
        D = self.head_dim
        rot = D if self.rot_dim is None else self.rot_dim
        hq, hk = _heads(self.q, D, "q"), _heads(self.k, D, "k")
        R = self._first().shape[0]
        wq, wk = hq * D, hk * D
        q, ld_q = _matrix(self.q, "q", R, wq, dtype, dev)
        k, ld_kv = _matrix(self.k, "k", R, wk, dtype, dev)
        dqo, ld_dqo = _matrix(self.dq_out, "dq_out", R, wq, dtype, dev)
        dko, ld_dko = _matrix(self.dk_out, "dk_out", R, wk, dtype, dev)
        dq, ld_dq = _matrix(self.dq, "dq", R, wq, grad_type, dev)
        dk, ld_dk = _matrix(self.dk, "dk", R, wk, grad_type, dev)
        f32 = _torch().float32
        pos = inv = 0
        if rot > 0:
            pos = _vector(self.pos, "pos", R, _torch().int32, dev)
            inv = _vector(self.inv_freq, "inv_freq", rot // 2, f32, dev)
        return _QNGSEG(q, k, dqo, dko, dq, dk, _vector(self.wq, "wq", D, f32, dev), _vector(self.wk, "wk", D, f32, dev),
                       pos, inv, R, ld_q, ld_kv, ld_dqo, ld_dko, ld_dq, ld_dk, D, rot, hq, hk,
                       1 if self.interleaved else 0, 1 if self.mean else 0)

    def to_c(self) -> ds_qngseg:
        return ds_qngseg.from_buffer_copy(self._pack())


@dataclass
class LSeg:
    """Rows of logits.  x [R, V] fp32 or bf16; ids int32 or int64 [R]
    (negative: not scored).  ds_logp_rows writes whichever of logp, lse,
    entropy (fp32 [R]), top_id (int32 [R, k]) and top_logp (fp32 [R, k]) are
    given.  ds_logp_rows_backward reads lse (and entropy), dlogp, dentropy,
    dlse (fp32 [R] or None) and writes dx [R, V].  scale: 1 / temperature."""

    x: Any
    ids: Any = None
    logp: Any = None
    lse: Any = None
    entropy: Any = None
    top_id: Any = None
    top_logp: Any = None
    dlogp: Any = None
    dentropy: Any = None
    dlse: Any = None
    dx: Any = None
    scale: float = 1.0

    def _first(self):
        return self.x

    def _pack(self, dev=None, dtype=None, grad_type=None) -> bytes:
        R, V = self.x.shape
        f32 = _torch().float32
        x, ld = _matrix(self.x, "x", R, V, dtype, dev)
        dx, ld_d = _matrix(self.dx, "dx", R, V, grad_type, dev)
        ids, wide = (0, 0) if self.ids is None else _id_vector(self.ids, "ids", R, dev)
        k = top = tlp = 0
        if self.top_id is not None:
            k = self.top_id.shape[1]
            top = _matrix(self.top_id, "top_id", R, k, _torch().int32, dev)[0]
            tlp = _matrix(self.top_logp, "top_logp", R, k, f32, dev)[0]
            if not self.top_id.is_contiguous() or not (self.top_logp is None or self.top_logp.is_contiguous()):
                raise ValueError("top_id and top_logp must be contiguous")
        elif self.top_logp is not None:
            raise ValueError("top_logp needs top_id")
        return _LSEG(x, ids, _vector(self.logp, "logp", R, f32, dev), _vector(self.lse, "lse", R, f32, dev),
                     _vector(self.entropy, "entropy", R, f32, dev), top, tlp, _vector(self.dlogp, "dlogp", R, f32, dev),
                     _vector(self.dentropy, "dentropy", R, f32, dev), _vector(self.dlse, "dlse", R, f32, dev), dx, R, V, ld,
                     ld_d, self.scale, k, wide)

    def to_c(self) -> ds_lseg:
        return ds_lseg.from_buffer_copy(self._pack())


def _table(segs, cls):
    items = [s if isinstance(s, cls) else s.to_c() for s in segs]
    arr = (cls * max(1, len(items)))(*items)
    return arr, len(items)


def ds_wn_forward(segs: Sequence, out_dtype="bf16", eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_wseg)
    _check(_lib.ds_wn_forward(arr, n, _dtype_code(out_dtype), eps, _stream_ptr(stream)), "ds_wn_forward")


def ds_wn_backward(segs: Sequence, gy_dtype="bf16", eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_wseg)
    _check(_lib.ds_wn_backward(arr, n, _dtype_code(gy_dtype), eps, _stream_ptr(stream)), "ds_wn_backward")


def ds_row_renorm(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_wseg)
    _check(_lib.ds_row_renorm(arr, n, eps, _stream_ptr(stream)), "ds_row_renorm")


def ds_grad_project(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_wseg)
    _check(_lib.ds_grad_project(arr, n, eps, _stream_ptr(stream)), "ds_grad_project")


def ds_renorm_momentum(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_wseg)
    _check(_lib.ds_renorm_momentum(arr, n, eps, _stream_ptr(stream)), "ds_renorm_momentum")


def ds_l2_rows(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_aseg)
    _check(_lib.ds_l2_rows(arr, n, eps, _stream_ptr(stream)), "ds_l2_rows")


def ds_slerp_rows(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_aseg)
    _check(_lib.ds_slerp_rows(arr, n, eps, _stream_ptr(stream)), "ds_slerp_rows")


def ds_gate_l2_rows(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_fseg)
    _check(_lib.ds_gate_l2_rows(arr, n, eps, _stream_ptr(stream)), "ds_gate_l2_rows")


def ds_swiglu_l2_rows(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_fseg)
    _check(_lib.ds_swiglu_l2_rows(arr, n, eps, _stream_ptr(stream)), "ds_swiglu_l2_rows")


def ds_row_norms(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_wseg)
    _check(_lib.ds_row_norms(arr, n, eps, _stream_ptr(stream)), "ds_row_norms")


def ds_gain_preserve(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_wseg)
    _check(_lib.ds_gain_preserve(arr, n, eps, _stream_ptr(stream)), "ds_gain_preserve")


def ds_qk_rows_l2(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_qkseg)
    _check(_lib.ds_qk_rows_l2(arr, n, eps, _stream_ptr(stream)), "ds_qk_rows_l2")


def ds_l2_rows_backward(segs: Sequence, eps: float = 1e-6, stream=None) -> None:
    arr, n = _table(segs, ds_agseg)
    _check(_lib.ds_l2_rows_backward(arr, n, eps, _stream_ptr(stream)), "ds_l2_rows_backward")


def ds_slerp_rows_backward_workspace(cols: int) -> int:
    """Workspace bytes ds_slerp_rows_backward needs for dalpha over `cols` columns."""
    return int(_lib.ds_slerp_rows_backward_workspace(cols))


def ds_slerp_rows_backward(segs: Sequence, eps: float = 1e-6, dalpha=None, workspace=None, stream=None) -> None:
    """dalpha: fp32 [cols] CUDA tensor or None.  workspace: a CUDA tensor of at
    least ds_slerp_rows_backward_workspace(cols) bytes (256-byte aligned), or
    None to have one allocated here for this call."""
    arr, n = _table(segs, ds_agseg)
    ws_ptr, ws_bytes = 0, 0
    if dalpha is not None:
        cols = int(arr[0].cols) if n else 0
        need = ds_slerp_rows_backward_workspace(cols) if cols else 0
        if workspace is None and need:
            import torch

            workspace = torch.empty(need, dtype=torch.uint8, device=dalpha.device)
        if workspace is not None:
            ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(_lib.ds_slerp_rows_backward(arr, n, eps, _vec(dalpha), ws_ptr, ws_bytes, _stream_ptr(stream)),
           "ds_slerp_rows_backward")


def ds_slerp_rows_backward_noalloc(segs: Sequence, eps: float = 1e-6, dalpha=None, stream=None) -> None:
    """ds_slerp_rows_backward for callers that cannot allocate device memory
    where they run the backward (their device memory all belongs to a pool
    of their own, or they must avoid the implicit synchronisation of
    cudaMalloc / cudaFree): dalpha's partial sums go to the library's
    built-in 64 MB scratch instead of a workspace.  Rows needing more than
    that are refused; calls must not overlap on the GPU."""
    arr, n = _table(segs, ds_agseg)
    _check(_lib.ds_slerp_rows_backward_noalloc(arr, n, eps, _vec(dalpha), _stream_ptr(stream)),
           "ds_slerp_rows_backward_noalloc")


def ds_embed_rows(segs: Sequence, w_dtype="f32", out_dtype="bf16", eps: float = 1e-6, stream=None) -> None:
    wd, od = _type_code(w_dtype), _type_code(out_dtype)
    table, n, dev = _packed(segs, ds_eseg, _tensor_type(wd), _tensor_type(od), "forward")
    _check(_lib.ds_embed_rows(table, n, wd, od, eps, _raw_stream(stream, dev)), "ds_embed_rows")


def ds_embed_rows_backward_workspace(tokens: int, vocab: int, cols: int) -> int:
    """Workspace bytes ds_embed_rows_backward needs for one segment."""
    return int(_lib.ds_embed_rows_backward_workspace(tokens, vocab, cols))


def ds_embed_rows_backward(segs: Sequence, w_dtype="f32", dy_dtype="bf16", eps: float = 1e-6, workspace=None,
                           stream=None) -> None:
    """workspace: a CUDA tensor of at least the largest
    ds_embed_rows_backward_workspace(tokens, vocab, cols) of the segments
    (256-byte aligned), or None to have one allocated here for this call."""
    wd, dd = _type_code(w_dtype), _type_code(dy_dtype)
    table, n, dev = _packed(segs, ds_eseg, _tensor_type(wd), _tensor_type(dd), "backward")
    need = 0
    if workspace is None and dev >= 0:
        need = max(ds_embed_rows_backward_workspace(s.tokens, s.vocab, s.cols)
                   for s in (ds_eseg * n).from_buffer_copy(table))
    ptr, size, workspace = _workspace(workspace, need, dev, stream)
    _check(_lib.ds_embed_rows_backward(table, n, wd, dd, eps, ptr, size, _raw_stream(stream, dev)),
           "ds_embed_rows_backward")


def ds_qk_norm_rows(segs: Sequence, dtype="bf16", eps: float = 1e-6, stream=None) -> None:
    dt = _type_code(dtype)
    table, n, dev = _packed(segs, ds_qnseg, _tensor_type(dt))
    _check(_lib.ds_qk_norm_rows(table, n, dt, eps, _raw_stream(stream, dev)), "ds_qk_norm_rows")


def ds_qk_norm_rows_backward_workspace(head_dim: int) -> int:
    """Workspace bytes ds_qk_norm_rows_backward needs for dwq and dwk."""
    return int(_lib.ds_qk_norm_rows_backward_workspace(head_dim))


def ds_qk_norm_rows_backward(segs: Sequence, dtype="bf16", grad_dtype="bf16", eps: float = 1e-6, dwq=None, dwk=None,
                             workspace=None, stream=None) -> None:
    """dwq, dwk: fp32 [head_dim] outputs or None.  workspace: a CUDA tensor of
    at least ds_qk_norm_rows_backward_workspace(head_dim) bytes (256-byte
    aligned), or None to have one allocated here for this call."""
    dt, gd = _type_code(dtype), _type_code(grad_dtype)
    table, n, dev = _packed(segs, ds_qngseg, _tensor_type(dt), _tensor_type(gd))
    need = 0
    if n and (dwq is not None or dwk is not None):
        D = ds_qngseg.from_buffer_copy(table).head_dim
        need = ds_qk_norm_rows_backward_workspace(D)
        f32, on = _torch().float32, dev if dev >= 0 else None
        dwq, dwk = _vector(dwq, "dwq", D, f32, on), _vector(dwk, "dwk", D, f32, on)
    else:
        dwq = dwk = 0
    ptr, size, workspace = _workspace(workspace, need, dev, stream)
    _check(_lib.ds_qk_norm_rows_backward(table, n, dt, gd, eps, dwq, dwk, ptr, size, _raw_stream(stream, dev)),
           "ds_qk_norm_rows_backward")


def ds_logp_rows(segs: Sequence, dtype="bf16", stream=None) -> None:
    dt = _type_code(dtype)
    table, n, dev = _packed(segs, ds_lseg, _tensor_type(dt))
    _check(_lib.ds_logp_rows(table, n, dt, _raw_stream(stream, dev)), "ds_logp_rows")


def ds_logp_rows_backward(segs: Sequence, dtype="bf16", grad_dtype=None, stream=None) -> None:
    """grad_dtype: dx's type (None: dtype)."""
    dt = _type_code(dtype)
    gd = dt if grad_dtype is None else _type_code(grad_dtype)
    table, n, dev = _packed(segs, ds_lseg, _tensor_type(dt), _tensor_type(gd))
    _check(_lib.ds_logp_rows_backward(table, n, dt, gd, _raw_stream(stream, dev)), "ds_logp_rows_backward")


def ds_get_device_status(stream=None) -> int:
    """Synchronise the stream; return (and clear) the device error word."""
    return int(_lib.ds_get_device_status(_stream_ptr(stream)))


def ds_launch_count() -> int:
    return int(_lib.ds_launch_count())


def ds_version() -> int:
    return int(_lib.ds_version())


def ds_status_string(status: int) -> str:
    return _lib.ds_status_string(status).decode()


def ds_last_error() -> str:
    return _lib.ds_last_error().decode()


def ds_row_class(op: int, cols: int) -> tuple[int, int, int]:
    """(path, threads per row, CTAs per row) the library picks for this row length."""
    p, g, c = ct.c_int(), ct.c_int(), ct.c_int()
    _check(_lib.ds_row_class(op, cols, ct.byref(p), ct.byref(g), ct.byref(c)), "ds_row_class")
    return p.value, g.value, c.value


def ds_debug_force_path(path: int) -> None:
    _check(_lib.ds_debug_force_path(path), "ds_debug_force_path")


def ds_debug_set_wait_limit_ns(limit_ns: int) -> None:
    _check(_lib.ds_debug_set_wait_limit_ns(limit_ns), "ds_debug_set_wait_limit_ns")


def ds_debug_wait_timeout_selftest(limit_ns: int, stream=None) -> None:
    _check(_lib.ds_debug_wait_timeout_selftest(limit_ns, _stream_ptr(stream)), "ds_debug_wait_timeout_selftest")


def ds_debug_division_check(stream=None) -> tuple[int, int, int, int]:
    """(reciprocal mismatches, quotient mismatches, reciprocal inputs checked,
    quotient inputs checked) of the Dory rows' fast division over every fp32
    input; synchronises the stream."""
    import torch

    counts = torch.zeros(4, dtype=torch.int64, device="cuda")
    _check(_lib.ds_debug_division_check(counts.data_ptr(), _stream_ptr(stream)), "ds_debug_division_check")
    torch.cuda.synchronize()
    return tuple(int(v) for v in counts.tolist())


class force_path:
    """Context manager: run the enclosed calls on one path (tests)."""

    def __init__(self, path: int):
        self.path = path

    def __enter__(self):
        ds_debug_force_path(self.path)
        return self

    def __exit__(self, *exc):
        ds_debug_force_path(DS_PATH_AUTO)
        return False
