"""The layer operators of include/libgdn_layer.h for ctypes: names, structures and
argument types.  (No torch here: the library loads without it.)"""
from __future__ import annotations

import ctypes

GDN_E4M3 = 2
LAYER_EXPORTS = ["gdn_norm_forward", "gdn_norm_backward", "gdn_workspace_bytes_norm_backward",
                 "gdn_conv_forward", "gdn_conv_backward", "gdn_workspace_bytes_conv_backward",
                 "gdn_conv_step", "gdn_ssm_forward", "gdn_workspace_bytes_ssm", "gdn_ssm_backward",
                 "gdn_workspace_bytes_ssm_backward", "gdn_ssm_step",
                 "gdn_layer_norm_forward", "gdn_layer_norm_backward", "gdn_workspace_bytes_layer_norm_backward",
                 "gdn_gate_norm_forward", "gdn_gate_norm_backward", "gdn_workspace_bytes_gate_norm_backward",
                 "gdn_glr_forward", "gdn_workspace_bytes_glr", "gdn_glr_backward", "gdn_workspace_bytes_glr_backward",
                 "gdn_glr_step"]

_I64, _I32, _F32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", _I64), ("D", _I64), ("x_stride", _I64), ("x_dtype", _I32), ("s_dtype", _I32),
                ("w_dtype", _I32), ("out_dtype", _I32), ("group", _I32), ("eps", _F32)]


class ConvProblem(ctypes.Structure):
    _fields_ = [("B", _I64), ("T", _I64), ("D", _I64), ("W", _I64), ("x_stride_b", _I64),
                ("x_stride_t", _I64), ("dy_stride_b", _I64), ("dy_stride_t", _I64), ("n_seqs", _I64),
                ("io_dtype", _I32), ("w_dtype", _I32), ("silu", _I32)]


class SsmProblem(ctypes.Structure):
    _fields_ = [("B", _I64), ("T", _I64), ("H", _I64), ("P", _I64), ("N", _I64), ("G", _I64),
                ("x_stride_b", _I64), ("x_stride_t", _I64), ("bc_stride_b", _I64), ("bc_stride_t", _I64),
                ("dt_stride_b", _I64), ("dt_stride_t", _I64), ("dxbc_stride_b", _I64),
                ("dxbc_stride_t", _I64), ("n_seqs", _I64), ("io_dtype", _I32), ("dt_dtype", _I32),
                ("softplus", _I32)]


class GateNormProblem(ctypes.Structure):
    _fields_ = [("T", _I64), ("H", _I64), ("D", _I64), ("x_stride_t", _I64), ("x_stride_h", _I64), ("z_stride_t", _I64),
                ("z_stride_h", _I64), ("dz_stride_t", _I64), ("dz_stride_h", _I64), ("io_dtype", _I32), ("w_dtype", _I32),
                ("each", _I32), ("gate_first", _I32), ("center", _I32), ("act", _I32), ("eps", _F32)]


class GlrProblem(ctypes.Structure):
    _fields_ = [("B", _I64), ("T", _I64), ("D", _I64), ("x_stride_b", _I64), ("x_stride_t", _I64), ("g_stride_b", _I64),
                ("g_stride_t", _I64), ("dy_stride_b", _I64), ("dy_stride_t", _I64), ("dx_stride_b", _I64), ("dx_stride_t", _I64),
                ("dg_stride_b", _I64), ("dg_stride_t", _I64), ("n_seqs", _I64), ("io_dtype", _I32), ("g_dtype", _I32),
                ("form", _I32), ("scale", _I32)]


def declare(lib):
    """Argument types of the layer operators' functions."""
    vp, sz, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
    n, c, s, g, r = (ctypes.POINTER(t) for t in (NormProblem, ConvProblem, SsmProblem, GateNormProblem, GlrProblem))
    lib.gdn_norm_forward.argtypes = [n] + [vp] * 7
    lib.gdn_norm_backward.argtypes = [n] + [vp] * 8 + [sz, vp]
    lib.gdn_conv_forward.argtypes = [c] + [vp] * 8
    lib.gdn_conv_backward.argtypes = [c] + [vp] * 12 + [sz, vp]
    lib.gdn_conv_step.argtypes = [c] + [vp] * 5 + [i64, vp, vp]
    lib.gdn_ssm_forward.argtypes = [s] + [vp] * 12 + [sz, vp]
    lib.gdn_ssm_backward.argtypes = [s] + [vp] * 20 + [sz, vp]
    lib.gdn_ssm_step.argtypes = [s] + [vp] * 9 + [i64, vp, vp]
    lib.gdn_layer_norm_forward.argtypes = [n] + [vp] * 8
    lib.gdn_layer_norm_backward.argtypes = [n] + [vp] * 9 + [sz, vp]
    lib.gdn_gate_norm_forward.argtypes = [g] + [vp] * 6
    lib.gdn_gate_norm_backward.argtypes = [g] + [vp] * 10 + [sz, vp]
    lib.gdn_glr_forward.argtypes = [r] + [vp] * 9 + [sz, vp]
    lib.gdn_glr_backward.argtypes = [r] + [vp] * 14 + [sz, vp]
    lib.gdn_glr_step.argtypes = [r] + [vp] * 6 + [i64, vp, vp]
    for name, arg in (("norm_backward", n), ("conv_backward", c), ("ssm", s), ("ssm_backward", s), ("layer_norm_backward", n),
                      ("gate_norm_backward", g), ("glr", r), ("glr_backward", r)):
        f = getattr(lib, "gdn_workspace_bytes_" + name)
        f.argtypes, f.restype = [arg], sz
    for name in LAYER_EXPORTS:
        if "workspace" not in name:
            getattr(lib, name).restype = ctypes.c_int
