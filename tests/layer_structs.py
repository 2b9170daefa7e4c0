"""The argument structs of include/sol_attn.h's layer operators, field by field, for tests that call the library itself."""
import ctypes

_vp, _i, _ll, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float


class Rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("dtype", _i), ("stride_b", _ll), ("stride_l", _ll)]


class Vectors(ctypes.Structure):
    _fields_ = [("data", _vp), ("dtype", _i), ("groups", _i), ("stride_b", _ll), ("stride_g", _ll)]


class NormArgs(ctypes.Structure):
    _fields_ = [("B", _i), ("L", _i), ("C", _i), ("x_inner", _i), ("x_stride_h", _ll), ("x", Rows), ("y", Rows),
                ("x_out", Rows), ("h", Rows), ("q", _vp), ("q_stride", _ll), ("q_scale", _vp),
                ("residual_scale", _f), ("norm", _i), ("eps", _f), ("post_norm", _i), ("post_eps", _f),
                ("scale", Vectors), ("shift", Vectors), ("gate", Vectors), ("weight", Vectors),
                ("bias", Vectors), ("post_weight", Vectors), ("post_bias", Vectors)]


class RopeTensor(ctypes.Structure):
    _fields_ = [("in_", _vp), ("stride_b", _ll), ("stride_l", _ll), ("stride_h", _ll), ("out", _vp),
                ("weight", _vp), ("weight_dtype", _i)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("B", _i), ("L", _i), ("H", _i), ("d", _i), ("dtype", _i), ("q", RopeTensor), ("k", RopeTensor),
                ("v", RopeTensor), ("norm", _i), ("eps", _f), ("pairing", _i), ("axes", _i), ("freqs", _vp),
                ("axis", _vp), ("pos_kind", _i), ("grid_f", _i), ("grid_h", _i), ("grid_w", _i), ("start", _ll),
                ("positions", _vp), ("pos_stride_b", _ll), ("pos_stride_l", _ll), ("pos_stride_a", _ll)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("M", _i), ("N", _i), ("K", _i), ("a", _vp), ("a_stride", _ll), ("a_scale", _vp), ("w", _vp),
                ("w_stride", _ll), ("w_scale", _vp), ("bias", _vp), ("bias_dtype", _i), ("out", _vp), ("out_dtype", _i),
                ("out_stride", _ll), ("flags", ctypes.c_uint)]
