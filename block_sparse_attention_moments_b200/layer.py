"""Operators around the attention of a diffusion-transformer layer.

Thin bindings of sol_attn_norm_modulate, sol_attn_rope and
sol_attn_quantized_linear in ``include/sol_attn.h``: they check tensor properties, allocate the outputs and
marshal pointers; all arithmetic runs in the library's CUDA kernels.  Forward
only, as the attention is: a call whose inputs ask for gradients is refused.

Every call works on the device of its tensors, on ``stream`` (a torch stream
of that device) or that device's current one, holds no workspace and can be
captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _check, forward, lib

__all__ = ["norm_modulate", "gate_residual", "gate_residual_norm", "quantize_rows", "rope", "rope_axes",
           "int8_linear", "linear_status", "AttentionLayer"]

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_NORMS = {"none": 0, "layer": 1, "rms": 2}
_ROPE_NORMS = {"none": 0, "head": 1, "token": 2}
_PAIRINGS = {"interleaved": 0, "half": 1}
_POSITIONS = {torch.int32: 1, torch.int64: 2, torch.float32: 3, torch.float64: 4}

_vp, _i, _ll, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float


class _Rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("dtype", _i), ("stride_b", _ll), ("stride_l", _ll)]


class _Vectors(ctypes.Structure):
    _fields_ = [("data", _vp), ("dtype", _i), ("groups", _i), ("stride_b", _ll), ("stride_g", _ll)]


class _NormArgs(ctypes.Structure):
    _fields_ = [("B", _i), ("L", _i), ("C", _i), ("x_inner", _i), ("x_stride_h", _ll), ("x", _Rows), ("y", _Rows),
                ("x_out", _Rows), ("h", _Rows), ("q", _vp), ("q_stride", _ll), ("q_scale", _vp),
                ("residual_scale", _f), ("norm", _i), ("eps", _f), ("post_norm", _i), ("post_eps", _f),
                ("scale", _Vectors), ("shift", _Vectors), ("gate", _Vectors), ("weight", _Vectors),
                ("bias", _Vectors), ("post_weight", _Vectors), ("post_bias", _Vectors)]


class _RopeTensor(ctypes.Structure):
    _fields_ = [("in_", _vp), ("stride_b", _ll), ("stride_l", _ll), ("stride_h", _ll), ("out", _vp),
                ("weight", _vp), ("weight_dtype", _i)]


class _RopeArgs(ctypes.Structure):
    _fields_ = [("B", _i), ("L", _i), ("H", _i), ("d", _i), ("dtype", _i), ("q", _RopeTensor), ("k", _RopeTensor),
                ("v", _RopeTensor), ("norm", _i), ("eps", _f), ("pairing", _i), ("axes", _i), ("freqs", _vp),
                ("axis", _vp), ("pos_kind", _i), ("grid_f", _i), ("grid_h", _i), ("grid_w", _i), ("start", _ll),
                ("positions", _vp), ("pos_stride_b", _ll), ("pos_stride_l", _ll), ("pos_stride_a", _ll)]


class _LinearArgs(ctypes.Structure):
    _fields_ = [("M", _i), ("N", _i), ("K", _i), ("a", _vp), ("a_stride", _ll), ("a_scale", _vp), ("w", _vp),
                ("w_stride", _ll), ("w_scale", _vp), ("bias", _vp), ("bias_dtype", _i), ("out", _vp), ("out_dtype", _i),
                ("out_stride", _ll)]


# ------------------------------------------------------------------ checks
def _input(t, name, device=None, dtypes=_DTYPES):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has the unsupported type {t.dtype}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and there is no backward pass: call under torch.no_grad()")


def _choice(value, choices, name):
    if value not in choices:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, choices))} (got {value!r})")
    return choices[value]


def _tokens(t, name):
    """(B, L, C, stride_b, stride_l) of a [B, L, C] or [L, C] tensor."""
    if t.dim() == 3:
        B, L, C = t.shape
        sb, sl, sc = t.stride()
    elif t.dim() == 2:
        (L, C), B, sb = t.shape, 1, 0
        sl, sc = t.stride()
    else:
        raise ValueError(f"{name} must be [B, L, C] or [L, C]")
    if C > 1 and sc != 1:
        raise ValueError(f"{name}: the channels of a token must be contiguous")
    return B, L, C, sb, sl


def _rows(t, name):
    _, _, _, sb, sl = _tokens(t, name)
    return _Rows(t.data_ptr(), _DTYPES[t.dtype], sb, sl)


def _vectors(t, name, B, L, C, device, plain=False):
    """[C], [B, C] or [B, G, C] (B may be 1: the same for every batch element); plain: [C] only."""
    if t is None:
        return _Vectors()
    _input(t, name, device)
    if t.dim() == 1 and t.shape[0] == C:
        G, sb, sg = 1, 0, 0
    elif t.dim() == 2 and not plain and t.shape[1] == C and t.shape[0] in (1, B):
        G, sb, sg = 1, t.stride(0) if t.shape[0] > 1 else 0, 0
    elif t.dim() == 3 and not plain and t.shape[2] == C and t.shape[0] in (1, B) and (t.shape[1] > 0 and L % t.shape[1] == 0):
        G, sb, sg = t.shape[1], t.stride(0) if t.shape[0] > 1 else 0, t.stride(1)
    else:
        want = f"[{C}]" if plain else f"[{C}], [{B}, {C}] or [{B}, G, {C}] with G dividing {L}"
        raise ValueError(f"{name} must be {want} (got {list(t.shape)})")
    if C > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels must be contiguous")
    return _Vectors(t.data_ptr(), _DTYPES[t.dtype], G, sb, sg)


def _output(out, name, like, dtype):
    if out is None:
        return torch.empty(like.shape, device=like.device, dtype=dtype)
    if not isinstance(out, torch.Tensor) or out.device != like.device or out.dtype != dtype or out.shape != like.shape:
        raise ValueError(f"{name} must be a {dtype} tensor {list(like.shape)} on {like.device}")
    if out.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and there is no backward pass: call under torch.no_grad()")
    return out


def _padded_rows(shape, device):
    """int8 [..., K] whose rows start at multiples of 16 bytes, and its row pitch."""
    pitch = (shape[-1] + 15) // 16 * 16
    return torch.empty(*shape[:-1], pitch, device=device, dtype=torch.int8)[..., :shape[-1]], pitch


def _placed(fn):
    """Runs fn with its first tensor's device current and, where a stream is given, with that stream current,
    so that outputs belong to it; the inputs are marked as used by it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        x = args[0] if args else next(iter(kw.values()), None)
        if isinstance(x, torch.Tensor) and x.is_cuda:
            if stream is not None:
                if stream.device != x.device:
                    raise ValueError(f"stream is on {stream.device}, the tensors on {x.device}")
                if stream != torch.cuda.current_stream(x.device):
                    for t in (*args, *kw.values()):
                        if isinstance(t, torch.Tensor) and t.is_cuda:
                            t.record_stream(stream)
                with torch.cuda.stream(stream):
                    return fn(*args, **kw)
            if x.device.index != torch.cuda.current_device():
                with torch.cuda.device(x.device):
                    return fn(*args, **kw)
        return fn(*args, **kw)
    return call


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# ------------------------------------------------------------------ norms
def _norm_call(x, y, gate, scale, shift, residual_scale, post_norm, post_weight, post_bias, post_eps, norm, weight, bias,
               eps, out_dtype, quantize, x_out, want_x, want_h, out):
    _input(x, "x")
    B, L, C, sb, sl = _tokens(x, "x")
    if C < 1:
        raise ValueError("x has no channels")
    dev = x.device
    a = _NormArgs(B=B, L=L, C=C, x_inner=C, x=_Rows(x.data_ptr(), _DTYPES[x.dtype], sb, sl), residual_scale=residual_scale,
                  norm=_choice(norm, _NORMS, "norm"), eps=eps, post_norm=_choice(post_norm, _NORMS, "post_norm"),
                  post_eps=post_eps)
    if weight is not None or bias is not None:
        a.weight = _vectors(weight, "weight", B, L, C, dev, True)
        a.bias = _vectors(bias, "bias", B, L, C, dev, True)
    a.scale = _vectors(scale, "scale", B, L, C, dev)
    a.shift = _vectors(shift, "shift", B, L, C, dev)
    h_dtype = x.dtype
    if y is not None:
        _input(y, "y", dev)
        if y.shape != x.shape:
            raise ValueError("x and y must share one shape")
        a.y = _rows(y, "y")
        a.gate = _vectors(gate, "gate", B, L, C, dev)
        if post_weight is not None or post_bias is not None:
            a.post_weight = _vectors(post_weight, "post_weight", B, L, C, dev, True)
            a.post_bias = _vectors(post_bias, "post_bias", B, L, C, dev, True)
        h_dtype = y.dtype
        if y.dtype != x.dtype and x.dtype != torch.float32:
            raise ValueError("y must have the type of x, or x must be float32")
    if out_dtype is not None and out_dtype != h_dtype:
        if y is not None:
            raise ValueError("out_dtype must be the type of y")
        if out_dtype not in _DTYPES or x.dtype != torch.float32:
            raise ValueError("out_dtype must be the type of x, or x must be float32")
        h_dtype = out_dtype
    if quantize and (out is not None or out_dtype is not None):
        raise ValueError("quantize=True takes neither out nor out_dtype")
    results = []
    if want_x:
        x_out = _output(x_out, "x_out", x, x.dtype)
        a.x_out = _rows(x_out, "x_out")
        results.append(x_out)
    if want_h and quantize:
        q, pitch = _padded_rows(x.shape, dev)
        s = torch.empty(x.shape[:-1], device=dev, dtype=torch.float32)
        a.q, a.q_stride, a.q_scale = q.data_ptr(), pitch, s.data_ptr()
        results += [q, s]
    elif want_h:
        h = _output(out, "out", x, h_dtype)
        a.h = _rows(h, "out")
        results.append(h)
    if B and L:
        _check(lib().sol_attn_norm_modulate(ctypes.byref(a), _stream(dev)))
    return results[0] if len(results) == 1 else tuple(results)


@_placed
def norm_modulate(x, scale=None, shift=None, *, norm="layer", weight=None, bias=None, eps=1e-6, out_dtype=None,
                  quantize=False, out=None):
    """norm(x) * (1 + scale) + shift, token by token.

    x: [B, L, C] or [L, C], bf16, fp16 or fp32, channels contiguous, any row strides.  norm: "layer", "rms" or
    "none", over the C channels, then weight and bias [C].  scale, shift: [C], [B, C] or [B, G, C], each group for
    L / G consecutive tokens (frames, or G = L: every token its own); a first dimension of 1 serves every batch
    element.  Vectors may have any of the three types.  Returns h in x's type (out_dtype: another one, where x is
    fp32), or with quantize=True (q, s): int8 [B, L, C] and fp32 [B, L] with h ~ q * s[..., None], the rows of q
    starting at multiples of 16 bytes as int8_linear reads them.  A row of zeros gives s = 0; a row with an
    infinity or a NaN gives an s that is not finite, and q = 0."""
    return _norm_call(x, None, None, scale, shift, 1.0, "none", None, None, 0.0, norm, weight, bias, eps, out_dtype,
                      quantize, None, False, True, out)


@_placed
def gate_residual(x, y, gate=None, *, residual_scale=1.0, post_norm="none", post_weight=None, post_bias=None,
                  post_eps=1e-6, out=None):
    """x' = residual_scale * x + gate * post_norm(y): the output y of a block joins the residual stream x.

    y has x's shape, and its type where x is not fp32.  gate: as scale in norm_modulate.  out=x updates x in place."""
    return _norm_call(x, y, gate, None, None, residual_scale, post_norm, post_weight, post_bias, post_eps, "none", None,
                      None, 0.0, None, False, out, True, False, None)


@_placed
def gate_residual_norm(x, y, gate=None, scale=None, shift=None, *, residual_scale=1.0, post_norm="none",
                       post_weight=None, post_bias=None, post_eps=1e-6, norm="layer", weight=None, bias=None, eps=1e-6,
                       out_dtype=None, quantize=False, x_out=None, out=None):
    """gate_residual and, in the same pass, the norm and modulation before the next block.

    Returns (x', h), or (x', q, s) with quantize=True; h has y's type and comes from x' before its rounding.
    x_out=x updates the stream in place."""
    return _norm_call(x, y, gate, scale, shift, residual_scale, post_norm, post_weight, post_bias, post_eps, norm, weight,
                      bias, eps, out_dtype, quantize, x_out, True, True, out)


@_placed
def quantize_rows(x):
    """8-bit rows of x: (q, s) with s = max|row| / 127 and x ~ q * s.

    x: [L, C] or [B, L, C], or [B, L, H, d] for the rows of H * d channels that the heads of a token make, such as
    the attention's output through out.transpose(1, 2); q is [..., C] with rows at multiples of 16 bytes."""
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        return _norm_call(x, None, None, None, None, 1.0, "none", None, None, 0.0, "none", None, None, 0.0, None, True,
                          None, False, True, None)
    _input(x, "x")
    B, L, H, d = x.shape
    sb, sl, sh, sd = x.stride()
    if d > 1 and sd != 1:
        raise ValueError("x: the channels of a head must be contiguous")
    if H * d < 1:
        raise ValueError("x has no channels")
    q, pitch = _padded_rows((B, L, H * d), x.device)
    s = torch.empty(B, L, device=x.device, dtype=torch.float32)
    a = _NormArgs(B=B, L=L, C=H * d, x_inner=d, x_stride_h=sh, x=_Rows(x.data_ptr(), _DTYPES[x.dtype], sb, sl),
                  q=q.data_ptr(), q_stride=pitch, q_scale=s.data_ptr(), residual_scale=1.0)
    if B and L:
        _check(lib().sol_attn_norm_modulate(ctypes.byref(a), _stream(x.device)))
    return q, s


# ------------------------------------------------------------------ rotary positions
def rope_axes(d):
    """Channels of a head's time, height and width axes: a third each for height and width, rounded down to an even
    number, and the rest for the time ((44, 42, 42) of 128)."""
    side = 2 * (d // 6)
    return (d - 2 * side, side, side)


@functools.lru_cache(maxsize=64)
def _rope_pairs(axes, theta, freqs):
    """The host arrays of a pair's frequency and axis, which depend on plain numbers only."""
    axis = [i for i, n in enumerate(axes) for _ in range(n // 2)]
    if freqs is None:
        freqs = [math.pow(theta, -2.0 * j / n) for n in axes for j in range(n // 2)]
    return (ctypes.c_double * len(freqs))(*freqs), (ctypes.c_ubyte * len(axis))(*axis)


@_placed
def rope(q, k, v=None, *, grid=None, positions=None, axes=None, start=0, theta=10000.0, freqs=None,
         pairing="interleaved", norm="none", q_weight=None, k_weight=None, eps=1e-6):
    """Rotary positions with several axes; returns (q, k) or (q, k, v), contiguous [B, H, L, d] as forward reads them.

    q, k, v: [B, L, H, d] of one type, such as views of one projection's [B, L, 3, H, d]; the channels of a head are
    contiguous, base address and other strides are multiples of 8 elements, d is a multiple of 16.  v is only laid out anew.
    Positions: grid=(frames, rows, columns) for tokens in raster order, the first one at raster index start (tokens
    behind the grid, such as text, do not turn); or positions [L, A] or [B, L, A] on the device, int32, int64,
    float32 or float64, with A axes of 1 to 4.  axes: channels of each axis, even numbers that sum to d (three axes:
    rope_axes(d)).  Pair j of an axis of n channels turns by position * theta**(-2 j / n), or freqs gives the d / 2
    frequencies.  pairing: "interleaved" pairs channels (2i, 2i + 1), "half" (i, i + d / 2).
    norm: RMS norm of q and k before the rotation over each head's channels ("head", weights [d]) or over all of a
    token's ("token", weights [H * d])."""
    _input(q, "q")
    if q.dim() != 4:
        raise ValueError("q, k and v must be [B, L, H, d]")
    B, L, H, d = q.shape
    dev = q.device
    kind = _choice(norm, _ROPE_NORMS, "norm")
    if (grid is None) == (positions is None):
        raise ValueError("give either grid or positions")
    A = 3
    a = _RopeArgs(B=B, L=L, H=H, d=d, dtype=_DTYPES[q.dtype], norm=kind, eps=eps,
                  pairing=_choice(pairing, _PAIRINGS, "pairing"))
    if grid is not None:
        if len(grid) != 3 or any(int(n) != n or not 1 <= n < 2 ** 31 for n in grid):
            raise ValueError(f"grid must be (frames, rows, columns), each at least 1 (got {grid!r})")
        if not 0 <= start < 2 ** 62:
            raise ValueError(f"start must not be negative (got {start!r})")
        a.grid_f, a.grid_h, a.grid_w = (int(n) for n in grid)
        a.start = start
    else:
        _input(positions, "positions", dev, _POSITIONS)
        if positions.dim() not in (2, 3) or positions.shape[-2] != L or (positions.dim() == 3 and positions.shape[0] not in (1, B)):
            raise ValueError(f"positions must be [{L}, A] or [{B}, {L}, A] (got {list(positions.shape)})")
        if start:
            raise ValueError("start goes with grid")
        A = positions.shape[-1]
        a.pos_kind = _POSITIONS[positions.dtype]
        a.positions = positions.data_ptr()
        a.pos_stride_b = positions.stride(0) if positions.dim() == 3 and positions.shape[0] > 1 else 0
        a.pos_stride_l, a.pos_stride_a = positions.stride(-2), positions.stride(-1)
    if axes is None:
        if A != 3:
            raise ValueError(f"axes must be given for {A} axes")
        axes = rope_axes(d)
    axes = tuple(int(n) for n in axes)
    if len(axes) != A or any(n < 0 or n % 2 for n in axes) or sum(axes) != d:
        raise ValueError(f"axes must be {A} even numbers that sum to {d} (got {axes})")
    if freqs is not None:
        freqs = tuple(float(f) for f in freqs)
        if len(freqs) != d // 2:
            raise ValueError(f"freqs must have {d // 2} values")
    elif not theta > 0:
        raise ValueError("theta must be positive")
    freq_array, axis_array = _rope_pairs(axes, float(theta), freqs)
    a.axes = A
    a.freqs, a.axis = ctypes.addressof(freq_array), ctypes.addressof(axis_array)
    outs = []
    for name, t, w in (("q", q, q_weight), ("k", k, k_weight), ("v", v, None)):
        if t is None and name == "v":
            continue
        _input(t, name, dev)
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError("q, k and v must share one shape [B, L, H, d] and one type")
        if t.stride(3) != 1:
            raise ValueError(f"{name}: the channels of a head must be contiguous")
        out = torch.empty(B, H, L, d, device=dev, dtype=q.dtype)
        outs.append(out)
        r = _RopeTensor(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2), out.data_ptr())
        if w is not None:
            _input(w, f"{name}_weight", dev)
            n = {0: 0, 1: d, 2: H * d}[kind]
            if not n:
                raise ValueError(f"{name}_weight goes with a norm")
            if w.dim() != 1 or w.shape[0] != n or not w.is_contiguous():
                raise ValueError(f"{name}_weight must be a contiguous [{n}]")
            r.weight, r.weight_dtype = w.data_ptr(), _DTYPES[w.dtype]
        setattr(a, name, r)
    if B and L and H:
        _check(lib().sol_attn_rope(ctypes.byref(a), _stream(dev)))
    return tuple(outs)


# ------------------------------------------------------------------ products of 8-bit integers
def _scales(t, name, n, device):
    _input(t, name, device, (torch.float32,))
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} contiguous values (got {list(t.shape)})")


@_placed
def int8_linear(a, a_scale, w, w_scale, bias=None, *, out_dtype=None, out=None):
    """(a @ w.T) * a_scale[:, None] * w_scale + bias for 8-bit a and w, summed exactly.

    a: int8 [M, K] or [B, L, K] with fp32 scales [M] or [B, L], such as (q, s) of quantize_rows or
    norm_modulate(quantize=True); w: int8 [N, K] with fp32 scales [N], such as quantize_rows of a weight matrix.  The
    rows of both start at multiples of 16 bytes (as those calls return them); K is at most 131071.  bias: [N], bf16,
    fp16 or fp32.  Returns [M, N] or [B, L, N] in out_dtype (bf16, fp16 or fp32; by default bf16)."""
    _input(a, "a", None, (torch.int8,))
    _input(w, "w", a.device, (torch.int8,))
    if a.dim() not in (2, 3) or w.dim() != 2 or w.shape[1] != a.shape[-1]:
        raise ValueError(f"a must be [M, K] or [B, L, K] and w [N, K] (got {list(a.shape)} and {list(w.shape)})")
    K, N = a.shape[-1], w.shape[0]
    M = a.numel() // K if K else 0
    if K < 1:
        raise ValueError("K must be at least 1")
    if (K > 1 and (a.stride(-1) != 1 or w.stride(1) != 1)) or \
            (a.dim() == 3 and a.shape[0] > 1 and a.shape[1] > 1 and a.stride(0) != a.shape[1] * a.stride(1)):
        raise ValueError("the rows of a and w must be contiguous, and those of a at one pitch")
    pitch = a.stride(-2) if a.shape[-2] > 1 else a.stride(0)
    _scales(a_scale, "a_scale", M, a.device)
    _scales(w_scale, "w_scale", N, a.device)
    if out is None:
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype not in _DTYPES:
            raise ValueError(f"out has the unsupported type {out_dtype}")
        out = torch.empty(*a.shape[:-1], N, device=a.device, dtype=out_dtype)
    else:
        _input(out, "out", a.device)
        if out.shape != (*a.shape[:-1], N) or out_dtype not in (None, out.dtype) or not out.is_contiguous():
            raise ValueError(f"out must be contiguous, {[*a.shape[:-1], N]} and of the type out_dtype")
    p = _LinearArgs(M, N, K, a.data_ptr(), pitch, a_scale.data_ptr(), w.data_ptr(), w.stride(0), w_scale.data_ptr(), None, 0,
                    out.data_ptr(), _DTYPES[out.dtype], N)
    if bias is not None:
        _input(bias, "bias", a.device)
        if bias.shape != (N,) or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous [{N}] (got {list(bias.shape)})")
        p.bias, p.bias_dtype = bias.data_ptr(), _DTYPES[bias.dtype]
    if M and N:
        _check(lib().sol_attn_quantized_linear(ctypes.byref(p), _stream(a.device)))
    return out


def linear_status(device=None, stream=None):
    """Synchronises the stream and raises SolAttnError if a product on this device gave up a bounded wait."""
    with torch.cuda.device(device if stream is None else stream.device):
        _check(lib().sol_attn_linear_status(_stream(None) if stream is None else stream.cuda_stream))


# ------------------------------------------------------------------ the layer
class AttentionLayer:
    """The self-attention of a diffusion-transformer block around ``forward``, its two projections in 8-bit integers:

      h        = norm(x) * (1 + scale) + shift, in 8 bits        norm_modulate
      q, k, v  = h w_qkv^T + b_qkv                               int8_linear
      q, k     : RMS norm, rotary positions; q, k, v head-major  rope
      o        = sparse attention, in 8 bits token by token      forward, quantize_rows
      y        = o w_out^T + b_out                               int8_linear
      x', h'   = x + gate * y, norm(x') * (1 + next_scale) + next_shift   gate_residual_norm

    w_qkv: [3 H d, C], the rows of q, k and v in that order; w_out: [C, H d]; b_qkv, b_out: their biases; C is the
    width of x, d = 64 or 128.  Both are quantised here, once, row by row.  norm, eps, qk_norm, q_weight, k_weight,
    pairing, theta and axes are those of norm_modulate and rope.  Forward only."""

    def __init__(self, w_qkv, w_out, heads, *, b_qkv=None, b_out=None, norm="layer", eps=1e-6, qk_norm="token",
                 q_weight=None, k_weight=None, pairing="interleaved", theta=10000.0, axes=None):
        if w_qkv.dim() != 2 or w_out.dim() != 2 or heads < 1 or w_qkv.shape[0] % (3 * heads) or \
                tuple(w_out.shape) != (w_qkv.shape[1], w_qkv.shape[0] // 3):
            raise ValueError(f"w_qkv must be [3 H d, C] and w_out [C, H d] for {heads} heads "
                             f"(got {list(w_qkv.shape)} and {list(w_out.shape)})")
        self.heads, self.d = heads, w_qkv.shape[0] // (3 * heads)
        if self.d not in (64, 128):
            raise ValueError(f"a head must have 64 or 128 channels (got {self.d})")
        self.w_qkv, self.w_qkv_scale = quantize_rows(w_qkv)
        self.w_out, self.w_out_scale = quantize_rows(w_out)
        self.b_qkv, self.b_out = b_qkv, b_out
        self.norm, self.eps = norm, eps
        self.rope = dict(norm=qk_norm, q_weight=q_weight, k_weight=k_weight, pairing=pairing, theta=theta, axes=axes,
                         eps=eps)

    def __call__(self, x, scale=None, shift=None, gate=None, *, beta, chunk, flags=0, grid=None, positions=None, start=0,
                 next_scale=None, next_shift=None, x_out=None):
        """x: [B, L, C], bf16 or fp32; scale, shift, gate, next_scale, next_shift: vectors as norm_modulate takes
        them; beta, chunk, flags: the attention's; grid, positions, start: rope's.  Returns (x', h') with h' in
        bf16; x_out=x updates the stream in place.  Runs on the current stream of x's device; the attention's
        workspace is the device's, so calls on one device must not overlap."""
        _input(x, "x", self.w_qkv.device, (torch.bfloat16, torch.float32))
        if x.dim() != 3 or x.shape[2] != self.w_qkv.shape[1]:
            raise ValueError(f"x must be [B, L, {self.w_qkv.shape[1]}] (got {list(x.shape)})")
        B, L, _ = x.shape
        with torch.cuda.device(x.device):
            h, h_scale = norm_modulate(x, scale, shift, norm=self.norm, eps=self.eps, quantize=True)
            qkv = int8_linear(h, h_scale, self.w_qkv, self.w_qkv_scale, self.b_qkv).view(B, L, 3, self.heads, self.d)
            q, k, v = rope(qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2], grid=grid, positions=positions, start=start, **self.rope)
            o = forward(q, k, v, beta, chunk, flags=flags)
            o8, o_scale = quantize_rows(o.transpose(1, 2))
            y = int8_linear(o8, o_scale, self.w_out, self.w_out_scale, self.b_out)
            return gate_residual_norm(x, y, gate, next_scale, next_shift, norm=self.norm, eps=self.eps, x_out=x_out)
