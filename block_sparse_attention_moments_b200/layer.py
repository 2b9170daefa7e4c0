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
import struct
from operator import index

import torch

from . import _check, forward, lib

__all__ = ["norm_modulate", "gate_residual", "gate_residual_norm", "quantize_rows", "rope", "rope_axes",
           "int8_linear", "linear_status", "AttentionLayer"]

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_INT8, _FP32 = (torch.int8,), (torch.float32,)
_NORMS = {"none": 0, "layer": 1, "rms": 2}
_ROPE_NORMS = {"none": 0, "head": 1, "token": 2}
_PAIRINGS = {"interleaved": 0, "half": 1}
_POSITIONS = {torch.int32: 1, torch.int64: 2, torch.float32: 3, torch.float64: 4}

# Argument structs of include/sol_attn.h, packed by struct in one call: a ctypes Structure of this many fields takes
# longer to fill than the smallest of these operators runs.  Native alignment gives the C layout.
_ROWS, _VECTORS, _ROPE_TENSOR = "Piqq", "Piiqq", "PqqqPPi4x"
_NORM_ARGS = struct.Struct("@iiiiq" + 4 * _ROWS + "PqPfifif" + 7 * _VECTORS)
_ROPE_ARGS = struct.Struct("@iiiii" + 3 * _ROPE_TENSOR + "ifiiPPiiiiqPqqq")
_LINEAR_ARGS = struct.Struct("@iiiPqPPqPPiPiqI4x")
_NO_ROWS, _NO_VECTORS = (0, 0, 0, 0), (0, 0, 0, 0, 0)
_NO_AFFINE = _NO_VECTORS + _NO_VECTORS


# ------------------------------------------------------------------ checks
def _input(t, name, device=None, dtypes=_DTYPES):
    """device: the index of the device that the tensor has to be on (None: any)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has the unsupported type {t.dtype}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and there is no backward pass: call under torch.no_grad()")


def _choice(value, choices, name):
    if value not in choices:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, choices))} (got {value!r})")
    return choices[value]


def _rows(t, name):
    """(data, dtype, stride_b, stride_l) of a [B, L, C] or [L, C] tensor."""
    strides = t.stride()
    if strides[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the channels of a token must be contiguous")
    return (t.data_ptr(), _DTYPES[t.dtype], strides[0] if len(strides) == 3 else 0, strides[-2])


def _vectors(t, name, B, L, C, device, plain=False):
    """[C], [B, C] or [B, G, C] (B may be 1: the same for every batch element); plain: [C] only."""
    if t is None:
        return _NO_VECTORS
    _input(t, name, device)
    shape, strides = t.shape, t.stride()
    n = len(shape)
    if n == 1 and shape[0] == C:
        G, sb, sg = 1, 0, 0
    elif n == 2 and not plain and shape[1] == C and shape[0] in (1, B):
        G, sb, sg = 1, strides[0] if shape[0] > 1 else 0, 0
    elif n == 3 and not plain and shape[2] == C and shape[0] in (1, B) and shape[1] > 0 and L % shape[1] == 0:
        G, sb, sg = shape[1], strides[0] if shape[0] > 1 else 0, strides[1]
    else:
        want = f"[{C}]" if plain else f"[{C}], [{B}, {C}] or [{B}, G, {C}] with G dividing {L}"
        raise ValueError(f"{name} must be {want} (got {list(shape)})")
    if C > 1 and strides[-1] != 1:
        raise ValueError(f"{name}: the channels must be contiguous")
    return (t.data_ptr(), _DTYPES[t.dtype], G, sb, sg)


def _output(out, name, like, dtype):
    if out is None:
        if like.is_contiguous():
            return torch.empty_like(like, dtype=dtype)
        return like.new_empty(like.shape, dtype=dtype)
    if not isinstance(out, torch.Tensor) or out.device != like.device or out.dtype != dtype or out.shape != like.shape:
        raise ValueError(f"{name} must be a {dtype} tensor {list(like.shape)} on {like.device}")
    if out.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and there is no backward pass: call under torch.no_grad()")
    return out


def _padded_rows(x, shape):
    """int8 [..., K] whose rows start at multiples of 16 bytes, and its row pitch."""
    K = shape[-1]
    pitch = (K + 15) // 16 * 16
    t = x.new_empty((*shape[:-1], pitch), dtype=torch.int8)
    return (t if pitch == K else t[..., :K]), pitch


def _placed(fn):
    """Runs fn with the device of its first parameter, a tensor, current and, where a stream is given, with that stream
    current, so that outputs belong to it; the inputs are marked as used by it.  The tensor is found by its name among
    keywords; fn refuses a call without one."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        x = args[0] if args else kw.get(name)
        if isinstance(x, torch.Tensor) and x.is_cuda:
            if stream is not None:
                return on_stream(x, stream, args, kw)
            if x.get_device() != _current_device():
                with torch.cuda.device(x.device):
                    return fn(*args, **kw)
        return fn(*args, **kw)

    def on_stream(x, stream, args, kw):
        if stream.device != x.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {x.device}")
        if stream != torch.cuda.current_stream(x.device):
            for t in (*args, *kw.values()):
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


# The current device without torch.cuda's lazy initialisation (a CUDA tensor is at hand), and the handle of a
# device's current stream without a Stream object in between.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


# ------------------------------------------------------------------ norms
def _norm_call(x, y, gate, scale, shift, residual_scale, post_norm, post_weight, post_bias, post_eps, norm, weight, bias,
               eps, out_dtype, quantize, x_out, want_x, want_h, out):
    _input(x, "x")
    shape = x.shape
    if len(shape) == 3:
        B, L, C = shape
    elif len(shape) == 2:
        B, (L, C) = 1, shape
    else:
        raise ValueError("x must be [B, L, C] or [L, C]")
    if C < 1:
        raise ValueError("x has no channels")
    dev, x_dtype = x.get_device(), x.dtype
    x_rows, y_rows, xo_rows, h_rows, q_rows = _rows(x, "x"), _NO_ROWS, _NO_ROWS, _NO_ROWS, (0, 0, 0)
    norm = _choice(norm, _NORMS, "norm")
    post_norm = _choice(post_norm, _NORMS, "post_norm")
    scale = _vectors(scale, "scale", B, L, C, dev)
    shift = _vectors(shift, "shift", B, L, C, dev)
    gates, affine, post_affine = _NO_VECTORS, _NO_AFFINE, _NO_AFFINE
    if weight is not None or bias is not None:
        affine = _vectors(weight, "weight", B, L, C, dev, True) + _vectors(bias, "bias", B, L, C, dev, True)
    h_dtype = x_dtype
    if y is not None:
        _input(y, "y", dev)
        if y.shape != shape:
            raise ValueError("x and y must share one shape")
        h_dtype = y.dtype
        if h_dtype != x_dtype and x_dtype != torch.float32:
            raise ValueError("y must have the type of x, or x must be float32")
        y_rows = _rows(y, "y")
        gates = _vectors(gate, "gate", B, L, C, dev)
        if post_weight is not None or post_bias is not None:
            post_affine = (_vectors(post_weight, "post_weight", B, L, C, dev, True) +
                           _vectors(post_bias, "post_bias", B, L, C, dev, True))
    if out_dtype is not None and out_dtype != h_dtype:
        if y is not None:
            raise ValueError("out_dtype must be the type of y")
        if out_dtype not in _DTYPES or x_dtype != torch.float32:
            raise ValueError("out_dtype must be the type of x, or x must be float32")
        h_dtype = out_dtype
    if quantize and (out is not None or out_dtype is not None):
        raise ValueError("quantize=True takes neither out nor out_dtype")
    results = ()
    if want_x:
        x_out = _output(x_out, "x_out", x, x_dtype)
        xo_rows = _rows(x_out, "x_out")
        results = (x_out,)
    if want_h and quantize:
        q, pitch = _padded_rows(x, shape)
        s = x.new_empty(shape[:-1], dtype=torch.float32)
        q_rows = (q.data_ptr(), pitch, s.data_ptr())
        results += (q, s)
    elif want_h:
        h = _output(out, "out", x, h_dtype)
        h_rows = _rows(h, "out")
        results += (h,)
    if B and L:
        args = _NORM_ARGS.pack(B, L, C, C, 0, *x_rows, *y_rows, *xo_rows, *h_rows, *q_rows, residual_scale, norm, eps,
                               post_norm, post_eps, *scale, *shift, *gates, *affine, *post_affine)
        rc = lib().sol_attn_norm_modulate(args, _raw_stream(dev))
        if rc:
            _check(rc)
    return results[0] if len(results) == 1 else results


@_placed
def norm_modulate(x, scale=None, shift=None, *, norm="layer", weight=None, bias=None, eps=1e-6, out_dtype=None,
                  quantize=False, out=None):
    """norm(x) * (1 + scale) + shift, token by token.

    x: [B, L, C] or [L, C], bf16, fp16 or fp32, C up to 16384, channels contiguous, any row strides.  norm: "layer",
    "rms" or "none", over the C channels, then weight and bias [C].  scale, shift: [C], [B, C] or [B, G, C], each group for
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
    q, pitch = _padded_rows(x, (B, L, H * d))
    s = x.new_empty((B, L), dtype=torch.float32)
    if B and L:
        args = _NORM_ARGS.pack(B, L, H * d, d, sh, x.data_ptr(), _DTYPES[x.dtype], sb, sl, *_NO_ROWS, *_NO_ROWS, *_NO_ROWS,
                               q.data_ptr(), pitch, s.data_ptr(), 1.0, 0, 0.0, 0, 0.0, *_NO_VECTORS, *_NO_VECTORS,
                               *_NO_VECTORS, *_NO_AFFINE, *_NO_AFFINE)
        rc = lib().sol_attn_norm_modulate(args, _raw_stream(x.get_device()))
        if rc:
            _check(rc)
    return q, s


# ------------------------------------------------------------------ rotary positions
def rope_axes(d):
    """Channels of a head's time, height and width axes: a third each for height and width, rounded down to an even
    number, and the rest for the time ((44, 42, 42) of 128)."""
    side = 2 * (d // 6)
    return (d - 2 * side, side, side)


@functools.lru_cache(maxsize=64)
def _rope_pairs(axes, theta, freqs, d):
    """The host arrays of a pair's frequency and axis, with their addresses; they depend on plain numbers only."""
    axes = tuple(index(n) for n in axes)
    if any(n < 0 or n % 2 for n in axes) or sum(axes) != d:
        raise ValueError(f"axes must be {len(axes)} even numbers that sum to {d} (got {axes})")
    axis = [i for i, n in enumerate(axes) for _ in range(n // 2)]
    if freqs is None:
        if not theta > 0:
            raise ValueError("theta must be positive")
        freqs = [math.pow(theta, -2.0 * j / n) for n in axes for j in range(n // 2)]
    elif len(freqs) != d // 2:
        raise ValueError(f"freqs must have {d // 2} values")
    freq_array, axis_array = (ctypes.c_double * len(freqs))(*freqs), (ctypes.c_ubyte * len(axis))(*axis)
    return ctypes.addressof(freq_array), ctypes.addressof(axis_array), freq_array, axis_array


def _rope_tensor(t, name, q, w, n, out):
    if t is not q:
        _input(t, name, q.get_device())
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError("q, k and v must share one shape [B, L, H, d] and one type")
    strides = t.stride()
    if strides[3] != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    if w is None:
        return (t.data_ptr(), *strides[:3], out.data_ptr(), 0, 0)
    _input(w, f"{name}_weight", q.get_device())
    if not n:
        raise ValueError(f"{name}_weight goes with a norm")
    if w.dim() != 1 or w.shape[0] != n or not w.is_contiguous():
        raise ValueError(f"{name}_weight must be a contiguous [{n}]")
    return (t.data_ptr(), *strides[:3], out.data_ptr(), w.data_ptr(), _DTYPES[w.dtype])


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
    dev = q.get_device()
    kind = _choice(norm, _ROPE_NORMS, "norm")
    pairing = _choice(pairing, _PAIRINGS, "pairing")
    if (grid is None) == (positions is None):
        raise ValueError("give either grid or positions")
    A = 3
    if grid is not None:
        try:
            F, R, C = grid
            F, R, C = index(F), index(R), index(C)
        except (TypeError, ValueError):
            F = 0
        if F < 1 or R < 1 or C < 1 or F >= 2 ** 31 or R >= 2 ** 31 or C >= 2 ** 31:
            raise ValueError(f"grid must be (frames, rows, columns), each at least 1 (got {grid!r})")
        start = index(start)
        if not 0 <= start < 2 ** 62:
            raise ValueError(f"start must not be negative (got {start!r})")
        where = (0, F, R, C, start, 0, 0, 0, 0)
    else:
        _input(positions, "positions", dev, _POSITIONS)
        shape, strides = positions.shape, positions.stride()
        if len(shape) not in (2, 3) or shape[-2] != L or (len(shape) == 3 and shape[0] not in (1, B)):
            raise ValueError(f"positions must be [{L}, A] or [{B}, {L}, A] (got {list(shape)})")
        if start:
            raise ValueError("start goes with grid")
        A = shape[-1]
        where = (_POSITIONS[positions.dtype], 0, 0, 0, 0, positions.data_ptr(),
                 strides[0] if len(shape) == 3 and shape[0] > 1 else 0, strides[-2], strides[-1])
    if axes is None:
        if A != 3:
            raise ValueError(f"axes must be given for {A} axes")
        axes = rope_axes(d)
    if len(axes) != A:
        raise ValueError(f"axes must be {A} even numbers that sum to {d} (got {tuple(axes)})")
    pairs = _rope_pairs(tuple(axes), float(theta), None if freqs is None else tuple(map(float, freqs)), d)
    n = 0 if kind == 0 else d if kind == 1 else H * d
    outs = (q.new_empty((B, H, L, d)), q.new_empty((B, H, L, d))) + (() if v is None else (q.new_empty((B, H, L, d)),))
    tensors = _rope_tensor(q, "q", q, q_weight, n, outs[0]) + _rope_tensor(k, "k", q, k_weight, n, outs[1])
    tensors += (0, 0, 0, 0, 0, 0, 0) if v is None else _rope_tensor(v, "v", q, None, n, outs[2])
    if B and L and H:
        args = _ROPE_ARGS.pack(B, L, H, d, _DTYPES[q.dtype], *tensors, kind, eps, pairing, A, pairs[0], pairs[1], *where)
        rc = lib().sol_attn_rope(args, _raw_stream(dev))
        if rc:
            _check(rc)
    return outs


# ------------------------------------------------------------------ products of 8-bit integers
def _scales(t, name, n, device):
    _input(t, name, device, _FP32)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} contiguous values (got {list(t.shape)})")


@_placed
def int8_linear(a, a_scale, w, w_scale, bias=None, *, out_dtype=None, out=None):
    """(a @ w.T) * a_scale[:, None] * w_scale + bias for 8-bit a and w, summed exactly.

    a: int8 [M, K] or [B, L, K] with fp32 scales [M] or [B, L], such as (q, s) of quantize_rows or
    norm_modulate(quantize=True); w: int8 [N, K] with fp32 scales [N], such as quantize_rows of a weight matrix.  The
    rows of both start at multiples of 16 bytes (as those calls return them); K is at most 131071.  bias: [N], bf16,
    fp16 or fp32.  Returns [M, N] or [B, L, N] in out_dtype (bf16, fp16 or fp32; by default bf16).  linear_status tells
    whether a product's bounded waits held; it is the only sign of one that gave up and left its output unwritten."""
    _input(a, "a", None, _INT8)
    dev = a.get_device()
    _input(w, "w", dev, _INT8)
    if a.dim() not in (2, 3) or w.dim() != 2 or w.shape[1] != a.shape[-1]:
        raise ValueError(f"a must be [M, K] or [B, L, K] and w [N, K] (got {list(a.shape)} and {list(w.shape)})")
    K, N = a.shape[-1], w.shape[0]
    if K < 1:
        raise ValueError("K must be at least 1")
    lead, strides, w_strides = a.shape[:-1], a.stride(), w.stride()
    M = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    if (K > 1 and (strides[-1] != 1 or w_strides[1] != 1)) or \
            (len(lead) == 2 and lead[0] > 1 and lead[1] > 1 and strides[0] != lead[1] * strides[1]):
        raise ValueError("the rows of a and w must be contiguous, and those of a at one pitch")
    pitch = strides[-2] if lead[-1] > 1 else strides[0]
    _scales(a_scale, "a_scale", M, dev)
    _scales(w_scale, "w_scale", N, dev)
    if out is None:
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype not in _DTYPES:
            raise ValueError(f"out has the unsupported type {out_dtype}")
        out = a.new_empty((*lead, N), dtype=out_dtype)
    else:
        _input(out, "out", dev)
        if out.shape != (*lead, N) or out_dtype not in (None, out.dtype) or not out.is_contiguous():
            raise ValueError(f"out must be contiguous, {[*lead, N]} and of the type out_dtype")
    b = (0, 0)
    if bias is not None:
        _input(bias, "bias", dev)
        if bias.shape != (N,) or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous [{N}] (got {list(bias.shape)})")
        b = (bias.data_ptr(), _DTYPES[bias.dtype])
    if M and N:
        args = _LINEAR_ARGS.pack(M, N, K, a.data_ptr(), pitch, a_scale.data_ptr(), w.data_ptr(), w_strides[0],
                                 w_scale.data_ptr(), *b, out.data_ptr(), _DTYPES[out.dtype], N, 0)
        rc = lib().sol_attn_quantized_linear(args, _raw_stream(dev))
        if rc:
            _check(rc)
    return out


def linear_status(device=None, stream=None):
    """Synchronises the stream (by default the device's current one; no other) and raises SolAttnError if a product gave
    up a bounded wait: one on that stream, or another of the device that has ended.  A report is given once."""
    with torch.cuda.device(device if stream is None else stream.device):
        _check(lib().sol_attn_linear_status((torch.cuda.current_stream() if stream is None else stream).cuda_stream))


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
        workspace is the device's, so calls on one device must not overlap, replays of captured ones among them, and
        the first call of a shape must not be captured.  linear_status tells whether the products' waits held."""
        _input(x, "x", self.w_qkv.get_device(), (torch.bfloat16, torch.float32))
        if x.dim() != 3 or x.shape[2] != self.w_qkv.shape[1]:
            raise ValueError(f"x must be [B, L, {self.w_qkv.shape[1]}] (got {list(x.shape)})")
        B, L, _ = x.shape
        with torch.cuda.device(x.device):
            h, h_scale = norm_modulate(x, scale, shift, norm=self.norm, eps=self.eps, quantize=True)
            qkv = int8_linear(h, h_scale, self.w_qkv, self.w_qkv_scale, self.b_qkv).view(B, L, 3, self.heads, self.d)
            q, k, v = rope(qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2], grid=grid, positions=positions, start=start, **self.rope)
            o = forward(q, k, v, beta, chunk, flags=flags) if B and L else q
            o8, o_scale = quantize_rows(o.transpose(1, 2))
            y = int8_linear(o8, o_scale, self.w_out, self.w_out_scale, self.b_out)
            return gate_residual_norm(x, y, gate, next_scale, next_shift, norm=self.norm, eps=self.eps, x_out=x_out)
