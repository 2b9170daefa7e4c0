"""Norms with modulation, gate, residual and 8-bit rows (norm_modulate,
gate_residual, gate_residual_norm, quantize_rows) against their formulas in
64 bits.

Tolerances.  An output is computed in fp32 and rounded once to its type t:
|error| <= eps(t)/2 |value| + K u M with u = 2^-24.  M is the size of the terms
that the value is a sum of, (|n| + |mean| / sigma + 1) |A| + |B| for
h = n A + B: the mean and the mean square are sums of C terms, a thread adds at
most 32 of them one after the other and trees add the rest, so their relative
errors are below (32 + 16) u, the reciprocal root halves one of them and adds 2
units, and the products and sums behind it add fewer than 8.  K = 64 covers the sum.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import block_sparse_attention_moments_b200 as sa  # noqa: E402

U = 2.0 ** -24
K = 64
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def norm64(v, kind, weight, bias, eps):
    """(n * weight + bias, size of its terms)"""
    if kind == "none":
        n, size = v, v.abs()
    else:
        mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
        c = v - mean
        r = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
        n, size = c * r, (c * r).abs() + mean.abs() * r + 1
    if weight is not None:
        n, size = n * weight.double(), size * weight.double().abs()
    if bias is not None:
        n, size = n + bias.double(), size + bias.double().abs()
    return n, size


def spread(t, B, L, C):
    """[C], [B, C] or [B, G, C] -> [B, L, C] in 64 bits."""
    t = t.double()
    t = t.expand(B, 1, C) if t.dim() == 1 else t[:, None].expand(B, 1, C) if t.dim() == 2 else t.expand(B, -1, C)
    return t.repeat_interleave(L // t.shape[1], dim=1)


def reference(x, y=None, gate=None, scale=None, shift=None, residual_scale=1.0, post_norm="none", post_weight=None,
              post_bias=None, post_eps=1e-6, norm="layer", weight=None, bias=None, eps=1e-6):
    """(x', its size, h, its size)"""
    B, L, C = x.shape
    v = x.double()
    xs = v.abs()
    if y is not None:
        n, size = norm64(y.double(), post_norm, post_weight, post_bias, post_eps)
        if gate is not None:
            g = spread(gate, B, L, C)
            n, size = n * g, size * g.abs()
        v = residual_scale * v + n
        xs = abs(residual_scale) * xs + size
    h, hs = norm64(v, norm, weight, bias, eps)
    if y is not None and norm != "none":
        # what x' is off by reaches h through the norm: by each channel's own
        # error over sigma, and by the row's mean error in the statistics
        c = v - v.mean(-1, keepdim=True) if norm == "layer" else v
        r = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
        w = 1 if weight is None else weight.double().abs()
        hs = hs + (xs + xs.mean(-1, keepdim=True)) * r * w * (1 + h.abs())
    elif y is not None:
        hs = hs + xs * (1 if weight is None else weight.double().abs())
    if scale is not None:
        s = spread(scale, B, L, C)
        h, hs = h * (1 + s), hs * (1 + s.abs())
    if shift is not None:
        s = spread(shift, B, L, C)
        h, hs = h + s, hs + s.abs()
    return v, xs, h, hs


def close(got, want, size, what):
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + K * U * size + torch.finfo(got.dtype).tiny
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float(((got.double() - want).abs() / tol).nan_to_num(9e9).max()):.3g} of the tolerance"


def randn(*shape, dtype=FP32, mean=0.0, std=1.0, seed=[0]):
    seed[0] += 1
    g = torch.Generator(device="cuda").manual_seed(seed[0])
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(mean, std, generator=g)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (FP16, FP16), (FP32, FP32), (FP32, BF16), (FP32, FP16)])
@pytest.mark.parametrize("B,L,C", [(1, 1, 64), (2, 5, 1), (1, 33, 7), (3, 17, 1000), (1, 9, 1285), (2, 40, 1536),
                                   (1, 21, 5120), (1, 3, 16384), (1, 2, 16383), (1, 700, 264), (2, 31, 4097)])
def test_norm_modulate(B, L, C, dtype, out_dtype, kind):
    x = randn(B, L, C, dtype=dtype, mean=0.7)
    scale, shift = randn(B, C, std=0.5), randn(B, C, std=0.5)
    weight, bias = randn(C, dtype=out_dtype, mean=1, std=0.2), randn(C, dtype=out_dtype)
    for kw in ({}, {"scale": scale, "shift": shift}, {"weight": weight, "bias": bias, "scale": scale, "shift": shift}):
        h = sa.norm_modulate(x, norm=kind, out_dtype=out_dtype, **kw)
        assert h.dtype == out_dtype and h.shape == x.shape
        _, _, want, size = reference(x, norm=kind, **kw)
        close(h, want, size, kw.keys())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ydtype", [(BF16, BF16), (FP16, FP16), (FP32, FP32), (FP32, BF16), (FP32, FP16)])
@pytest.mark.parametrize("post", ["none", "layer", "rms"])
@pytest.mark.parametrize("B,L,C", [(1, 1, 5120), (2, 19, 1285), (1, 130, 512), (1, 300, 2048)])
def test_gate_residual_norm(B, L, C, post, dtype, ydtype):
    x, y = randn(B, L, C, dtype=dtype, mean=0.2), randn(B, L, C, dtype=ydtype, mean=-0.4)
    gate, scale, shift = (randn(B, 1, C, std=0.5) for _ in range(3))
    kw = dict(residual_scale=0.5, post_norm=post, post_weight=randn(C, dtype=ydtype, mean=1, std=0.2),
              post_bias=randn(C, dtype=ydtype), norm="layer", weight=randn(C, mean=1, std=0.1), bias=randn(C))
    xn, h = sa.gate_residual_norm(x, y, gate, scale, shift, **kw)
    assert xn.dtype == dtype and h.dtype == ydtype
    want_x, size_x, want_h, size_h = reference(x, y, gate, scale, shift, **kw)
    close(xn, want_x, size_x, "x'")
    close(h, want_h, size_h, "h")
    only = sa.gate_residual(x, y, gate, residual_scale=0.5, post_norm=post, post_weight=kw["post_weight"],
                            post_bias=kw["post_bias"])
    assert torch.equal(only, xn)
    inplace = x.clone()
    got, h2 = sa.gate_residual_norm(inplace, y, gate, scale, shift, x_out=inplace, **kw)
    assert got.data_ptr() == inplace.data_ptr() and torch.equal(inplace, xn) and torch.equal(h2, h)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [64, 99, 5120])
@pytest.mark.parametrize("G,per", [(1, 40), (5, 8), (40, 1), (2, 20)])
def test_groups_of_tokens(C, G, per):
    """A modulation for each frame, for each token, and vectors cut out of one [B, G, 6, C] tensor."""
    B = 3
    x, y = randn(B, G * per, C, dtype=BF16), randn(B, G * per, C, dtype=BF16)
    six = randn(B, G, 6, C, std=0.4)
    gate, scale, shift = six[:, :, 2], six[:, :, 1], six[:, :, 0]
    xn, h = sa.gate_residual_norm(x, y, gate, scale, shift)
    want_x, size_x, want_h, size_h = reference(x, y, gate, scale, shift)
    close(xn, want_x, size_x, "x'")
    close(h, want_h, size_h, "h")
    # groups of different lengths in one call, and one group for the whole batch
    one = randn(1, 1, C, std=0.4)
    h = sa.norm_modulate(x, scale, one)
    _, _, want_h, size_h = reference(x, scale=scale, shift=one)
    close(h, want_h, size_h, "broadcast shift")


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 97])
def test_strides(C):
    """Slices of larger tensors, transposed batches, 2-D rows, and outputs into slices; what lies between stays."""
    big = randn(2, 50, 3 * C, dtype=BF16)
    x = big[:, 5:45, C:2 * C]
    h = sa.norm_modulate(x)
    assert torch.equal(h, sa.norm_modulate(x.contiguous()))
    xt = randn(40, 2, C, dtype=BF16).transpose(0, 1)
    assert torch.equal(sa.norm_modulate(xt), sa.norm_modulate(xt.contiguous()))
    assert torch.equal(sa.norm_modulate(x[1]), h[1])
    buf = torch.full((2, 50, 3 * C), 7.0, device="cuda", dtype=BF16)
    out = buf[:, 5:45, C:2 * C]
    assert sa.norm_modulate(x, out=out) is out
    assert torch.equal(out, h)
    buf[:, 5:45, C:2 * C] = 7.0
    assert (buf == 7.0).all()
    # neighbouring columns of one buffer, read and written
    two = torch.cat([x, torch.zeros_like(x)], -1).contiguous()
    sa.norm_modulate(two[..., :C], out=two[..., C:])
    assert torch.equal(two[..., C:], h) and torch.equal(two[..., :C], x)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [0, 1])
def test_no_tokens_and_one(rows):
    for shape in ((rows, 8), (1, rows, 8), (rows, 3, 8)):
        x = randn(*shape, dtype=BF16)
        h = sa.norm_modulate(x)
        assert h.shape == x.shape
        xn, q, s = sa.gate_residual_norm(x, x, quantize=True)
        assert xn.shape == x.shape and q.shape == x.shape and s.shape == x.shape[:-1]


@pytest.mark.gpu
def test_large_offsets_keep_the_variance():
    """Rows near 1000 with a spread of 1: the variance is taken of centred values."""
    x = randn(4, 64, 2048, mean=1000.0)
    h = sa.norm_modulate(x)
    _, _, want, size = reference(x)
    close(h, want, size, "h")


@pytest.mark.gpu
def test_rows_do_not_touch_each_other():
    """NaN and infinities stay in their rows; constant rows and rows of zeros are finite."""
    x, y = randn(1, 64, 520, dtype=BF16), randn(1, 64, 520, dtype=BF16)
    clean_x, clean_h = sa.gate_residual_norm(x, y)
    x[0, 3, 100], x[0, 9, 0], y[0, 20, 519] = math.nan, math.inf, -math.inf
    xn, h = sa.gate_residual_norm(x, y)
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[3, 9, 20]] = True
    assert torch.equal(h[0, ~bad], clean_h[0, ~bad]) and torch.equal(xn[0, ~bad], clean_x[0, ~bad])
    assert h[0, bad].isnan().all()
    _, q, s = sa.gate_residual_norm(x, y, quantize=True)
    assert not s[0, bad].isfinite().any() and s[0, ~bad].isfinite().all() and not q[0, bad].any()
    for kind in ("layer", "rms"):
        assert (sa.norm_modulate(torch.zeros(3, 520, device="cuda"), norm=kind) == 0).all()
    assert (sa.norm_modulate(torch.full((3, 520), 2.5, device="cuda")) == 0).all()


def check_quantised(q, s, v, size):
    """s within its rounding of max|v| / 127, and q the nearest whole number of v / s, or the next one where v / s
    is within its error of a half: v is off by K u M, the scale by 2 u of itself and as much as v, and the
    quotient by 2 u more, so v / s by K u M / s + 127 (K M / max + 4) u."""
    amax = v.abs().amax(-1)
    off = K * U * size.amax(-1)
    assert ((s.double() - amax / 127).abs() <= (off + 2 * U * amax) / 127 + 1e-44).all()
    live = amax > 0
    ratio = torch.where(live[..., None], v / (amax / 127).clamp_min(1e-300)[..., None], 0.0)
    slack = torch.where(live[..., None], (K * U * size + off[..., None]) / (amax / 127).clamp_min(1e-300)[..., None] + 127 * 4 * U, 0.0)
    assert ((q.double() - ratio).abs() <= 0.5 + slack).all()
    assert q.abs().amax() <= 127


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("L,C", [(1, 16), (37, 1000), (5, 1285), (64, 5120), (3, 5)])
def test_quantised_rows(L, C, dtype):
    x = randn(2, L, C, dtype=dtype)
    scale, shift = randn(2, C, std=0.3), randn(2, C, std=0.3)
    q, s = sa.norm_modulate(x, scale, shift, quantize=True)
    assert q.dtype == torch.int8 and s.dtype == FP32 and q.stride(-2) % 16 == 0
    _, _, want, size = reference(x, scale=scale, shift=shift)
    check_quantised(q, s, want, size)
    q, s = sa.quantize_rows(x)
    check_quantised(q, s, x.double(), torch.zeros_like(x, dtype=torch.float64))
    y = randn(2, L, C, dtype=dtype)
    xn, q, s = sa.gate_residual_norm(x, y, None, scale, shift, quantize=True)
    want_x, size_x, want, size = reference(x, y, None, scale, shift)
    close(xn, want_x, size_x, "x'")
    check_quantised(q, s, want, size)


@pytest.mark.gpu
def test_quantised_rows_exactly():
    """Whole numbers come back, ties go to the even one, and rows of zeros, tiny and huge values are held."""
    x = torch.zeros(6, 32, device="cuda")
    x[0, :5] = torch.tensor([127.0, -127.0, 2.5, 3.5, -0.5])
    x[1, :3] = torch.tensor([254.0, 1.0, 3.0])
    x[3, :2] = torch.tensor([1e-42, -1e-42])
    x[4, :2] = torch.tensor([3e38, -1.5e38])
    x[5, :2] = torch.tensor([1e-37, 5e-38])
    q, s = sa.quantize_rows(x)
    assert q[0, :5].tolist() == [127, -127, 2, 4, 0] and s[0] == 1
    assert q[1, :3].tolist() == [127, 0, 2] and s[1] == 2
    assert s[2] == 0 and not q[2].any()
    assert q[3, :2].tolist() == [127, -127]
    assert q[4, 0] == 127 and abs(int(q[4, 1])) in (63, 64) and q[5, 0] == 127


@pytest.mark.gpu
@pytest.mark.parametrize("H,d", [(8, 128), (3, 64), (5, 7)])
def test_quantised_heads(H, d):
    """The rows that the heads of a token make, read from the attention's head-major output."""
    o = randn(2, H, 45, d, dtype=BF16)
    q, s = sa.quantize_rows(o.transpose(1, 2))
    q2, s2 = sa.quantize_rows(o.transpose(1, 2).flatten(2))
    assert q.shape == (2, 45, H * d) and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.gpu
def test_streams_and_graphs():
    x, y = randn(2, 100, 640, dtype=BF16), randn(2, 100, 640, dtype=BF16)
    gate = randn(2, 640)
    want = sa.gate_residual_norm(x, y, gate)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sa.gate_residual_norm(x, y, gate, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xn, h = sa.gate_residual_norm(x, y, gate)
        xn2, q, s = sa.gate_residual_norm(xn, h, gate, quantize=True)
    x.copy_(randn(2, 100, 640, dtype=BF16))
    for _ in range(2):
        graph.replay()
    want = sa.gate_residual_norm(x, y, gate)
    want2 = sa.gate_residual_norm(want[0], want[1], gate, quantize=True)
    torch.cuda.synchronize()
    assert torch.equal(xn, want[0]) and torch.equal(h, want[1])
    assert all(torch.equal(a, b) for a, b in zip((xn2, q, s), want2))


# ------------------------------------------------------------------ refusals
def test_refusals_without_a_device():
    x = torch.zeros(2, 4, 8)
    for call in (lambda: sa.norm_modulate(x), lambda: sa.quantize_rows(x), lambda: sa.gate_residual(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_entry_point_refusals():
    """The library's own checks, which come before anything is read or enqueued."""
    import layer_structs as ly
    lib, byref = sa.lib(), ly.ctypes.byref

    def args(**kw):
        a = ly.NormArgs(B=2, L=4, C=64, x_inner=64, x=ly.Rows(0x10000, 0, 256, 64), h=ly.Rows(0x90000, 0, 256, 64),
                         residual_scale=1.0, norm=1, eps=1e-6)
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    call = lambda **kw: lib.sol_attn_norm_modulate(byref(args(**kw)), None)
    assert lib.sol_attn_norm_modulate(None, None) == -1
    assert call(C=0) == -1 and call(B=-1) == -1 and call(C=16385, x_inner=16385) == -2
    assert call(B=0) == 0 and call(L=0) == 0
    assert call(norm=3) == -1 and call(post_norm=-1) == -1
    assert call(eps=-1.0) == -1 and call(eps=math.nan) == -1
    assert call(x=ly.Rows(None, 0, 256, 64)) == -1
    assert call(x=ly.Rows(0x10001, 0, 256, 64)) == -3
    assert call(x=ly.Rows(0x10000, 5, 256, 64)) == -1
    assert call(x=ly.Rows(0x10000, 0, 256, -64)) == -1
    assert call(h=ly.Rows(0x10000, 0, 256, 64)) == -1            # h is x
    assert call(h=ly.Rows(0x90000, 0, 256, 63)) == -1            # rows of h share elements
    assert call(h=ly.Rows(0x90000, 2, 256, 64)) == -2            # fp32 from bf16
    assert call(h=ly.Rows()) == -1                               # nothing to write
    assert call(x_out=ly.Rows(0xA0000, 0, 256, 64)) == -1        # x' without y
    assert call(y=ly.Rows(0x50000, 0, 256, 64), x_out=ly.Rows(0x50000, 0, 256, 64)) == -1
    assert call(y=ly.Rows(0x50000, 0, 256, 64), x_out=ly.Rows(0x10080, 0, 256, 64)) == -1
    assert call(y=ly.Rows(0x50000, 0, 256, 64), x_out=ly.Rows(0x90000, 0, 256, 64)) == -1
    assert call(scale=ly.Vectors(0x50000, 0, 3, 64, 64)) == -1   # 3 groups of 4 tokens
    assert call(scale=ly.Vectors(0x50000, 0, 0, 64, 64)) == -1
    assert call(scale=ly.Vectors(0x50000, 9, 1, 64, 64)) == -1
    assert call(scale=ly.Vectors(0x50002, 2, 1, 64, 64)) == -3
    assert call(scale=ly.Vectors(0x50000, 0, 2, 64, -64)) == -1 and call(gate=ly.Vectors(0x50000, 0, 1, -64, 0)) == -1
    assert call(scale=ly.Vectors(0x90010, 0, 1, 64, 64)) == -1    # h overlaps scale
    assert call(q=0xB0000, q_stride=64) == -1                     # no scales
    assert call(q=0xB0000, q_stride=32, q_scale=0xC0000) == -1
    assert call(x_inner=48) == -1
    assert "x_inner" in lib.sol_attn_error_string(-1).decode()


@pytest.mark.gpu
def test_refusals():
    x = randn(2, 4, 64, dtype=BF16)
    vec = randn(64)

    def refused(match, call):
        with pytest.raises((ValueError, sa.SolAttnError), match=match):
            call()

    refused("unsupported type", lambda: sa.norm_modulate(x.double()))
    refused("must be", lambda: sa.norm_modulate(x[0, 0]))
    refused("contiguous", lambda: sa.norm_modulate(x.transpose(1, 2)))
    refused("scale must be", lambda: sa.norm_modulate(x, vec[:32]))
    refused("scale must be", lambda: sa.norm_modulate(x, randn(2, 3, 64)))
    refused("scale must be", lambda: sa.norm_modulate(x, randn(2, 0, 64)))
    refused("scale must be", lambda: sa.norm_modulate(x, randn(3, 64)))
    refused("weight must be", lambda: sa.norm_modulate(x, weight=randn(2, 64)))
    refused("norm must be", lambda: sa.norm_modulate(x, norm="batch"))
    refused("share one shape", lambda: sa.gate_residual(x, x[:1]))
    refused("type of x", lambda: sa.gate_residual(x, x.float()))
    refused("out_dtype", lambda: sa.norm_modulate(x, out_dtype=FP32))
    refused("out_dtype", lambda: sa.norm_modulate(x.float(), out_dtype=torch.float64))
    refused("quantize", lambda: sa.norm_modulate(x, quantize=True, out=x.clone()))
    refused("out must be", lambda: sa.norm_modulate(x, out=torch.empty_like(x)[:1]))
    refused("overlaps", lambda: sa.norm_modulate(x, out=x))
    refused("overlap", lambda: sa.gate_residual_norm(x, x.clone(), x_out=(b := x.clone()), out=b))
    refused("x_out overlaps", lambda: sa.gate_residual(x, b := x.clone(), out=b))
    refused("share elements", lambda: sa.norm_modulate(x, out=torch.empty(2, 1, 64, device="cuda", dtype=BF16).expand(2, 4, 64)))
    refused("no backward", lambda: sa.norm_modulate(x, vec.clone().requires_grad_()))
    with torch.no_grad():
        sa.norm_modulate(x, vec.clone().requires_grad_())
    refused("eps", lambda: sa.norm_modulate(x, eps=-1.0))
    refused("exceeds", lambda: sa.norm_modulate(randn(1, 16392, dtype=BF16)))
    refused("no channels", lambda: sa.norm_modulate(x[..., :0]))


# ------------------------------------------------------------------ many rows
# From four rows of a block on (592 on 148 SMs), in groups of eight and more,
# another kernel takes the rows, with folded factors in shared memory, some two
# at a time and groups whose ends may lie between the two.
MANY = [(1, 100, 9, 512), (3, 41, 8, 1544), (1, 37, 17, 5120), (2, 300, 1, 264), (1, 1, 593, 99), (3, 1, 1601, 64), (1, 13, 391, 264), (2, 3, 801, 1024), (5, 1, 1001, 1544), (1, 1, 4737, 2048), (2, 7, 343, 2056),
        (1, 1, 4800, 5120), (3, 50, 33, 1000), (1, 5, 961, 8192)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,G,per,C", MANY)
@pytest.mark.parametrize("dtype,ydtype", [(BF16, BF16), (FP16, FP16), (FP32, FP32), (FP32, BF16)])
def test_many_rows(B, G, per, C, dtype, ydtype):
    L = G * per
    x = randn(B, L, C, dtype=dtype, mean=0.3)
    six = randn(B, G, 6, C, std=0.4)
    gate, scale, shift = six[:, :, 2], six[:, :, 1], six[:, :, 0]
    weight, bias = randn(C, dtype=ydtype, mean=1, std=0.2), randn(C, dtype=ydtype)
    h = sa.norm_modulate(x, scale, shift, norm="layer", weight=weight, bias=bias, out_dtype=ydtype)
    _, _, want, size = reference(x, scale=scale, shift=shift, weight=weight, bias=bias)
    close(h, want, size, "h")
    q, s = sa.norm_modulate(x, scale, shift, norm="rms", quantize=True)
    _, _, want, size = reference(x, scale=scale, shift=shift, norm="rms")
    check_quantised(q, s, want, size)
    y = randn(B, L, C, dtype=ydtype, mean=-0.2)
    for post, post_bias in (("none", None), ("rms", None), ("layer", bias)):
        kw = dict(residual_scale=0.5, post_norm=post, post_weight=weight, post_bias=post_bias, norm="rms")
        want_x, size_x, want, size = reference(x, y, gate, scale, shift, **kw)
        xn, h = sa.gate_residual_norm(x, y, gate, scale, shift, **kw)
        close(xn, want_x, size_x, "x'")
        close(h, want, size, "h")
    inplace = x.clone()
    got, h2 = sa.gate_residual_norm(inplace, y, gate, scale, shift, x_out=inplace, **kw)
    assert torch.equal(got, xn) and torch.equal(h2, h)


@pytest.mark.gpu
@pytest.mark.parametrize("H,d", [(8, 128), (16, 64), (40, 128), (5, 8), (3, 24)])
def test_many_rows_of_heads(H, d):
    o = randn(2, H, 2500, d, dtype=BF16)
    q, s = sa.quantize_rows(o.transpose(1, 2))
    rows = o.transpose(1, 2).flatten(2)
    check_quantised(q, s, rows.double(), torch.zeros_like(rows, dtype=torch.float64))
    q2, s2 = sa.quantize_rows(rows)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [520, 1024, 1544])
def test_many_rows_do_not_touch_each_other(C):
    """Bad rows at a pair's first and second place, at a group's and at a batch element's border."""
    B, G, per = 3, 5, 333
    x, y = randn(B, G * per, C, dtype=BF16), randn(B, G * per, C, dtype=BF16)
    scale = randn(B, G, C, std=0.3)
    clean = sa.gate_residual_norm(x, y, None, scale)
    clean_q = sa.norm_modulate(x, scale, quantize=True)
    bad = torch.zeros(B, G * per, dtype=torch.bool, device="cuda")
    for b, l in ((0, 0), (0, 332), (0, 333), (0, 700), (0, 1664), (1, 0), (1, 999), (1, 1001), (2, 1664)):
        bad[b, l] = True
        x[b, l, (7 * l) % C] = math.nan if l % 2 else math.inf
    xn, h = sa.gate_residual_norm(x, y, None, scale)
    assert torch.equal(h[~bad], clean[1][~bad]) and torch.equal(xn[~bad], clean[0][~bad]) and h[bad].isnan().all()
    q, s = sa.norm_modulate(x, scale, quantize=True)
    assert torch.equal(q[~bad], clean_q[0][~bad]) and torch.equal(s[~bad], clean_q[1][~bad])
    assert not s[bad].isfinite().any() and not q[bad].any()
    x[:] = 0
    q, s = sa.quantize_rows(x)
    assert not q.any() and not s.any()


@pytest.mark.gpu
def test_many_rows_and_few_give_the_same_values():
    """The same row through both kernels: each within its tolerance, so they differ by two tolerances at most; and
    the larger kernel's result does not depend on what comes before or behind a row."""
    x = randn(1, 6000, 640, dtype=FP32)
    scale = randn(640, std=0.3)
    a = sa.norm_modulate(x, scale)
    assert torch.equal(a[:, 500:5500], sa.norm_modulate(x[:, 500:5500], scale))
    b = sa.norm_modulate(x[:, :100], scale)
    _, _, want, size = reference(x[:, :100], scale=scale)
    close(b, want, size, "few")
    close(a[:, :100], want, size, "many")


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows that lie more than 2^31 elements from the first one, read, written and modulated."""
    C, L = 8, 6000
    big = torch.empty(1 + 2 ** 31 // 1024 + 4000, 1024, device="cuda", dtype=BF16)     # 4.3 GB
    x = big.as_strided((2, L, C), (2 ** 31 + 16, 64, 1))
    v = randn(2, L, C, dtype=BF16)
    x.copy_(v)
    assert torch.equal(sa.norm_modulate(x), sa.norm_modulate(v))
    out = big.as_strided((2, L, C), (2 ** 31 + 16, 64, 1), 8)
    sa.norm_modulate(v, out=out)
    assert torch.equal(out, sa.norm_modulate(v)) and torch.equal(x, v)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [1024, 5120])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_many_rows_at_any_alignment(C, dtype):
    """Rows at multiples of 32, 16 and 2 bytes, in and out, and groups that end at odd rows: the same values."""
    B, G, per = 2, 3, 1601
    L = G * per
    x, y = randn(B, L, C, dtype=dtype), randn(B, L, C, dtype=dtype)
    scale = randn(B, G, C, std=0.3)
    want_x, size_x, want, size = reference(x, y, None, scale, scale)
    for off in (0, 16, 8, 4, 1):
        a, b = (torch.zeros(B, L, C + 16, device="cuda", dtype=dtype)[..., off:off + C] for _ in range(2))
        a.copy_(x), b.copy_(y)
        out, x_out = (torch.full((B, L, C + 16), 3.0, device="cuda", dtype=dtype) for _ in range(2))
        sa.gate_residual_norm(a, b, None, scale, scale, x_out=x_out[..., off:off + C], out=out[..., off:off + C])
        close(x_out[..., off:off + C], want_x, size_x, f"x' at {off}")
        close(out[..., off:off + C], want, size, f"h at {off}")
        assert (out[..., :off] == 3).all() and (out[..., off + C:] == 3).all()
        q, s = sa.quantize_rows(a)
        check_quantised(q, s, x.double(), torch.zeros_like(x, dtype=torch.float64))


# ------------------------------------------------------------------ 8-bit values, exactly
def whole(v):
    """127 v / max|row| to the nearest whole number, ties to the even one, exactly, and where another neighbour will do.
    Products of values of 24 bits or fewer by whole numbers below 2^8 are exact in 64 bits, and so is their difference
    wherever its sign decides.  The quotient is formed with two roundings of half a unit each: what is within a unit of
    a half c / 2, and not a half, may take either neighbour; a unit is 2^-23 of it at most, so |254 v - c max| <=
    2^-23 c max there (and 1e-3 of that for terms of 2^-44).  Values of 16 bits are never that near: the difference is
    zero or two units of v's last place (2^-11 of it or more, v = c max / 254) at least, 2^-18 c max."""
    v = v.double()
    a, amax = v.abs(), v.abs().amax(-1, keepdim=True)
    k = torch.where(amax > 0, torch.floor(127 * a / amax.clamp_min(1e-300)), 0.0)
    beyond = 254 * a - (2 * k + 1) * amax
    either = (beyond != 0) & (beyond.abs() <= 1.001 * 2.0 ** -23 * (2 * k + 1) * amax)
    k = k + ((beyond > 0) | ((beyond == 0) & (k % 2 == 1) & (amax > 0)))
    return (k * v.sign()).to(torch.int8), either


def check_whole(q, want, either, dtype):
    assert dtype == FP32 or not either.any()
    assert torch.equal(q[~either], want[~either]), f"{int(((q != want) & ~either).sum())} of {q.numel()} values"
    assert ((q.int() - want.int()).abs() <= 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("L,C", [(3, 64), (5, 1285), (40, 5120), (3, 16384), (2000, 1024), (2000, 1000), (1500, 5120), (700, 99)])
def test_whole_numbers_with_ties(L, C, dtype):
    """Rows of 16-bit values hold exact halves of the 8-bit step; fp32 rows hold them too, and values a unit beside
    them.  Rows of very small and very large values hold them at their own scale."""
    x = randn(2, L, C, dtype=BF16 if dtype == FP32 else dtype)
    x[0, 0], x[1, L - 1] = x[0, 0] * 2.0 ** (-8 if dtype == FP16 else -115), x[1, L - 1] * 2.0 ** (8 if dtype == FP16 else 115)
    x = x.to(dtype)
    if dtype == FP32:
        row = x[1, 0]
        row[1:] = row[0].abs() * (2 * (torch.arange(1, C, device="cuda") % 127) + 1) / 254 * row[1:].sign()
        row[1:] = torch.nextafter(row[1:], torch.where(torch.arange(1, C, device="cuda") % 3 == 0, row[1:], 1e30 * row[1:].sign()))
    want, either = whole(x)
    if dtype == BF16 and L >= 700 and C >= 1000:     # there are ties, and some of them have to go down
        a, amax = x.double().abs(), x.double().abs().amax(-1, keepdim=True)
        half = (254 * a == (2 * torch.floor(127 * a / amax) + 1) * amax)
        assert (half & (want.abs() < 127 * a / amax)).any() and (half & (want.abs() > 127 * a / amax)).any()
    q, _ = sa.quantize_rows(x)
    check_whole(q, want, either, dtype)
    if C % 8 == 0:
        q2, _ = sa.quantize_rows(x.unflatten(2, (8, C // 8)).transpose(1, 2).contiguous().transpose(1, 2))   # by heads
        assert torch.equal(q2, q)
    _, q2, _ = sa.gate_residual_norm(torch.zeros_like(x), x, norm="none", quantize=True)
    assert torch.equal(q2, q)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,bits", [(BF16, 8), (FP16, 11)])
def test_every_ratio_of_16_bit_values(dtype, bits):
    """A row for each leading part of the largest value, and in it every smaller value that is not rounded to zero."""
    m = torch.arange(2 ** (bits - 1), 2 ** bits, device="cuda", dtype=torch.float64)
    smaller = torch.cat([m * 2.0 ** -i for i in range(9)])
    x = torch.where(smaller <= m[:, None], smaller, 0.0)
    x = torch.cat([m[:, None], x * torch.where(torch.arange(len(smaller), device="cuda") % 3 == 0, -1, 1)], 1)
    assert torch.equal(x.to(dtype).double(), x)
    x = x.to(dtype)
    want, either = whole(x)
    check_whole(sa.quantize_rows(x)[0], want, either, dtype)


# ------------------------------------------------------------------ memory that inputs and outputs share
@pytest.mark.gpu
@pytest.mark.parametrize("B,L", [(3, 1), (1, 1), (1, 4), (3, 4)])
@pytest.mark.parametrize("batch_first", [True, False])
def test_slices_of_one_buffer(B, L, batch_first):
    """Columns side by side in one buffer, token-major or batch-major, are read and written; columns that meet are not."""
    C = 40
    buf = randn(B, L, 2 * C, dtype=BF16) if batch_first else randn(L, B, 2 * C, dtype=BF16).transpose(0, 1)
    x, out = buf[..., :C], buf[..., C:]
    kept = x.clone()
    want = sa.norm_modulate(kept)
    assert sa.norm_modulate(x, out=out) is out
    assert torch.equal(out, want) and torch.equal(x, kept)
    want_x, want_h = sa.gate_residual_norm(kept, kept)
    both = torch.zeros(B, L, 4 * C, device="cuda", dtype=BF16)
    sa.gate_residual_norm(both[..., :C].copy_(kept), kept, x_out=both[..., C:2 * C], out=both[..., 3 * C:])
    assert torch.equal(both[..., C:2 * C], want_x) and torch.equal(both[..., 3 * C:], want_h) and not both[..., 2 * C:3 * C].any()
    with pytest.raises(sa.SolAttnError, match="overlap"):
        sa.norm_modulate(x, out=buf[..., C - 1:2 * C - 1])
    with pytest.raises(sa.SolAttnError, match="overlap"):
        sa.norm_modulate(out, out=buf[..., 1:C + 1])
    with pytest.raises(sa.SolAttnError, match="overlap"):
        sa.gate_residual_norm(kept, kept, x_out=both[..., C:2 * C], out=both[..., 2 * C - 1:3 * C - 1])


def test_the_scales_of_rows_overlap_nothing():
    """Refused before anything is read."""
    import layer_structs as ly

    def call(q_scale):
        a = ly.NormArgs(B=2, L=4, C=64, x_inner=64, x=ly.Rows(0x10000, 0, 256, 64), y=ly.Rows(0x30000, 0, 256, 64),
                        x_out=ly.Rows(0x50000, 0, 256, 64), h=ly.Rows(0x70000, 0, 256, 64), q=0x90000, q_stride=64,
                        q_scale=q_scale, residual_scale=1.0, norm=1, eps=1e-6, scale=ly.Vectors(0xB0000, 2, 1, 64, 0))
        return sa.lib().sol_attn_norm_modulate(ly.ctypes.byref(a), None)

    for at in (0x10000, 0x303FC, 0x50010, 0x703F0, 0x90100, 0xB0080):
        assert call(at) == -1 and "overlap" in sa.lib().sol_attn_error_string(-1).decode()
