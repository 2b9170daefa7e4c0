"""Rotary positions with several axes, query/key norm and head-major layout
(rope) against the formula in 64 bits.

Tolerances.  |error| <= eps(t)/2 |value| + 64 u M, u = 2^-24, for an output of
type t: M = |a'| + |b'| of the normalised pair.  The turn's fraction is rounded
to fp32 (an angle error of pi u at most), sine and cosine add 2 u each, the sum
of squares 48 u (a thread adds 32 terms in a row, trees the rest), its root's
reciprocal 2 u, weight, products and sum 6 u."""
import math

import pytest

torch = pytest.importorskip("torch")

import block_sparse_attention_moments_b200 as sa  # noqa: E402

U = 2.0 ** -24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def grid_positions(L, grid, start):
    f, h, w = grid
    i = start + torch.arange(L)
    return torch.stack([i // (h * w), i // w % h, i % w], -1) * (i < f * h * w)[:, None]


def reference(x, pos, axes, weight, norm, pairing, theta=10000.0, freqs=None, eps=1e-6):
    """([B, H, L, d], size of its terms) in 64 bits."""
    B, L, H, d = x.shape
    x = x.double()
    if norm != "none":
        v = x.flatten(2) if norm == "token" else x
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
        v = v if weight is None else v * weight.double()
        x = v.view(B, L, H, d)
    axis = sum(([i] * (n // 2) for i, n in enumerate(axes)), [])
    f = [theta ** (-2 * j / n) for n in axes for j in range(n // 2)] if freqs is None else freqs
    t = pos.double().cuda()[..., axis] * torch.tensor(f, device="cuda", dtype=torch.float64)
    t = (t if t.dim() == 3 else t[None])[:, :, None]
    a, b = (x[..., :d // 2], x[..., d // 2:]) if pairing == "half" else (x[..., 0::2], x[..., 1::2])
    u, v, m = a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos(), a.abs() + b.abs()
    out, size = ((torch.cat([u, v], -1), torch.cat([m, m], -1)) if pairing == "half" else
                 (torch.stack([u, v], -1).flatten(-2), torch.stack([m, m], -1).flatten(-2)))
    return out.transpose(1, 2), size.transpose(1, 2)


def close(got, want_size, what):
    want, size = want_size
    assert got.shape == want.shape and got.is_contiguous()
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + 64 * U * size + torch.finfo(got.dtype).tiny
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float(((got.double() - want).abs() / tol).nan_to_num(9e9).max()):.3g} of the tolerance"


def make(B, L, H, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.empty(B, L, 3, H, d, device="cuda", dtype=dtype).normal_(0, 1, generator=g)
    return qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]


def weights(norm, H, d, dtype, seed):
    if norm == "none":
        return None, None
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.empty(d if norm == "head" else H * d, device="cuda", dtype=dtype).normal_(1, 0.3, generator=g)
                 for _ in range(2))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("norm", ["none", "head", "token"])
@pytest.mark.parametrize("B,H,d,grid,extra,start", [
    (1, 1, 16, (1, 1, 1), 0, 0), (2, 3, 64, (2, 3, 5), 0, 0), (1, 40, 128, (3, 5, 8), 7, 0), (2, 5, 96, (4, 4, 4), 3, 11),
    (1, 2, 256, (2, 9, 7), 0, 100), (1, 64, 256, (1, 2, 3), 1, 0), (3, 7, 48, (1, 6, 6), 0, 20), (1, 17, 80, (5, 2, 2), 0, 0)])
def test_grid(B, H, d, grid, extra, start, norm, pairing, dtype):
    L = max(1, math.prod(grid) - start) + extra
    q, k, v = make(B, L, H, d, dtype, 1)
    wq, wk = weights(norm, H, d, dtype, 2)
    q2, k2, v2 = sa.rope(q, k, v, grid=grid, start=start, pairing=pairing, norm=norm, q_weight=wq, k_weight=wk)
    pos, axes = grid_positions(L, grid, start), sa.rope_axes(d)
    assert sum(axes) == d and not any(n % 2 for n in axes)
    close(q2, reference(q, pos, axes, wq, norm, pairing), "q")
    close(k2, reference(k, pos, axes, wk, norm, pairing), "k")
    assert torch.equal(v2, v.transpose(1, 2)) and v2.is_contiguous()
    pair = sa.rope(q, k, grid=grid, start=start, pairing=pairing, norm=norm, q_weight=wq, k_weight=wk)
    assert len(pair) == 2 and torch.equal(pair[0], q2) and torch.equal(pair[1], k2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64, torch.float32, torch.float64])
@pytest.mark.parametrize("axes", [(64,), (32, 32), (16, 24, 24), (8, 8, 16, 32), (0, 32, 32)])
def test_positions(axes, dtype):
    """Positions of each token, far ones among them, with one to four axes, in every type and any strides."""
    B, L, H, d, A = 2, 37, 3, 64, len(axes)
    q, k, _ = make(B, L, H, d, FP32, 3)
    g = torch.Generator().manual_seed(4)
    pos = torch.randint(0, 1_000_000, (B, L, A), generator=g)
    pos[:, 5] = 0
    pos[0, 0] = 2 ** 24 - 1
    pos = (pos.double() + (0.25 if dtype.is_floating_point else 0)).to(dtype)
    where = pos.cuda()
    q2, k2 = sa.rope(q, k, positions=where, axes=axes)
    close(q2, reference(q, pos, axes, None, "none", "interleaved"), "q")
    close(k2, reference(k, pos, axes, None, "none", "interleaved"), "k")
    strided = torch.zeros(L, 2 * A, B, device="cuda", dtype=dtype).permute(2, 0, 1)[..., ::2]
    strided.copy_(where)
    assert torch.equal(sa.rope(q, k, positions=strided, axes=axes)[0], q2)
    same = sa.rope(q, k, positions=where[1], axes=axes)[0]
    assert torch.equal(same[1], q2[1])
    assert torch.equal(same, sa.rope(q, k, positions=where[1:2], axes=axes)[0])


@pytest.mark.gpu
def test_frequencies_and_theta():
    q, k, _ = make(1, 30, 2, 64, FP32, 5)
    pos = torch.arange(90).view(30, 3)
    f = [0.5 / (1 + i) for i in range(32)]
    a = sa.rope(q, k, positions=pos.cuda(), freqs=f, pairing="half")
    close(a[0], reference(q, pos, sa.rope_axes(64), None, "none", "half", freqs=f), "freqs")
    a = sa.rope(q, k, positions=pos.cuda(), theta=256.0)
    close(a[1], reference(k, pos, sa.rope_axes(64), None, "none", "interleaved", theta=256.0), "theta")


@pytest.mark.gpu
def test_layouts():
    """Separate tensors, head-major inputs and slices give the same bits as one projection's views."""
    q, k, v = make(2, 50, 4, 64, BF16, 6)
    kw = dict(grid=(2, 5, 5), norm="head")
    want = sa.rope(q, k, v, **kw)
    for f in (lambda t: t.contiguous(), lambda t: t.transpose(1, 2).contiguous().transpose(1, 2),
              lambda t: torch.cat([t, t], 1)[:, :50], lambda t: torch.cat([t, t], 3)[..., 64:]):
        got = sa.rope(f(q), f(k), f(v), **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_shards_of_a_sequence_meet():
    """A sequence cut into pieces, each with its start, gives what the whole gives."""
    q, k, _ = make(1, 75, 2, 128, BF16, 7)
    whole = sa.rope(q, k, grid=(3, 5, 4), norm="token")
    cut = [sa.rope(q[:, a:b], k[:, a:b], grid=(3, 5, 4), start=a, norm="token") for a, b in ((0, 1), (1, 40), (40, 75))]
    for i in range(2):
        assert torch.equal(torch.cat([c[i] for c in cut], 2), whole[i])


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ["head", "token"])
def test_rows_do_not_touch_each_other(norm):
    q, k, v = make(1, 40, 3, 64, BF16, 8)
    clean = sa.rope(q, k, v, grid=(1, 5, 8), norm=norm)
    q = q.clone()
    q[0, 7, 1, 3], q[0, 30, 2, 0], q[0, 12] = math.nan, math.inf, 0
    got = sa.rope(q, k, v, grid=(1, 5, 8), norm=norm)
    other = [i for i in range(40) if i not in (7, 12, 30)]
    assert torch.equal(got[0][:, :, other], clean[0][:, :, other])
    assert torch.equal(got[1], clean[1]) and torch.equal(got[2], clean[2])
    assert got[0][0, 1, 7].isnan().any() and (got[0][0, :, 12] == 0).all()
    if norm == "head":
        assert torch.equal(got[0][0, 0, 7], clean[0][0, 0, 7])


@pytest.mark.gpu
def test_empty_streams_and_graphs():
    q, k, v = make(2, 0, 3, 64, BF16, 9)
    assert [t.shape for t in sa.rope(q, k, v, grid=(1, 1, 1))] == [(2, 3, 0, 64)] * 3
    q, k, v = make(2, 60, 3, 64, BF16, 10)
    kw = dict(grid=(3, 4, 5), norm="token")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sa.rope(q, k, v, stream=side, **kw)
    side.synchronize()
    want = sa.rope(q, k, v, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sa.rope(q, k, v, **kw)
    q.mul_(2)
    graph.replay()
    want = sa.rope(q, k, v, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_into_the_attention():
    """A projection's output through rope and the attention: the same as the attention of the 64-bit form's q and k
    in bf16, up to the roundings of q and k (the rotation's outputs differ from them in no more than one unit)."""
    q, k, v = make(1, 200, 2, 128, BF16, 11)
    a, b, c = sa.rope(q, k, v, grid=(2, 10, 10), norm="head")
    pos, axes = grid_positions(200, (2, 10, 10), 0), sa.rope_axes(128)
    a2 = reference(q, pos, axes, None, "head", "interleaved")[0].to(BF16).contiguous()
    b2 = reference(k, pos, axes, None, "head", "interleaved")[0].to(BF16).contiguous()
    got = sa.forward(a, b, c, -math.inf, 4, flags=sa.FLAG_SELECT_ALL)
    want = sa.forward(a2, b2, v.transpose(1, 2).contiguous(), -math.inf, 4, flags=sa.FLAG_SELECT_ALL)
    assert (got.float() - want.float()).abs().max() <= 2e-2


# ------------------------------------------------------------------ refusals
def test_entry_point_refusals():
    """The library's own checks, which come before anything is read or enqueued."""
    import layer_structs as ly
    lib, c = sa.lib(), ly.ctypes
    freqs, axis = (c.c_double * 32)(*[1.0] * 32), (c.c_ubyte * 32)()
    keep = []

    def args(**kw):
        t = lambda i, o: ly.RopeTensor(i, 4 * 128, 128, 64, o)
        a = ly.RopeArgs(B=2, L=4, H=2, d=64, dtype=0, q=t(0x10000, 0x90000), k=t(0x20000, 0xA0000), axes=3,
                         freqs=c.addressof(freqs), axis=c.addressof(axis), grid_f=1, grid_h=2, grid_w=2)
        for k, v in kw.items():
            setattr(a, k, v)
        keep.append(a)
        return c.byref(a)

    call = lambda **kw: lib.sol_attn_rope(args(**kw), None)
    assert lib.sol_attn_rope(None, None) == -1
    assert call(H=0) == -1 and call(d=0) == -1 and call(d=72) == -2 and call(d=272) == -2 and call(H=257) == -2
    assert call(L=0) == 0 and call(B=0) == 0 and call(L=-1) == -1
    assert call(dtype=3) == -1 and call(norm=3) == -1 and call(eps=-1.0) == -1 and call(pairing=2) == -1
    assert call(axes=5) == -2 and call(axes=0) == -2 and call(axes=2) == -1
    assert call(freqs=None) == -1 and call(axis=None) == -1
    assert call(grid_f=0) == -1 and call(grid_f=1 << 16, grid_h=1 << 16) == -1 and call(start=-1) == -1
    assert call(pos_kind=5) == -1 and call(pos_kind=1) == -1 and call(pos_kind=2, positions=0x30004) == -3
    assert call(q=ly.RopeTensor(0x10008, 512, 128, 64, 0x90000)) == -3
    assert call(q=ly.RopeTensor(0x10000, 512, 124, 64, 0x90000)) == -3
    assert call(q=ly.RopeTensor(0x10000, 512, -128, 64, 0x90000)) == -1
    assert call(q=ly.RopeTensor(0x10000, 512, 128, 64, 0x10000)) == -1
    assert call(q=ly.RopeTensor(0x10000, 512, 128, 64, 0xA0000)) == -1
    assert call(q=ly.RopeTensor(0x10000, 512, 128, 64, 0x90000, 0x50000, 0)) == -1    # a weight without a norm
    assert call(norm=1, q=ly.RopeTensor(0x10000, 512, 128, 64, 0x90000, 0xA0000, 0)) == -1     # k's output over q's weight
    assert call(pos_kind=1, positions=0x90000) == -1 and call(pos_kind=1, positions=0x30000, pos_stride_l=-3) == -1
    bad = (c.c_double * 32)(*[math.nan] * 32)
    assert call(freqs=c.addressof(bad)) == -1
    far = (c.c_ubyte * 32)(*[3] * 32)
    assert call(axis=c.addressof(far)) == -1


@pytest.mark.gpu
def test_refusals():
    q, k, v = make(2, 12, 2, 64, BF16, 12)
    kw = dict(grid=(1, 3, 4))

    def refused(match, call):
        with pytest.raises((ValueError, sa.SolAttnError), match=match):
            call()

    pos = torch.zeros(12, 3, device="cuda", dtype=torch.int32)
    refused("either grid or positions", lambda: sa.rope(q, k, v))
    refused("either grid or positions", lambda: sa.rope(q, k, v, positions=pos, **kw))
    refused("grid must be", lambda: sa.rope(q, k, v, grid=(1, 0, 4)))
    refused("grid must be", lambda: sa.rope(q, k, v, grid=(3, 4)))
    refused("bad grid", lambda: sa.rope(q, k, v, grid=(2 ** 20, 2 ** 20, 1)))
    refused("start", lambda: sa.rope(q, k, v, start=-1, **kw))
    refused("start goes", lambda: sa.rope(q, k, v, start=1, positions=pos))
    refused("positions must be", lambda: sa.rope(q, k, v, positions=pos[:5]))
    refused("unsupported type", lambda: sa.rope(q, k, v, positions=pos.to(torch.int16)))
    refused("axes must be", lambda: sa.rope(q, k, v, axes=(32, 32), **kw))
    refused("axes must be", lambda: sa.rope(q, k, v, axes=(21, 21, 22), **kw))
    refused("axes must be given", lambda: sa.rope(q, k, v, positions=pos[:, :2]))
    refused("freqs", lambda: sa.rope(q, k, v, freqs=[1.0] * 31, **kw))
    refused("not finite", lambda: sa.rope(q, k, v, freqs=[math.inf] * 32, **kw))
    refused("theta", lambda: sa.rope(q, k, v, theta=-1.0, **kw))
    refused("pairing", lambda: sa.rope(q, k, v, pairing="both", **kw))
    refused("norm must be", lambda: sa.rope(q, k, v, norm="layer", **kw))
    refused("share one shape", lambda: sa.rope(q, k[:, :5], v, **kw))
    refused("share one shape", lambda: sa.rope(q, k, v.float(), **kw))
    refused("goes with a norm", lambda: sa.rope(q, k, v, q_weight=torch.ones(64, device="cuda"), **kw))
    refused("contiguous", lambda: sa.rope(q, k, v, norm="head", k_weight=torch.ones(63, device="cuda"), **kw))
    refused("multiple of 16", lambda: sa.rope(q[..., :40], k[..., :40], axes=(8, 16, 16), **kw))
    refused("16-byte|multiples of 8", lambda: sa.rope(q[..., 4:52], k[..., 4:52], axes=(16, 16, 16), **kw))
    refused("contiguous", lambda: sa.rope(q.transpose(2, 3), k.transpose(2, 3), axes=(0, 0, 2), **kw))
    refused("no backward", lambda: sa.rope(q.clone().requires_grad_(), k, v, **kw))
    refused("CUDA", lambda: sa.rope(q.cpu(), k, v, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("norm", ["none", "head", "token"])
@pytest.mark.parametrize("B,H,d,grid,extra", [(2, 40, 128, (5, 9, 14), 3), (1, 8, 64, (7, 30, 41), 0), (1, 3, 96, (9, 31, 20), 11),
                                              (1, 70, 96, (3, 20, 13), 0)])
def test_more_tokens_than_teams(B, H, d, grid, extra, norm, pairing):
    """Teams that go through several tokens: rings and tables that come round."""
    L = math.prod(grid) + extra
    q, k, v = make(B, L, H, d, BF16, 20)
    wq, wk = weights(norm, H, d, BF16, 21)
    q2, k2, v2 = sa.rope(q, k, v, grid=grid, pairing=pairing, norm=norm, q_weight=wq, k_weight=wk)
    pos, axes = grid_positions(L, grid, 0), sa.rope_axes(d)
    close(q2, reference(q, pos, axes, wq, norm, pairing), "q")
    close(k2, reference(k, pos, axes, wk, norm, pairing), "k")
    assert torch.equal(v2, v.transpose(1, 2))
    q2, k2 = sa.rope(q, k, positions=pos.cuda(), pairing=pairing, norm=norm, q_weight=wq, k_weight=wk)
    close(k2, reference(k, pos, axes, wk, norm, pairing), "k without v")


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ["head", "token"])
@pytest.mark.parametrize("H,d", [(64, 256), (341, 48), (68, 240), (1024, 16), (204, 80)])
def test_the_widest_rows(H, d, norm):
    """fp32 rows of up to 16384 channels with v: less of them fits shared memory."""
    q, k, v = make(1, 200, H, d, FP32, 22)
    wq, wk = weights(norm, H, d, FP32, 23)
    for pairing in ("interleaved", "half"):
        q2, k2, v2 = sa.rope(q, k, v, grid=(4, 5, 10), pairing=pairing, norm=norm, q_weight=wq, k_weight=wk)
        pos, axes = grid_positions(200, (4, 5, 10), 0), sa.rope_axes(d)
        close(q2, reference(q, pos, axes, wq, norm, pairing), "q")
        close(k2, reference(k, pos, axes, wk, norm, pairing), "k")
        assert torch.equal(v2, v.transpose(1, 2))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Inputs whose tokens and heads lie more than 2^31 elements from the first one, and an output of that size."""
    B, L, H, d = 1, 40, 2, 64
    big = torch.zeros(2 ** 31 // 1024 + 8000, 1024, device="cuda", dtype=BF16)
    q, k, v = make(B, L, H, d, BF16, 24)
    far = [big.as_strided((B, L, H, d), (2 ** 31, 64, 2 ** 31 + 4096, 1), i * 8192) for i in range(3)]
    for f, t in zip(far, (q, k, v)):
        f.copy_(t)
    kw = dict(grid=(2, 4, 5), norm="head")
    assert all(torch.equal(a, b) for a, b in zip(sa.rope(*far, **kw), sa.rope(q, k, v, **kw)))
    del big, far
    L = 300_000
    q = torch.randn(1, 1, 128, 64, device="cuda", dtype=BF16).expand(1, L, 128, 64)     # 2.46e9 values out
    out, _ = sa.rope(q, q, grid=(300, 40, 25))
    for l in (0, 1, 262_143, 262_144, L - 1):
        one, _ = sa.rope(q[:, :1], q[:, :1], grid=(300, 40, 25), start=l)
        assert torch.equal(out[:, :, l], one[:, :, 0])
