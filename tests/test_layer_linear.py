"""Products of 8-bit integers with scales for tokens and channels (int8_linear)
against exact sums, alone and behind the operators that make its rows.

Tolerances.  The integer sum is exact.  Its conversion to fp32, two products
and a sum round once each, relative to the size P + |bias| of the terms,
P = |sum| a_scale w_scale; then the output rounds once to its type:
|error| <= eps(t)/2 |value| + 4 u (P + |bias|), u = 2^-24."""
import math

import pytest

torch = pytest.importorskip("torch")

import block_sparse_attention_moments_b200 as sa  # noqa: E402

U = 2.0 ** -24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def rows(n, K, seed, full=False):
    """int8 [n, K] over the whole range, -128 among it, in rows at multiples of 16 bytes; what pads them is noise."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(-128, 128, (n, (K + 15) // 16 * 16), device="cuda", dtype=torch.int8, generator=g)
    if full:
        t.fill_(-128)
    return t[:, :K]


def scales(n, seed, mean):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(n, device="cuda").uniform_(0.2 * mean, 1.8 * mean, generator=g)


def check(got, a, sa_, w, sw, bias):
    acc = a.double() @ w.double().t()       # below 2^53: exact
    p = acc * sa_.double().reshape(-1, 1) * sw.double()
    want = p if bias is None else p + bias.double()
    size = p.abs() if bias is None else p.abs() + bias.double().abs()
    got = got.reshape(want.shape)
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + 4 * U * size + torch.finfo(got.dtype).tiny
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values off, first at {bad.nonzero()[0].tolist()}"


SIZES = [(1, 1, 1), (1, 16, 16), (1, 5120, 5120), (2, 777, 1000), (3, 130, 48), (5, 4096, 128), (8, 1001, 4096),
         (9, 33, 33), (16, 512, 1024), (17, 2048, 640), (31, 1543, 96), (33, 300, 5120), (64, 640, 1111), (65, 129, 256),
         (100, 5120, 5120), (127, 257, 127), (128, 128, 128), (129, 130, 129), (200, 1024, 1024), (256, 256, 256),
         (257, 511, 384), (500, 96, 2000), (1000, 1000, 1000), (1031, 1543, 1000), (2048, 5120, 512), (3000, 16, 64),
         (4097, 768, 4096), (20000, 264, 160)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K, dtype):
    a, w = rows(M, K, 1), rows(N, K, 2)
    s, t = scales(M, 3, 0.01), scales(N, 4, 0.01 / math.sqrt(K))
    for bias in (None, torch.randn(N, device="cuda").to(dtype)):
        out = sa.int8_linear(a, s, w, t, bias, out_dtype=dtype)
        assert out.shape == (M, N) and out.dtype == dtype
        check(out, a, s, w, t, bias)
    sa.linear_status(a.device)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 300])
def test_the_longest_sums(M):
    """-128 * -128 added up K = 131071 times stays below 2^31; one term more could not."""
    K, N = 131071, 40
    a, w = rows(M, K, 0, full=True), rows(N, K, 0, full=True)
    one = torch.ones(max(M, N), device="cuda")
    out = sa.int8_linear(a, one[:M], w, one[:N], out_dtype=FP32)
    assert (out == float(128 * 128 * K)).all()   # a multiple of 2^14 below 2^31: exact in fp32
    with pytest.raises(sa.SolAttnError, match="131071"):
        sa.int8_linear(rows(1, K + 1, 0), one[:1], rows(1, K + 1, 0), one[:1])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 7, 50, 400])
def test_strides_and_slices(M):
    """Rows cut out of wider ones, batches, outputs into a given tensor whose neighbours stay."""
    N, K = 300, 200
    big = rows(M, 640, 5)
    a, w = big[:, 208:408], rows(N, 400, 6)[:, 16:216]
    s, t = scales(M, 7, 1.0), scales(N, 8, 0.01)
    want = sa.int8_linear(a, s, w, t, out_dtype=FP32)
    check(want, a, s, w, t, None)
    buf = torch.full((M + 2, N), 5.0, device="cuda")
    out = sa.int8_linear(a, s, w, t, out=buf[1:-1])
    assert torch.equal(out, want) and (buf[0] == 5).all() and (buf[-1] == 5).all()
    odd = torch.full((M * N + 2,), 5.0, device="cuda", dtype=BF16)
    got = sa.int8_linear(a, s, w, t, out=odd[1:-1].view(M, N))     # not aligned to 16 bytes
    assert torch.equal(got, sa.int8_linear(a, s, w, t)) and odd[0] == 5 and odd[-1] == 5
    if M > 1 and M % 2 == 0:
        three = sa.int8_linear(a.unflatten(0, (2, M // 2)), s.view(2, -1), w, t, out_dtype=FP32)
        assert three.shape == (2, M // 2, N) and torch.equal(three.flatten(0, 1), want)


@pytest.mark.gpu
def test_rows_do_not_depend_on_their_neighbours():
    """A token's output has the same bits whatever the number of tokens beside it."""
    a, w = rows(700, 1000, 9), rows(520, 1000, 10)
    s, t = scales(700, 11, 0.1), scales(520, 12, 0.01)
    whole = sa.int8_linear(a, s, w, t)
    for n in (1, 2, 5, 8, 9, 40, 128, 129, 300):
        assert torch.equal(sa.int8_linear(a[:n], s[:n], w, t), whole[:n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 12, 300])
def test_scales_that_are_not_finite(M):
    a, w = rows(M, 64, 13), rows(40, 64, 14)
    s, t = torch.ones(M, device="cuda"), torch.ones(40, device="cuda")
    a[0], s[0] = 0, math.inf
    out = sa.int8_linear(a, s, w, t, out_dtype=FP32)
    assert out[0].isnan().all() and out[1:].isfinite().all()
    s[0] = 0
    assert (sa.int8_linear(a, s, w, t, out_dtype=FP32)[0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(0, 16), (5, 0)])
def test_empty(M, N):
    a, w = torch.empty(M, 32, device="cuda", dtype=torch.int8), torch.empty(N, 32, device="cuda", dtype=torch.int8)
    assert sa.int8_linear(a, torch.empty(M, device="cuda"), w, torch.empty(N, device="cuda")).shape == (M, N)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 60, 500])
def test_streams_and_graphs(M):
    a, w = rows(M, 512, 15), rows(640, 512, 16)
    s, t = scales(M, 17, 0.1), scales(640, 18, 0.01)
    want = sa.int8_linear(a, s, w, t)
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [sa.int8_linear(a, s, w, t, stream=(side, other)[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sa.int8_linear(a, s, w, t)
    a.neg_()
    for _ in range(3):
        graph.replay()
    want = sa.int8_linear(a, s, w, t)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    sa.linear_status(stream=side)


@pytest.mark.gpu
@pytest.mark.parametrize("L,C,N", [(1, 256, 768), (40, 1000, 99), (333, 640, 512)])
def test_behind_the_norm(L, C, N):
    """norm_modulate(quantize=True) into int8_linear: exactly the product of the rows that the norm gives."""
    g = torch.Generator(device="cuda").manual_seed(19)
    x = torch.empty(2, L, C, device="cuda", dtype=BF16).normal_(0, 1, generator=g)
    q, s = sa.norm_modulate(x, quantize=True)
    wq, ws = sa.quantize_rows(torch.empty(N, C, device="cuda").normal_(0, 0.02, generator=g))
    y = sa.int8_linear(q, s, wq, ws)
    assert y.shape == (2, L, N)
    check(y, q.flatten(0, 1), s, wq, ws, None)


# ------------------------------------------------------------------ refusals
def test_entry_point_refusals():
    """The library's own checks, which come before anything is read or enqueued."""
    import layer_structs as ly
    lib = sa.lib()

    def call(**kw):
        p = ly.LinearArgs(4, 32, 64, 0x10000, 64, 0x20000, 0x30000, 64, 0x40000, None, 0, 0x50000, 0, 32)
        for k, v in kw.items():
            setattr(p, k, v)
        return lib.sol_attn_quantized_linear(ly.ctypes.byref(p), None)

    assert lib.sol_attn_quantized_linear(None, None) == -1
    assert call(M=-1) == -1 and call(N=-1) == -1 and call(K=0) == -1 and call(K=131072, a_stride=1 << 18, w_stride=1 << 18) == -2
    assert call(M=0) == 0 and call(N=0) == 0
    assert call(a=None) == -1 and call(w=None) == -1 and call(a_scale=None) == -1 and call(w_scale=None) == -1
    assert call(out=None) == -1 and call(out_dtype=3) == -1
    assert call(a=0x10008) == -3 and call(w=0x30001) == -3 and call(a_stride=72) == -3 and call(w_stride=65) == -3
    assert call(a_stride=48) == -1 and call(w_stride=48) == -1 and call(out_stride=31) == -1
    assert call(out=0x50001) == -3 and call(a_scale=0x20002) == -3
    assert call(bias=0x60001, bias_dtype=0) == -3 and call(bias=0x60000, bias_dtype=7) == -1
    assert call(flags=1) == -1 and call(M=2 ** 31 - 1) == -2
    assert call(out=0x10000) == -1 and call(out=0x30000) == -1 and call(out=0x40040) == -1


@pytest.mark.gpu
def test_refusals():
    a, w = rows(4, 64, 20), rows(32, 64, 21)
    s, t = scales(4, 22, 1.0), scales(32, 23, 1.0)

    def refused(match, call):
        with pytest.raises((ValueError, sa.SolAttnError), match=match):
            call()

    refused("unsupported type", lambda: sa.int8_linear(a.float(), s, w, t))
    refused("CUDA", lambda: sa.int8_linear(a, s, w.cpu(), t))
    refused("must be", lambda: sa.int8_linear(a, s, w[:, :32], t))
    refused("a_scale must hold", lambda: sa.int8_linear(a, s[:3], w, t))
    refused("w_scale must hold", lambda: sa.int8_linear(a, s, w, t[:3]))
    refused("unsupported type", lambda: sa.int8_linear(a, s.half(), w, t))
    refused("bias must be", lambda: sa.int8_linear(a, s, w, t, t[:5]))
    refused("unsupported type", lambda: sa.int8_linear(a, s, w, t, out_dtype=torch.float64))
    refused("out must be", lambda: sa.int8_linear(a, s, w, t, out=torch.empty(4, 31, device="cuda", dtype=BF16)))
    refused("multiples of 16", lambda: sa.int8_linear(torch.zeros(4, 40, device="cuda", dtype=torch.int8), s,
                                                      torch.zeros(32, 40, device="cuda", dtype=torch.int8), t))
    refused("aligned", lambda: sa.int8_linear(a[:, 8:40], s, w[:, 8:40], t))
    refused("contiguous", lambda: sa.int8_linear(a.t().contiguous().t(), s, w, t))
    refused("no backward", lambda: sa.int8_linear(a, s.clone().requires_grad_(), w, t))
    refused("at least 1", lambda: sa.int8_linear(a[:, :0], s, w[:, :0], t))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(10, 300, 600), (40, 20000, 256), (100, 512, 2000), (300, 300, 500), (4000, 5000, 512)])
def test_waits_that_run_out(M, N, K):
    """Products whose tiles never come: every wait gives up, the kernel ends, its output stays as it was, the status
    says so once, and the next product is right."""
    import layer_structs as ly
    from block_sparse_attention_moments_b200 import FLAG_TEST_STALL
    a, w = rows(M, K, 30), rows(N, K, 31)
    s, t = scales(M, 32, 0.1), scales(N, 33, 0.01)
    out = torch.full((M, N), 7.0, device="cuda", dtype=BF16)
    p = ly.LinearArgs(M, N, K, a.data_ptr(), a.stride(0), s.data_ptr(), w.data_ptr(), w.stride(0), t.data_ptr(), None, 0,
                      out.data_ptr(), 0, N, FLAG_TEST_STALL)
    assert sa.lib().sol_attn_quantized_linear(ly.ctypes.byref(p), torch.cuda.current_stream().cuda_stream) == 0
    with pytest.raises(sa.SolAttnError, match="gave up") as e:
        sa.linear_status(a.device)
    assert e.value.code == -5
    assert (out == 7).all()
    sa.linear_status(a.device)
    check(sa.int8_linear(a, s, w, t), a, s, w, t, None)
    sa.linear_status(a.device)


# ------------------------------------------------------------------ the status
def stall(M, N, K, stream):
    """Enqueues a product whose tiles never come; returns what it reads, to be kept until it has ended."""
    import layer_structs as ly
    from block_sparse_attention_moments_b200 import FLAG_TEST_STALL
    a, w = rows(M, K, 34), rows(N, K, 35)
    s, t = scales(M, 36, 0.1), scales(N, 37, 0.01)
    out = torch.zeros((M, N), device="cuda", dtype=BF16)
    torch.cuda.synchronize()
    p = ly.LinearArgs(M, N, K, a.data_ptr(), a.stride(0), s.data_ptr(), w.data_ptr(), w.stride(0), t.data_ptr(), None, 0,
                      out.data_ptr(), 0, N, FLAG_TEST_STALL)
    assert sa.lib().sol_attn_quantized_linear(ly.ctypes.byref(p), stream.cuda_stream) == 0
    return a, w, s, t, out


@pytest.mark.gpu
def test_status_waits_for_its_stream_only():
    """The status of one stream, while the default stream is busy for about a second."""
    side = torch.cuda.Stream()
    keep = stall(300, 300, 500, side)
    torch.cuda._sleep(2_000_000_000)
    busy = torch.cuda.Event()
    busy.record()
    with pytest.raises(sa.SolAttnError, match="gave up"):
        sa.linear_status(stream=side)
    sa.linear_status(stream=side)
    assert not busy.query()
    torch.cuda.synchronize()
    del keep


@pytest.mark.gpu
def test_status_of_products_that_end_while_it_is_read():
    """Readings on another stream while a product gives up: it is reported by one of them, or by the one behind it."""
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        keep = stall(300, 300, 500, side)
        reports = 0
        for stream in [other] * 50 + [side]:
            try:
                sa.linear_status(stream=stream)
            except sa.SolAttnError as e:
                assert e.code == -5
                reports += 1
        assert reports
        del keep
    sa.linear_status(stream=side)


@pytest.mark.gpu
def test_status_is_refused_in_a_capture():
    """And the capture goes on."""
    a, w = rows(40, 64, 38), rows(32, 64, 39)
    s, t = scales(40, 40, 1.0), scales(32, 41, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sa.int8_linear(a, s, w, t)
        with pytest.raises(sa.SolAttnError, match="captured") as e:
            sa.linear_status(a.device)
        assert e.value.code == -6
    graph.replay()
    assert torch.equal(y, sa.int8_linear(a, s, w, t))
    sa.linear_status(a.device)


# ------------------------------------------------------------------ large products
# Of these sizes the tiles of two SMs are taken (on 148 SMs), in several bands of tokens, with ragged edges.  The weights
# of the second one are larger than what is kept in L2 beside the rest.
LARGE = [(4099, 5001, 384), (4500, 6001, 6000), (5003, 4001, 1000)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_and_ragged(M, N, K, dtype):
    """Odd numbers of channels, so that output rows are at no multiple of 16 bytes, rows at such multiples with an odd
    end, and an output tensor at an odd place; the same bits in all."""
    a, w = rows(M, K, 50), rows(N, K, 51)
    s, t = scales(M, 52, 0.01), scales(N, 53, 0.01 / math.sqrt(K))
    bias = torch.randn(N, device="cuda").to(dtype)
    out = sa.int8_linear(a, s, w, t, bias, out_dtype=dtype)
    check(out, a, s, w, t, bias)
    even = N // 8 * 8
    assert torch.equal(sa.int8_linear(a, s, w[:even], t[:even], bias[:even], out_dtype=dtype), out[:, :even])
    odd = torch.full((M * N + 2,), 5.0, device="cuda", dtype=dtype)
    assert torch.equal(sa.int8_linear(a, s, w, t, bias, out=odd[1:-1].view(M, N)), out) and odd[0] == 5 and odd[-1] == 5
    sa.linear_status(a.device)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", LARGE)
def test_rows_of_large_products_do_not_depend_on_their_neighbours(M, N, K):
    """The same bits through the kernels for one to four tokens, for up to 128, for single SMs and for pairs."""
    a, w = rows(M, K, 54), rows(N, K, 55)
    s, t = scales(M, 56, 0.1), scales(N, 57, 0.01)
    whole = sa.int8_linear(a, s, w, t)
    for first, n in ((0, 1), (255, 2), (M - 4, 4), (250, 12), (1000, 30), (M - 128, 128), (127, 130), (4095, 4), (M - 300, 300)):
        assert torch.equal(sa.int8_linear(a[first:first + n], s[first:first + n], w, t), whole[first:first + n]), (first, n)
    n = 520
    assert torch.equal(sa.int8_linear(a, s, w[:n], t[:n]), whole[:, :n])


@pytest.mark.gpu
def test_the_longest_sums_of_large_products():
    M, N, K = 513, 9000, 131071
    a, w = rows(M, K, 0, full=True), rows(N, K, 0, full=True)
    one = torch.ones(N, device="cuda")
    assert (sa.int8_linear(a, one[:M], w, one, out_dtype=FP32) == float(128 * 128 * K)).all()


@pytest.mark.gpu
def test_bands_of_tokens():
    """Many tokens and few weights, which go through narrow bands: the last band is half full."""
    M, N, K = 40_500, 777, 1000
    a, w = rows(M, K, 58), rows(N, K, 59)
    s, t = scales(M, 60, 0.01), scales(N, 61, 0.01 / math.sqrt(K))
    out = sa.int8_linear(a, s, w, t)
    check(out, a, s, w, t, None)
    assert torch.equal(sa.int8_linear(a[-300:], s[-300:], w, t), out[-300:])
