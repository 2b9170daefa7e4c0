"""A whole attention layer (AttentionLayer): its operators together, as they are used."""
import math

import pytest

torch = pytest.importorskip("torch")

import block_sparse_attention_moments_b200 as sa  # noqa: E402

BF16, FP32 = torch.bfloat16, torch.float32


def make(B, L, H, d, dtype, seed=0):
    C = H * d
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *shape, std=1.0, mean=0.0, dtype=FP32: torch.empty(shape, device="cuda", dtype=dtype).normal_(mean, std, generator=g)
    w = dict(w_qkv=rnd(3 * C, C, std=C ** -0.5), w_out=rnd(C, C, std=C ** -0.5), b_qkv=rnd(3 * C, std=0.1),
             b_out=rnd(C, std=0.1), q_weight=rnd(C, mean=1, std=0.1), k_weight=rnd(C, mean=1, std=0.1))
    vectors = [t for t in rnd(B, 5, C, std=0.3).unbind(1)]
    return rnd(B, L, C, dtype=dtype), w, vectors


def plain(x, w, vectors, H, grid, quantised):
    """The layer in 64 bits with dense attention; quantised: its four 8-bit operands rounded as the layer rounds them."""
    B, L, C = x.shape
    d = C // H
    shift, scale, gate, next_shift, next_scale = (v.double()[:, None] for v in vectors)

    def eight(t):
        if not quantised:
            return t
        s = t.abs().amax(-1, keepdim=True) / 127
        return torch.round(t / s) * s

    def norm(t):
        c = t - t.mean(-1, keepdim=True)
        return c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-6)

    def rms(t, weight):
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * weight.double()

    x = x.double()
    h = eight(norm(x) * (1 + scale) + shift)
    q, k, v = (h @ eight(w["w_qkv"].double()).t() + w["b_qkv"].double()).chunk(3, -1)
    f, r, c = grid
    i = torch.arange(L, device="cuda")
    pos = (torch.stack([i // (r * c), i // c % r, i % c], -1) * (i < f * r * c)[:, None]).double()
    axes = sa.rope_axes(d)
    t = torch.cat([pos[:, a, None] * torch.tensor([10000.0 ** (-2 * j / n) for j in range(n // 2)], device="cuda", dtype=torch.float64)
                   for a, n in enumerate(axes)], -1)
    turn = torch.polar(torch.ones_like(t), t)

    def heads(u):
        return u.view(B, L, H, d).transpose(1, 2)

    def rotate(u):
        return torch.view_as_real(torch.view_as_complex(heads(u).reshape(B, H, L, d // 2, 2)) * turn).flatten(-2)

    q, k = rotate(rms(q, w["q_weight"])), rotate(rms(k, w["k_weight"]))
    o = torch.softmax(q @ k.transpose(-1, -2) / math.sqrt(d), -1) @ heads(v)
    y = eight(o.transpose(1, 2).flatten(2)) @ eight(w["w_out"].double()).t() + w["b_out"].double()
    xn = x + gate * y
    return xn, norm(xn) * (1 + next_scale) + next_shift, gate * y


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,H,d,grid,dtype", [(1, 1, 1, 64, (1, 1, 1), FP32), (2, 150, 3, 64, (2, 5, 13), FP32),
                                                (1, 333, 2, 128, (3, 10, 11), BF16), (1, 640, 4, 128, (4, 10, 16), FP32)])
def test_layer_against_the_formulas(B, L, H, d, grid, dtype):
    """With every block selected, against dense attention in 64 bits on the same 8-bit weights and activations.
    What the layer rounds besides: q, k, v, o and y to bf16 (2^-9 of the value each, root mean square 2^-9/sqrt(3) or
    less), the attention's own probabilities to bf16, and 8-bit values that those roundings move across a half: an
    operand that is off by the relative error e moves that many of its values by one step, which adds no more than e
    again.  Five such steps in a row, each within 2^-8 of the whole in the 2-norm: 2 * 5 * 2^-8 = 4e-2 bounds the
    block's own part gate * y, and h' is off by as much of its unit size, besides its own bf16."""
    x, w, vectors = make(B, L, H, d, dtype)
    layer = sa.AttentionLayer(w["w_qkv"], w["w_out"], H, b_qkv=w["b_qkv"], b_out=w["b_out"], q_weight=w["q_weight"],
                              k_weight=w["k_weight"])
    shift, scale, gate, next_shift, next_scale = vectors
    xn, h = layer(x, scale, shift, gate, beta=-math.inf, chunk=4, flags=sa.FLAG_SELECT_ALL, grid=grid,
                  next_scale=next_scale, next_shift=next_shift)
    assert xn.dtype == dtype and h.dtype == BF16
    want_x, want_h, branch = plain(x, w, vectors, H, grid, True)
    rounding = 2.0 ** -8 * want_x.norm() if dtype == BF16 else 0
    assert (xn.double() - want_x).norm() <= 4e-2 * branch.norm() + rounding
    assert (h.double() - want_h).norm() <= (4e-2 + 2.0 ** -7) * want_h.norm()


@pytest.mark.gpu
def test_layer_is_its_operators():
    """The layer gives the bits of its operators called one by one, sparse, in place and over again."""
    B, L, H, d, grid = 2, 700, 2, 128, (7, 10, 10)
    x, w, vectors = make(B, L, H, d, BF16, 1)
    shift, scale, gate, next_shift, next_scale = vectors
    layer = sa.AttentionLayer(w["w_qkv"], w["w_out"], H, b_qkv=w["b_qkv"], b_out=w["b_out"], q_weight=w["q_weight"],
                              k_weight=w["k_weight"])
    kw = dict(beta=0.5, chunk=8, grid=grid, next_scale=next_scale, next_shift=next_shift)
    xn, h = layer(x, scale, shift, gate, **kw)
    a, s = sa.norm_modulate(x, scale, shift, quantize=True)
    wq, ws = sa.quantize_rows(w["w_qkv"])
    qkv = sa.int8_linear(a, s, wq, ws, w["b_qkv"]).view(B, L, 3, H, d)
    q, k, v = sa.rope(*qkv.unbind(2), grid=grid, norm="token", q_weight=w["q_weight"], k_weight=w["k_weight"])
    o = sa.forward(q, k, v, 0.5, 8)
    counts = sa.stats(B, H, L)
    assert 0 < int(counts.sum()) < B * H * 11 * 11
    a, s = sa.quantize_rows(o.transpose(1, 2))
    wq, ws = sa.quantize_rows(w["w_out"])
    y = sa.int8_linear(a, s, wq, ws, w["b_out"])
    want = sa.gate_residual_norm(x, y, gate, next_scale, next_shift)
    assert torch.equal(xn, want[0]) and torch.equal(h, want[1])
    again = layer(x, scale, shift, gate, x_out=x, **kw)
    assert again[0] is x and torch.equal(x, xn) and torch.equal(again[1], h)
    sa.linear_status(x.device)


@pytest.mark.gpu
def test_refusals():
    x, w, _ = make(1, 20, 2, 64, BF16)
    with pytest.raises(ValueError, match="w_qkv must be"):
        sa.AttentionLayer(w["w_qkv"], w["w_qkv"], 2)
    with pytest.raises(ValueError, match="64 or 128"):
        sa.AttentionLayer(w["w_qkv"], w["w_out"], 4)
    layer = sa.AttentionLayer(w["w_qkv"], w["w_out"], 2)
    with pytest.raises(ValueError, match="x must be"):
        layer(x[..., :64], beta=1.0, chunk=4, grid=(1, 4, 5))
    with pytest.raises(ValueError, match="unsupported type"):
        layer(x.half(), beta=1.0, chunk=4, grid=(1, 4, 5))
    with pytest.raises(ValueError, match="grid or positions"):
        layer(x, beta=1.0, chunk=4)


def test_packed_arguments_are_the_structs():
    """The bindings pack their arguments in one go; the bytes are the header's structs, field by field."""
    import ctypes

    import layer_structs as st
    from block_sparse_attention_moments_b200 import layer

    def flat(cls, prefix=""):
        for name, kind in cls._fields_:
            if issubclass(kind, ctypes.Structure):
                yield from flat(kind, f"{prefix}{name}.")
            else:
                yield f"{prefix}{name}", kind

    for packer, cls in ((layer._NORM_ARGS, st.NormArgs), (layer._ROPE_ARGS, st.RopeArgs), (layer._LINEAR_ARGS, st.LinearArgs)):
        fields = list(flat(cls))
        assert packer.size == ctypes.sizeof(cls)
        got = cls.from_buffer_copy(packer.pack(*range(1, len(fields) + 1)))
        for value, (name, _) in enumerate(fields, 1):
            x = got
            for part in name.split("."):
                x = getattr(x, part)
            assert x == value, name


FIRST_CALLS = """
import torch
import block_sparse_attention_moments_b200 as sa
x = torch.randn(2, 300, 512, device="cuda", dtype=torch.bfloat16)
wide = torch.randn(1, 5000, 1024, device="cuda", dtype=torch.bfloat16)
w = torch.randint(-127, 128, (1536, 512), device="cuda", dtype=torch.int8)
ws = torch.rand(1536, device="cuda")
static = [torch.zeros(n, 512, device="cuda", dtype=torch.int8) for n in (2, 40)]
scales = [torch.ones(n, device="cuda") for n in (2, 40)]
def calls():
    q, s = sa.norm_modulate(x, quantize=True)
    qkv = sa.int8_linear(q, s, w, ws).view(2, 300, 3, 4, 128)
    return (*sa.rope(*qkv.unbind(2), grid=(3, 10, 10), norm="token"), *sa.gate_residual_norm(wide, wide),
            *(sa.int8_linear(a, s, w, ws) for a, s in zip(static, scales)))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
sa.linear_status("cuda")
print("the first calls were captured")
"""


@pytest.mark.gpu
def test_first_calls_may_be_captured():
    """In a process of its own: no operator needs a call before the capture."""
    import os
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "were captured" in r.stdout, r.stdout + r.stderr


# ------------------------------------------------------------------ streams and devices by keyword
class OnDevice(torch.Tensor):
    """A CPU tensor that says that it lies on the second GPU."""
    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1

    def record_stream(self, stream):
        stream.recorded.append(self)


@pytest.mark.parametrize("order", [("t", "grid"), ("grid", "t"), ("none", "other", "t"), ("stream", "grid", "other", "t")])
@pytest.mark.parametrize("positional", [False, True])
def test_the_named_tensor_decides_where_a_call_runs(monkeypatch, order, positional):
    """Without a GPU: whatever comes first among the keywords, the stream and the device are those of the operator's
    first parameter, and a call without it runs nowhere."""
    import contextlib

    from block_sparse_attention_moments_b200 import layer
    current = []

    @contextlib.contextmanager
    def entered(x):
        current.append(x)
        yield
        current.pop()

    class Stream:
        device, recorded = OnDevice.device, []

    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "device", entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(layer, "_current_device", lambda: 0)
    seen = []

    @layer._placed
    def operator(t, other=None, *, grid=None, none=None):
        seen.append(list(current))
        return t

    t = torch.zeros(4).as_subclass(OnDevice)
    kw = {"t": t, "other": torch.zeros(2), "grid": (1, 2, 3), "none": None}
    stream = Stream()
    kw = {name: stream if name == "stream" else kw[name] for name in order}
    args = (kw.pop("t"),) if positional else ()
    kw.pop("stream", None)
    assert operator(*args, **kw) is t and seen.pop() == [OnDevice.device]
    assert operator(*args, **kw, stream=stream) is t and seen.pop() == [stream]
    assert any(r is t for r in stream.recorded)
    Stream.device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="stream is on"):
        operator(*args, **kw, stream=stream)
    with pytest.raises(TypeError):
        operator(grid=(1, 2, 3), stream=stream)
    assert not seen and not current


def test_a_stream_is_not_dropped_without_a_tensor():
    for call in (lambda: sa.norm_modulate(norm="rms", x=torch.zeros(2, 8), stream=object()),
                 lambda: sa.rope(grid=(1, 1, 1), q=torch.zeros(1, 1, 1, 16), k=None, stream=object()),
                 lambda: sa.quantize_rows(stream=object(), x=torch.zeros(2, 8))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_keywords_only_on_a_side_stream(monkeypatch):
    """Every operator called with keywords only, one that is no tensor first: the library gets the given stream."""
    from block_sparse_attention_moments_b200 import layer
    streams, handle = [], layer._raw_stream
    monkeypatch.setattr(layer, "_raw_stream", lambda device: streams.append(handle(device)) or streams[-1])
    x = torch.randn(1, 40, 128, device="cuda").to(BF16)
    q = x.view(1, 40, 2, 64)
    w, ws = sa.quantize_rows(x[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls = {"norm_modulate": (sa.norm_modulate, dict(norm="rms", scale=None, x=x)),
             "gate_residual": (sa.gate_residual, dict(residual_scale=0.5, gate=None, y=x, x=x)),
             "gate_residual_norm": (sa.gate_residual_norm, dict(norm="rms", gate=None, y=x, x=x)),
             "quantize_rows": (sa.quantize_rows, dict(x=x)),
             "rope": (sa.rope, dict(grid=(2, 4, 5), norm="head", v=None, k=q, q=q)),
             "int8_linear": (sa.int8_linear, dict(out_dtype=BF16, w_scale=ws, w=w, a_scale=ws, a=w))}
    for name, (fn, kw) in calls.items():
        streams.clear()
        got = fn(**kw, stream=side)
        assert streams == [side.cuda_stream], name
        torch.cuda.synchronize()
        want = fn(**kw)
        assert streams[1:] == [torch.cuda.current_stream().cuda_stream], name
        for a, b in zip(*(t if isinstance(t, tuple) else (t,) for t in (got, want))):
            assert torch.equal(a, b), name


@pytest.mark.gpu
def test_a_captured_layer_outlives_a_larger_call():
    """A captured layer is replayed after a forward that needs a larger workspace, and after smaller ones."""
    B, L, H, d, grid = 1, 700, 2, 128, (7, 10, 10)
    x, w, vectors = make(B, L, H, d, BF16, 2)
    shift, scale, gate, next_shift, next_scale = vectors
    layer = sa.AttentionLayer(w["w_qkv"], w["w_out"], H, b_qkv=w["b_qkv"], b_out=w["b_out"])
    kw = dict(beta=0.5, chunk=8, grid=grid, next_scale=next_scale, next_shift=next_shift)
    torch.cuda.synchronize()
    sa.release()
    want = layer(x, scale, shift, gate, **kw)        # the workspace is this shape's
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x, scale, shift, gate, **kw)
    for shape in ((1, 8, 5000, 128), (1, 1, 70, 64), (2, 8, 9000, 128)):
        q, k, v = (torch.randn(shape, device="cuda").to(BF16) for _ in range(3))
        first = sa.forward(q, k, v, 0.5, 8)
        for t in got:
            t.zero_()
        graph.replay()
        assert torch.equal(sa.forward(q, k, v, 0.5, 8), first)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    del graph
    sa.release()


def no_room():
    """A workspace of terabytes: the allocator refuses it before anything is read or enqueued."""
    B, H, L, d = 1, 65535, 2 ** 20, 128
    assert sa.workspace_bytes(B, H, L, d) > 2 ** 40
    far = [2 ** 40 + i * 2 * B * H * L * d for i in range(3)]
    with pytest.raises(sa.SolAttnError) as e:
        sa._check(sa.lib().sol_attn_stage_pool(*far, B, H, L, d, 64, None, torch.cuda.current_stream().cuda_stream))
    assert e.value.code == -4 and "memory" in str(e.value)


@pytest.mark.gpu
def test_a_failed_call_does_not_fail_the_next():
    x = torch.randn(3, 64, device="cuda")
    want = sa.norm_modulate(x)
    torch.cuda.synchronize()
    sa.release()
    no_room()
    assert torch.equal(sa.norm_modulate(x), want)
    no_room()
    x.add_(1)
    torch.cuda.synchronize()
    sa.release()


@pytest.mark.gpu
def test_a_shape_that_finds_no_room_leaves_no_views():
    """The shape before it then gets a block, and views, of its own."""
    q, k, v = (torch.randn(1, 2, 300, 64, device="cuda").to(BF16) for _ in range(3))
    torch.cuda.synchronize()
    sa.release()
    want = sa.forward(q, k, v, 0.5, 8)
    no_room()
    with pytest.raises(sa.SolAttnError) as e:
        sa.stats(1, 2, 300)
    assert e.value.code == -6
    assert torch.equal(sa.forward(q, k, v, 0.5, 8), want)
    torch.cuda.synchronize()
    sa.release()


@pytest.mark.gpu
@pytest.mark.parametrize("B,L", [(1, 0), (0, 5), (0, 0)])
def test_layer_without_tokens(B, L):
    x, w, _ = make(1, 1, 2, 64, FP32)
    layer = sa.AttentionLayer(w["w_qkv"], w["w_out"], 2)
    xn, h = layer(torch.empty(B, L, 128, device="cuda"), beta=1.0, chunk=4, grid=(1, 1, 1))
    assert xn.shape == h.shape == (B, L, 128) and xn.dtype == FP32 and h.dtype == BF16


@pytest.mark.gpu
def test_host_threads_on_streams_of_their_own():
    """The operators called by several threads at once, each on its stream: the bits of one thread's calls."""
    import threading

    def calls(x, w, ws):
        a, s = sa.norm_modulate(x, quantize=True)
        y = sa.int8_linear(a, s, w, ws)
        q, k = sa.rope(y.view(2, -1, 3, 2, 64)[:, :, 0], y.view(2, -1, 3, 2, 64)[:, :, 1], grid=(2, 5, 30), norm="token")
        return (y, q, k, *sa.gate_residual_norm(y, y, quantize=True))

    inputs = []
    for i, L in enumerate((1, 60, 300, 1000)):
        g = torch.Generator(device="cuda").manual_seed(i)
        rnd = lambda *shape: torch.empty(shape, device="cuda").normal_(generator=g)
        inputs.append((rnd(2, L, 128).to(BF16), *sa.quantize_rows(rnd(384, 128))))
    want = [calls(*t) for t in inputs]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = calls(*inputs[i])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    sa.linear_status("cuda")
