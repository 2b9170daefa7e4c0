"""The operators around the sparse attention of a diffusion-transformer layer: cases, plain forms and calls.

Four groups, in the order in which a layer runs them:
  norm        layer or RMS norm of the residual stream, modulated by a scale and a shift;
  rope        q, k and v of one projection: query/key RMS norm, rotary positions with several axes, and the
              [B, H, L, d] layout that the attention reads;
  linear      product of 8-bit integers with a scale for each token and each output channel, alone
              ("linear"), behind the norm that quantises its rows ("normlinear") and behind the attention,
              whose head-major output is quantised token by token ("attnlinear");
  gate        the block's output, normed or not, gated and added to the residual stream, with the norm and
              modulation of the next block in the same pass.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _norm(name, B, L, C, G, x, p, h, kind, affine, mod):
    return {"name": name, "op": "norm", "B": B, "L": L, "C": C, "G": G, "x": x, "p": p, "h": h, "kind": kind,
            "affine": affine, "mod": mod}


def _gate(name, B, L, C, G, x, y, p, h, kind, affine, mod, gate, post, rscale):
    return {"name": name, "op": "gate", "B": B, "L": L, "C": C, "G": G, "x": x, "y": y, "p": p, "h": h,
            "kind": kind, "affine": affine, "mod": mod, "gate": gate, "post": post, "rscale": rscale}


def _rope(name, B, L, H, d, grid, start, dt, pairing, norm, v):
    """grid: "FxHxW", or "" for explicit positions of every token."""
    return {"name": name, "op": "rope", "B": B, "L": L, "H": H, "d": d, "grid": grid, "start": start, "x": dt,
            "pairing": pairing, "norm": norm, "v": v}


def listed():
    return [
        # the last norm of a step that works on one token, fp32 modulation: latency
        _norm("norm one token", 1, 1, 5120, 1, "bf16", "fp32", "bf16", "layer", False, True),
        # the norm before attention at the Wan-like length: 21 x 45 x 80 tokens of 40 heads of 128
        _norm("norm video", 1, 75600, 5120, 1, "bf16", "fp32", "bf16", "layer", False, True),
        # a modulation of its own for each of 13 frames of 391 tokens, batch of 2 (guidance), RMS norm
        _norm("norm frames", 2, 13 * 391, 1544, 13, "fp16", "fp16", "fp16", "rms", True, True),
        # between two blocks, residual stream in fp32, Wan-like length
        _gate("gate video", 1, 75600, 5120, 1, "fp32", "bf16", "fp32", "bf16", "layer", False, True, True, "none", 1.0),
        # sandwich norm with an odd width, so that no row but the first is aligned
        _gate("gate odd width", 2, 1031, 1285, 1, "bf16", "bf16", "bf16", "bf16", "rms", True, True, True, "rms", 0.5),
        # a single frame's pooled token: latency
        _rope("rope one token", 1, 1, 40, 128, "21x45x80", 3600, "bf16", "interleaved", "token", True),
        # the Wan-like projection: query/key norm over the whole width, three axes
        _rope("rope video", 1, 75600, 40, 128, "21x45x80", 0, "bf16", "interleaved", "token", True),
        # image and text tokens in one sequence, positions given for each token, per-head norm, halves paired
        _rope("rope positions", 2, 4096 + 77, 16, 64, "", 0, "fp16", "half", "head", True),
        # the modulation's own projection of two guidance branches: six vectors of 5120
        {"name": "linear two rows", "op": "linear", "M": 2, "N": 6 * 5120, "K": 5120, "bias": True, "h": "fp32"},
        # q, k and v of the Wan-like length
        {"name": "linear video", "op": "linear", "M": 75600, "N": 3 * 5120, "K": 5120, "bias": True, "h": "bf16"},
        # a small latent with an odd number of tokens and odd widths, from the norm to the projection
        {"name": "normlinear ragged", "op": "normlinear", "B": 2, "L": 517, "C": 1000, "N": 1543, "x": "bf16",
         "kind": "layer", "bias": True, "h": "bf16"},
        # the output projection behind 8 heads over 16384 tokens
        {"name": "attnlinear image", "op": "attnlinear", "B": 1, "L": 16384, "H": 8, "d": 128, "N": 1024,
         "x": "bf16", "bias": True, "h": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gate", "rope", "linear", "normlinear", "attnlinear"])
    x = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    B = rng.choice([1, 1, 2, 3])
    if op in ("norm", "gate"):
        C = _log(rng, 64, 8192)
        C = C if rng.random() < 0.3 else (C + 7) // 8 * 8
        per = _log(rng, 1, max(1, 200_000_000 // C // B // 16))     # tokens of a modulation group
        G = rng.choice([1, 1, rng.randint(2, 16)])
        h = x if x != "fp32" else rng.choice(["fp32", "bf16", "fp16"])
        p = rng.choice([h, "fp32"])
        kind, affine, mod = rng.choice(["layer", "rms"]), rng.random() < 0.5, rng.random() < 0.8
        c = _norm("", B, per * G, C, G, x, p, h, kind, affine, mod)
        if op == "gate":
            c = _gate("", B, per * G, C, G, x, h, p, h, kind, affine, mod, rng.random() < 0.8,
                      rng.choice(["none", "layer", "rms"]), rng.choice([1.0, 0.5, 0.70710678]))
    elif op == "rope":
        d, H = rng.choice([32, 64, 96, 128]), rng.randint(1, 40)
        f, h, w = rng.randint(1, 24), rng.randint(1, 48), rng.randint(1, 80)
        L = f * h * w + rng.choice([0, 0, rng.randint(1, 300)])
        L = min(L, max(1, 300_000_000 // (B * H * d * 3)))
        c = _rope("", B, L, H, d, rng.choice(["", "%dx%dx%d" % (f, h, w)]), rng.choice([0, 0, rng.randint(1, 5000)]), x,
                  rng.choice(["interleaved", "half"]), rng.choice(["none", "head", "token"]), rng.random() < 0.7)
    elif op == "linear":
        c = {"name": "", "op": op, "M": _log(rng, 1, 30000), "N": _log(rng, 16, 16384), "K": _log(rng, 16, 14336),
             "bias": rng.random() < 0.5, "h": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    elif op == "normlinear":
        c = {"name": "", "op": op, "B": B, "L": _log(rng, 1, 10000), "C": _log(rng, 64, 6144), "N": _log(rng, 16, 8192),
             "x": x, "kind": rng.choice(["layer", "rms"]), "bias": rng.random() < 0.5, "h": "bf16" if x == "fp32" else x}
    else:
        c = {"name": "", "op": op, "B": B, "L": _log(rng, 1, 10000), "H": rng.randint(1, 40), "d": rng.choice([64, 128]),
             "N": _log(rng, 16, 8192), "x": "bf16", "bias": rng.random() < 0.5, "h": "bf16"}
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _axes(d):
    """Channels of the time, height and width axes of a head: two thirds split evenly between height and
    width, an even number each, and the rest for the time."""
    hw = 2 * (d // 6)
    return (d - 2 * hw, hw, hw)


def _grid(c):
    return tuple(int(n) for n in c["grid"].split("x")) if c["grid"] else None


class _Make:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, shape, dtype, mean=0.0, std=1.0):
        t = torch.empty(shape, device="cuda", dtype=dtype)
        return t.normal_(mean, std, generator=self.g)

    def int8(self, rows, K):
        """Quantised rows: bell-shaped values that reach 127, in rows that start at multiples of 16 bytes."""
        t = torch.zeros(rows, (K + 15) // 16 * 16, device="cuda", dtype=torch.int8)
        for i in range(0, rows, 16384):
            part = t[i:i + 16384]
            part.copy_(torch.empty(part.shape, device="cuda").normal_(0, 32, generator=self.g).round_().clamp_(-127, 127))
        t[:, K:] = 0
        return t[:, :K]

    def scales(self, n, mean):
        return torch.empty(n, device="cuda").uniform_(0.5 * mean, 1.5 * mean, generator=self.g)


def _norm_inputs(m, c, s):
    B, L, C, G, p = c["B"], c["L"], c["C"], c["G"], DTYPES[c["p"]]
    # a residual stream has channels of quite different sizes, and a mean
    x = m.normal((B, L, C), DTYPES[c["x"]])
    x *= m.normal((C,), torch.float32, 0.0, 0.6).exp_().to(x.dtype)
    x += 0.25
    s["x"] = x
    s["scale"] = s["shift"] = s["weight"] = s["bias"] = None
    if c["mod"]:
        six = m.normal((B, G, 6, C), p, 0.0, 0.3)     # the six vectors of a block: shift, scale and gate, twice
        s["shift"], s["scale"], s["gate"] = six[:, :, 0], six[:, :, 1], six[:, :, 2]
    else:
        s["gate"] = m.normal((B, G, C), p, 0.0, 0.3)
    if c["affine"]:
        s["weight"] = m.normal((C,), p, 1.0, 0.1)
        s["bias"] = m.normal((C,), p, 0.0, 0.1) if c["kind"] == "layer" else None


def prepare(case, seed):
    c, m, s = case, _Make(seed), {"c": case}
    if c["op"] in ("norm", "gate"):
        _norm_inputs(m, c, s)
        if c["op"] == "gate":
            s["y"] = m.normal(tuple(s["x"].shape), DTYPES[c["y"]], 0.1, 0.7)
            s["post_weight"] = m.normal((c["C"],), DTYPES[c["p"]], 1.0, 0.1) if c["post"] != "none" else None
            s["gate"] = s["gate"] if c["gate"] else None
    elif c["op"] == "rope":
        B, L, H, d, t = c["B"], c["L"], c["H"], c["d"], DTYPES[c["x"]]
        qkv = m.normal((B, L, 3, H, d), t)            # one projection's output
        s["q"], s["k"], s["v"] = qkv[:, :, 0], qkv[:, :, 1], (qkv[:, :, 2] if c["v"] else None)
        n = {"none": 0, "head": d, "token": H * d}[c["norm"]]
        s["q_weight"] = m.normal((n,), t, 1.0, 0.2) if n else None
        s["k_weight"] = m.normal((n,), t, 1.0, 0.2) if n else None
        s["positions"] = None
        if not c["grid"]:
            s["positions"] = torch.randint(0, 20000, (B, L, 3), device="cuda", dtype=torch.int32, generator=m.g)
            s["positions"][:, L - L // 50:] = 0       # text tokens
    else:
        M = c["M"] if c["op"] == "linear" else c["B"] * c["L"]
        K = {"linear": c.get("K"), "normlinear": c.get("C"), "attnlinear": c.get("H", 0) * c.get("d", 0)}[c["op"]]
        s["w"], s["w_scale"] = m.int8(c["N"], K), m.scales(c["N"], 1.0 / (32 * math.sqrt(K)))
        s["b"] = m.normal((c["N"],), torch.float32) if c["bias"] else None
        if c["op"] == "linear":
            s["a"], s["a_scale"] = m.int8(M, K), m.scales(M, 1.0 / 32)
        elif c["op"] == "normlinear":
            _norm_inputs(m, {**c, "G": 1, "p": c["h"], "affine": False, "mod": True}, s)
        else:
            s["o"] = m.normal((c["B"], c["H"], c["L"], c["d"]), DTYPES[c["x"]])
    return s


# ------------------------------------------------------------------ plain forms, in 32 bits
def _normed(x, kind, weight, bias):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    x = x if weight is None else x * weight.float()
    return x if bias is None else x + bias.float()


def _per_token(t, L):
    """[B, G, C] -> [B, L, C] (or [B, 1, C]) in 32 bits."""
    t = t.float()
    return t if t.shape[1] == 1 else t.repeat_interleave(L // t.shape[1], dim=1)


def _modulated(x, kind, weight, bias, scale, shift):
    h = _normed(x, kind, weight, bias)
    L = x.shape[1]
    return h if scale is None else h * (1 + _per_token(scale, L)) + _per_token(shift, L)


def _quantised(h):
    """Rows in 8 bits: the values as whole numbers in 32-bit floats, and each row's scale."""
    scale = h.abs().amax(-1) / 127
    return torch.round(h / scale.clamp_min(1e-38)[..., None]), scale


def _product(a, a_scale, w, w_scale, b):
    y = a.reshape(-1, a.shape[-1]).float() @ w.float().t()
    y = y * a_scale.reshape(-1, 1) * w_scale
    return y if b is None else y + b


def _angles(c, s):
    """[B or 1, L, d / 2] in 64 bits: position along the pair's axis, times the pair's frequency."""
    axes, dev = _axes(c["d"]), s["q"].device
    j = torch.cat([torch.arange(n // 2, device=dev, dtype=torch.float64) / (n / 2) for n in axes])
    axis = torch.cat([torch.full((n // 2,), i, device=dev) for i, n in enumerate(axes)])
    if s["positions"] is None:
        f, h, w = _grid(c)
        i = c["start"] + torch.arange(c["L"], device=dev)
        pos = torch.stack([i // (h * w), i // w % h, i % w], -1) * (i < f * h * w)[:, None]
        pos = pos[None]
    else:
        pos = s["positions"]
    return pos.double()[..., axis] * torch.pow(torch.tensor(10000.0, device=dev, dtype=torch.float64), -j)


def _rotated(x, weight, cos, sin, c):
    x = x.float()
    if c["norm"] == "head":
        x = _normed(x, "rms", weight, None)
    elif c["norm"] == "token":
        x = _normed(x.flatten(2), "rms", weight, None).view_as(x)
    cos, sin = cos[:, :, None], sin[:, :, None]
    if c["pairing"] == "half":
        a, b = x.chunk(2, -1)
        x = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return x.transpose(1, 2)


def _plain(s):
    c, op = s["c"], s["c"]["op"]
    out = DTYPES[c["h"]] if "h" in c else None
    if op == "norm":
        return _modulated(s["x"].float(), c["kind"], s["weight"], s["bias"], s["scale"], s["shift"]).to(out)
    if op == "gate":
        y = s["y"].float()
        y = y if c["post"] == "none" else _normed(y, c["post"], s["post_weight"], None)
        y = y if s["gate"] is None else y * _per_token(s["gate"], c["L"])
        x = c["rscale"] * s["x"].float() + y
        h = _modulated(x, c["kind"], s["weight"], s["bias"], s["scale"], s["shift"])
        return x.to(s["x"].dtype), h.to(out)
    if op == "rope":
        angle = _angles(c, s)
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        t = s["q"].dtype
        q = _rotated(s["q"], s["q_weight"], cos, sin, c).to(t).contiguous()
        k = _rotated(s["k"], s["k_weight"], cos, sin, c).to(t).contiguous()
        return (q, k) if s["v"] is None else (q, k, s["v"].transpose(1, 2).contiguous())
    if op == "linear":
        return _product(s["a"], s["a_scale"], s["w"], s["w_scale"], s["b"]).to(out)
    if op == "normlinear":
        h = _modulated(s["x"].float(), c["kind"], None, None, s["scale"], s["shift"])
    else:
        h = s["o"].float().transpose(1, 2).flatten(2)
    a, a_scale = _quantised(h)
    return _product(a, a_scale, s["w"], s["w_scale"], s["b"]).to(out).view(c["B"], c["L"], -1)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import block_sparse_attention_moments_b200 as sa
    c, op = s["c"], s["c"]["op"]
    out = DTYPES[c["h"]] if "h" in c else None
    if op == "norm":
        return sa.norm_modulate(s["x"], s["scale"], s["shift"], norm=c["kind"], weight=s["weight"], bias=s["bias"],
                                eps=EPS, out_dtype=out)
    if op == "gate":
        return sa.gate_residual_norm(s["x"], s["y"], s["gate"], s["scale"], s["shift"], residual_scale=c["rscale"],
                                     post_norm=c["post"], post_weight=s["post_weight"], post_eps=EPS, norm=c["kind"],
                                     weight=s["weight"], bias=s["bias"], eps=EPS, out_dtype=out)
    if op == "rope":
        return sa.rope(s["q"], s["k"], s["v"], grid=_grid(c), axes=_axes(c["d"]), positions=s["positions"],
                       start=c["start"] if c["grid"] else 0, theta=10000.0, pairing=c["pairing"], norm=c["norm"],
                       q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    if op == "linear":
        return sa.int8_linear(s["a"], s["a_scale"], s["w"], s["w_scale"], s["b"], out_dtype=out)
    if op == "normlinear":
        a, a_scale = sa.norm_modulate(s["x"], s["scale"], s["shift"], norm=c["kind"], eps=EPS, quantize=True)
    else:
        a, a_scale = sa.quantize_rows(s["o"].transpose(1, 2))
    return sa.int8_linear(a, a_scale, s["w"], s["w_scale"], s["b"], out_dtype=out)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    if op in ("norm", "gate"):
        n, per = c["B"] * c["L"] * c["C"], SIZE[c["p"]] * c["B"] * c["G"] * c["C"]
        vectors = (2 * per if c["mod"] else 0) + (SIZE[c["p"]] * c["C"] * 2 if c["affine"] else 0)
        if op == "norm":
            return {"bytes": n * (SIZE[c["x"]] + SIZE[c["h"]]) + vectors, "flops": 8 * n}
        vectors += per if c["gate"] else 0
        return {"bytes": n * (2 * SIZE[c["x"]] + SIZE[c["y"]] + SIZE[c["h"]]) + vectors, "flops": 12 * n}
    if op == "rope":
        n, m = c["B"] * c["L"] * c["H"] * c["d"], 3 if c["v"] else 2
        return {"bytes": 2 * m * n * SIZE[c["x"]] + (0 if c["grid"] else 12 * c["B"] * c["L"]), "flops": 2 * n * 6}
    M = c["M"] if op == "linear" else c["B"] * c["L"]
    K = {"linear": c.get("K"), "normlinear": c.get("C"), "attnlinear": c.get("H", 0) * c.get("d", 0)}[op]
    a = M * K + 4 * M if op == "linear" else M * K * SIZE[c["x"]]
    return {"bytes": a + c["N"] * (K + 4) + M * c["N"] * SIZE[c["h"]], "flops": 2 * M * c["N"] * K}


# ------------------------------------------------------------------ 64 bits
def _norm64(x, kind, weight, bias):
    var, mean = torch.var_mean(x, dim=-1, unbiased=False, keepdim=True)
    n = (x - mean) / torch.sqrt(var + EPS) if kind == "layer" else x / torch.sqrt(var + mean ** 2 + EPS)
    n = n * (1 if weight is None else weight.double())
    return n + (0 if bias is None else bias.double())


def _mod64(h, scale, shift):
    if scale is None:
        return h
    B, L, C = h.shape
    G = scale.shape[1]
    h = h.view(B, G, L // G, C)
    return (h + h * scale.double()[:, :, None] + shift.double()[:, :, None]).view(B, L, C)


def exact(case, seed):
    """What run() returns, in 64 bits: norms through the library's variance, rotations as products of complex
    numbers, products in doubles."""
    c, op, s = case, case["op"], prepare(case, seed)
    if op == "norm":
        return _mod64(_norm64(s["x"].double(), c["kind"], s["weight"], s["bias"]), s["scale"], s["shift"])
    if op == "gate":
        y = s["y"].double()
        if c["post"] != "none":
            y = _norm64(y, c["post"], s["post_weight"], None)
        if s["gate"] is not None:
            B, L, C = y.shape
            y = (y.view(B, c["G"], -1, C) * s["gate"].double()[:, :, None]).view(B, L, C)
        x = s["x"].double() * c["rscale"] + y
        return x, _mod64(_norm64(x, c["kind"], s["weight"], s["bias"]), s["scale"], s["shift"])
    if op == "rope":
        B, L, H, d = s["q"].shape
        if s["positions"] is None:
            f, h, w = _grid(c)
            every = torch.cartesian_prod(*(torch.arange(n, dtype=torch.float64) for n in (f, h, w))).view(-1, 3)
            pos = torch.zeros(L, 3, dtype=torch.float64)
            there = max(0, min(L, f * h * w - c["start"]))
            pos[:there] = every[c["start"]:c["start"] + there]
            pos = pos[None].cuda()
        else:
            pos = s["positions"].double()
        parts = []
        for i, n in enumerate(_axes(d)):
            freq = torch.tensor([math.pow(10000.0, -2.0 * j / n) for j in range(n // 2)], dtype=torch.float64, device="cuda")
            parts.append(pos[..., i, None] * freq)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.cat(parts, -1))[:, None]
        out = []
        for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.double()
            if c["norm"] == "head":
                x = _norm64(x, "rms", weight, None)
            if c["norm"] == "token":
                x = _norm64(x.reshape(B, L, H * d), "rms", weight, None).view(B, L, H, d)
            x = x.transpose(1, 2)
            if c["pairing"] == "half":
                z = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous()) * turn
                out.append(torch.cat([z.real, z.imag], -1))
            else:
                z = torch.view_as_complex(x.reshape(B, H, L, d // 2, 2).contiguous()) * turn
                out.append(torch.view_as_real(z).reshape(B, H, L, d))
        return tuple(out) if s["v"] is None else (*out, s["v"].double().transpose(1, 2).contiguous())
    if op == "linear":
        a, a_scale = s["a"].double(), s["a_scale"].double()
    else:
        if op == "normlinear":
            h = _mod64(_norm64(s["x"].double(), c["kind"], None, None), s["scale"], s["shift"])
        else:
            h = s["o"].double().permute(0, 2, 1, 3).reshape(c["B"], c["L"], -1)
        h = h.reshape(-1, h.shape[-1])
        a_scale = torch.linalg.vector_norm(h, ord=math.inf, dim=-1) / 127
        a = (h / torch.where(a_scale > 0, a_scale, 1.0)[:, None]).round()
    y = torch.mm(a, s["w"].double().t()).mul_(a_scale[:, None]).mul_(s["w_scale"].double())
    y = y if s["b"] is None else y.add_(s["b"].double())
    return y if op == "linear" else y.view(c["B"], c["L"], -1)
