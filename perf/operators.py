"""Cases of the 8-bit linear layers (quantisation, forward, backward) and of the
norms around a block (norm after * gate + scaled residual, norm before of the
next block), with their plain forms.

Layouts (as the library documents them): tokens T by features C row-major;
``rows`` groups are 128 features of one token, their scales [ceil(C/128), T];
``cols`` groups are 128 tokens of one feature, their scales [ceil(T/128), C];
a weight shard [in, out] has a scale per 128 x 128 block.  A scale is the
smallest power of two (at least 2^-119) that brings the group's largest
magnitude within the format; a group that holds an infinity or a NaN has the
scale NaN and zeros.
"""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
#: the largest exponent step of each format: its largest value is 0.875 * 2^TOP
TOP = {"e4m3": 9, "e5m2": 16}
DTYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
EPS = 1e-5


# ---- the cases ------------------------------------------------------------------------

def listed():
    return [
        # one token through the QKV projection of the 4096-wide layer: latency, the weight's bytes
        {"name": "linear decode 1 token", "op": "linear", "split": "column", "tokens": 1, "fin": 4096,
         "fout": 12288, "t": 1, "chunks": 1},
        # a decode batch through the 175B-class output projection, eight row shards
        {"name": "linear decode 48 tokens", "op": "linear", "split": "row", "tokens": 48, "fin": 12288,
         "fout": 12288, "t": 8, "chunks": 1},
        # a ragged prefill: no size a multiple of the tiles
        {"name": "linear ragged 777 tokens", "op": "linear", "split": "column", "tokens": 777,
         "fin": 2064, "fout": 8240, "t": 1, "chunks": 1},
        # the QKV projection of the 175B-class layer, eight column shards
        {"name": "linear 175B QKV", "op": "linear", "split": "column", "tokens": 2048, "fin": 12288,
         "fout": 36864, "t": 8, "chunks": 1},
        # training, backward: the output projection of the 4096-wide layer, token chunks
        {"name": "backward 16384 x 4096", "op": "linear_backward", "split": "row", "tokens": 16384,
         "fin": 4096, "fout": 4096, "t": 8, "chunks": 8, "dy": "e5m2"},
        # training, backward: a small layer with a ragged batch
        {"name": "backward ragged 333 tokens", "op": "linear_backward", "split": "column",
         "tokens": 333, "fin": 1040, "fout": 2064, "t": 1, "chunks": 1, "dy": "e4m3"},
        # training: the activations of the 4096-wide layer, both groupings in one pass
        {"name": "quantize 16384 x 4096", "op": "quantize", "tokens": 16384, "fin": 4096, "chunks": 8,
         "rows": True, "cols": True, "fmt": "e4m3"},
        # serving: a weight shard laid out once (after a weight update, every step)
        {"name": "quantize weight 12288 x 4608", "op": "weight", "fin": 12288, "fout": 4608,
         "fmt": "e4m3"},
        # one token's norm after, gate, residual and next norm, ready for the 8-bit product
        {"name": "norm decode 1 token", "op": "norm", "tokens": 1, "hidden": 12288, "post": "rms",
         "pre": "rms", "gate_rows": 1, "alpha": 0.5, "quantize": True},
        # training: eight sequences of 2048 tokens with a gate row each
        {"name": "norm 16384 x 4096", "op": "norm", "tokens": 16384, "hidden": 4096, "post": "rms",
         "pre": "rms", "gate_rows": 2048, "alpha": 1.0, "quantize": True},
        # training, backward, of the same
        {"name": "norm backward 16384 x 4096", "op": "norm_backward", "tokens": 16384, "hidden": 4096,
         "post": "rms", "pre": "rms", "gate_rows": 2048, "alpha": 1.0},
        # LayerNorm on both sides, wide rows, a ragged batch of seven sequences
        {"name": "norm backward 7 x 131 x 9000", "op": "norm_backward", "tokens": 917,
         "hidden": 9000, "post": "layer", "pre": "layer", "gate_rows": 131, "alpha": 0.7},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "quantize", "weight", "norm",
                     "norm_backward"])
    if op in ("linear", "linear_backward"):
        limit = 2048 * 12288 * 36864 if op == "linear" else 16384 * 4096 * 4096
        while True:
            t = rng.choice([1, 1, 2, 8])
            split = rng.choice(["column", "row"])
            shard, other = 16 * _log(rng, 16, 1536 // t), 16 * _log(rng, 16, 768)
            fin, fout = (other, shard * t) if split == "column" else (shard * t, other)
            tokens, chunks = _log(rng, 1, 16384), 1
            if tokens >= 1024 and rng.random() < 0.5:
                chunks = rng.choice([2, 4, 8])
                tokens -= tokens % (128 * chunks)
            if tokens * fin * fout <= limit:
                break
        case = {"op": op, "split": split, "tokens": tokens, "fin": fin, "fout": fout, "t": t,
                "chunks": chunks}
        if op == "linear_backward":
            case["dy"] = rng.choice(["e4m3", "e5m2"])
        return case
    if op == "quantize":
        tokens, fin = _log(rng, 1, 16384), 16 * _log(rng, 16, 256)
        rows = rng.random() < 0.8
        return {"op": op, "tokens": tokens, "fin": fin, "chunks": 1, "rows": rows,
                "cols": not rows or rng.random() < 0.6, "fmt": rng.choice(["e4m3", "e5m2"])}
    if op == "weight":
        return {"op": op, "fin": 16 * _log(rng, 16, 768), "fout": 16 * _log(rng, 16, 288),
                "fmt": rng.choice(["e4m3", "e5m2"])}
    hidden = 8 * _log(rng, 32, 2048)
    tokens = _log(rng, 1, max(1, min(16384, 16384 * 4096 // hidden)))
    per = _log(rng, 1, tokens)
    gate = rng.choice(["none", "one", "sequences", "sequences"])
    if gate == "sequences":
        tokens = max(1, tokens // per) * per
    case = {"op": op, "tokens": tokens, "hidden": hidden,
            "post": rng.choice(["rms", "rms", "layer", "none"]), "pre": rng.choice(["rms", "layer"]),
            "gate_rows": {"none": 0, "one": tokens, "sequences": per}[gate],
            "alpha": rng.choice([1.0, 0.5, 0.83])}
    if op == "norm":
        case["quantize"] = hidden % 16 == 0 and rng.random() < 0.5
    return case


# ---- inputs ---------------------------------------------------------------------------

def _randn(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 11)
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        # activations: a few features much larger than the rest, as trained layers have them
        X = _randn(gen, case["tokens"], case["fin"])
        X[:, ::97] *= 16.0
        s["X"] = X.chunk(case["chunks"])
        return s
    if op == "weight":
        s["W"] = _randn(gen, case["fin"], case["fout"], std=0.02)
        return s
    if op in ("linear", "linear_backward"):
        T, t = case["tokens"], case["t"]
        column = case["split"] == "column"
        win, wout = (case["fin"], case["fout"] // t) if column else (case["fin"] // t, case["fout"])
        # the quantised weight shards that the layer keeps
        W = _randn(gen, t, win, wout, std=0.02)
        s["Wq"], s["Ws"] = _quantize_blocks(W, "e4m3")
        s["b"] = _randn(gen, case["fout"], std=0.02)
        X = _randn(gen, T, win) if column else _randn(gen, t, T, win)
        if op == "linear":
            # the tokens, in chunks (column) or as one tensor for each shard (row)
            s["X"] = X.chunk(case["chunks"]) if column else list(X)
        else:
            # the tokens quantised along columns in the forward pass, kept for this one
            s["Xq"], s["Xs"] = _quantize(X, "e4m3", along_tokens=True)
            dY = _randn(gen, t, T, wout) if column else _randn(gen, T, wout)
            s["dY"] = list(dY) if column else dY.chunk(case["chunks"])
        return s
    T, h = case["tokens"], case["hidden"]
    s["Z"] = _randn(gen, T, h, std=0.7)
    s["post_gamma"] = (1 + 0.1 * torch.randn(h, generator=gen, device=DEV)).to(torch.bfloat16)
    s["pre_gamma"] = (1 + 0.1 * torch.randn(h, generator=gen, device=DEV)).to(torch.bfloat16)
    s["post_beta"] = _randn(gen, h, std=0.02)
    s["pre_beta"] = _randn(gen, h, std=0.02)
    if case["gate_rows"]:
        s["gate"] = _randn(gen, T // case["gate_rows"], h, std=0.5)
    X = _randn(gen, T, h, std=2.0)
    if op == "norm":
        s["X"] = X
        return s
    # what the forward pass kept: its output and the rows' means and reciprocal deviations
    s["Out"], _, s["stats"] = _norm_forward(s, X)
    s["dOut"], s["dXn"] = _randn(gen, T, h), _randn(gen, T, h)
    return s


# ---- plain forms ------------------------------------------------------------------------

def _scale(amax, fmt):
    """The power of two of a group and its reciprocal, from the group's largest magnitude."""
    m, e = torch.frexp(amax)
    k = e - TOP[fmt] + (m > 0.875)
    k = torch.where(amax > 0, k, -119).clamp(min=-119).to(torch.int32)
    scale, inverse = ((k + 127) << 23).view(torch.float32), ((127 - k) << 23).view(torch.float32)
    fine = torch.isfinite(amax)
    return torch.where(fine, scale, math.nan), torch.where(fine, inverse, 0.0)


def _to8(x, fmt):
    return torch.nan_to_num(x, nan=0.0).to(DTYPE[fmt])


def _quantize(X, fmt, along_tokens):
    """X [..., T, C] in groups of 128 of a token's features, or of a feature's tokens."""
    x = X.float()
    T, C = x.shape[-2:]
    if along_tokens:
        x = F.pad(x, (0, 0, 0, -T % 128)).unflatten(-2, (-1, 128))
        scale, inverse = _scale(x.abs().amax(-2), fmt)
        return _to8(x * inverse.unsqueeze(-2), fmt).flatten(-3, -2)[..., :T, :].contiguous(), scale
    x = F.pad(x, (0, -C % 128)).unflatten(-1, (-1, 128))
    scale, inverse = _scale(x.abs().amax(-1), fmt)
    return (_to8(x * inverse.unsqueeze(-1), fmt).flatten(-2)[..., :C].contiguous(),
            scale.transpose(-1, -2).contiguous())


def _quantize_blocks(W, fmt):
    w = W.float()
    r, c = w.shape[-2:]
    w = F.pad(w, (0, -c % 128, 0, -r % 128)).unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    scale, inverse = _scale(w.abs().amax((-3, -1)), fmt)
    q = _to8(w * inverse[..., None, :, None], fmt)
    return q.flatten(-2).flatten(-3, -2)[..., :r, :c].contiguous(), scale


def _spread(s, dim, size):
    return s.repeat_interleave(128, dim).narrow(dim, 0, size)


def _rows(q, s):
    return q.float() * _spread(s.transpose(-1, -2), -1, q.shape[-1])


def _cols(q, s):
    return q.float() * _spread(s, -2, q.shape[-2])


def _blocks(q, s):
    return q.float() * _spread(_spread(s, -2, q.shape[-2]), -1, q.shape[-1])


def _linear(s):
    W = _blocks(s["Wq"], s["Ws"])
    if s["split"] == "column":
        X = _rows(*_quantize(torch.cat(s["X"]), "e4m3", False))
        return list((X @ W + s["b"].float().view(s["t"], 1, -1)).to(torch.bfloat16))
    X = _rows(*_quantize(torch.stack(s["X"]), "e4m3", False))
    Z = (X @ W).sum(0) + s["b"].float()
    return list(Z.to(torch.bfloat16).chunk(s["chunks"]))


def _linear_backward(s):
    W, X = _blocks(s["Wq"], s["Ws"]), _cols(s["Xq"], s["Xs"])
    column = s["split"] == "column"
    dY = torch.stack(s["dY"]) if column else torch.cat(s["dY"])
    rows = _rows(*_quantize(dY, s["dy"], False))
    dX = rows @ W.transpose(-1, -2)
    dX = list(dX.sum(0).to(torch.bfloat16).chunk(s["chunks"])) if column else list(dX.to(torch.bfloat16))
    dW = X.transpose(-1, -2) @ _cols(*_quantize(dY, s["dy"], True))
    return {"dX": dX, "dW": list(dW), "db": dY.float().sum(-2).flatten()}


def _normed(x, kind, gamma, beta):
    """N(x), the rows' means and reciprocal deviations, and the normalised rows."""
    if kind == "none":
        return x, None, None, x
    mean = x.mean(-1) if kind == "layer" else torch.zeros_like(x[:, 0])
    c = x - mean[:, None]
    rstd = (c.square().mean(-1) + EPS).rsqrt()
    hat = c * rstd[:, None]
    return hat * gamma + (beta if kind == "layer" else 0), mean, rstd, hat


def _gate(s):
    return s["gate"].repeat_interleave(s["gate_rows"], 0) if s["gate_rows"] else None


def _norm_forward(s, X):
    u, m1, r1, _ = _normed(s["Z"].float(), s["post"], s["post_gamma"].float(), s["post_beta"].float())
    gate = _gate(s)
    out = (s["alpha"] * X.float() + (u if gate is None else gate.float() * u)).to(torch.bfloat16)
    xn, m2, r2, _ = _normed(out.float(), s["pre"], s["pre_gamma"].float(), s["pre_beta"].float())
    zero = torch.zeros_like(m2)
    return out, xn.to(torch.bfloat16), torch.stack([zero if v is None else v for v in (m1, r1, m2, r2)])


def _norm(s):
    out, xn, stats = _norm_forward(s, s["X"])
    if not s["quantize"]:
        return {"Out": out, "Xn": xn}
    q, scale = _quantize(xn, "e4m3", False)
    return {"Out": out, "q": q, "scale": _as8(scale)}


def _as8(scale):
    # a scale is a power of two: its 8-bit exponent stands for it
    return scale.to(torch.float8_e8m0fnu)


def _through(w, hat, rstd, kind):
    """The gradient of a normalised row's input from that of the normalised row."""
    w = w - hat * (w * hat).mean(-1, keepdim=True) - (w.mean(-1, keepdim=True) if kind == "layer" else 0)
    return w * rstd[:, None]


def _norm_backward(s):
    m1, r1, m2, r2 = s["stats"]
    T, h = s["tokens"], s["hidden"]
    dxn, g = s["dXn"].float(), s["dOut"].float()
    hat = (s["Out"].float() - m2[:, None]) * r2[:, None]
    got = {"dpre_gamma": (dxn * hat).sum(0)}
    if s["pre"] == "layer":
        got["dpre_beta"] = dxn.sum(0)
    g = g + _through(dxn * s["pre_gamma"].float(), hat, r2, s["pre"])
    got["dX"] = (s["alpha"] * g).to(torch.bfloat16)
    z, gate = s["Z"].float(), _gate(s)
    if s["post"] != "none":
        z = (z - m1[:, None]) * r1[:, None]
        u = z * s["post_gamma"].float() + (s["post_beta"].float() if s["post"] == "layer" else 0)
    else:
        u = z
    if gate is not None:
        got["dgate"] = (g * u).view(T // s["gate_rows"], s["gate_rows"], h).sum(1)
        g = g * gate.float()
    if s["post"] != "none":
        got["dpost_gamma"] = (g * z).sum(0)
        if s["post"] == "layer":
            got["dpost_beta"] = g.sum(0)
        g = _through(g * s["post_gamma"].float(), z, r1, s["post"])
    got["dZ"] = g.to(torch.bfloat16)
    return got


# ---- the framework's calls ----------------------------------------------------------------

def _own_layer(s):
    """The layer object a program makes once and keeps with its weights and buffers."""
    if "layer" not in s:
        if s["op"] in ("linear", "linear_backward"):
            from tensor_transformer_mlp_gemm_gb300.fp8 import DeviceFp8Linear
            from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear
            w = custom_linear(s["tokens"], s["fin"], s["fout"], s["t"], s["split"],
                              seq_chunks=s["chunks"])
            s["layer"] = DeviceFp8Linear(w, list(s["Wq"]), list(s["Ws"]), s["b"],
                                         dy_format=s.get("dy", "e4m3"))
        else:
            from tensor_transformer_mlp_gemm_gb300.norm import DeviceNormResidual
            s["layer"] = DeviceNormResidual(
                s["tokens"], s["hidden"], post=s["post"], pre=s["pre"], gate_rows=s["gate_rows"],
                residual_scale=s["alpha"], eps=EPS, post_gamma=s["post_gamma"],
                post_beta=s["post_beta"], pre_gamma=s["pre_gamma"], pre_beta=s["pre_beta"],
                quantize="e4m3" if s.get("quantize") else None)
    return s["layer"]


def _own(s):
    op = s["op"]
    if op in ("quantize", "weight"):
        from tensor_transformer_mlp_gemm_gb300 import fp8
        if op == "weight":
            q, scale = fp8.quantize_weight(s["W"], s["fmt"])
            return {"q": q, "scale": scale}
        x = fp8.quantize_tokens(s["X"], s["fmt"], rows=s["rows"], cols=s["cols"])
        got = {"rows": x.rows, "row_scale": x.row_scale} if s["rows"] else {}
        return dict(got, cols=x.cols, col_scale=x.col_scale) if s["cols"] else got
    layer = _own_layer(s)
    if op == "linear":
        layer.forward(layer.quantize(s["X"]))
        return layer.Y
    if op == "linear_backward":
        from tensor_transformer_mlp_gemm_gb300.fp8 import Fp8Tokens
        shards = [(s["Xq"], s["Xs"])] if s["split"] == "column" else list(zip(s["Xq"], s["Xs"]))
        layer.backward(s["dY"], [Fp8Tokens(cols=q, col_scale=c) for q, c in shards])
        return {"dX": layer.dX, "dW": layer.dW, "db": layer.db}
    if op == "norm":
        layer.forward(s["X"], s["Z"], gate=s.get("gate"))
        if s["quantize"]:
            return {"Out": layer.Out, "q": layer.q, "scale": _as8(layer.q_scale)}
        return {"Out": layer.Out, "Xn": layer.Xn}
    layer.backward(s["dOut"], s["dXn"], s["Z"], s["Out"], s["stats"], gate=s.get("gate"))
    got = {"dX": layer.dX, "dZ": layer.dZ, "dpre_gamma": layer.dpre_gamma}
    if s["pre"] == "layer":
        got["dpre_beta"] = layer.dpre_beta
    if s["gate_rows"]:
        got["dgate"] = layer.dgate
    if s["post"] != "none":
        got["dpost_gamma"] = layer.dpost_gamma
        if s["post"] == "layer":
            got["dpost_beta"] = layer.dpost_beta
    return got


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "quantize":
        X = torch.cat(state["X"])
        got = {}
        if state["rows"]:
            got["rows"], got["row_scale"] = _quantize(X, state["fmt"], False)
        if state["cols"]:
            got["cols"], got["col_scale"] = _quantize(X, state["fmt"], True)
        return got
    if op == "weight":
        q, scale = _quantize_blocks(state["W"], state["fmt"])
        return {"q": q, "scale": scale}
    return {"linear": _linear, "linear_backward": _linear_backward, "norm": _norm,
            "norm_backward": _norm_backward}[op](state)


# ---- work and the definition in 64 bits ----------------------------------------------------

def work(case):
    op = case["op"]
    up = lambda n: -(-n // 128)  # noqa: E731
    if op in ("linear", "linear_backward"):
        T, i, o = case["tokens"], case["fin"], case["fout"]
        if op == "linear":
            return {"bytes": 2 * T * i + i * o + 2 * T * o + 2 * o, "flops": 2 * T * i * o}
        return {"bytes": 2 * T * o + T * i + 4 * up(T) * i + i * o + 2 * T * i + 4 * i * o + 4 * o,
                "flops": 4 * T * i * o}
    if op == "quantize":
        T, C = case["tokens"], case["fin"]
        b = 2 * T * C
        if case["rows"]:
            b += T * C + 4 * up(C) * T
        if case["cols"]:
            b += T * C + 4 * up(T) * C
        return {"bytes": b, "flops": 2 * T * C}
    if op == "weight":
        i, o = case["fin"], case["fout"]
        return {"bytes": 3 * i * o + 4 * up(i) * up(o), "flops": 2 * i * o}
    T, h = case["tokens"], case["hidden"]
    gate = 2 * h * (T // case["gate_rows"]) if case["gate_rows"] else 0
    if op == "norm":
        each = 7 * T * h + 4 * T * up(h) if case["quantize"] else 8 * T * h
        return {"bytes": each + gate + 4 * h, "flops": 12 * T * h}
    return {"bytes": 12 * T * h + 16 * T + 3 * gate + 12 * h, "flops": 30 * T * h}


def _groups64(x, fmt, dim):
    """The values that stand for x in 64 bits: each group of 128 along `dim` at its power of two."""
    x = x.double().movedim(dim, -1)
    n = x.shape[-1]
    g = F.pad(x, (0, -n % 128)).reshape(*x.shape[:-1], -1, 128)
    scale = _scale64(g.abs().amax(-1, keepdim=True), fmt)
    values = (_round64(g / scale, fmt) * scale).reshape(*x.shape[:-1], -1)[..., :n].movedim(-1, dim)
    return values, scale[..., 0].movedim(-1, dim)


def _scale64(amax, fmt):
    top = 448.0 if fmt == "e4m3" else 57344.0
    k = torch.ceil(torch.log2(amax.clamp(min=1e-300) / top))
    k = torch.where(torch.exp2(k - 1) * top >= amax, k - 1, k)
    k = torch.where(torch.exp2(k) * top < amax, k + 1, k)
    return torch.exp2(k.clamp(min=-119))


def _round64(x, fmt):
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.floor(torch.log2(x.abs().clamp(min=1e-300))).clamp(min=low)
    step = torch.exp2(e - bits)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        X, got = torch.cat(s["X"]), {}
        if case["rows"]:
            v, sc = _groups64(X, case["fmt"], -1)
            got["rows"], got["row_scale"] = v / sc.repeat_interleave(128, -1)[:, : X.shape[1]], sc.T
        if case["cols"]:
            v, sc = _groups64(X, case["fmt"], 0)
            got["cols"], got["col_scale"] = v / sc.repeat_interleave(128, 0)[: X.shape[0]], sc
        return got
    if op == "weight":
        W = s["W"].double()
        r, c = W.shape
        full = torch.zeros(-(-r // 128) * 128, -(-c // 128) * 128, dtype=torch.float64, device=DEV)
        full[:r, :c] = W.abs()
        scale = _scale64(F.max_pool2d(full[None, None], 128)[0, 0], case["fmt"])
        big = torch.kron(scale, torch.ones(128, 128, dtype=torch.float64, device=DEV))[:r, :c]
        return {"q": _round64(W / big, case["fmt"]), "scale": scale}
    if op in ("linear", "linear_backward"):
        t, column = case["t"], case["split"] == "column"
        ones = torch.ones(128, 128, dtype=torch.float64, device=DEV)
        W = [torch.kron(s["Ws"][i].double(), ones)[: q.shape[0], : q.shape[1]] * q.double()
             for i, q in enumerate(s["Wq"])]
        b = s["b"].double()
        if op == "linear":
            if column:
                X = _groups64(torch.cat(s["X"]), "e4m3", -1)[0]
                return [X @ w + v for w, v in zip(W, b.chunk(t))]
            Z = sum(_groups64(x, "e4m3", -1)[0] @ w for x, w in zip(s["X"], W)) + b
            return list(Z.chunk(case["chunks"]))
        X = [q.double() * sc.double().repeat_interleave(128, 0)[: q.shape[0]]
             for q, sc in ([(s["Xq"], s["Xs"])] if column else zip(s["Xq"], s["Xs"]))]
        dY = s["dY"] if column else [torch.cat(s["dY"])]
        rows = [_groups64(d, case["dy"], -1)[0] for d in dY]
        cols = [_groups64(d, case["dy"], 0)[0] for d in dY]
        if column:
            dX = list(sum(d @ w.T for d, w in zip(rows, W)).chunk(case["chunks"]))
            dW = [X[0].T @ d for d in cols]
        else:
            dX = [rows[0] @ w.T for w in W]
            dW = [x.T @ cols[0] for x in X]
        return {"dX": dX, "dW": dW, "db": torch.cat([d.double().sum(0) for d in dY])}
    # the norms
    h = case["hidden"]
    gate = s["gate"].double().repeat_interleave(case["gate_rows"], 0) if case["gate_rows"] else None

    def norm(x, kind, which):
        if kind == "none":
            return x
        y = F.layer_norm(x, (h,), eps=EPS) if kind == "layer" else x / (x.square().mean(-1, True) + EPS).sqrt()
        return y * p[which + "_gamma"] + (p[which + "_beta"] if kind == "layer" else 0.0)

    p = {k: s[k].double().requires_grad_() for k in ("post_gamma", "post_beta", "pre_gamma", "pre_beta")}
    Z = s["Z"].double()
    if op == "norm":
        u = norm(Z, case["post"], "post")
        out = case["alpha"] * s["X"].double() + (u if gate is None else gate * u)
        # the next norm reads the rounded output
        xn = norm(out.to(torch.bfloat16).double(), case["pre"], "pre")
        # rounding to 8 bits turns on the last bit of what is rounded: no value of its own
        return {"Out": out, "q": None, "scale": None} if case["quantize"] else {"Out": out, "Xn": xn.detach()}
    Z.requires_grad_()
    Out = s["Out"].double().requires_grad_()
    norm(Out, case["pre"], "pre").backward(s["dXn"].double())
    g = s["dOut"].double() + Out.grad
    got = {"dX": case["alpha"] * g, "dpre_gamma": p["pre_gamma"].grad}
    if case["pre"] == "layer":
        got["dpre_beta"] = p["pre_beta"].grad
    u = norm(Z, case["post"], "post")
    if gate is not None:
        got["dgate"] = (g * u.detach()).view(-1, case["gate_rows"], h).sum(1)
    u.backward(g if gate is None else g * gate)
    got["dZ"] = Z.grad
    if case["post"] != "none":
        got["dpost_gamma"] = p["post_gamma"].grad
        if case["post"] == "layer":
            got["dpost_beta"] = p["post_beta"].grad
    return got
