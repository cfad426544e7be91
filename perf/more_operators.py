"""Cases of the 4-bit linear layers (quantisation and back, forward, a training
step) and of the global gradient norm with clipping, with their plain forms.

Definitions (as the library documents them): a 4-bit value is a sign, two
exponent bits and one mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6), rounded to
nearest even.  A group lies along the axis that a product sums over.

  mxfp4   groups of 32; the scale is the smallest power of two, at least 2^-126,
          with which the group's largest magnitude is at most 6
  nvfp4   groups of 16 and one scale g for the tensor: the smallest power of two, at
          least 2^-110, with which its largest magnitude is at most 6 * 448 g (or the
          one that a calibration gave); the group's scale is g times its largest
          magnitude / (6 g), rounded to e4m3 and at least 2^-9

Gradients are clipped to max_norm as g * min(1, max_norm / (norm + 1e-6)), the
norm being that of all tensors together.
"""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
GROUP = {"mxfp4": 32, "nvfp4": 16}
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ---- the cases ------------------------------------------------------------------------

def listed():
    return [
        # one token through the QKV projection of the 4096-wide layer: latency, the weight's bytes
        {"name": "linear decode 1 token", "op": "linear", "fmt": "nvfp4", "split": "column",
         "tokens": 1, "fin": 4096, "fout": 12288, "t": 1, "chunks": 1},
        # a decode batch through the 175B-class output projection, eight row shards
        {"name": "linear decode 48 tokens", "op": "linear", "fmt": "mxfp4", "split": "row",
         "tokens": 48, "fin": 12288, "fout": 12288, "t": 8, "chunks": 1},
        # a ragged prefill: no size a multiple of the tiles
        {"name": "linear ragged 777 tokens", "op": "linear", "fmt": "nvfp4", "split": "column",
         "tokens": 777, "fin": 2080, "fout": 8224, "t": 1, "chunks": 1},
        # the QKV projection of the 175B-class layer, eight column shards
        {"name": "linear 175B QKV", "op": "linear", "fmt": "nvfp4", "split": "column",
         "tokens": 2048, "fin": 12288, "fout": 36864, "t": 8, "chunks": 1},
        # training: the output projection of the 4096-wide layer, forward and backward, token chunks
        {"name": "step 16384 x 4096", "op": "step", "fmt": "mxfp4", "split": "row",
         "tokens": 16384, "fin": 4096, "fout": 4096, "t": 8, "chunks": 8},
        # training: a small layer with a ragged batch
        {"name": "step ragged 333 tokens", "op": "step", "fmt": "nvfp4", "split": "column",
         "tokens": 333, "fin": 1056, "fout": 2080, "t": 1, "chunks": 1},
        # what 4 bits leave of the 4096-wide layer's activations, along features and along tokens
        {"name": "quantize 16384 x 4096", "op": "quantize", "fmt": "mxfp4", "tokens": 16384,
         "fin": 4096, "rows": True, "cols": True},
        # and of a weight shard, as training with simulated rounding takes it each step
        {"name": "weight 12288 x 4608", "op": "weight", "fmt": "nvfp4", "fin": 12288, "fout": 4608},
        # the gradients of the smallest MLP block: latency
        {"name": "clip tiny block", "op": "clip", "layers": 1, "hidden": 256, "ffn": 1024, "t": 2,
         "type": "fp32", "clip": True},
        # a whole small model, bf16 weight gradients and fp32 bias gradients, no size even
        {"name": "clip 24 odd layers", "op": "clip", "layers": 24, "hidden": 771, "ffn": 2053 * 2,
         "t": 2, "type": "bf16", "clip": True},
        # the 4096-wide block in eight shards
        {"name": "clip 4096 x 16384 block", "op": "clip", "layers": 1, "hidden": 4096, "ffn": 16384,
         "t": 8, "type": "fp32", "clip": True},
        # the 175B-class block in eight shards, a norm that is below the limit
        {"name": "clip 175B block", "op": "clip", "layers": 1, "hidden": 12288, "ffn": 49152,
         "t": 8, "type": "fp32", "clip": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "step", "step", "quantize", "weight", "clip", "clip"])
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op in ("linear", "step"):
        limit = 2048 * 12288 * 36864 if op == "linear" else 16384 * 4096 * 4096
        while True:
            t = rng.choice([1, 1, 2, 8])
            split = rng.choice(["column", "row"])
            shard, other = 32 * _log(rng, 8, 768 // t), 32 * _log(rng, 8, 384)
            fin, fout = (other, shard * t) if split == "column" else (shard * t, other)
            tokens, chunks = _log(rng, 1, 16384), 1
            if tokens >= 1024 and rng.random() < 0.5:
                chunks = rng.choice([2, 4, 8])
                tokens -= tokens % (128 * chunks)
            if tokens * fin * fout <= limit:
                break
        return {"op": op, "fmt": fmt, "split": split, "tokens": tokens, "fin": fin, "fout": fout,
                "t": t, "chunks": chunks}
    if op == "quantize":
        rows = rng.random() < 0.8
        return {"op": op, "fmt": fmt, "tokens": _log(rng, 1, 16384), "fin": 32 * _log(rng, 8, 128),
                "rows": rows, "cols": not rows or rng.random() < 0.6}
    if op == "weight":
        return {"op": op, "fmt": fmt, "fin": 32 * _log(rng, 8, 384), "fout": 32 * _log(rng, 8, 144)}
    while True:
        t = rng.choice([1, 2, 8])
        hidden, ffn, layers = _log(rng, 16, 12288), t * _log(rng, 16, 49152 // t), _log(rng, 1, 96)
        if layers * hidden * ffn <= 12288 * 49152 // 2:
            break
    return {"op": op, "layers": layers, "hidden": hidden, "ffn": ffn, "t": t,
            "type": rng.choice(["fp32", "bf16"]), "clip": rng.random() < 0.75}


# ---- inputs ---------------------------------------------------------------------------

def _randn(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def _activations(gen, *shape):
    # a few features much larger than the rest, as trained layers have them
    X = _randn(gen, *shape)
    X[..., ::97] *= 16.0
    return X


def _shapes(case):
    """The weights' and the biases' gradients of the MLP blocks, in order."""
    h, f, t = case["hidden"], case["ffn"], case["t"]
    weights = ([(h, f // t)] * t + [(f // t, h)] * t) * case["layers"]
    return weights, [(f,), (h,)] * case["layers"]


def _views(flat, shapes):
    """Tensors of these shapes in a flat buffer, each on 256 bytes."""
    step = 256 // flat.element_size()
    views, at = [], 0
    for s in shapes:
        n = math.prod(s)
        views.append(flat[at:at + n].view(s))
        at += -(-n // step) * step
    return views


def _flat(shapes, dtype):
    step = 256 // dtype.itemsize
    return torch.zeros(sum(-(-math.prod(s) // step) * step for s in shapes), dtype=dtype, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 11)
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        s["X"] = _activations(gen, case["tokens"], case["fin"])
        return s
    if op == "weight":
        s["W"] = _randn(gen, case["fin"], case["fout"], std=0.02)
        return s
    if op in ("linear", "step"):
        T, t, fmt = case["tokens"], case["t"], case["fmt"]
        column = case["split"] == "column"
        win, wout = (case["fin"], case["fout"] // t) if column else (case["fin"] // t, case["fout"])
        s["W"] = _randn(gen, t, win, wout, std=0.02)
        # the values that the 4-bit weights stand for, which a plain layer keeps in their place: grouped
        # along the inputs for the forward pass, along the outputs for the backward pass
        g = _tensor_scale(s["W"]) if fmt == "nvfp4" else None
        s["W_forward"] = _along(s["W"], fmt, -2, g)
        if op == "step":
            s["W_backward"] = _along(s["W"], fmt, -1, g)
            dY = _randn(gen, t, T, wout, std=1e-4) if column else _randn(gen, T, wout, std=1e-4)
            s["dY"] = list(dY) if column else list(dY.chunk(case["chunks"]))
        s["b"] = _randn(gen, case["fout"], std=0.02)
        # the activations' scale that a calibration gave (their largest magnitude is near 75)
        s["x_scale"] = torch.full((1,), 2.0 ** -5, device=DEV) if fmt == "nvfp4" else None
        X = _activations(gen, T, win) if column else _activations(gen, t, T, win)
        s["X"] = list(X.chunk(case["chunks"])) if column else list(X)
        return s
    weights, biases = _shapes(case)
    s["weights"], s["biases"] = _flat(weights, TYPES[case["type"]]), _flat(biases, torch.float32)
    total = 0
    for flat, shapes in ((s["weights"], weights), (s["biases"], biases)):
        for v in _views(flat, shapes):
            v.copy_(torch.randn(v.shape, generator=gen, device=DEV) * 1e-3)
            total += v.numel()
    # gradients of 1e-3: the norm is near 1e-3 sqrt(values)
    s["max_norm"] = (0.5 if case["clip"] else 2.0) * 1e-3 * math.sqrt(total)
    # where the clipped gradients go
    s["weights_out"], s["biases_out"] = torch.zeros_like(s["weights"]), torch.zeros_like(s["biases"])
    return s


# ---- plain forms ------------------------------------------------------------------------

def _power(k):
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _tensor_scale(x):
    m, e = torch.frexp(x.float().abs().amax())
    # 6 * 448 = 0.65625 * 2^12
    return _power(torch.where(m > 0, e - 12 + (m > 0.65625).to(e.dtype), -110).clamp(min=-110)).view(1)


def _to4(x):
    """x in 32 bits to the nearest of the 4-bit values, ties to even."""
    a = x.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6.0) * torch.sign(x)


def _grouped(x, fmt, g):
    """The values of x [..., groups, size], a scale for each group, g for all."""
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        m, e = torch.frexp(amax)
        s = _power(torch.where(m > 0, e - 3 + (m > 0.75).to(e.dtype), -126).clamp(min=-126))
        return _to4(x / s) * s
    s = ((amax / g) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
    return _to4((x / g) / s) * s * g


def _along(X, fmt, dim, g):
    """The values of the 4-bit X grouped along `dim`, in bf16, which holds them exactly."""
    x = X.float().movedim(dim, -1)
    n, size = x.shape[-1], GROUP[fmt]
    x = _grouped(F.pad(x, (0, -n % size)).unflatten(-1, (-1, size)), fmt, g)
    return x.flatten(-2)[..., :n].movedim(-1, dim).to(torch.bfloat16)


def _linear(s):
    """Y_i = X W_i + b_i, or Z = sum_i X_i W_i + b."""
    W, b = s["W_forward"].float(), s["b"].float()
    if s["split"] == "column":
        X = _along(torch.cat(s["X"]), s["fmt"], -1, s["x_scale"]).float()
        return list((X @ W + b.view(s["t"], 1, -1)).to(torch.bfloat16))
    X = _along(torch.stack(s["X"]), s["fmt"], -1, s["x_scale"]).float()
    return list(((X @ W).sum(0) + b).to(torch.bfloat16).chunk(s["chunks"]))


def _step(s):
    column, fmt = s["split"] == "column", s["fmt"]
    X = torch.cat(s["X"]) if column else torch.stack(s["X"])
    dY = torch.stack(s["dY"]) if column else torch.cat(s["dY"])
    g = _tensor_scale(dY) if fmt == "nvfp4" else None
    dX = _along(dY, fmt, -1, g).float() @ s["W_backward"].float().transpose(-1, -2)
    dX = list(dX.sum(0).to(torch.bfloat16).chunk(s["chunks"])) if column else list(dX.to(torch.bfloat16))
    Xc = _along(X, fmt, -2, s["x_scale"]).float().transpose(-1, -2)
    dW = Xc @ _along(dY, fmt, -2, g).float()
    return {"Y": _linear(s), "dX": dX, "dW": list(dW), "db": dY.double().sum(-2).flatten().float()}


def _clip(s):
    norm = (s["weights"].double().square().sum() + s["biases"].double().square().sum()).sqrt()
    c = (s["max_norm"] / (norm + EPS)).clamp(max=1.0).float()
    return {"norm": norm.float().view(1), "weights": (s["weights"].float() * c).to(s["weights"].dtype),
            "biases": s["biases"] * c}


# ---- the framework's calls ----------------------------------------------------------------

def _own_layer(s):
    """The layer, or the list of gradients, that a program makes once and keeps."""
    if "layer" not in s:
        if s["op"] == "clip":
            from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
            weights, biases = _shapes(s)
            s["layer"] = DeviceGradients(
                _views(s["weights"], weights) + _views(s["biases"], biases),
                out=_views(s["weights_out"], weights) + _views(s["biases_out"], biases))
        else:
            from tensor_transformer_mlp_gemm_gb300 import fp4
            from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear
            w = custom_linear(s["tokens"], s["fin"], s["fout"], s["t"], s["split"],
                              seq_chunks=s["chunks"])
            s["layer"] = fp4.DeviceFp4Linear(
                w, fp4.quantize_weight(list(s["W"]), s["fmt"], backward=s["op"] == "step"), s["b"],
                x_scale=s["x_scale"])
    return s["layer"]


def _own(s):
    op = s["op"]
    if op == "quantize":
        from tensor_transformer_mlp_gemm_gb300 import fp4
        x = fp4.quantize_tokens(s["X"], s["fmt"], rows=s["rows"], cols=s["cols"])
        got = {"rows": x.rows.values()} if s["rows"] else {}
        return dict(got, cols=x.cols.values()) if s["cols"] else got
    if op == "weight":
        from tensor_transformer_mlp_gemm_gb300 import fp4
        w = fp4.quantize_weight(s["W"], s["fmt"], backward=True)
        return {"forward": w.forward[0].values(), "backward": w.backward[0].values()}
    layer = _own_layer(s)
    if op == "clip":
        layer.clip(s["max_norm"])
        return {"norm": layer.norm, "weights": s["weights_out"], "biases": s["biases_out"]}
    if op == "linear":
        layer.forward(s["X"])
        return layer.Y
    layer.forward(s["X"], save=True)
    layer.backward(s["dY"])
    return {"Y": layer.Y, "dX": layer.dX, "dW": layer.dW, "db": layer.db}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op in ("quantize", "weight"):
        X, fmt = state["X" if op == "quantize" else "W"], state["fmt"]
        g = _tensor_scale(X) if fmt == "nvfp4" else None
        got = {}
        # grouped along tokens (a weight: along its inputs) the matrix lies transposed
        if op == "weight" or state["rows"]:
            got["backward" if op == "weight" else "rows"] = _along(X, fmt, 1, g)
        if op == "weight" or state["cols"]:
            got["forward" if op == "weight" else "cols"] = _along(X, fmt, 0, g).t().contiguous()
        return got
    return {"linear": _linear, "step": _step, "clip": _clip}[op](state)


# ---- work and the definition in 64 bits ----------------------------------------------------

def work(case):
    op = case["op"]
    if op == "clip":
        weights, biases = _shapes(case)
        w, b = (sum(math.prod(s) for s in shapes) for shapes in (weights, biases))
        return {"bytes": 2 * (TYPES[case["type"]].itemsize * w + 4 * b), "flops": 3 * (w + b)}
    # bytes of a 4-bit value with its share of the scale
    q = 0.5 + 1 / GROUP[case["fmt"]]
    if op in ("linear", "step"):
        T, i, o = case["tokens"], case["fin"], case["fout"]
        once = 2 * T * i + q * i * o + 2 * T * o + 2 * o
        if op == "linear":
            return {"bytes": once, "flops": 2 * T * i * o}
        return {"bytes": once + 2 * T * o + q * i * o + 2 * T * i + 4 * i * o + 4 * o,
                "flops": 6 * T * i * o}
    # the 4-bit form is written and read between
    n = case["fin"] * (case["tokens"] if op == "quantize" else case["fout"])
    ways = 2 if op == "weight" else case["rows"] + case["cols"]
    return {"bytes": n * (2 + ways * (2 * q + 2)), "flops": 4 * ways * n}


def _floor_log2(x):
    e = torch.floor(torch.log2(x))
    e = torch.where(torch.exp2(e) > x, e - 1, e)
    return torch.where(torch.exp2(e + 1) <= x, e + 1, e)


def _least_power(amax, top, low):
    """The smallest power of two that brings amax to `top` or below."""
    k = torch.ceil(torch.log2(amax.clamp(min=1e-300) / top))
    k = torch.where(torch.exp2(k - 1) * top >= amax, k - 1, k)
    k = torch.where(torch.exp2(k) * top < amax, k + 1, k)
    return torch.exp2(k.clamp(min=low))


def _round64(x, bits, low, top):
    step = torch.exp2(_floor_log2(x.abs().clamp(min=2.0 ** low)) - bits)
    return (torch.round(x / step) * step).clamp(-top, top)


def _exact_values(X, fmt, dim, g=None):
    x = X.double().movedim(dim, -1)
    n, size = x.shape[-1], GROUP[fmt]
    x = F.pad(x, (0, -n % size)).reshape(*x.shape[:-1], -1, size)
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        s = _least_power(amax, 6.0, -126)
    else:
        s = g * _round64(amax / (6.0 * g), 3, -6, 448.0).clamp(min=2.0 ** -9)
    v = _round64(x / s, 1, 0, 6.0) * s
    return v.reshape(*v.shape[:-2], -1)[..., :n].movedim(-1, dim)


def _exact_g(X, fmt):
    return _least_power(X.double().abs().amax(), 2688.0, -110) if fmt == "nvfp4" else None


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        squares = sum(torch.dot(v, v) for v in (s["weights"].double(), s["biases"].double()))
        norm = math.sqrt(float(squares))
        c = min(1.0, s["max_norm"] / (norm + EPS))
        return {"norm": torch.full((1,), norm, dtype=torch.float64, device=DEV),
                "weights": s["weights"].double() * c, "biases": s["biases"].double() * c}
    fmt = case["fmt"]
    if op in ("quantize", "weight"):
        X = s["X"] if op == "quantize" else s["W"]
        names = ("rows", "cols") if op == "quantize" else ("backward", "forward")
        got, g = {}, _exact_g(X, fmt)
        if op == "weight" or case["rows"]:
            got[names[0]] = _exact_values(X, fmt, 1, g)
        if op == "weight" or case["cols"]:
            got[names[1]] = _exact_values(X.t(), fmt, 1, g)
        return got
    t, column = case["t"], case["split"] == "column"
    # a 64-bit product runs at about 1 TFLOP/s
    if 2 * case["tokens"] * case["fin"] * case["fout"] * (3 if op == "step" else 1) > 1e13:
        return None
    gw, gx = _exact_g(s["W"], fmt), None if s["x_scale"] is None else s["x_scale"].double()
    W = [_exact_values(w, fmt, 0, gw) for w in s["W"]]
    X = [torch.cat(s["X"])] if column else s["X"]
    Xr = [_exact_values(x, fmt, 1, gx) for x in X]
    b = s["b"].double()
    if column:
        Y = [torch.addmm(v, Xr[0], w) for w, v in zip(W, b.chunk(t))]
    else:
        Y = list((sum(x @ w for x, w in zip(Xr, W)) + b).chunk(case["chunks"]))
    if op == "linear":
        return Y
    dY = s["dY"] if column else [torch.cat(s["dY"])]
    gd = _exact_g(torch.stack(s["dY"]), fmt)
    rows, cols = ([_exact_values(d, fmt, k, gd) for d in dY] for k in (1, 0))
    back = [_exact_values(w, fmt, 1, gw) for w in s["W"]]
    if column:
        dX = list(sum(d @ w.T for d, w in zip(rows, back)).chunk(case["chunks"]))
    else:
        dX = [rows[0] @ w.T for w in back]
    Xc = [_exact_values(x, fmt, 0, gx) for x in X]
    dW = [Xc[0].T @ d for d in cols] if column else [x.T @ cols[0] for x in Xc]
    return {"Y": Y, "dX": dX, "dW": dW, "db": torch.cat([d.double().sum(0) for d in dY])}
