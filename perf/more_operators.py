"""The operators between a layer's attention and its matrices in 8 bits, as they are measured.

  norm      root-mean-square norm in groups of the residual stream with a layer's output added, as E4M3 codes and a scale per row
  quantize  rows as E4M3 codes and a scale per row
  linear    matrix product (E4M3 codes with their scales, bf16 or fp16) with bias, activation and residual

``run`` computes them in plain torch operations, or, where ``own`` is true, with this repository's operators.  The shapes
are those of the 3.7B model (hidden 2560 in two norm groups, 32 query heads over 8 KV heads of 128, intermediate 10240)
and of the ragged test model (hidden 640, intermediate 1664).

E4M3 codes are returned as float8 tensors, next to their scales.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}
EPS = 1e-6
TOP = 448.0  # the largest finite E4M3 value


# ---- cases -----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one conversation's decode step: the residual stream in fp32, a layer's output added; latency counts
        {"name": "norm 1 x 2560", "op": "norm", "tokens": 1, "hidden": 2560, "groups": 2, "type": "f32", "stream": "f32", "wide": False},
        # a batch of 64 requests, everything in bf16, the layer's output a column slice of wider rows
        {"name": "norm 64 x 2560 bf16", "op": "norm", "tokens": 64, "hidden": 2560, "groups": 2, "type": "bf16", "stream": "bf16", "wide": True},
        # a prompt block of the ragged model behind the embedding: no residual to add yet
        {"name": "norm 509 x 640 f16", "op": "norm", "tokens": 509, "hidden": 640, "groups": 2, "type": "f16", "stream": "none", "wide": False},
        # a full prefill block over the fp32 residual stream
        {"name": "norm 2048 x 2560", "op": "norm", "tokens": 2048, "hidden": 2560, "groups": 2, "type": "f32", "stream": "f32", "wide": False},
        # the SwiGLU output of 16 requests, ahead of the down projection
        {"name": "quantize 16 x 10240", "op": "quantize", "tokens": 16, "hidden": 10240, "type": "bf16", "wide": False},
        # the same of a large prompt
        {"name": "quantize 8192 x 10240", "op": "quantize", "tokens": 8192, "hidden": 10240, "type": "bf16", "wide": False},
        # one conversation's q | k | v
        {"name": "linear 1 qkv f8", "op": "linear", "tokens": 1, "rows": 6144, "cols": 2560, "type": "f8", "out": "f32",
         "activation": "none", "bias": False, "residual": False},
        # the gate and up projections of 16 requests
        {"name": "linear 16 gate up f8", "op": "linear", "tokens": 16, "rows": 20480, "cols": 2560, "type": "f8", "out": "bf16",
         "activation": "swiglu", "bias": False, "residual": False},
        # the down projection of 64 requests, added to the fp32 residual stream
        {"name": "linear 64 down f8", "op": "linear", "tokens": 64, "rows": 2560, "cols": 10240, "type": "f8", "out": "f32",
         "activation": "none", "bias": False, "residual": True},
        # a prompt chunk of the ragged model with a bias and a GELU
        {"name": "linear 333 ragged f16", "op": "linear", "tokens": 333, "rows": 1664, "cols": 640, "type": "f16", "out": "f16",
         "activation": "gelu", "bias": True, "residual": False},
        # the gate and up projections of a full prefill block
        {"name": "linear 2048 gate up f8", "op": "linear", "tokens": 2048, "rows": 20480, "cols": 2560, "type": "f8", "out": "bf16",
         "activation": "swiglu", "bias": False, "residual": False},
        # the down projection of a large prompt in bf16, added to a bf16 residual stream
        {"name": "linear 4096 down bf16", "op": "linear", "tokens": 4096, "rows": 2560, "cols": 10240, "type": "bf16", "out": "bf16",
         "activation": "none", "bias": False, "residual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "linear", "linear"])
    if op == "norm":
        groups = rng.choice([1, 2, 2, 4])
        return {"op": op, "tokens": _log(rng, 1, 2048), "hidden": groups * rng.choice([16, 160, 320, 1280, _log(rng, 7, 1280)]), "groups": groups,
                "type": rng.choice(["f32", "bf16", "f16"]), "stream": rng.choice(["none", "f32", "bf16", "f16"]), "wide": rng.random() < 0.3}
    if op == "quantize":
        return {"op": op, "tokens": _log(rng, 1, 8192), "hidden": rng.choice([640, 1664, 2560, 4096, 10240, _log(rng, 5, 10240)]),
                "type": rng.choice(["bf16", "bf16", "f16"]), "wide": rng.random() < 0.3}
    rows = rng.choice([640, 2560, 6144, 20480, 2 * _log(rng, 4, 10240)])
    cols = rng.choice([640, 1664, 2560, 4096, _log(rng, 16, 4096)])
    kind = rng.choice(["f8", "f8", "bf16", "f16"])
    activation = rng.choice(["none", "none", "swiglu", "silu", "gelu", "gelu_tanh", "relu"])
    return {"op": op, "tokens": _log(rng, 1, max(1, min(8192, 2 ** 36 // (rows * cols)))), "rows": rows, "cols": cols, "type": kind,
            "out": rng.choice(["f32", "bf16", "f16"]), "activation": activation, "bias": rng.random() < 0.4, "residual": rng.random() < 0.4}


def _size(kind):
    return {"none": 0, "f32": 4, "bf16": 2, "f16": 2, "f8": 1}[kind]


def work(case):
    t = case["tokens"]
    if case["op"] == "linear":
        n, k = case["rows"], case["cols"]
        outs = t * (n // 2 if case["activation"] == "swiglu" else n) * _size(case["out"])
        scales = 4 * (n + t) if case["type"] == "f8" else 0
        return {"bytes": (n + t) * k * _size(case["type"]) + outs * (2 if case["residual"] else 1) + scales + (4 * n if case["bias"] else 0),
                "flops": 2 * t * n * k}
    h = case["hidden"]
    # a row read, codes and a scale written; the residual stream read and written, and the gain read
    each = _size(case["type"]) + 1 + 2 * _size(case.get("stream", "none"))
    return {"bytes": t * (h * each + 4) + (2 * h if case["op"] == "norm" else 0), "flops": t * h * (8 if case["op"] == "norm" else 3)}


# ---- inputs ----------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (_prepare_linear if case["op"] == "linear" else _prepare_rows)(case, gen)


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _activations(gen, tokens, hidden):
    """Rows of a layer: some channels are larger than others, and so are some tokens."""
    x = _randn(gen, tokens, hidden)
    x *= (_randn(gen, hidden) * 0.6).exp_()
    x *= (_randn(gen, tokens, 1) * 0.5).exp_()
    return x


def _prepare_rows(case, gen):
    t, h = case["tokens"], case["hidden"]
    x = _activations(gen, t, h).to(TYPES[case["type"]])
    if case["wide"]:  # a column slice of wider rows
        x = torch.cat([x, x[:, :h // 2], x], 1)[:, h + h // 2:]
    s = {"op": case["op"], "x": x, "codes": torch.zeros(t, -(-h // 16) * 16, dtype=torch.float8_e4m3fn, device="cuda")[:, :h],
         "scales": torch.zeros(t, device="cuda")}
    if case["op"] == "norm":
        s["groups"] = case["groups"]
        s["gain"] = (1 + 0.1 * _randn(gen, h)).bfloat16()
        s["stream"] = s["stream_out"] = None
        if case["stream"] != "none":
            s["stream"] = (_activations(gen, t, h) * 4).to(TYPES[case["stream"]])
            s["stream_out"] = torch.zeros_like(s["stream"])
    return s


def _codes(x):
    """Rows [n, k] as E4M3 codes, 16-byte rows apart, and a scale for each."""
    n, k = x.shape
    scale = x.abs().amax(1) / TOP
    codes = torch.zeros(n, -(-k // 16) * 16, dtype=torch.float8_e4m3fn, device=x.device)
    codes[:, :k] = (x / scale[:, None]).to(torch.float8_e4m3fn)
    return codes[:, :k], scale


def _spaced(x):
    """16-bit rows [n, k] whose starts are 16-byte aligned."""
    n, k = x.shape
    wide = torch.zeros(n, -(-k // 8) * 8, dtype=x.dtype, device=x.device)
    wide[:, :k] = x
    return wide[:, :k]


def _prepare_linear(case, gen):
    t, n, k, out = case["tokens"], case["rows"], case["cols"], TYPES[case["out"]]
    x = _activations(gen, t, k) / math.sqrt(1.5)
    w = _randn(gen, n, k) * (1 / math.sqrt(k))
    s = {"op": "linear", "activation": case["activation"], "x_scale": None, "w_scale": None, "bias": None, "residual": None}
    if case["type"] == "f8":
        (s["x"], s["x_scale"]), (s["w"], s["w_scale"]) = _codes(x), _codes(w)
    else:
        s["x"], s["w"] = _spaced(x.to(TYPES[case["type"]])), _spaced(w.to(TYPES[case["type"]]))
    if case["bias"]:
        s["bias"] = 0.3 * _randn(gen, n)
    width = n // 2 if case["activation"] == "swiglu" else n
    if case["residual"]:
        s["residual"] = (3 * _randn(gen, t, width)).to(out)
    s["out"] = torch.zeros(t, width, dtype=out, device="cuda")
    return s


# ---- one pass --------------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return {"norm": _own_norm, "quantize": _own_quantize, "linear": _own_linear}[state["op"]](state)
    return {"norm": _norm, "quantize": _quantize, "linear": _linear}[state["op"]](state)


def _own_norm(s):
    from dense_gqa_decoder_gb300 import k2
    k2.norm_quantize(s["x"], s["gain"], s["codes"], s["scales"], residual=s["stream"], residual_out=s["stream_out"], groups=s["groups"], eps=EPS)
    return [s["codes"], s["scales"]] + ([] if s["stream"] is None else [s["stream_out"]])


def _own_quantize(s):
    from dense_gqa_decoder_gb300 import k2
    k2.quantize_rows(s["x"], s["codes"], s["scales"])
    return [s["codes"], s["scales"]]


def _own_linear(s):
    from dense_gqa_decoder_gb300 import k2
    k2.linear(s["w"], s["x"], s["out"], w_scale=s["w_scale"], x_scale=s["x_scale"], bias=s["bias"], activation=s["activation"],
              residual=s["residual"])
    return s["out"]


def _as_codes(y):
    scale = y.abs().amax(1) / TOP
    q = torch.where(scale[:, None] > 0, y / scale[:, None], 0.0)
    return [q.clamp(-TOP, TOP).to(torch.float8_e4m3fn), scale]


def _norm(s):
    h = s["x"].float()
    if s["stream"] is not None:
        h = h + s["stream"].float()
    t, n = h.shape
    parts = h.view(t, s["groups"], n // s["groups"])
    y = parts / torch.sqrt((parts * parts).mean(2, keepdim=True) + EPS)
    got = _as_codes(y.reshape(t, n) * s["gain"].float())
    return got + ([] if s["stream"] is None else [h.to(s["stream"].dtype)])


def _quantize(s):
    return _as_codes(s["x"].float())


def _linear(s):
    z = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["w_scale"] is not None:
        z = z * s["w_scale"] * s["x_scale"][:, None]
    if s["bias"] is not None:
        z = z + s["bias"]
    a = s["activation"]
    if a == "swiglu":  # row 2j of the matrix is the gate of output j, row 2j + 1 its factor
        gate, up = z[:, 0::2], z[:, 1::2]
        z = gate / (1 + torch.exp(-gate)) * up
    elif a == "silu":
        z = z / (1 + torch.exp(-z))
    elif a == "gelu":
        z = 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    elif a == "gelu_tanh":
        z = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    elif a == "relu":
        z = torch.where(z < 0, 0.0, z)
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(s["out"].dtype)


# ---- in 64 bits ------------------------------------------------------------------------------------------------------

def exact(case, seed):
    """Codes stand for their values: the quotients before they are rounded."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(s, case)
    x = s["x"].double()
    sums = []
    if case["op"] == "norm":
        if s["stream"] is not None:
            x = x + s["stream"].double()
            sums = [x]
        size = case["hidden"] // case["groups"]
        power = torch.stack([x[:, g * size:(g + 1) * size].square().sum(1) / size for g in range(case["groups"])], 1)
        x = x * (power + EPS).rsqrt().repeat_interleave(size, 1) * s["gain"].double()
    scale = x.abs().max(1).values / TOP
    return [x / scale.clamp(min=1e-300)[:, None], scale] + sums


def _exact_linear(s, case):
    w = s["w"].double()
    if case["type"] == "f8":
        w *= s["w_scale"].double()[:, None]
    got = []
    for lo in range(0, case["tokens"], 1024):
        x = s["x"][lo:lo + 1024].double()
        if case["type"] == "f8":
            x = x * s["x_scale"][lo:lo + 1024, None].double()
        y = x @ w.T
        if case["bias"]:
            y += s["bias"].double()
        kind = case["activation"]
        if kind == "swiglu":
            y = y.unflatten(1, (-1, 2))
            y = y[..., 0] * torch.sigmoid(y[..., 0]) * y[..., 1]
        elif kind == "silu":
            y = y * torch.sigmoid(y)
        elif kind == "gelu":
            y = y * (1 + torch.erf(y / math.sqrt(2))) / 2
        elif kind == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        elif kind == "relu":
            y = y.clamp(min=0)
        if case["residual"]:
            y += s["residual"][lo:lo + 1024].double()
        got.append(y)
    return torch.cat(got)
