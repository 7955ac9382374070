"""The 8-bit operators as they are measured: cases, inputs, plain forms, exact values.

Four operators of a W8A8 transformer layer:

* ``norm``     RMS norm of x (+ residual), output in 8 bits with one scale per token;
* ``tokens``   x / s in 8 bits with one scale per token;
* ``weights``  W * s in 8 bits with one scale per row (output channel);
* ``gemm``     Y = X W^T of 8-bit integers, rescaled per token and per channel.

The 8-bit values are whole numbers in [-127, 127] and are returned as such: the operators'
definition fixes every fp32 rounding that decides them, so both sides have to agree exactly.
"""
import math

import torch

own = False

EPS = 1e-5
TINY = 2.0 ** -100  # a row whose largest magnitude is below this counts as zero
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one token of a decoding step, 7B-shaped layer: latency
        {"name": "norm 1x4096 bf16 residual", "op": "norm", "rows": 1, "d": 4096, "type": "bf16", "residual": True, "scales": True},
        # a small ragged batch with an fp32 residual stream, the first norm (nothing to add yet)
        {"name": "norm 77x2048 f32", "op": "norm", "rows": 77, "d": 2048, "type": "f32", "residual": False, "scales": False},
        # a batch of prompts, 13B-shaped layer
        {"name": "norm 8192x5120 bf16 residual", "op": "norm", "rows": 8192, "d": 5120, "type": "bf16", "residual": True, "scales": True},
        # input of the MLP's down projection: 16 sequences decoding, no channel scales
        {"name": "tokens 16x11008 bf16", "op": "tokens", "rows": 16, "d": 11008, "type": "bf16", "scales": False},
        # the same for a ragged prompt batch of a 13B-shaped layer
        {"name": "tokens 4001x13824 bf16 scales", "op": "tokens", "rows": 4001, "d": 13824, "type": "bf16", "scales": True},
        # encoding an attention projection, and a down projection kept in fp32
        {"name": "weights 4096x4096 bf16 scales", "op": "weights", "rows": 4096, "d": 4096, "type": "bf16", "scales": True},
        {"name": "weights 4096x11008 f32 scales", "op": "weights", "rows": 4096, "d": 11008, "type": "f32", "scales": True},
        # decoding one sequence: an attention projection
        {"name": "gemm 1x4096 to 4096", "op": "gemm", "rows": 1, "d": 4096, "out": 4096, "type": "bf16"},
        # the output head over an odd vocabulary for five sequences, logits in fp32
        {"name": "gemm 5x4096 to 32001 f32", "op": "gemm", "rows": 5, "d": 4096, "out": 32001, "type": "f32"},
        # a large decoding batch through the down projection
        {"name": "gemm 100x11008 to 4096", "op": "gemm", "rows": 100, "d": 11008, "out": 4096, "type": "bf16"},
        # one ragged prompt through a 13B-shaped gate projection
        {"name": "gemm 777x5120 to 13824", "op": "gemm", "rows": 777, "d": 5120, "out": 13824, "type": "bf16"},
        # a batch of prompts through a 7B-shaped gate projection
        {"name": "gemm 8192x4096 to 11008", "op": "gemm", "rows": 8192, "d": 4096, "out": 11008, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "tokens", "weights", "gemm", "gemm"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "gemm":
        d, out = 64 * _log(rng, 1, 216), _log(rng, 1, 33000)
        most = 8192 * 4096 * 11008 // (d * out)
        return {"op": op, "rows": _log(rng, 1, max(1, min(8192, most))), "d": d, "out": out, "type": kind}
    d = 64 * _log(rng, 1, 512)
    rows = _log(rng, 1, max(1, min(20000, 8192 * 5120 // d)))
    case = {"op": op, "rows": rows, "d": d, "type": kind, "scales": rng.random() < 0.6}
    if op == "norm":
        case["residual"] = rng.random() < 0.7
    return case


def _heavy(rows, cols, scale, g):
    """Student-t (5 degrees of freedom) times `scale`: trained weights' heavy tails."""
    z = torch.randn((6, rows, cols), generator=g, device="cuda")
    return z[0] * z[1:].square_().mean(0).rsqrt_().mul_(scale)


def _activations(rows, cols, g):
    """N(0, 1) with 1% outlier channels x20; the last token of a batch of eight or more is padding (zeros)."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    if rows >= 8:
        x[-1] = 0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rows, d, t = case["rows"], case["d"], TYPES[case["type"]]
    s = {"op": case["op"], "type": t}
    if case["op"] == "gemm":
        s["xq"], s["x_scale"] = _quantise(_activations(rows, d, g))
        s["wq"], s["w_scale"] = _quantise(_heavy(case["out"], d, 0.02, g))
        return s
    s["x"] = (_heavy(rows, d, 0.02, g) if case["op"] == "weights" else _activations(rows, d, g)).to(t)
    s["scale"] = None
    if case["scales"]:  # lognormal activation statistics to the power 1/2, in binary16
        s["scale"] = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda")).to(torch.float16)
    if case["op"] == "norm":
        s["gain"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(t)
        s["residual"] = _activations(rows, d, g).mul_(2).to(t) if case["residual"] else None
    return s


def _quantise(v):
    """q and the largest magnitude over 127 of each row of v (fp32, one rounding a step)."""
    a = v.abs().amax(-1, keepdim=True)
    inv = torch.where(a >= TINY, torch.full_like(a, 127.0) / a, torch.zeros_like(a))
    scale = torch.where(a >= TINY, a / torch.full_like(a, 127.0), torch.zeros_like(a))
    return (v * inv).round().to(torch.int8), scale.squeeze(-1)


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "gemm":
        acc = state["xq"].float() @ state["wq"].float().t()
        return (acc * state["x_scale"][:, None] * state["w_scale"][None, :]).to(state["type"])
    x, s = state["x"].float(), state["scale"]
    if op == "weights":
        return _quantise(x if s is None else x * s.float())
    one = torch.ones(x.shape[1], device=x.device)
    if op == "tokens":
        return _quantise(x if s is None else x * (one / s.float()))
    added = state["residual"] is not None
    h = (x + state["residual"].float()).to(state["type"]) if added else state["x"]
    c = state["gain"].float()
    if s is not None:
        c = c / s.float()
    q, scale = _quantise(h.float() * c)
    rstd = 1 / torch.sqrt(h.float().square().mean(-1) + EPS)
    return (h, q, scale * rstd) if added else (q, scale * rstd)


def _own(state):
    from vector_quantization_codec_b200 import qamw
    op = state["op"]
    if op == "gemm":
        return qamw.qamw_int8_gemm(state["xq"], state["x_scale"], state["wq"], state["w_scale"], dtype=state["type"])
    if op == "weights":
        return qamw.qamw_int8_encode_weights(state["x"], state["scale"])
    if op == "tokens":
        return qamw.qamw_int8_encode_tokens(state["x"], state["scale"])
    return qamw.qamw_rmsnorm_int8(state["x"], state["gain"], EPS, residual=state["residual"], chan_scale=state["scale"])


def work(case):
    rows, d, b = case["rows"], case["d"], SIZE[case["type"]]
    if case["op"] == "gemm":
        n = case["out"]
        return {"bytes": rows * d + n * d + 4 * (rows + n) + b * rows * n, "flops": 2 * rows * d * n}
    n, columns = rows * d, (2 * d if case["scales"] else 0)
    if case["op"] == "norm":
        streams = b * (3 if case["residual"] else 1) + 1
        return {"bytes": n * streams + 4 * rows + b * d + columns, "flops": 7 * n}
    return {"bytes": n * (b + 1) + 4 * rows + columns, "flops": 4 * n}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "gemm":
        y = torch.empty((case["rows"], case["out"]), dtype=torch.float64, device="cuda")
        w = state["wq"].double() * state["w_scale"].double()[:, None]
        for i in range(0, case["rows"], 1024):
            x = state["xq"][i:i + 1024].double() * state["x_scale"][i:i + 1024].double()[:, None]
            torch.matmul(x, w.T, out=y[i:i + 1024])
        return y
    x = state["x"].double()
    s = 1.0 if state["scale"] is None else state["scale"].double()
    if case["op"] == "norm":
        h = x
        if state["residual"] is not None:
            h = (x + state["residual"].double()).to(state["type"]).double()  # the stream keeps its type
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * state["gain"].double() / s
    else:
        y = x * s if case["op"] == "weights" else x / s
    largest = y.abs().max(1).values
    unit = torch.where(largest > 0, largest / 127, 1.0)
    q = torch.round(y / unit[:, None]).to(torch.int8)
    if case["op"] == "norm" and state["residual"] is not None:
        return h, q, largest / 127
    return q, largest / 127
