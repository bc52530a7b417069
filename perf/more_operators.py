"""The dense operators of a decoder block: what is measured, and their plain forms.

What stands between attention and the routed experts in serving:

  norm     the residual stream takes up a block's output (normed or not, gated, scaled) and is normed for the next
           block in the same pass; or the heads of queries and keys are normed by themselves
  linear   rows quantized to 8-bit floating point with a power of two for each block of 128, times weights held so
  block    both in a row: the normed stream goes into the product as 8-bit rows

`run` with own = False computes them by elementary torch operations in 32 bits (the norm before a quantization in 64:
a value next to a border would round to the other side); with own = True it calls the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 128    # values that share a scale
MOST = 448.0   # the largest e4m3 value
EPS = 1e-6


# --------------------------------------------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decoded token between attention and the experts: latency
        dict(name="norm_token", op="norm", dtype="bf16", tokens=1, heads=1, dim=4096, block=True, post=True, gate="none", scale=1.0),
        # the streams of a decode batch in a wide model, a gate for each channel
        dict(name="norm_batch", op="norm", dtype="fp16", tokens=200, heads=1, dim=7168, block=True, post=True, gate="channel", scale=1.0),
        # queries and keys of a prefill batch, each head by itself, out of the rows of one product
        dict(name="norm_heads", op="norm", dtype="bf16", tokens=3001, heads=40, dim=128, block=False, post=False, gate="none", scale=1.0),
        # an odd width, the block's output added as it is behind a gate for each element
        dict(name="norm_odd", op="norm", dtype="fp16", tokens=777, heads=1, dim=2184, block=True, post=False, gate="element", scale=0.22),
        # a large prefill batch, a gate for each token
        dict(name="norm_prefill", op="norm", dtype="bf16", tokens=16384, heads=1, dim=4096, block=True, post=True, gate="token", scale=0.5),
        # queries, keys and values of one decoded token: latency
        dict(name="linear_token", op="linear", dtype="bf16", out="bf16", tokens=1, n=5120, k=4096),
        # drafted tokens through a projection back to the stream
        dict(name="linear_drafts", op="linear", dtype="fp16", out="fp16", tokens=19, n=4096, k=11008),
        # logits of a decode batch over an odd vocabulary
        dict(name="linear_logits", op="linear", dtype="bf16", out="fp32", tokens=32, n=100003, k=4096),
        # a ragged batch through a small projection, nothing of it a multiple of 128
        dict(name="linear_odd", op="linear", dtype="bf16", out="bf16", tokens=333, n=1000, k=2064),
        # a long prompt through a wide projection
        dict(name="linear_prefill", op="linear", dtype="bf16", out="bf16", tokens=8192, n=10240, k=4096),
        # the end of one block and the start of the next for a decode batch
        dict(name="block_decode", op="block", dtype="bf16", out="bf16", tokens=16, dim=4096, n=6144, post=True, gate="none", scale=1.0),
        # the same for a prefill batch
        dict(name="block_prefill", op="block", dtype="bf16", out="bf16", tokens=4001, dim=5120, n=5120, post=True, gate="channel", scale=0.5),
    ]


MOST_VALUES = 16384 * 4096             # of a norm
MOST_PRODUCTS = 8192 * 10240 * 4096    # of a product
MOST_WEIGHTS = 100003 * 4096


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "block"])
    dtype = rng.choice(["bf16", "fp16"])
    blocks = dict(post=rng.random() < 0.6, gate=rng.choice(["none", "token", "channel", "element"]), scale=rng.choice([1.0, 0.5, 0.22]))
    if op == "norm" and rng.random() < 0.3:
        heads, dim = rng.choice([5, 8, 12, 40]), rng.choice([64, 80, 128])
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, MOST_VALUES // (heads * dim) // 2), heads=heads, dim=dim, block=False, post=False,
                    gate="none", scale=1.0)
    if op == "norm":
        dim = 8 * _log(rng, 16, 1536)
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, min(16384, MOST_VALUES // dim)), heads=1, dim=dim, block=True, **blocks)
    k = 16 * _log(rng, 8, 1024)
    n = _log(rng, 64, min(32768, MOST_WEIGHTS // k))
    tokens = _log(rng, 1, min(8192, MOST_PRODUCTS // (n * k)))
    if op == "linear":
        return dict(op=op, dtype=dtype, out=rng.choice([dtype, dtype, "fp32"]), tokens=tokens, n=n, k=k)
    return dict(op=op, dtype=dtype, out=dtype, tokens=tokens, dim=min(k, 12288), n=n, **blocks)


# --------------------------------------------------------------------------------------------------------------
# the inputs
# --------------------------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g):
    return torch.randn(shape, device="cuda", generator=g, dtype=torch.float32)


def _activations(rows, dim, dtype, g):
    """Normal values, a few channels far larger than the others."""
    x = _normal((rows, dim), g)
    return (x * torch.exp(1.5 * _normal((dim,), g).clamp_min(0.0))).to(DTYPES[dtype])


def _weights(case, k, g):
    """8-bit weights [n, k] as a program holds them: codes, and the scales' exponents + 127, four of them at least in a row."""
    codes, scales = _quantized(_normal((case["n"], k), g) * k ** -0.5)
    exponents = (torch.frexp(scales).exponent + 126).to(torch.uint8)
    held = torch.full((case["n"], 4 * -(-exponents.shape[1] // 4)), 127, dtype=torch.uint8, device="cuda")
    held[:, :exponents.shape[1]] = exponents
    return codes.to(torch.float8_e4m3fn), held


def prepare(case, seed):
    g, dtype = _generator(seed), DTYPES[case["dtype"]]
    t = case["tokens"]
    s = dict(case=case)
    if case["op"] in ("norm", "block"):
        h, d = case.get("heads", 1), case["dim"]
        if h > 1:  # the first heads of wider rows: the last four hold what is not normed
            s["x"] = _normal((t, h + 4, d), g).to(dtype)[:, :h]
        else:
            s["x"] = _activations(t, d, case["dtype"], g)[:, None]
        if case.get("block", True):
            s["block"] = (0.3 * _normal((t, h, d), g)).to(dtype)
        shape = {"none": None, "token": (t, h, 1), "channel": (1, 1, d), "element": (t, h, d)}[case["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(_normal(shape, g)).to(dtype)
        s["pre_weight"] = 1 + 0.2 * _normal((d,), g)
        s["post_weight"] = 1 + 0.2 * _normal((d,), g) if case["post"] else None
        if case.get("block", True):
            s["y"] = torch.empty((t, h, d), dtype=dtype, device="cuda")
        if case["op"] == "norm":
            s["normed"] = torch.empty((t, h, d), dtype=dtype, device="cuda")
    if case["op"] in ("linear", "block"):
        k = case["k"] if case["op"] == "linear" else case["dim"]
        s["codes"], s["scales"] = _weights(case, k, g)
        s["out"] = torch.empty((t, case["n"]), dtype=DTYPES[case["out"]], device="cuda")
        if case["op"] == "linear":
            s["x"] = _activations(t, k, case["dtype"], g)
    return s


# --------------------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "block": _own_block}[op](s)
    return {"norm": _plain_norm, "linear": _plain_linear, "block": _plain_block}[op](s)


def _own_residual(s, **outputs):
    from nvfp4_block_scaled_gather_gb300 import dense as D
    c = s["case"]
    if not c.get("block", True):
        D.moe_residual_norm(s["x"], normed=s["normed"], pre_weight=s["pre_weight"], eps=EPS)
        return
    D.moe_residual_norm(s["x"], s["block"], y=s["y"], pre_weight=s["pre_weight"], post_norm=c["post"], post_weight=s["post_weight"],
                        gate=s["gate"], residual_scale=c["scale"], eps=EPS, **outputs)


def _own_norm(s):
    _own_residual(s, normed=s["normed"])
    return {n: s[n] for n in ("y", "normed") if n in s}


def _handle(s):
    """The handle that a program keeps over its weights."""
    if "weights" not in s:
        from nvfp4_block_scaled_gather_gb300 import dense as D
        s["weights"] = D.Fp8Rows(s["codes"], s["scales"])
    return s["weights"]


def _own_linear(s):
    from nvfp4_block_scaled_gather_gb300 import dense as D
    w = _handle(s)
    if "workspace" not in s:
        s["workspace"] = D.linear_workspace(s["x"].shape[0], s["x"].shape[1])
    D.moe_fp8_linear(s["x"], w, s["out"], s["workspace"])
    return {"out": s["out"]}


def _own_block(s):
    from nvfp4_block_scaled_gather_gb300 import dense as D
    w = _handle(s)
    if "rows" not in s:
        s["rows"] = D.Fp8Rows.empty(s["x"].shape[0], s["x"].shape[2])
    _own_residual(s, quantized=s["rows"])
    D.moe_fp8_gemm(s["rows"], w, s["out"])
    return {"y": s["y"], "out": s["out"]}


# --------------------------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------------------------

def _plain_residual(s, to):
    """The stream after the block and its norm, in the type `to`."""
    c = s["case"]

    def norm(v, w):
        v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        return v if w is None else v * w.to(to)

    y = s["x"].to(to)
    if "block" in s:
        b = s["block"].to(to)
        if c["post"]:
            b = norm(b, s["post_weight"])
        if s["gate"] is not None:
            b = b * s["gate"].to(to)
        y = y + c["scale"] * b
    return y, norm(y, s["pre_weight"])


def _plain_norm(s):
    y, normed = _plain_residual(s, torch.float32)
    out = {"normed": normed.to(s["x"].dtype)}
    return {"y": y.to(s["x"].dtype), **out} if "block" in s else out


def _quantized(x):
    """Rows as e4m3 values [rows, k] and the scale of each block of 128 [rows, blocks], both in 32 bits: the smallest
    power of two (2^-127 at least) with which the block's largest value is at most 448."""
    rows, k = x.shape
    padded = torch.nn.functional.pad(x, (0, -k % BLOCK)).reshape(rows, -1, BLOCK)
    most, exponent = torch.frexp(padded.abs().amax(-1).float())
    exponent = (exponent - 9 + (most > 0.875).int()).clamp_min(-127)
    exponent = torch.where(most == 0, torch.full_like(exponent, -127), exponent)
    scale = torch.ldexp(torch.ones_like(most), exponent)
    codes = (padded / scale[..., None]).to(torch.float8_e4m3fn).float()
    return codes.reshape(rows, -1)[:, :k], scale


def _times_weights(s, rows, scale):
    """Dequantized rows times dequantized weights."""
    k = s["codes"].shape[1]

    def wide(values, scales):
        return values * scales.repeat_interleave(BLOCK, dim=1)[:, :k]

    weights = wide(s["codes"].float(), torch.ldexp(torch.ones((), device="cuda"), s["scales"].int() - 127))
    return (wide(rows, scale) @ weights.T).to(s["out"].dtype)


def _plain_linear(s):
    return {"out": _times_weights(s, *_quantized(s["x"].float()))}


def _plain_block(s):
    y, normed = _plain_residual(s, torch.float64)
    return {"y": y.to(s["x"].dtype), "out": _times_weights(s, *_quantized(normed[:, 0]))}


# --------------------------------------------------------------------------------------------------------------
# the definition in 64 bits, and the work
# --------------------------------------------------------------------------------------------------------------

def _root_mean_square(v):
    return torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS)


def _exact_residual(s):
    c = s["case"]
    y = s["x"].double()
    if "block" in s:
        add = s["block"].double()
        if c["post"]:
            add = add / _root_mean_square(add) * s["post_weight"].double()
        if s["gate"] is not None:
            add = add * s["gate"].double()
        y = y + add * c["scale"]
    return y, y / _root_mean_square(y) * s["pre_weight"].double()


def _exact_blocks(x):
    """x [rows, k] in 64 bits, as the e4m3 values times their block's scale that stand for it."""
    rows, k = x.shape
    out = torch.empty_like(x)
    for at in range(0, k, BLOCK):
        v = x[:, at:at + BLOCK]
        scale = torch.exp2(torch.ceil(torch.log2(v.abs().amax(1, keepdim=True) / MOST)).clamp(-127, 127))
        scale = torch.where(v.abs().amax(1, keepdim=True) > MOST * scale, 2 * scale, scale)              # (a logarithm next
        scale = torch.where(v.abs().amax(1, keepdim=True) <= MOST * scale / 2, (scale / 2).clamp_min(2.0 ** -127), scale)  # to a border)
        v = v / scale
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)  # normal values have three bits behind the first
        out[:, at:at + BLOCK] = torch.round(v / step) * step * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        y, normed = _exact_residual(s)
        return {"y": y, "normed": normed} if "block" in s else {"normed": normed}
    k = s["codes"].shape[1]
    power = torch.exp2(s["scales"].double() - 127)
    found = {}
    if case["op"] == "linear":
        rows = s["x"].double()
    else:
        found["y"], rows = _exact_residual(s)
        rows = rows[:, 0]
    rows = _exact_blocks(rows)
    out = torch.zeros((rows.shape[0], case["n"]), dtype=torch.float64, device="cuda")
    for at in range(0, k, 16 * BLOCK):  # (the weights in 64 bits would be large)
        part = s["codes"][:, at:at + 16 * BLOCK].to(torch.float32).double()
        part *= power[:, at // BLOCK:at // BLOCK + 16].repeat_interleave(BLOCK, dim=1)[:, :part.shape[1]]
        out += rows[:, at:at + 16 * BLOCK] @ part.T
    return {**found, "out": out}


def work(case):
    t, held = case["tokens"], 4 if case.get("out") == "fp32" else 2
    moved = flops = 0
    if case["op"] in ("norm", "block"):
        h, d = case.get("heads", 1), case["dim"]
        values = t * h * d
        gates = {"none": 0, "token": t * h, "channel": d, "element": values}[case["gate"]]
        reads = values * (2 if case.get("block", True) else 1)
        writes = values * ((1 if case["op"] == "norm" else 0) + (1 if case.get("block", True) else 0))
        moved += 2 * (reads + writes + gates) + 4 * d * (2 if case["post"] else 1)
        flops += 12 * values
    if case["op"] in ("linear", "block"):
        n, k = case["n"], case["k"] if case["op"] == "linear" else case["dim"]
        moved += n * (k + -(-k // BLOCK)) + t * n * held + (2 * t * k if case["op"] == "linear" else 0)
        flops += 2 * t * n * k
    return {"bytes": moved, "flops": flops}
