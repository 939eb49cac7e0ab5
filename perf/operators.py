"""The training operators around the blockwise-FP8 linears: what they compute and on which sizes they are timed.

Embedding lookup and its gradient, LayerNorm's two passes, RMSNorm's backward pass (the forward pass is the
library's quantizing producer), and the clipping of all gradients by their global norm.  `run` computes an
operator on what `prepare` made: with elementary torch operations, or, where `own` is set, through the
library.  `exact` computes the same from the definitions in 64 bits.

The workload sizes are the synthetic Qwen3-1.7B-like model's (hidden 2048, MLP 6144, vocabulary 151936, batches of
16384 tokens: four sequences of 4096) and the odd and ragged sizes the tests use.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}

# One transformer layer's gradients: QKV, O, gate/up and down projections, and the two norms' weights.
LAYER = [(4096, 2048), (2048, 2048), (12288, 2048), (2048, 6144), (2048,), (2048,)]


def listed():
    return [
        # a generation step of a small batch through the trained model: one id per sequence
        dict(name="embed_fwd_8", op="embed_fwd", tokens=8, vocab=151936, dim=2048, dtype="bf16", scale=1.0),
        # a training step's four sequences, with the sqrt(dim) scaling some models put on the lookup
        dict(name="embed_fwd_16384", op="embed_fwd", tokens=16384, vocab=151936, dim=2048, dtype="bf16",
             scale=45.254833995939045),
        # a small model's ragged batch, its table's gradient in the table's own type
        dict(name="embed_bwd_509", op="embed_bwd", tokens=509, vocab=1031, dim=640, dtype="bf16", grad="bf16",
             scale=1.0, padding=0),
        # a training step's whole FP32 table gradient
        dict(name="embed_bwd_16384", op="embed_bwd", tokens=16384, vocab=151936, dim=2048, dtype="bf16", grad="fp32",
             scale=1.0, padding=-1),
        # a ragged batch of a small model with an odd hidden size
        dict(name="ln_fwd_200x1283", op="ln_fwd", rows=200, cols=1283, dtype="fp32"),
        # the norm before a layer's projections, a training step's tokens
        dict(name="ln_fwd_16384x2048", op="ln_fwd", rows=16384, cols=2048, dtype="bf16"),
        # a short sequence's backward pass
        dict(name="ln_bwd_509x2048", op="ln_bwd", rows=509, cols=2048, dtype="bf16", residual=False),
        # the same norm's backward pass over a training step, joined with the residual stream's gradient
        dict(name="ln_bwd_16384x2048", op="ln_bwd", rows=16384, cols=2048, dtype="bf16", residual=True),
        # RMSNorm of FP32 rows as wide as the MLP, a ragged batch
        dict(name="rms_bwd_777x6144", op="rms_bwd", rows=777, cols=6144, dtype="fp32", residual=False),
        # the block input's RMSNorm over a training step, joined with the residual stream's gradient
        dict(name="rms_bwd_16384x2048", op="rms_bwd", rows=16384, cols=2048, dtype="bf16", residual=True),
        # a small model's gradients, odd sizes among them
        dict(name="clip_small", op="clip", sizes="640x1283,512x512,1283,509,1,384x640,200x77", dtype="bf16", most=1.0),
        # eight layers' FP32 gradients
        dict(name="clip_8_layers", op="clip", sizes=",".join("x".join(map(str, s)) for s in LAYER * 8), dtype="fp32",
             most=1.0),
    ]


def spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "ln_fwd", "ln_bwd", "rms_bwd", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "embed_fwd":
        dim = spread(rng, 64, 8192)
        dim -= dim % rng.choice([1, 8, 64])
        return dict(op=op, tokens=min(spread(rng, 1, 32768), 64000000 // dim), vocab=min(spread(rng, 500, 151936), 300000000 // dim),
                    dim=dim, dtype=dtype, scale=rng.choice([1.0, dim ** 0.5]))
    if op == "embed_bwd":
        dim = spread(rng, 64, 8192)
        dim -= dim % rng.choice([1, 8, 64])
        vocab = min(spread(rng, 500, 151936), 300000000 // dim)
        return dict(op=op, tokens=min(spread(rng, 1, 32768), 33000000 // dim), vocab=vocab, dim=dim, dtype=dtype,
                    grad=rng.choice([dtype, "fp32"]), scale=rng.choice([1.0, dim ** 0.5]), padding=rng.choice([-1, 0]))
    if op == "clip":
        count, total = rng.randint(1, 60), spread(rng, 10000, 300000000)
        parts = [rng.random() ** 3 + 1e-6 for _ in range(count)]
        sizes = [max(1, int(total * p / sum(parts))) for p in parts]
        return dict(op=op, sizes=",".join(map(str, sizes)), dtype=dtype, most=rng.choice([0.5, 1.0, 1e9]))
    cols = spread(rng, 64, 16384)
    cols -= cols % rng.choice([1, 8, 64])
    case = dict(op=op, rows=min(spread(rng, 1, 32768), 48000000 // cols), cols=cols, dtype=dtype)
    if op != "ln_fwd":
        case["residual"] = rng.random() < 0.5
    return case


def shapes(case):
    return [tuple(int(n) for n in s.split("x")) for s in case["sizes"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).add_(mean)

    state = dict(case=case)
    op = case["op"]
    if op in ("embed_fwd", "embed_bwd"):
        # token ids as texts have them: the r-th most frequent about as often as 1 / r
        u = torch.rand(case["tokens"], generator=gen, device="cuda", dtype=torch.float64)
        ids = torch.exp(u * math.log(case["vocab"] + 1.0)).floor().long().sub_(1).clamp_(0, case["vocab"] - 1)
        state["ids"] = ids
        if op == "embed_fwd":
            state["w"] = normal(case["vocab"], case["dim"], std=0.02).to(dt)
        else:
            state["dy"] = normal(case["tokens"], case["dim"], std=1e-3).to(dt)
    elif op == "clip":
        state["grads"] = [normal(*s, std=1e-3).to(dt) for s in shapes(case)]
        state["out"] = [torch.empty_like(g) for g in state["grads"]]
    else:
        rows, cols = case["rows"], case["cols"]
        x = normal(rows, cols)
        x[:, :: max(1, cols // 20)] *= 10.0  # outlier channels, as a residual stream has them
        x = x.add_(normal(rows, 1, std=0.5)).to(dt)
        state["x"] = x
        state["gamma"] = normal(cols, std=0.1, mean=1.0).to(dt)
        if op == "ln_fwd":
            state["beta"] = normal(cols, std=0.1).to(dt)
        else:
            # what the forward pass kept: the rows' statistics in FP32
            x64 = x.double()
            mean = x64.mean(1) if op == "ln_bwd" else torch.zeros(rows, device="cuda", dtype=torch.float64)
            state["mean"] = mean.float()
            state["rstd"] = torch.rsqrt((x64 - mean[:, None]).square().mean(1) + 1e-6).float()
            state["dy"] = normal(rows, cols, std=1e-3).to(dt)
            state["residual"] = normal(rows, cols, std=1e-3).to(dt) if case["residual"] else None
    return state


def run(state):
    if own:
        return run_library(state)
    case = state["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "embed_fwd":
        return {"y": (state["w"][state["ids"]].float() * case["scale"]).to(dt)}
    if op == "embed_bwd":
        ids = state["ids"]
        rows = state["dy"].float() * case["scale"] * (ids != case["padding"]).float()[:, None]
        dw = torch.zeros(case["vocab"], case["dim"], device=ids.device).index_add_(0, ids, rows)
        return {"dw": dw.to(DTYPES[case["grad"]])}
    if op == "clip":
        squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in state["grads"]])
        norm = squares.sum().sqrt()
        factor = (case["most"] / (norm + 1e-6)).clamp(max=1.0).float()
        return {"norm": norm.float(), "clipped": [(g.float() * factor).to(dt) for g in state["grads"]]}
    x, gamma = state["x"].float(), state["gamma"].float()
    if op == "ln_fwd":
        mean = x.mean(1)
        centred = x - mean[:, None]
        rstd = torch.rsqrt(centred.square().mean(1) + 1e-5)
        y = centred * rstd[:, None] * gamma + state["beta"].float()
        return {"y": y.to(dt), "mean": mean, "rstd": rstd}
    dy, rstd = state["dy"].float(), state["rstd"][:, None]
    centred = x - state["mean"][:, None] if op == "ln_bwd" else x
    xhat = centred * rstd
    dxhat = dy * gamma
    dx = dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True)
    if op == "ln_bwd":
        dx = dx - dxhat.mean(1, keepdim=True)
    dx = dx * rstd
    if state["residual"] is not None:
        dx = dx + state["residual"].float()
    grads = {"dx": dx.to(dt), "dgamma": (dy * xhat).sum(0)}
    if op == "ln_bwd":
        grads["dbeta"] = dy.sum(0)
    return grads


def run_library(state):
    import blockwise_fp8_linear_fp8bq_b200 as fp

    case = state["case"]
    op = case["op"]
    if op == "embed_fwd":
        return {"y": fp.embedding_forward(state["w"], state["ids"], scale=case["scale"])}
    if op == "embed_bwd":
        padding = case["padding"] if case["padding"] >= 0 else None
        return {"dw": fp.embedding_backward(state["dy"], state["ids"], case["vocab"], scale=case["scale"],
                                            padding_id=padding, dtype=DTYPES[case["grad"]])}
    if op == "clip":
        norm = fp.clip_grads(state["grads"], case["most"], out=state["out"])
        return {"norm": norm, "clipped": state["out"]}
    if op == "ln_fwd":
        y, mean, rstd = fp.layernorm_forward(state["x"], state["gamma"], state["beta"], eps=1e-5)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx, dgamma, dbeta = fp.layernorm_backward(state["dy"], state["x"], state["mean"], state["rstd"],
                                                  state["gamma"], dres=state["residual"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    dx, dgamma = fp.rmsnorm_backward(state["dy"], state["x"], state["rstd"], state["gamma"], dres=state["residual"])
    return {"dx": dx, "dgamma": dgamma}


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("embed_fwd", "embed_bwd"):
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        if op == "embed_fwd":
            # each distinct id's row once: at the ids' distribution, about this many of them
            bins = [math.log((r + 2.0) / (r + 1.0)) / math.log(v + 1.0) for r in range(min(v, 4096))]
            rest = max(0, v - 4096)
            tail = max(0.0, 1.0 - sum(bins))
            distinct = sum(1.0 - (1.0 - p) ** t for p in bins) + (rest * (1.0 - (1.0 - tail / rest) ** t) if rest else 0)
            return {"bytes": int(distinct * d * e + t * d * e + t * 8), "flops": t * d}
        return {"bytes": t * d * e + t * 8 + v * d * SIZE[case["grad"]], "flops": 2 * t * d}
    if op == "clip":
        n = sum(math.prod(s) for s in shapes(case))
        return {"bytes": 2 * n * e + 4, "flops": 3 * n}
    m, n = case["rows"], case["cols"]
    if op == "ln_fwd":
        return {"bytes": 2 * m * n * e + 2 * n * e + 8 * m, "flops": 8 * m * n}
    tensors = 4 if case["residual"] else 3
    params = 2 if op == "ln_bwd" else 1
    return {"bytes": tensors * m * n * e + n * e + 4 * params * (m + n), "flops": (12 if op == "ln_bwd" else 10) * m * n}


def exact(case, seed):
    """The definitions in 64 bits: sums over the axis as products with a vector of ones, the lookup's gradient as
    sums over runs of equal ids."""
    state = prepare(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        return {"y": torch.index_select(state["w"], 0, state["ids"]).double().mul_(case["scale"])}
    if op == "embed_bwd":
        order = torch.argsort(state["ids"], stable=True)
        ids, counts = torch.unique_consecutive(state["ids"][order], return_counts=True)
        sums = torch.segment_reduce(state["dy"].double()[order], "sum", lengths=counts, axis=0).mul_(case["scale"])
        sums[ids == case["padding"]] = 0.0
        dw = torch.zeros(case["vocab"], case["dim"], device="cuda", dtype=torch.float64)
        dw[ids] = sums
        return {"dw": dw}
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in state["grads"]))
        factor = min(1.0, case["most"] / (norm + 1e-6))
        return {"norm": norm, "clipped": [g.double().mul_(factor) for g in state["grads"]]}
    x, gamma = state["x"].double(), state["gamma"].double()
    ones = torch.ones(case["cols"], 1, device="cuda", dtype=torch.float64) / case["cols"]
    if op == "ln_fwd":
        mean = x @ ones
        rstd = 1.0 / torch.sqrt((x - mean).pow_(2) @ ones + 1e-5)
        return {"y": torch.addcmul(state["beta"].double(), (x - mean) * rstd, gamma), "mean": mean[:, 0],
                "rstd": rstd[:, 0]}
    dy, rstd, mean = state["dy"].double(), state["rstd"].double()[:, None], state["mean"].double()[:, None]
    h = (x - mean) * rstd
    g = dy * gamma
    inner = g if op == "rms_bwd" else g - g @ ones
    dx = rstd * (inner - h * ((g * h) @ ones))
    if state["residual"] is not None:
        dx += state["residual"].double()
    rows = torch.ones(1, case["rows"], device="cuda", dtype=torch.float64)
    grads = {"dx": dx, "dgamma": (rows @ (dy * h))[0]}
    if op == "ln_bwd":
        grads["dbeta"] = (rows @ dy)[0]
    return grads
