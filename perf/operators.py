"""Cases of the gradient-clipping operators: the global gradient norm over many
tensors, clipping them in place, the reduce that yields the norm of the shard
it writes, and the AdamW step that applies the clip.

Where `own` is false, run() is the plain form, elementary torch operations;
where it is true, run() makes the library's calls on the same state.  exact()
is the operators' definition in 64 bits.

With total = the sum of squares of all gradients (norm "2") or their largest
magnitude (norm "inf"):
    norm    = sqrt(total), or total
    coef    = min(1, max_norm / (norm + 1e-6)), rounded to fp32
    clip    : g <- g * coef
    reduce  : out = (sum of the A*N slices) / N, and out's total and norm
    adamw   : the AdamW update with g * coef as the gradient
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1   # the optimizer's settings in every case
NORM_EPS = 1e-6


# ------------------------------------------------------------------ sizes --

def _block(d, f):
    """A Llama-like block's parameter shapes: q, k, v, o, gate, up, down, two norms."""
    return [(d, d)] * 4 + [(f, d)] * 2 + [(d, f)] + [(d,)] * 2


def _sizes(case):
    """Element counts of one rank's local tensors (the dim-0 chunk of each parameter)."""
    kind, world = case["layout"], case["world"]
    if kind == "mlp":        # W_in, W_out, bias, norm
        shapes = [(64, 256), (256, 64), (256,), (64,)]
    elif kind == "llama":    # `layers` blocks, and the embedding and head where there is a vocabulary
        shapes = [(case["vocab"], case["dim"])] * (2 if case["vocab"] else 0) + _block(case["dim"], case["ffn"]) * case["layers"]
    else:                    # "spread": `count` parameters, their counts spread evenly over the logarithm up to `most`
        u = torch.rand(case["count"], generator=torch.Generator().manual_seed(case["count"]), dtype=F64)
        return [max(1, int(v)) for v in torch.exp(u * math.log(case["most"])).tolist()]
    return [-(-s[0] // world) * math.prod(s[1:]) for s in shapes]


def listed():
    """Sizes: the tiny 2-layer MLP on 4 ranks; one 7B block, and the whole 7B model's shard (842,301,440
    elements), on 8; 97 parameters of 1 to 4M elements, whose starts fall on any element."""
    llama7 = {"layout": "llama", "dim": 4096, "ffn": 11008, "world": 8}
    return [
        # the norm of a small model's shard: all launch latency
        {"name": "norm_mlp", "op": "norm", "layout": "mlp", "world": 4, "dtype": "fp32", "norm": "2"},
        # one block's bf16 gradients, as a per-group norm reads them
        {"name": "norm_block_bf16", "op": "norm", **llama7, "layers": 1, "vocab": 0, "dtype": "bf16", "norm": "2"},
        # largest magnitude over many odd parameters, matrices in bf16 beside fp32 ones
        {"name": "norm_spread_inf", "op": "norm", "layout": "spread", "count": 97, "most": 4194304, "world": 1, "dtype": "mixed", "norm": "inf"},
        # the whole model's fp32 gradient shard, one tensor per parameter
        {"name": "norm_model", "op": "norm", **llama7, "layers": 32, "vocab": 32000, "dtype": "fp32", "norm": "2"},
        # clipping many odd parameters of both types in place
        {"name": "clip_spread_mixed", "op": "clip", "layout": "spread", "count": 97, "most": 4194304, "world": 1, "dtype": "mixed", "norm": "2"},
        # clipping the whole model's fp32 gradient shard in place
        {"name": "clip_model", "op": "clip", **llama7, "layers": 32, "vocab": 32000, "dtype": "fp32", "norm": "2"},
        # a small model's reduce, 4 ranks, one micro-step: latency
        {"name": "reduce_mlp", "op": "reduce", "n": 8272, "world": 4, "acc": 1, "norm": "2"},
        # one block's reduce, 8 ranks, one micro-step
        {"name": "reduce_block", "op": "reduce", "n": 25297920, "world": 8, "acc": 1, "norm": "2"},
        # three blocks and an odd tail, 8 ranks, 4 micro-steps: 32 slices
        {"name": "reduce_acc_inf", "op": "reduce", "n": 75893763, "world": 8, "acc": 4, "norm": "inf"},
        # a small model's optimizer step: latency
        {"name": "adamw_mlp", "op": "adamw", "n": 8272, "dtype": "fp32", "norm": "2"},
        # the 97 parameters' flat shard on 8 ranks, gradients still in bf16
        {"name": "adamw_spread_bf16", "op": "adamw", "n": 2680548, "dtype": "bf16", "norm": "inf"},
        # the whole model's shard
        {"name": "adamw_model", "op": "adamw", "n": 842301440, "dtype": "fp32", "norm": "2"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, norm = rng.choice(["norm", "clip", "reduce", "adamw"]), rng.choice(["2", "2", "inf"])
    if op == "adamw":
        return {"op": op, "n": _log(rng, 1000, 400_000_000), "dtype": rng.choice(["fp32", "fp32", "bf16"]), "norm": norm}
    if op == "reduce":
        world, acc = rng.choice([2, 4, 8, 16]), rng.choice([1, 2, 3, 4])
        return {"op": op, "n": _log(rng, 5000, 1_600_000_000 // (world * acc)), "world": world, "acc": acc, "norm": norm}
    dtype = rng.choice(["fp32", "bf16", "mixed"])
    if rng.random() < 0.5:
        return {"op": op, "layout": "spread", "count": _log(rng, 1, 300), "most": _log(rng, 1000, 16_000_000), "world": 1, "dtype": dtype, "norm": norm}
    dim = 128 * rng.randint(1, 32)
    return {"op": op, "layout": "llama", "dim": dim, "ffn": 32 * (dim // 12) + 32, "layers": rng.randint(1, 16), "vocab": rng.choice([0, 32000]),
            "world": rng.choice([2, 3, 8]), "dtype": dtype, "norm": norm}


# ------------------------------------------------------------------ state --

def _grad(gen, n, dtype):
    """Gradients: normal, 1e-3, one in a thousand 30 times as large."""
    g = torch.randn(n, generator=gen, device="cuda", dtype=F32).mul_(1e-3)
    at = torch.randint(0, n, (n // 1000 + 1,), generator=gen, device="cuda")
    g[at] = g[at] * 30
    return g.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"op": case["op"], "norm_type": case["norm"], "total": torch.empty(1, dtype=F64, device="cuda"),
             "norm": torch.empty(1, dtype=F32, device="cuda"), "max_norm": 1.0}
    # clipping reads the total that all ranks' shards gave, a little over the limit: a step is scaled by 0.98 to 0.995
    over = 1.005 + 0.015 * float(torch.rand(1, generator=torch.Generator().manual_seed(seed), dtype=F64))
    if case["op"] in ("clip", "adamw"):
        state["total"].fill_(over if case["norm"] == "inf" else over * over)
    if case["op"] in ("norm", "clip"):
        # one rank's gradients, as a sharded engine holds them: one flat buffer (one for each type), and each parameter's view of it
        sizes = _sizes(case)
        of = [BF16 if case["dtype"] == "bf16" or (case["dtype"] == "mixed" and i % 3) else F32 for i in range(len(sizes))]
        state["flats"], views = [], [None] * len(sizes)
        for t in (F32, BF16):
            mine = [i for i in range(len(sizes)) if of[i] == t]
            if mine:
                flat = _grad(gen, sum(sizes[i] for i in mine), t)
                state["flats"].append(flat)
                for i, v in zip(mine, torch.split(flat, [sizes[i] for i in mine])):
                    views[i] = v
        if own:   # the handle that a program keeps for its gradient tensors
            import fsdp_sharded_state_amd as fs
            state["grads"] = fs.fs_grad_list(views)
    elif case["op"] == "reduce":
        n, terms = case["n"], case["world"] * case["acc"]
        pitch = -(-n // 8) * 8   # every slice starts on 16 bytes
        state["slices"] = torch.empty(terms, pitch, dtype=BF16, device="cuda")
        for k in range(terms):
            state["slices"][k, :n] = _grad(gen, n, BF16)
        state["slices"] = state["slices"][:, :n]
        state["out"] = torch.empty(n, dtype=F32, device="cuda")
        state["world"], state["acc"] = case["world"], case["acc"]
        if own:
            import fsdp_sharded_state_amd as fs
            state["grads"] = fs.fs_grad_list(list(state["slices"]))
    else:
        n = case["n"]
        state["grad"] = _grad(gen, n, F32 if case["dtype"] == "fp32" else BF16)
        state["master"] = torch.randn(n, generator=gen, device="cuda").mul_(0.02)
        state["m"] = torch.randn(n, generator=gen, device="cuda").mul_(1e-3)
        state["v"] = torch.randn(n, generator=gen, device="cuda").mul_(1e-3).square_()
        state["p16"] = torch.empty(n, dtype=BF16, device="cuda")
        state["step"] = 1000
    return state


# -------------------------------------------------------------- plain form --

# the settings as the boundary takes them, in fp32
LR32, BETA1_32, BETA2_32, EPS32, DECAY32, NORM_EPS32 = torch.tensor([LR, BETA1, BETA2, EPS, DECAY, NORM_EPS], dtype=F32).tolist()


def _coef(state):
    norm = state["total"] if state["norm_type"] == "inf" else state["total"].sqrt()
    return norm, (state["max_norm"] / (norm + NORM_EPS32)).clamp(max=1.0).to(F32)


def _measure(state, flats):
    """The total of the flats' elements, in 64 bits, and its norm."""
    if state["norm_type"] == "inf":
        parts = [f.abs().max().to(F64) for f in flats]
        state["total"].copy_(parts[0] if len(parts) == 1 else torch.maximum(*parts))
        state["norm"].copy_(state["total"])
    else:
        parts = [f.to(F64).square_().sum() for f in flats]
        state["total"].copy_(parts[0] if len(parts) == 1 else parts[0] + parts[1])
        state["norm"].copy_(state["total"].sqrt())


def _norm(state):
    _measure(state, state["flats"])
    return state["total"], state["norm"]


def _clip(state):
    norm, coef = _coef(state)
    state["norm"].copy_(norm)
    for flat in state["flats"]:   # one buffer for each type
        flat.copy_(flat.to(F32) * coef)
    return state["flats"], state["norm"]


def _reduce(state):
    state["out"].copy_(state["slices"].to(F32).sum(0) / state["world"])
    _measure(state, [state["out"]])
    return state["out"], state["total"], state["norm"]


def _adamw(state):
    lr, b1, b2, eps, wd = LR32, BETA1_32, BETA2_32, EPS32, DECAY32
    g = state["grad"].to(F32) * _coef(state)[1]
    th, m, v, t = state["master"], state["m"], state["v"], state["step"]
    m.mul_(b1).add_(g * (1 - b1))
    v.mul_(b2).add_(g * g * (1 - b2))
    den = (v / (1 - b2 ** t)).sqrt() + eps
    th.mul_(1 - lr * wd).sub_(m / (1 - b1 ** t) / den * lr)
    state["p16"].copy_(th)
    return th, m, v, state["p16"]


# --------------------------------------------------------- library's calls --

def _own(state):
    import fsdp_sharded_state_amd as fs
    op, kind = state["op"], state["norm_type"]
    if op == "norm":
        fs.fs_grad_norm(state["grads"], state["total"], state["norm"], norm_type=kind)
        return state["total"], state["norm"]
    if op == "clip":
        fs.fs_clip_grads(state["grads"], state["total"], state["max_norm"], state["norm"], norm_type=kind, norm_eps=NORM_EPS)
        return state["flats"], state["norm"]
    if op == "reduce":
        fs.fs_reduce_shard_norm(state["grads"], state["out"], state["total"], state["norm"], world=state["world"], grad_acc=state["acc"], norm_type=kind)
        return state["out"], state["total"], state["norm"]
    fs.fs_adamw_step_clip(state["master"], state["m"], state["v"], state["grad"], state["p16"], total=state["total"], max_norm=state["max_norm"],
                          norm_type=kind, norm_eps=NORM_EPS, lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, step=state["step"])
    return state["master"], state["m"], state["v"], state["p16"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "clip": _clip, "reduce": _reduce, "adamw": _adamw}[state["op"]](state)


# ------------------------------------------------------------- definitions --

def _total64(norm_type, xs):
    """Sum of squares, or largest magnitude, of 64-bit values, in pieces of 16M."""
    pieces = [p for x in xs for p in torch.split(x, 1 << 24)]
    if norm_type == "inf":
        return torch.stack([p.double().abs().amax() for p in pieces]).amax().reshape(1)
    return torch.stack([torch.dot(p.double(), p.double()) for p in pieces]).sum().reshape(1)


def exact(case, seed):
    s = prepare(case, seed)
    root = (lambda t: t) if case["norm"] == "inf" else torch.sqrt
    if case["op"] == "norm":
        total = _total64(case["norm"], s["flats"])
        return total, root(total)
    if case["op"] == "reduce":
        mean = torch.zeros(case["n"], dtype=F64, device="cuda")
        for k in range(s["slices"].shape[0]):
            mean += s["slices"][k]
        mean /= case["world"]
        total = _total64(case["norm"], [mean])
        return mean, total, root(total)
    norm = float(root(s["total"]))
    scale = min(1.0, s["max_norm"] / (norm + NORM_EPS))
    if case["op"] == "clip":
        return [f.double() * scale for f in s["flats"]], root(s["total"])
    lr, b1, b2, eps, wd = torch.tensor([LR, BETA1, BETA2, EPS, DECAY], dtype=F32).double().tolist()
    g = s["grad"].double() * scale
    m = b1 * s["m"].double() + (1 - b1) * g
    v = b2 * s["v"].double() + (1 - b2) * g ** 2
    del g
    step = lr * (m / (1 - b1 ** s["step"])) / (torch.sqrt(v / (1 - b2 ** s["step"])) + eps)
    theta = s["master"].double() * (1 - lr * wd) - step
    return theta, m, v, theta


def work(case):
    """Each gradient, slice and state element read once, each result written once."""
    if case["op"] in ("norm", "clip"):
        sizes = _sizes(case)
        size = sum(n * (2 if case["dtype"] == "bf16" or (case["dtype"] == "mixed" and i % 3) else 4) for i, n in enumerate(sizes))
        return {"bytes": size * (2 if case["op"] == "clip" else 1) + 12, "flops": sum(sizes) * (1 if case["op"] == "clip" else 2)}
    if case["op"] == "reduce":
        terms = case["world"] * case["acc"]
        return {"bytes": case["n"] * (2 * terms + 4) + 12, "flops": case["n"] * (terms + 2)}
    return {"bytes": case["n"] * (26 + (4 if case["dtype"] == "fp32" else 2)) + 8, "flops": case["n"] * 18}
