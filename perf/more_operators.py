"""Cases of the microscaled 4-bit operators: quantising a matrix and back, the
all-gather's copy-in and copy-out in 4 bits, the reduce of 4-bit gradient
slices, and the product of two 4-bit matrices, also with a weight that lies in
the gathered buffer.

Where `own` is false, run() is the plain form, elementary torch operations;
where it is true, run() makes the library's calls on the same state.  exact()
is the operators' definition in 64 bits.

A block is 32 consecutive elements: codes of 4 bits (sign, and one of 0, 0.5,
1, 1.5, 2, 3, 4, 6), the first element in the low half of the first byte, and
one byte s that scales them by 2^(s - 127).  With amax the block's largest
magnitude, a in [1, 2) and amax = a * 2^E:
    nearest    : s - 127 = max(E - 2, -127), codes rounded to nearest even, at most 6
    stochastic : one more where a > 1.5 (nothing exceeds 6); a value that lies
                 a share f of the way from one code to the next goes up where
                 f > (r + 0.5) / 65536, r 16 random bits from (seed, position)
A quantised shard of a group (one rank's part): every parameter's piece starts
on a multiple of 8 blocks; all codes, then all scales, zeros up to 128 bytes.
"""
import math

import torch

own = False

BF16, F32, F64, I64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int64, torch.uint8
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
BLOCK, PIECE, LINE = 32, 8, 128     # elements of a block, blocks a piece starts on, bytes a shard is a multiple of


# ------------------------------------------------------------------ sizes --

def _shapes(case):
    if case["layout"] == "mlp":        # W_in, W_out, bias, norm
        return [(64, 256), (256, 64), (256,), (64,)]
    if case["layout"] == "llama":      # blocks of q, k, v, o, gate, up, down and two norms
        d, f = case["dim"], case["ffn"]
        return ([(d, d)] * 4 + [(f, d)] * 2 + [(d, f)] + [(d,)] * 2) * case["layers"]
    u = torch.rand(case["count"], generator=torch.Generator().manual_seed(case["count"]), dtype=F64)   # "spread": over the logarithm
    return [(max(1, int(v)),) for v in torch.exp(u * math.log(case["most"])).tolist()]


def _up(n, a):
    return -(-n // a) * a


def _layout(case):
    """The group's pieces, one per parameter and rank that holds some of it: (parameter, rank, first element of the
    parameter, element count, first block in the rank's quantised shard, first element in its plain shard); then the
    quantised shard's blocks and bytes and the plain shard's elements."""
    shapes, world = _shapes(case), case["world"]
    numels = [math.prod(s) for s in shapes]
    pieces, blocks = [], 0
    if case["mode"] == "fsdp2":        # each parameter's rows in `world` chunks
        at = 0
        for p, s in enumerate(shapes):
            part = -(-s[0] // world) * math.prod(s[1:])
            for r in range(world):
                n = min(part, numels[p] - r * part)
                if n > 0:
                    pieces.append((p, r, r * part, n, blocks, at))
            at, blocks = at + part, blocks + _up(-(-part // BLOCK), PIECE)
        shard = at
    else:                              # one flat, each parameter on 16 bytes of it, cut into `world` equal shards
        starts, at = [], 0
        for n in numels:
            starts.append(at)
            at = _up(at + n, 16 // _width(case))
        shard = -(-(starts[-1] + numels[-1]) // world)
        used = [0] * world
        for p, (start, n) in enumerate(zip(starts, numels)):
            for r in range(start // shard, (start + n - 1) // shard + 1):
                lo, hi = max(start, r * shard), min(start + n, (r + 1) * shard)
                pieces.append((p, r, lo - start, hi - lo, used[r], lo - r * shard))
                used[r] += _up(-(-(hi - lo) // BLOCK), PIECE)
        blocks = max(used)
    return pieces, blocks, _up(17 * blocks, LINE), shard


def _width(case):
    return 4 if case.get("dtype") == "fp32" else 2


def _type(name):
    return F32 if name == "fp32" else BF16


def listed():
    """Sizes: the tiny 2-layer MLP on 4 ranks; one and three 7B blocks on 8; 97 parameters of 1 to 4M elements."""
    llama7 = {"layout": "llama", "dim": 4096, "ffn": 11008, "world": 8, "mode": "fsdp2"}
    mlp = {"layout": "mlp", "world": 4, "mode": "fsdp1"}
    spread = {"layout": "spread", "count": 97, "most": 4194304, "world": 8, "mode": "fsdp1"}
    return [
        # one token's activation before a product: all launch latency
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 4096, "pad": 0, "dtype": "bf16", "both": False, "random": False},
        # the gradient of a feed-forward's inner activations, for both of the layer's gradient products
        {"name": "quantize_train", "op": "quantize", "rows": 8192, "cols": 11008, "pad": 0, "dtype": "bf16", "both": True, "random": True},
        # a small model's gather: latency
        {"name": "gather_mlp", "op": "gather", **mlp, "dtype": "bf16", "random": False},
        # one block's gather, bf16 parameters
        {"name": "gather_block", "op": "gather", **llama7, "layers": 1, "dtype": "bf16", "random": False},
        # the gradients of odd parameters in fp32, unbiased, whose pieces start and end anywhere
        {"name": "gather_spread", "op": "gather", **spread, "dtype": "fp32", "random": True},
        # a small model's reduce, one micro-step: latency
        {"name": "reduce_mlp", "op": "reduce", **mlp, "acc": 1, "rank": 1},
        # one block's reduce, one micro-step
        {"name": "reduce_block", "op": "reduce", **llama7, "layers": 1, "acc": 1, "rank": 0},
        # three blocks, 4 micro-steps: 32 slices
        {"name": "reduce_acc", "op": "reduce", **llama7, "layers": 3, "acc": 4, "rank": 7},
        # one token through a feed-forward's gate, the weight where the all-gather left it
        {"name": "product_token", "op": "product", "m": 1, "n": 11008, "k": 4096, "world": 8, "out": "bf16"},
        # odd sizes throughout: a short batch, a ragged last block
        {"name": "product_odd", "op": "product", "m": 333, "n": 1000, "k": 1377, "world": 0, "out": "bf16"},
        # a batch of training tokens through the gate
        {"name": "product_train", "op": "product", "m": 8192, "n": 11008, "k": 4096, "world": 8, "out": "bf16"},
        # the gate's weight gradient over the batch, in fp32
        {"name": "product_wgrad", "op": "product", "m": 11008, "n": 4096, "k": 8192, "world": 0, "out": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gather", "reduce", "product"])
    if op == "quantize":
        rows = _log(rng, 1, 16384)
        return {"op": op, "rows": rows, "cols": min(_log(rng, 16, 16384), 80_000_000 // rows), "pad": rng.choice([0, 0, 8, 37]),
                "dtype": rng.choice(["bf16", "fp32"]), "both": rng.random() < 0.6, "random": rng.random() < 0.5}
    if op == "product":
        n, k = _log(rng, 16, 11008), _log(rng, 32, 11008)
        world = rng.choice([0, 0, 2, 3, 8])
        if world:                      # a weight's rows are whole blocks in the gathered buffer
            k = _up(k, BLOCK)
        return {"op": op, "m": _log(rng, 1, 8192), "n": n, "k": min(k, 11008), "world": world, "out": rng.choice(["bf16", "bf16", "fp32"])}
    if rng.random() < 0.5:
        group = {"layout": "spread", "count": _log(rng, 1, 150), "most": _log(rng, 1000, 4_000_000)}
    else:
        dim = 64 * rng.randint(1, 48)
        dim += 64 * (dim == 3008)
        group = {"layout": "llama", "dim": dim, "ffn": 32 * (dim // 12) + 32, "layers": 1}
    group |= {"world": rng.choice([2, 3, 4, 8]), "mode": rng.choice(["fsdp1", "fsdp2"])}
    if op == "reduce":
        return {"op": op, **group, "acc": rng.choice([1, 1, 2, 4]), "rank": rng.randrange(group["world"])}
    return {"op": op, **group, "dtype": rng.choice(["bf16", "fp32"]), "random": rng.random() < 0.5}


# ------------------------------------------------------------------ state --

def _normal(gen, shape, scale, dtype=F32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=F32).mul_(scale).to(dtype)


def _wire(case, pieces, blocks, nbytes):
    """Where each parameter element lies among the gathered buffer's elements, in parameter order."""
    at = []
    for p, r, first, n, b, _ in sorted(pieces, key=lambda x: (x[0], x[2])):
        lo = (r * blocks + b) * BLOCK
        at.append(torch.arange(lo, lo + n, device="cuda"))
    return torch.cat(at)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"op": case["op"], "case": dict(case)}
    if case.get("random"):             # the seed of the random bits is on the GPU, as a captured step needs it
        state["seed"] = torch.randint(0, 2 ** 62, (1,), generator=gen, device="cuda", dtype=I64)
    if case["op"] == "quantize":
        rows, cols = case["rows"], case["cols"]
        x = _normal(gen, (rows, cols + case["pad"]), 1.0)
        x *= torch.exp(0.5 * torch.randn(cols + case["pad"], generator=gen, device="cuda"))   # columns of unlike size
        state["x"] = x.to(_type(case["dtype"]))[:, :cols]
        state["out"] = torch.empty(rows, cols, dtype=_type(case["dtype"]), device="cuda")
        state["out_t"] = torch.empty(cols, rows, dtype=_type(case["dtype"]), device="cuda") if case["both"] else None
        if own:   # the buffers that a program keeps
            import fsdp_sharded_state_amd as fs
            state["by_row"] = fs.fs_mx4_empty(rows, cols)
            state["by_col"] = fs.fs_mx4_empty(cols, rows) if case["both"] else None
        return state
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        state["a"] = _encode(_blocks(_normal(gen, (m, k), 1.0)))
        state["out"] = torch.empty(m, n, dtype=_type(case["out"]), device="cuda")
        if not case["world"]:
            state["b"] = _encode(_blocks(_normal(gen, (n, k), 0.02)))
        else:      # the weight between two norms in a gathered group
            group = [(k,), (n, k), (k,)]
            world, chunk = case["world"], -(-n // case["world"])
            b0 = _up(-(-(-(-k // world)) // BLOCK), PIECE)
            nb = _up(chunk * k // BLOCK, PIECE)
            blocks = 2 * b0 + nb
            nbytes = _up(17 * blocks, LINE)
            buf = torch.zeros(world, nbytes, dtype=U8, device="cuda")
            w = torch.zeros(world * chunk, k, device="cuda")
            w[:n] = _normal(gen, (n, k), 0.02)
            codes, scales = _encode(w.view(world, -1, BLOCK))
            used = chunk * k // BLOCK
            buf[:, b0 * 16:(b0 + used) * 16] = codes.reshape(world, -1)
            buf[:, blocks * 16 + b0:blocks * 16 + b0 + used] = scales.reshape(world, -1)
            state["gathered"], state["at"] = buf.view(-1), (world, chunk, b0, used, blocks)
            if own:
                import fsdp_sharded_state_amd as fs
                state["plan"] = fs.fs_mx4_plan(fs.fs_plan(group, "bf16", world, False, "fsdp2"))
        if own:
            import fsdp_sharded_state_amd as fs
            state["A"] = fs.Mx4Matrix(*state["a"], k)
            state["B"] = fs.Mx4Matrix(*state["b"], k) if not case["world"] else state["plan"].matrix(state["gathered"], 1)
        return state
    shapes = _shapes(case)
    pieces, blocks, nbytes, shard = _layout(case)
    if own:
        import fsdp_sharded_state_amd as fs
        plan = fs.fs_plan(shapes, "fp32" if case.get("dtype") == "fp32" else "bf16", case["world"], case["mode"] == "fsdp1", case["mode"])
        state["plan"] = fs.fs_mx4_plan(plan).upload()
    if case["op"] == "gather":
        t = _type(case["dtype"])
        # matrices 0.02 (as gradients or weights are spread), vectors about 1 as norms are
        state["params"] = [_normal(gen, s, 0.02, t) if len(s) > 1 else (1 + _normal(gen, s, 0.1)).to(t) for s in shapes]
        starts, at = [], 0
        for s in shapes:
            starts.append(at)
            at = _up(at + math.prod(s), 16 // t.itemsize)
        state["flat"] = torch.zeros(at, dtype=t, device="cuda")      # the outputs, each on 16 bytes of one buffer
        state["outs"] = [state["flat"][a:a + math.prod(s)].view(s) for a, s in zip(starts, shapes)]
        state["gathered"] = torch.empty(case["world"] * nbytes, dtype=U8, device="cuda")
        if not own:
            state["wire"], state["blocks"], state["nbytes"] = _wire(case, pieces, blocks, nbytes), blocks, nbytes
            state["home"] = torch.cat([torch.arange(a, a + math.prod(s), device="cuda") for a, s in zip(starts, shapes)])
        return state
    mine = [x for x in pieces if x[1] == case["rank"]]
    terms = case["world"] * case["acc"]
    state["slices"] = torch.zeros(terms, nbytes, dtype=U8, device="cuda")
    for k in range(terms):             # each rank's gradients, 1e-3, one in a thousand 30 times as large
        for p, _, _, n, b, _ in mine:
            g = _normal(gen, n, 1e-3)
            at = torch.randint(0, n, (n // 1000 + 1,), generator=gen, device="cuda")
            g[at] = g[at] * 30
            codes, scales = _encode(_blocks(g))
            state["slices"][k, b * 16:b * 16 + codes.numel()] = codes.view(-1)
            state["slices"][k, blocks * 16 + b:blocks * 16 + b + scales.numel()] = scales.view(-1)
    state["out"] = torch.empty(shard, dtype=F32, device="cuda")
    if not own:
        state["blocks"] = blocks
        state["from"] = torch.cat([torch.arange(b * BLOCK, b * BLOCK + n, device="cuda") for _, _, _, n, b, _ in mine] or [torch.zeros(0, dtype=I64, device="cuda")])
        state["to"] = torch.cat([torch.arange(e, e + n, device="cuda") for _, _, _, n, _, e in mine] or [torch.zeros(0, dtype=I64, device="cuda")])
    return state


# -------------------------------------------------------------- plain form --

def _blocks(x):
    """The last dimension in blocks, the last one filled up with zeros."""
    pad = -x.shape[-1] % BLOCK
    x = torch.nn.functional.pad(x.to(F32), (0, pad)) if pad else x.to(F32)
    return x.unflatten(-1, (-1, BLOCK))


def _pow2(e):
    """2^e in fp32, -127 <= e <= 127, from its bits."""
    return torch.where(e > -127, (e + 127).to(torch.int32) << 23, 0x00400000).view(F32)


def _mulhilo(a, b):
    p = a * b                          # wraps: the low 64 bits are those of the unsigned product
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _random16(seed, blocks, orientation):
    """16 random bits for each element of `blocks` blocks: Philox4x32, 7 rounds, one call for 8 elements."""
    n = torch.arange(blocks * 4, device=seed.device)
    c0, c1 = n & 0xFFFFFFFF, n >> 32
    c2, c3 = torch.full_like(n, orientation), torch.zeros_like(n)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(7):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0, c1, c2, c3], -1)
    return torch.stack([words & 0xFFFF, words >> 16], -1).view(blocks, BLOCK)


def _encode(x, seed=None, orientation=0):
    """Codes (rows, 16 bytes a block) and scales (rows, blocks) of fp32 blocks (rows, blocks, 32)."""
    amax = x.abs().amax(-1, keepdim=True)
    a, e = torch.frexp(amax)           # amax = a * 2^e, a in [0.5, 1)
    e = torch.where(amax > 0, e - 3, -127)
    if seed is not None:
        e = e + ((a > 0.75) & (amax > 0)).to(e.dtype)
    e = e.clamp(min=-127)
    y = x.abs() * _pow2(-e)
    grid = torch.tensor(GRID, device=x.device)
    if seed is None:                   # the code's index is the number of midpoints below; a tie goes to the even index
        mid = (grid[1:] + grid[:-1]) / 2
        up = torch.bucketize(y, mid, out_int32=True)               # midpoints < y
        tie = torch.bucketize(y, mid, out_int32=True, right=True)  # midpoints <= y
        code = torch.where(up % 2 == 1, tie, up)
    else:
        code = torch.bucketize(y, grid, out_int32=True, right=True) - 1   # of the value at or below
        code = code.clamp(max=6)
        low, high = grid[code], grid[code + 1]
        r = _random16(seed, x.numel() // BLOCK, orientation).view(x.shape)
        code = code + ((y - low) / (high - low) > (r.to(F32) + 0.5) / 65536).to(code.dtype)
    code = (code + torch.signbit(x) * 8).to(U8)
    codes = code[..., 0::2] + code[..., 1::2] * 16
    return codes.flatten(-2), (e + 127).squeeze(-1).to(U8)


def _decode(codes, scales):
    """fp32 values (rows, 32 a block) of codes (rows, 16 a block) and scales (rows, blocks)."""
    grid = torch.tensor(GRID, device=codes.device)
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, BLOCK)) * _pow2(scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _quantize(state):
    x, seed = state["x"], state.get("seed")
    rows, cols = x.shape
    state["out"].copy_(_decode(*_encode(_blocks(x), seed, 0))[:, :cols])
    if state["out_t"] is None:
        return state["out"]
    state["out_t"].copy_(_decode(*_encode(_blocks(x.t()), seed, 1))[:, :rows])
    return state["out"], state["out_t"]


def _gather(state):
    world, blocks, nbytes = state["case"]["world"], state["blocks"], state["nbytes"]
    x = torch.zeros(world * blocks * BLOCK, device="cuda")
    x[state["wire"]] = torch.cat([p.reshape(-1) for p in state["params"]]).to(F32)
    codes, scales = _encode(x.view(world, blocks, BLOCK), state.get("seed"))
    buf = state["gathered"].view(world, nbytes)
    buf[:, :blocks * 16] = codes
    buf[:, blocks * 16:blocks * 17] = scales
    buf[:, blocks * 17:] = 0
    values = _decode(buf[:, :blocks * 16], buf[:, blocks * 16:blocks * 17]).view(-1)
    state["flat"][state["home"]] = values[state["wire"]].to(state["flat"].dtype)
    return state["flat"]


def _reduce(state):
    blocks = state["blocks"]
    s = state["slices"]
    total = _decode(s[:, :blocks * 16], s[:, blocks * 16:blocks * 17]).sum(0) / state["case"]["world"]
    state["out"].zero_()
    state["out"][state["to"]] = total[state["from"]]
    return state["out"]


def _product(state):
    k, n = state["case"]["k"], state["case"]["n"]
    a = _decode(*state["a"])[:, :k]
    if "b" in state:
        b = _decode(*state["b"])[:, :k]
    else:
        world, chunk, b0, used, blocks = state["at"]
        buf = state["gathered"].view(world, -1)
        b = _decode(buf[:, b0 * 16:(b0 + used) * 16], buf[:, blocks * 16 + b0:blocks * 16 + b0 + used]).view(world * chunk, k)[:n]
    state["out"].copy_(a @ b.t())
    return state["out"]


# --------------------------------------------------------- library's calls --

def _own(state):
    import fsdp_sharded_state_amd as fs
    op = state["op"]
    if op == "quantize":
        fs.fs_mx4_quantize(state["x"], state["by_row"], state["by_col"], seed=state.get("seed"))
        fs.fs_mx4_dequantize(state["by_row"], state["out"])
        if state["by_col"] is None:
            return state["out"]
        fs.fs_mx4_dequantize(state["by_col"], state["out_t"])
        return state["out"], state["out_t"]
    if op == "gather":
        fs.fs_pack_mx4(state["plan"], state["params"], state["gathered"], seed=state.get("seed"))
        fs.fs_unpack_mx4(state["plan"], state["gathered"], state["outs"])
        return state["flat"]
    if op == "reduce":
        fs.fs_reduce_shard_mx4(state["plan"], state["slices"], state["out"], rank=state["case"]["rank"], grad_acc=state["case"]["acc"])
        return state["out"]
    fs.fs_mx4_matmul(state["A"], state["B"], state["out"])
    return state["out"]


def run(state):
    if own:
        return _own(state)
    return {"quantize": _quantize, "gather": _gather, "reduce": _reduce, "product": _product}[state["op"]](state)


# ------------------------------------------------------------- definitions --

def _power64(e):
    """2^e in 64 bits: a power function may be off in the last bit."""
    return ((e.to(I64) + 1023) << 52).view(F64)


def _values64(codes, scales):
    """64-bit values of flat codes and scales: magnitude from the two exponent bits and the mantissa bit."""
    c = torch.stack([codes.reshape(-1) % 16, codes.reshape(-1) // 16], 1).reshape(-1).to(I64)
    exponent, mantissa = (c % 8) // 2, (c % 2).to(F64)
    v = torch.where(exponent == 0, mantissa / 2, _power64(exponent - 1) * (1 + mantissa / 2))
    v = torch.where(c >= 8, -v, v).view(-1, BLOCK)
    return (v * _power64(scales.reshape(-1, 1).to(I64) - 127)).reshape(-1)


def _philox64(seed, first, count, orientation):
    """The 16 random bits of `count` blocks from block `first` on, by 16-bit limbs."""
    def product(a, b):                 # of 32-bit numbers: (high, low)
        low, mid = (a & 0xFFFF) * b, (a >> 16) * b
        s = (low >> 16) + (mid & 0xFFFFFFFFFFFF)
        return s >> 16, ((s & 0xFFFF) << 16) | (low & 0xFFFF)

    group = torch.arange(first * 4, (first + count) * 4, device="cuda")
    x = [group % 2 ** 32, group // 2 ** 32, torch.full_like(group, orientation), torch.zeros_like(group)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for i in range(7):
        (h0, l0), (h1, l1) = product(x[0], 0xD2511F53), product(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return torch.stack([h for w in x for h in (w % 65536, w // 65536)], 1).reshape(count, BLOCK)


def _round64(x, seed=None, first=0, orientation=0):
    """64-bit values that a flat run of elements has after quantisation, block by block from block `first` on."""
    n = x.numel()
    v = torch.cat([x.reshape(-1).to(F64), torch.zeros(-n % BLOCK, dtype=F64, device=x.device)]).view(-1, BLOCK)
    amax = v.abs().max(1, keepdim=True).values
    # floor(log2), put right where the logarithm's rounding passed a whole number
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    e = e + (_power64(e + 1) <= amax).to(F64) - (_power64(e) > amax).to(F64) * (amax > 0)
    e = torch.where(amax > 0, e - 2, torch.full_like(e, -127))
    if seed is not None:
        e = e + (amax > 6 * _power64(e)).to(F64)
    scale = _power64(e.clamp(min=-127))
    y = v.abs() / scale
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).to(F64)
    if seed is None:                   # torch.round takes ties to even; so do the codes, whose last bit is that of value / step
        q = torch.round(y / step) * step
    else:
        low = torch.floor(y / step)
        r = _philox64(seed, first, v.shape[0], orientation)
        q = (low + ((y / step - low) * 65536 > r + 0.5).to(F64)) * step
    return (torch.copysign(q.clamp(max=6.0), v) * scale).reshape(-1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    bits = s["seed"].item() if "seed" in s else None
    if case["op"] == "quantize":
        outs = []
        for orientation, x in enumerate([s["x"], s["x"].t()][:1 + case["both"]]):
            full = torch.nn.functional.pad(x.to(F64), (0, -x.shape[1] % BLOCK))
            outs.append(_round64(full, bits, 0, orientation).view(full.shape)[:, :x.shape[1]])
        return tuple(outs) if case["both"] else outs[0]
    if case["op"] == "gather":
        flat = torch.zeros(s["flat"].numel(), dtype=F64, device="cuda")
        pieces, blocks, _, _ = _layout(case)
        start = [o.storage_offset() for o in s["outs"]]
        for p, r, first, n, b, _ in pieces:
            flat[start[p] + first:start[p] + first + n] = _round64(s["params"][p].reshape(-1)[first:first + n], bits, r * blocks + b)
        return flat
    if case["op"] == "reduce":
        pieces, blocks, _, shard = _layout(case)
        out = torch.zeros(shard, dtype=F64, device="cuda")
        for p, r, _, n, b, e in pieces:
            if r == case["rank"]:
                nb = -(-n // BLOCK)
                for t in s["slices"]:
                    out[e:e + n] += _values64(t[b * 16:(b + nb) * 16], t[blocks * 16 + b:blocks * 16 + b + nb])[:n]
        return out / case["world"]
    m, n, k = case["m"], case["n"], case["k"]
    a = _values64(*s["a"]).view(m, -1)
    if not case["world"]:
        b = _values64(*s["b"]).view(n, -1)
    else:
        world, chunk, b0, used, blocks = s["at"]
        ranks = s["gathered"].view(world, -1)
        b = torch.cat([_values64(r[b0 * 16:(b0 + used) * 16], r[blocks * 16 + b0:blocks * 16 + b0 + used]) for r in ranks]).view(-1, k)[:n]
    return torch.matmul(a, b.t())


def work(case):
    """Each input read once, each result written once; what is quantised and read back is both."""
    if case["op"] == "quantize":
        n, ways = case["rows"] * case["cols"], 2 if case["both"] else 1
        size = _width(case)
        return {"bytes": n * (size + ways * (2 * 17 / 32 + size)), "flops": 4 * n * ways}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k * 17 / 32 + m * n * (4 if case["out"] == "fp32" else 2), "flops": 2 * m * n * k}
    pieces, _, nbytes, shard = _layout(case)
    if case["op"] == "gather":
        n = sum(math.prod(s) for s in _shapes(case))
        return {"bytes": n * (2 * _width(case) + 2 * 17 / 32), "flops": 4 * n}
    n, terms = sum(x[3] for x in pieces if x[1] == case["rank"]), case["world"] * case["acc"]
    return {"bytes": max(1, n * terms * 17 / 32 + 4 * shard), "flops": 2 * n * terms}
