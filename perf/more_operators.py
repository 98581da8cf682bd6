"""The 4-bit exchange and products of a sharded step, measured operator by operator.

Values travel in microscaled 4-bit floating point: blocks of 32 consecutive
values share a power of two (8 bits), each value keeps a sign, two bits of
exponent and one of mantissa.  Four operators, and the runs they are used in:
  quantize  bf16 or fp32 values to 4 bits (parameter shards before the
            all-gather, activations and gradients before a product), rounded to
            nearest or at random, and the receiver's way back to bf16
  reduce    R peers' 4-bit gradient chunks summed in fp32, scaled
  exchange  the sender's and the receiver's half of a 4-bit reduce-scatter:
            R bf16 chunks quantized at random, then reduced
  product   C = A B' of two 4-bit operands: one token, a few, a training batch,
            a weight's gradient added to its fp32 accumulator
  linear    one layer's training step: its output and both gradients, all three
            products of 4-bit operands
Each case runs one of them: in plain torch operations, or (own = True) through
the package's calls.
"""

import math

import torch

own = False

BLOCK = 32
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
M32 = 0xFFFFFFFF


# ---- cases -------------------------------------------------------------------

def _quantize(name, rows, cols, dtype="bf16", along="rows", random=False, pad=0):
    """pad: the rows lie in a wider buffer, this many elements apart beyond their length."""
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype,
            "along": along, "random": random, "pad": pad}


def _reduce(name, n, peers, acc=False):
    return {"name": name, "op": "reduce", "n": n, "peers": peers, "acc": acc}


def _exchange(name, n, peers):
    return {"name": name, "op": "exchange", "n": n, "peers": peers}


def _product(name, m, n, k, accumulate=False):
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "accumulate": accumulate}


def _linear(name, tokens, d_in, d_out):
    return {"name": name, "op": "linear", "tokens": tokens, "d_in": d_in, "d_out": d_out}


def listed():
    return [
        # a small network's fp32 master shard before the all-gather: the latency of two calls
        _quantize("quantize small shard", 1, 262784, "fp32"),
        # a 124M model's master shard over 8 ranks
        _quantize("quantize 124M / 8", 1, 15554976, "fp32"),
        # one layer's gradient of a training batch, for both of its products, rounded at random
        _quantize("quantize both ways", 8192, 4096, "bf16", "both", True),
        # a small network's reduce-scatter share
        _reduce("reduce small shard", 262784, 2),
        # a 7.5B model's share over 64 ranks, earlier microbatches accumulated
        _reduce("reduce 7.5B / 64", 103890048, 8, acc=True),
        # a 124M model's reduce-scatter over 8 ranks, both halves
        _exchange("exchange 124M / 8", 15554976, 8),
        # one token through a d = 4096 projection: the weight read once
        _product("product one token", 1, 4096, 4096),
        # 16 tokens through the two stacked weights of a gated 4096-wide layer
        _product("product 16 tokens", 16, 28672, 4096),
        # odd and ragged on every side
        _product("product odd", 509, 1021, 777),
        # an attention weight's gradient over 8192 tokens, added to its accumulator
        _product("product weight gradient", 4096, 4096, 8192, True),
        # a training batch through the feed-forward's first weight
        _product("product feed-forward", 8192, 14336, 4096),
        # that layer's whole training step: the largest
        _linear("linear feed-forward", 8192, 4096, 14336),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _side(rng, lo, hi):
    """Half the sizes are multiples of 64, as real layers' are."""
    x = _log(rng, lo, hi)
    return max(64, x // 64 * 64) if rng.random() < 0.5 else x


def draw(rng):
    op = rng.choice(["quantize", "quantize", "reduce", "exchange", "product", "product",
                     "product", "linear"])
    if op == "quantize":
        dtype, random = rng.choice(["bf16", "fp32"]), rng.random() < 0.5
        if rng.random() < 0.5:
            c = _quantize(None, 1, _log(rng, 1000, 1 << 25), dtype, "rows", random)
        else:
            c = _quantize(None, _side(rng, 16, 8192), _side(rng, 32, 8192), dtype,
                          rng.choice(["rows", "cols", "both"]), random,
                          rng.choice([0, 0, 8, rng.randrange(1, 100)]))
    elif op == "reduce":
        R = rng.choice([1, 2, 3, 4, 8, 16])
        c = _reduce(None, _log(rng, 1000, (1 << 29) // max(R, 8)), R, rng.random() < 0.5)
    elif op == "exchange":
        c = _exchange(None, _log(rng, 1000, 1 << 24), rng.choice([2, 3, 4, 8]))
    elif op == "product":
        if rng.random() < 0.4:  # one token to a few
            c = _product(None, _log(rng, 1, 64), _side(rng, 256, 28672), _side(rng, 256, 14336))
        else:
            c = _product(None, _side(rng, 64, 8192), _side(rng, 64, 14336), _side(rng, 32, 8192),
                         rng.random() < 0.3)
    else:
        c = _linear(None, _side(rng, 64, 8192), _side(rng, 64, 4096), _side(rng, 64, 8192))
    del c["name"]
    return c


def _bits4(rows, cols):
    """Bytes of a 4-bit matrix: codes and scales of whole blocks."""
    return rows * -(-cols // BLOCK) * (BLOCK // 2 + 1)


def work(case):
    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        both = {"rows": [(r, c)], "cols": [(c, r)], "both": [(r, c), (c, r)]}[case["along"]]
        # in, the 4 bits that are sent or multiplied, and the receiver's values
        return {"bytes": r * c * (4 if case["dtype"] == "fp32" else 2)
                + sum(_bits4(*x) for x in both) + len(both) * r * c * 2, "flops": 0}
    if op == "reduce":
        n, R = case["n"], case["peers"]
        return {"bytes": R * _bits4(1, n) + n * (8 if case["acc"] else 4), "flops": n * (R + 1)}
    if op == "exchange":
        n, R = case["n"], case["peers"]
        return {"bytes": R * (2 * n + _bits4(1, n)) + n * 4, "flops": n * (R + 1)}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _bits4(m, k) + _bits4(n, k) + m * n * (8 if case["accumulate"] else 2),
                "flops": 2 * m * n * k}
    t, i, o = case["tokens"], case["d_in"], case["d_out"]
    # x, w and dy in bf16; y and dx in bf16; dw read and written in fp32
    return {"bytes": 2 * (t * i + i * o + t * o) + 2 * (t * o + t * i) + 8 * i * o,
            "flops": 6 * t * i * o}


# ---- the plain form --------------------------------------------------------------

def _philox(index, upper, seed, offset):
    """Philox4x32-10 (Salmon et al., 2011) of the counters (index, offset), the
    index's highest bit set where `upper`: four words each, [n, 4]."""
    def mul(a, c):  # high and low word of a 64-bit product
        u, v = (a >> 16) * c, (a & 0xFFFF) * c
        return (u + (v >> 16)) >> 16, (((u & 0xFFFF) << 16) + v) & M32

    c0, c1 = index & M32, (index >> 32) | (int(upper) << 31)
    c2, c3 = torch.full_like(c0, offset & M32), torch.full_like(c0, offset >> 32)
    k0, k1 = seed & M32, seed >> 32
    for _ in range(10):
        h0, l0 = mul(0xD2511F53, c0)
        h1, l1 = mul(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return torch.stack([c0, c1, c2, c3], 1)


def _plain_quantize(x, seed=None, offset=0, upper=False):
    """Codes 0..15 [rows, blocks, 32] and scale bytes [rows, blocks] of a matrix,
    blocks along its rows.  The scale is the block's largest power of two over 4
    (rounded to nearest: the top of the block, up to 8, saturates at 6), or the
    least power of two that holds all of it within 6 (at random)."""
    rows, cols = x.shape
    kb = -(-cols // BLOCK)
    x = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - cols)).view(rows, kb, BLOCK)
    bits = x.abs().amax(-1).view(torch.int32)  # NaN is the largest
    s = (bits >> 23) - 2
    if seed is not None:
        s = s + ((bits & 0x7FFFFF) > 0x400000).int()
    s = s.clamp(min=0)
    bad = (bits >> 23) == 255
    y = x.abs() * ((254 - s).clamp(min=0) << 23).view(torch.float32)[..., None]
    if seed is None:
        code = ((y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5)
                + (y >= 3.5) + (y > 5))
    else:
        words = _philox(torch.arange(rows * kb * 4, device=x.device), upper, seed, offset)
        r = torch.stack([words & 0xFFFF, words >> 16], 2).view(rows, kb, BLOCK)
        high = (y >= 2).long() + (y >= 4)
        y = torch.where(bad[..., None], torch.zeros_like(y), y)
        code = (((y * 131072).long() + (r << high)) >> (16 + high)) + 2 * high
    code = torch.where(bad[..., None], torch.zeros_like(code), code + 8 * (x < 0))
    return code.to(torch.uint8), torch.where(bad, torch.full_like(s, 255), s).to(torch.uint8)


def _packed(code, scale):
    """The bytes that travel: two codes a byte, the first in the low half."""
    rows, kb, _ = code.shape
    c = code.view(rows, kb * BLOCK // 2, 2)
    return (c[..., 0] | (c[..., 1] << 4)).contiguous(), scale.contiguous()


def _values(code, scale, cols, dtype=torch.float32):
    """fp32 values of codes [rows, blocks, 32] and their scales."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=code.device)
    s = scale.int()
    f = torch.where(s > 0, s << 23, torch.full_like(s, 1 << 22)).view(torch.float32)
    f = torch.where(s == 255, torch.full_like(f, float("nan")), f)
    return (grid[code.long()] * f[..., None]).flatten(1)[:, :cols].to(dtype)


def _unpacked(packed, cols, dtype=torch.float32):
    b, scale = packed
    code = torch.stack([b & 15, b >> 4], 2).view(b.shape[0], -1, BLOCK)
    return _values(code, scale, cols, dtype)


def _plain_matrix(x, seed=None, offset=0, upper=False):
    """The values that a quantized matrix stands for, fp32."""
    return _values(*_plain_quantize(x, seed, offset, upper), x.shape[1])


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def activations(*shape):
        """Normal values, every 64th column 8 times larger."""
        x = normal(*shape)
        x[:, ::64] *= 8
        return x.bfloat16()

    def sent(x):
        return _packed(*_plain_quantize(x))

    s = {"case": case, "seed": (seed * 0x9E3779B97F4A7C15 + 1) & (1 << 64) - 1,
         "offset": seed & 0xFFFF}
    op = case["op"]
    if op == "quantize":
        x = normal(case["rows"], case["cols"])
        if case["rows"] > 1:  # a batch's gradient: rows of very different sizes
            x = x * normal(case["rows"], 1).exp()
        x = (x * 0.02).to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)
        if case["pad"]:
            wide = torch.zeros(case["rows"], case["cols"] + case["pad"], dtype=x.dtype, device=dev)
            wide[:, :case["cols"]] = x
            x = wide[:, :case["cols"]]
        return {**s, "x": x}
    if op in ("reduce", "exchange"):
        n, R = case["n"], case["peers"]
        s["scale"] = 1.0 / R
        if op == "reduce":
            s["peers"] = [sent(normal(1, n) * 1e-3) for _ in range(R)]
            s["acc"] = normal(n).mul_(2e-3) if case["acc"] else None
        else:
            s["chunks"] = [normal(n).mul_(1e-3).bfloat16() for _ in range(R)]
        return {**s, "out": torch.empty(n, device=dev)}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {**s, "a": sent(activations(m, k)), "b": sent(normal(n, k) * 0.02),
                "c": normal(m, n) if case["accumulate"] else None}
    t, i, o = case["tokens"], case["d_in"], case["d_out"]
    return {**s, "x": activations(t, i), "w": (normal(o, i) * 0.02).bfloat16(),
            "dy": (normal(t, o) * normal(t, 1).exp() * 1e-3).bfloat16(),
            "dw": normal(o, i).mul_(1e-2)}


# ---- one pass ----------------------------------------------------------------

def _own(s):
    import sharded_bucket_plan_amd as sbp
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        q = sbp.mx_quantize(s["x"], along=case["along"],
                             seed=s["seed"] if case["random"] else None, offset=s["offset"])
        return [sbp.mx_dequantize(x) for x in (q if case["along"] == "both" else [q])]
    if op == "reduce":
        peers = [sbp.Mx4(c, f, (1, case["n"])) for c, f in s["peers"]]
        sbp.mx_reduce_shard(peers, s["acc"], s["scale"], s["out"])
        return s["out"]
    if op == "exchange":
        peers = [sbp.mx_quantize(c, seed=s["seed"], offset=s["offset"] + r)
                 for r, c in enumerate(s["chunks"])]
        sbp.mx_reduce_shard(peers, None, s["scale"], s["out"])
        return s["out"]
    if op == "product":
        a = sbp.Mx4(*s["a"], (case["m"], case["k"]))
        b = sbp.Mx4(*s["b"], (case["n"], case["k"]))
        return sbp.mx_matmul(a, b, out=s["c"], accumulate=case["accumulate"])
    x, xt = sbp.mx_quantize(s["x"], along="both")
    w, wt = sbp.mx_quantize(s["w"], along="both")
    y = sbp.mx_matmul(x, w)
    dy, dyt = sbp.mx_quantize(s["dy"], along="both", seed=s["seed"], offset=s["offset"])
    dx = sbp.mx_matmul(dy, wt)
    sbp.mx_matmul(dyt, xt, out=s["dw"], accumulate=True)
    return {"y": y, "dx": dx, "dw": s["dw"]}


def _plain(s):
    case = s["case"]
    op, bf = case["op"], torch.bfloat16
    if op == "quantize":
        x, seed, got = s["x"], s["seed"] if case["random"] else None, []
        if case["along"] != "cols":
            got.append(_plain_matrix(x, seed, s["offset"]).to(bf))
        if case["along"] != "rows":
            got.append(_plain_matrix(x.T.contiguous(), seed, s["offset"], True).to(bf))
        return got
    if op in ("reduce", "exchange"):
        total = None
        for r in range(case["peers"]):
            if op == "reduce":
                v = _unpacked(s["peers"][r], case["n"])[0]
            else:
                v = _plain_matrix(s["chunks"][r][None], s["seed"], s["offset"] + r)[0]
            total = v if total is None else total + v
        if op == "reduce" and s["acc"] is not None:
            total = s["acc"] + total
        return torch.mul(total, s["scale"], out=s["out"])
    if op == "product":
        c = _unpacked(s["a"], case["k"]) @ _unpacked(s["b"], case["k"]).T
        return s["c"].add_(c) if case["accumulate"] else c.to(bf)
    x, xt = _plain_matrix(s["x"]), _plain_matrix(s["x"].T.contiguous())
    w, wt = _plain_matrix(s["w"]), _plain_matrix(s["w"].T.contiguous())
    y = (x @ w.T).to(bf)
    dy = _plain_matrix(s["dy"], s["seed"], s["offset"])
    dyt = _plain_matrix(s["dy"].T.contiguous(), s["seed"], s["offset"], True)
    dx = (dy @ wt.T).to(bf)
    s["dw"].add_(dyt @ xt.T)
    return {"y": y, "dx": dx, "dw": s["dw"]}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---- the definition in 64 bits ---------------------------------------------------

def _power(e):
    """2^e in float64, exactly (a power function may be off in the last place)."""
    return ((e + 1023) << 52).view(torch.float64)


def _uniform(blocks, upper, seed, offset):
    """16 random bits a value, [blocks, 32]: words of Philox4x32-10, each value's
    half word in order, the low half first.  Products by 16-bit digits."""
    n = blocks * 4
    i = torch.arange(n, device="cuda")
    state = [i % 2 ** 32, i // 2 ** 32 + (2 ** 31 if upper else 0),
             torch.zeros_like(i) + offset % 2 ** 32, torch.zeros_like(i) + offset // 2 ** 32]
    key = [seed % 2 ** 32, seed // 2 ** 32]

    def digits(a, w):
        a0, a1, w0, w1 = a % 65536, a // 65536, w % 65536, w // 65536
        mid = a0 * w1 + a0 * w0 // 65536
        cross = a1 * w0 + mid % 65536
        return a1 * w1 + mid // 65536 + cross // 65536, cross % 65536 * 65536 + a0 * w0 % 65536

    for _ in range(10):
        first, second = digits(0xD2511F53, state[0]), digits(0xCD9E8D57, state[2])
        state = [second[0] ^ state[1] ^ key[0], second[1], first[0] ^ state[3] ^ key[1], first[1]]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    halves = [h for w in state for h in (w % 65536, w // 65536)]
    return torch.stack(halves, 1).reshape(blocks, BLOCK)


def _exact_matrix(x, seed=None, offset=0, upper=False):
    """The values that x quantized stands for.  All inputs here are finite."""
    rows, cols = x.shape
    kb = -(-cols // BLOCK)
    v = torch.zeros(rows, kb * BLOCK, dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    v = v.reshape(-1, BLOCK)
    top = v.abs().max(1, keepdim=True).values
    part = torch.frexp(top)  # top = mantissa * 2^exponent, the mantissa in [1/2, 1)
    e = torch.where(top > 0, part.exponent.long() - 1, torch.full_like(top, -200).long())
    if seed is not None:
        e = e + (part.mantissa > 0.75).long()
    unit = _power((e - 2).clamp(min=-127))
    y = v.abs() / unit
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    if seed is None:
        q = torch.round(y / step) * step  # ties to the even multiple of the step
        q = q.clamp(max=6.0)
    else:
        u = _uniform(rows * kb, upper, seed, offset).double() / 65536
        share = torch.floor(y * 131072) / 131072 / step
        q = torch.floor(share + u) * step
    return (torch.sign(v) * q * unit).reshape(rows, -1)[:, :cols]


def _exact_unpacked(packed, cols):
    b, scale = packed
    b = b.long()
    c = torch.stack([b % 16, b // 16], 2).reshape(b.shape[0], -1)
    m, p = c % 2, c // 2 % 4
    v = torch.where(p > 0, (2.0 + m) * _power(p - 2), m * 0.5)
    v = torch.where(c >= 8, -v, v).double()
    f = _power(scale.long() - 127)
    return (v * f.repeat_interleave(BLOCK, 1))[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x, r, got = s["x"], s["seed"] if case["random"] else None, []
        if case["along"] != "cols":
            got.append(_exact_matrix(x, r, s["offset"]))
        if case["along"] != "rows":
            got.append(_exact_matrix(x.T, r, s["offset"], True))
        return got
    if op in ("reduce", "exchange"):
        total = torch.zeros(case["n"], dtype=torch.float64, device="cuda")
        for r in range(case["peers"]):
            if op == "reduce":
                total += _exact_unpacked(s["peers"][r], case["n"])[0]
            else:
                total += _exact_matrix(s["chunks"][r][None], s["seed"], s["offset"] + r)[0]
        if op == "reduce" and s["acc"] is not None:
            total += s["acc"].double()
        return total * s["scale"]
    if op == "product":
        c = _exact_unpacked(s["a"], case["k"]) @ _exact_unpacked(s["b"], case["k"]).T
        return c + s["c"].double() if case["accumulate"] else c
    x, xt = _exact_matrix(s["x"]), _exact_matrix(s["x"].T)
    w, wt = _exact_matrix(s["w"]), _exact_matrix(s["w"].T)
    y = x @ w.T
    del x, w
    dx = _exact_matrix(s["dy"], s["seed"], s["offset"]) @ wt.T
    del wt
    dyt = _exact_matrix(s["dy"].T, s["seed"], s["offset"], True)
    return {"y": y, "dx": dx, "dw": s["dw"].double() + dyt @ xt.T}
