"""The momentum-orthogonalising shard step, measured operator by operator.

Three operators that a rank's optimizer step uses one after the other:
  momentum   R bf16 peer gradient chunks summed in fp32, scaled, folded into an
             fp32 momentum and emitted as the bf16 update direction
  ns         the update matrices orthogonalised by Newton-Schulz products
  update     decoupled weight decay and the update on the fp32 master, with the
             bf16 parameters emitted
Each case runs one of them: in plain torch operations, or (own = True) through
the package's calls.
"""

import math

import torch

own = False

COEFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


# ---- cases -------------------------------------------------------------------

def _ns(name, mats, steps=5, pad=0):
    """mats: "BxRxC" groups of B matrices of R rows and C columns; pad: the rows
    lie in a wider buffer, this many elements apart beyond their length."""
    return {"name": name, "op": "ns", "mats": mats, "steps": steps, "pad": pad}


def _momentum(name, n, peers, acc=False, nesterov=True):
    return {"name": name, "op": "momentum", "n": n, "peers": peers, "acc": acc,
            "nesterov": nesterov}


def _update(name, n):
    return {"name": name, "op": "update", "n": n}


def listed():
    return [
        # the two weights of a small two-layer network: the latency of one call
        _ns("ns two small weights", "1x256x1024,1x1024x256"),
        # column blocks of a fused projection, odd sizes, rows further apart than they are long
        _ns("ns odd strided", "3x509x1021", pad=79),
        # one d = 4096 projection split by attention head: many flat matrices
        _ns("ns per head", "32x128x4096"),
        # every attention weight of a 12-layer d = 768 model, in one call
        _ns("ns 12 layers d768", "12x768x2304,12x768x768"),
        # one layer's attention weights at d = 4096 with 8 kv heads of 128
        _ns("ns attention d4096", "2x4096x4096,2x1024x4096"),
        # one layer's feed-forward weights at d = 4096, tall and wide: the largest
        _ns("ns feed-forward d4096", "2x14336x4096,1x4096x14336"),
        # a small network's shard
        _momentum("momentum small shard", 262784, 2),
        # a 124M model's shard over 8 ranks
        _momentum("momentum 124M / 8", 15554976, 8),
        # a 7.5B model's shard over 64 ranks, earlier microbatches accumulated
        _momentum("momentum 7.5B / 64", 103890048, 8, acc=True),
        # the matrices of one 4096-wide layer owned whole by this rank
        _update("update 124M / 8", 15554976),
        _update("update one layer", 218103808),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ns", "ns", "ns", "momentum", "update"])
    if op == "ns":
        r, c = _log(rng, 16, 8192), _log(rng, 16, 8192)
        if rng.random() < 0.5:  # sizes of real layers are multiples of 64 half the time
            r, c = max(64, r // 64 * 64), max(64, c // 64 * 64)
        # as many as keep the products under the largest listed case's
        most = int(2.5e12 / (5 * _ns_flops(r, c)))
        b = max(1, min(_log(rng, 1, 64), most))
        c2 = _ns(None, f"{b}x{r}x{c}", steps=rng.choice([5, 5, 5, 4, 6]),
                 pad=rng.choice([0, 0, 8, rng.randrange(1, 100)]))
    elif op == "momentum":
        c2 = _momentum(None, _log(rng, 1000, 1 << 27), rng.choice([1, 2, 3, 4, 8]),
                       acc=rng.random() < 0.5, nesterov=rng.random() < 0.7)
    else:
        c2 = _update(None, _log(rng, 1000, 1 << 27))
    del c2["name"]
    return c2


def _groups(case):
    return [tuple(int(x) for x in g.split("x")) for g in case["mats"].split(",")]


def _ns_flops(r, c):
    """One step on one matrix: the Gram matrix and its square have only half
    their entries to compute, the last product all of them."""
    m, n = min(r, c), max(r, c)
    return m * m * n + m * m * m + 2 * m * m * n


def work(case):
    if case["op"] == "ns":
        g = _groups(case)
        return {"bytes": sum(4 * b * r * c for b, r, c in g),
                "flops": case["steps"] * sum(b * _ns_flops(r, c) for b, r, c in g)}
    n = case["n"]
    if case["op"] == "momentum":
        R = case["peers"]
        return {"bytes": n * (2 * R + (4 if case["acc"] else 0) + 4 + 4 + 2),
                "flops": n * (R + 8)}
    return {"bytes": n * (2 + 4 + 4 + 2), "flops": 4 * n}


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "ns":
        # momentum of a weight matrix: a few strong directions of falling
        # strength over the noise of the batch, at a gradient's size
        mats = []
        for b, r, c in _groups(case):
            k = min(32, r, c)
            fall = torch.arange(1, k + 1, device=dev).float().pow(-0.5)
            strong = torch.matmul(normal(b, r, k) * fall, normal(b, k, c))
            u = (strong + normal(b, r, c)).mul_(1e-3).bfloat16()
            if case["pad"]:
                wide = torch.zeros(b, r, c + case["pad"], dtype=torch.bfloat16, device=dev)
                wide[:, :, :c] = u
                u = wide[:, :, :c]
            mats.append(u)
        return {"case": case, "mats": mats}
    n = case["n"]
    if case["op"] == "momentum":
        return {"case": case, "scale": 1.0 / case["peers"], "mu": 0.95,
                "peers": [normal(n).mul_(1e-3).bfloat16() for _ in range(case["peers"])],
                "acc": normal(n).mul_(2e-3) if case["acc"] else None,
                "m": normal(n).mul_(3e-4),
                "u": torch.empty(n, dtype=torch.bfloat16, device=dev)}
    # an orthogonalised direction's entries are of the size 1 / sqrt(columns)
    return {"case": case, "lr": 0.02, "wd": 0.1,
            "u": normal(n).mul_(1 / 64).bfloat16(), "master": normal(n).mul_(0.02),
            "param": torch.empty(n, dtype=torch.bfloat16, device=dev)}


# ---- one pass ----------------------------------------------------------------

def _plain_ns(u, steps):
    """One group [B, rows, cols], on the side with the smaller Gram matrix."""
    tall = u.shape[1] > u.shape[2]
    x = (u.mT if tall else u).float().contiguous()
    x = x / x.square().sum((1, 2), keepdim=True).sqrt().clamp(min=EPS)
    a, b, c = COEFS
    for _ in range(steps):
        gram = torch.matmul(x, x.mT.contiguous())
        poly = b * gram + c * torch.matmul(gram, gram)
        x = a * x + torch.matmul(poly, x)
    return (x.mT if tall else x).bfloat16().contiguous()


def _plain_momentum(s):
    g = torch.stack(s["peers"]).float().sum(0) if len(s["peers"]) > 1 else s["peers"][0].float()
    if s["acc"] is not None:
        g = s["acc"] + g
    g = g * s["scale"]
    mu = s["mu"]
    s["m"].mul_(mu).add_(g, alpha=1 - mu)
    s["u"].copy_((1 - mu) * g + mu * s["m"] if s["case"]["nesterov"] else s["m"])


def _plain_update(s):
    s["master"].mul_(1 - s["lr"] * s["wd"]).sub_(s["lr"] * s["u"].float())
    s["param"].copy_(s["master"])


def run(state):
    case = state["case"]
    if own:
        import sharded_bucket_plan_amd as sbp
    if case["op"] == "ns":
        if own:
            return sbp.newton_schulz(state["mats"], steps=case["steps"], coefs=COEFS, eps=EPS)
        return [_plain_ns(u, case["steps"]) for u in state["mats"]]
    if case["op"] == "momentum":
        if own:
            sbp.momentum_shard(state["peers"], state["acc"], state["scale"], state["m"],
                               state["u"], state["mu"], nesterov=case["nesterov"])
        else:
            _plain_momentum(state)
        return {"m": state["m"], "u": state["u"]}
    if own:
        sbp.update_shard(state["u"], state["master"], state["param"], state["lr"], state["wd"])
    else:
        _plain_update(state)
    return {"master": state["master"], "param": state["param"]}


# ---- the definition in 64 bits ---------------------------------------------------

def _exact_ns(u, steps):
    """X <- a X + b (X X') X + c (X X')^2 X from X = U / max(|U|, eps), written
    for X' where the matrix is tall (the iteration is the same on both sides)."""
    w = u.double()
    w = w / torch.linalg.vector_norm(w).clamp(min=EPS)
    a, b, c = COEFS
    left = w.shape[0] <= w.shape[1]
    for _ in range(steps):
        if left:
            s = w @ w.T.contiguous()
            w = a * w + b * (s @ w) + c * (s @ (s @ w))
        else:
            s = w.T.contiguous() @ w
            w = a * w + b * (w @ s) + c * ((w @ s) @ s)
    return w


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ns":
        return [torch.stack([_exact_ns(x, case["steps"]) for x in u]) for u in s["mats"]]
    if case["op"] == "momentum":
        g = torch.zeros(case["n"], dtype=torch.float64, device="cuda")
        for p in s["peers"]:
            g += p.double()
        if s["acc"] is not None:
            g += s["acc"].double()
        g *= s["scale"]
        m = s["mu"] * s["m"].double() + (1 - s["mu"]) * g
        return {"m": m, "u": (1 - s["mu"]) * g + s["mu"] * m if case["nesterov"] else m}
    th = (1 - s["lr"] * s["wd"]) * s["master"].double() - s["lr"] * s["u"].double()
    return {"master": th, "param": th}
