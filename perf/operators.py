"""Cases of the Muon step's operators: the momentum step of an owner's shard,
alone and fused with the reduce-scatter, the orthogonalisation of update
matrices by Newton-Schulz products, and the owner update that applies them.

Each case can run in a plain form (elementary torch operations in FP32, one
rounding at the end) or, with `own` set, through the package's entry points.
"""
import math

import torch

own = False

COEFS = ((3.4445, -4.7750, 2.0315),) * 5   # the quintic's a, b, c, five times
MOMENTUM, NESTEROV = 0.95, True
LR, DECAY = 1e-3, 0.1
DEV = "cuda"


def listed():
    return [
        # one small projection: the call is a matter of latency
        dict(name="ns small 64x256", op="ns", mats=1, rows=64, cols=256, dtype="bf16", pad=0),
        # 32 experts' matrices of one layer in one call
        dict(name="ns experts 32x512x1024", op="ns", mats=32, rows=512, cols=1024, dtype="bf16", pad=0),
        # FP32 momentum matrices with odd sides inside a wider buffer
        dict(name="ns odd f32 3x777x1301", op="ns", mats=3, rows=777, cols=1301, dtype="f32", pad=11),
        # k and v of a layer of the 8B Llama-like chain
        dict(name="ns kv 2x1024x4096", op="ns", mats=2, rows=1024, cols=4096, dtype="bf16", pad=0),
        # q of the 7B-class layer and of the chain
        dict(name="ns q 4096x4096", op="ns", mats=1, rows=4096, cols=4096, dtype="bf16", pad=0),
        # gate and up of a layer of the chain: tall, the largest product
        dict(name="ns gate/up 2x14336x4096", op="ns", mats=2, rows=14336, cols=4096, dtype="bf16", pad=0),
        # an owner's shard of the tiny flat unit
        dict(name="momentum tiny shard", op="momentum", n=262144, clip=False),
        # an owner's shard of a chain layer, with the clip coefficient on the device
        dict(name="momentum layer shard", op="momentum", n=54525952, clip=True),
        # the last micro-batch of an odd-sized owner share: two ranks, accumulated gradient
        dict(name="reduce+momentum odd", op="reduce", ranks=2, shards=1, n=1000003, acc=True),
        # the whole 7B-class layer: four ranks, four owners
        dict(name="reduce+momentum layer", op="reduce", ranks=4, shards=4, n=202375168, acc=False),
        # the owner update on the same shards as the momentum step's
        dict(name="update tiny shard", op="update", n=262144, device_lr=False),
        dict(name="update layer shard", op="update", n=54525952, device_lr=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm; half of them odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, v | 1) if rng.random() < 0.5 else max(lo, v & ~7)


def draw(rng):
    op = rng.choice(("ns", "ns", "momentum", "reduce", "update"))
    if op == "ns":
        most = work(listed()[5])["flops"]
        k = _spread(rng, 24, 4096)
        l = max(k, int(k * rng.uniform(1.0, 4.0)))
        if rng.random() < 0.5:
            l = -(-l // 16) * 16
        rows, cols = (k, l) if rng.random() < 0.5 else (l, k)
        mats = rng.choice((1, 1, 2, 3, 8, 16))
        case = dict(op=op, mats=mats, rows=rows, cols=cols, dtype=rng.choice(("bf16", "bf16", "f32")),
                    pad=rng.choice((0, 0, 5, 64)))
        while work(case)["flops"] > 0.5 * most:
            case["mats"] = max(1, case["mats"] // 2)
            if case["mats"] == 1:
                break
        return case
    n = _spread(rng, 1000, 30000000)
    if op == "momentum":
        return dict(op=op, n=n, clip=rng.random() < 0.5)
    if op == "update":
        return dict(op=op, n=n, device_lr=rng.random() < 0.5)
    shards = rng.choice((1, 2, 4))
    return dict(op=op, ranks=rng.choice((1, 2, 3, 4, 8)), shards=shards, n=n * shards, acc=rng.random() < 0.5)


def work(case):
    if case["op"] == "ns":
        k, l = sorted((case["rows"], case["cols"]))
        size = 2 if case["dtype"] == "bf16" else 4
        # Symmetric products at half their price. Step by step each step is a
        # Gram product, its square and the product with X; the factors
        # are polynomials of the same matrix, so two steps can also share one
        # product with X: the cheaper of the two for each pair of steps.
        steps = len(COEFS)
        alone = 2 * (3 * k * k * l + k ** 3)
        pair = 3 * k * k * l + 5 * k ** 3
        flops = (steps // 2) * min(alone, pair) + (steps % 2) * alone / 2
        return dict(bytes=case["mats"] * k * l * (size + 2), flops=case["mats"] * flops)
    n = case["n"]
    if case["op"] == "momentum":
        return dict(bytes=14 * n, flops=(7 if case["clip"] else 6) * n)
    if case["op"] == "update":
        return dict(bytes=12 * n, flops=4 * n)
    r = case["ranks"]
    return dict(bytes=n * (2 * r + 10 + (4 if case["acc"] else 0)), flops=n * (2 * r - 1 + 6 + case["acc"]))


def _normal(gen, n, sigma):
    return torch.empty(n, dtype=torch.float32, device=DEV).normal_(0.0, sigma, generator=gen)


def _matrices(gen, case):
    """Momentum-like matrices: noise, and a few stronger directions of
    falling strength, as gradients of many tokens have."""
    b, m, n = case["mats"], case["rows"], case["cols"]
    r = max(1, min(32, min(m, n) // 4))
    strength = torch.arange(1, r + 1, dtype=torch.float32, device=DEV).rsqrt() / math.sqrt(r)
    left = _normal(gen, b * m * r, 1.0).view(b, m, r) * strength
    right = _normal(gen, b * r * n, 1.0).view(b, r, n)
    return (left @ right + _normal(gen, b * m * n, 1.0).view(b, m, n)) * 1e-3


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(op=case["op"])
    if case["op"] == "ns":
        b, m, n = case["mats"], case["rows"], case["cols"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        wide = torch.zeros(b, m, n + case["pad"], dtype=dtype, device=DEV)
        s["g"] = wide[:, :, :n]
        s["g"].copy_(_matrices(gen, case))
        s["scale"] = 0.2 * math.sqrt(max(m, n))   # the update's RMS near Adam's
        s["out"] = torch.empty(b, m, n, dtype=torch.bfloat16, device=DEV)
        return s
    n = case["n"]
    s["hp"] = dict(lr=LR, momentum=MOMENTUM, weight_decay=DECAY, nesterov=NESTEROV)
    if case["op"] == "update":
        s["master"] = _normal(gen, n, 0.02)
        s["o"] = _normal(gen, n, 0.2).to(torch.bfloat16)
        s["bf16"] = torch.empty(n, dtype=torch.bfloat16, device=DEV)
        s["lr"] = torch.full((1,), 3e-4, dtype=torch.float32, device=DEV) if case["device_lr"] else None
        return s
    if case["op"] == "momentum":
        s["m"] = _normal(gen, n, 3e-4)
        s["u"] = torch.empty(n, dtype=torch.bfloat16, device=DEV)
        s["g"] = _normal(gen, n, 1e-3)
        s["clip"] = torch.full((1,), 0.37, dtype=torch.float32, device=DEV) if case["clip"] else None
        return s
    k, r = case["shards"], case["ranks"]
    s["x"] = [_normal(gen, n, 1e-3).to(torch.bfloat16) for _ in range(r)]
    s["w"] = _weights(r)
    s["m"] = [_normal(gen, n // k, 3e-4) for _ in range(k)]
    s["u"] = [torch.empty(n // k, dtype=torch.bfloat16, device=DEV) for _ in range(k)]
    s["acc"] = [_normal(gen, n // k, 1e-3) for _ in range(k)] if case["acc"] else None
    return s


def _weights(ranks):
    """Rank weights by token counts, as FP32 values."""
    counts = torch.tensor([4096.0, 2048.0, 1024.0, 4096.0, 512.0, 2048.0, 4096.0, 1024.0][:ranks], dtype=torch.float64)
    return (counts / counts.sum()).to(torch.float32).tolist()


# ------------------------------------------------------------------ plain forms
def _plain_ns(g, scale):
    x = g.to(torch.float32)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    norm = x.double().square().sum(dim=(1, 2), keepdim=True).sqrt()
    x = (x.double() / norm).to(torch.float32)
    for a, b, c in COEFS:
        gram = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if tall:
        x = x.transpose(1, 2)
    return (x * scale).to(torch.bfloat16).contiguous()


def _plain_momentum(m, g, hp):
    beta = torch.tensor(hp["momentum"], dtype=torch.float32)
    rest = 1.0 - beta   # an FP32 subtraction
    fresh = rest * g
    m.mul_(beta).add_(fresh)
    return (fresh + beta * m if hp["nesterov"] else m).to(torch.bfloat16)


def _plain(s):
    if s["op"] == "ns":
        return _plain_ns(s["g"], s["scale"])
    hp = s["hp"]
    if s["op"] == "momentum":
        g = s["g"] if s["clip"] is None else s["g"] * s["clip"]
        return [s["m"], _plain_momentum(s["m"], g, hp)]
    if s["op"] == "update":
        p = s["master"]
        lr = s["lr"] if s["lr"] is not None else hp["lr"]
        p.sub_((s["o"].to(torch.float32) + p * hp["weight_decay"]) * lr)
        return [p, p.to(torch.bfloat16)]
    n = s["m"][0].numel()
    red = s["x"][0].to(torch.float32) * s["w"][0]
    for x, w in zip(s["x"][1:], s["w"][1:]):
        red += x.to(torch.float32) * w
    parts = list(red.split(n))
    if s["acc"] is not None:
        parts = [a + p for a, p in zip(s["acc"], parts)]
    return [s["m"], [_plain_momentum(m, p, hp) for m, p in zip(s["m"], parts)]]


# ------------------------------------------------------------------ the package's entry points
def _package(s):
    import zero_sharded_optimizer_reduce_amd as z
    if s["op"] == "ns":
        if "workspace" not in s:
            s["workspace"] = z.zero_newton_schulz_workspace(s["g"])
        z.zero_newton_schulz(s["g"], s["out"], s["workspace"], coefs=COEFS, scale=s["scale"])
        return s["out"]
    if s["op"] == "momentum":
        z.zero_muon_momentum(s["m"], s["u"], s["g"], s["hp"], grad_scale=s["clip"])
        return [s["m"], s["u"]]
    if s["op"] == "update":
        z.zero_muon_shard_step(s["master"], s["bf16"], s["o"], s["hp"], lr_dev=s["lr"])
        return [s["master"], s["bf16"]]
    z.zero_reduce_scatter_muon(s["x"], s["w"], s["m"], s["u"], s["hp"], grad_acc=s["acc"])
    return [s["m"], s["u"]]


def run(state):
    return _package(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "ns":
        outs = []
        for g in s["g"]:
            y = g.double()
            y = y / torch.linalg.matrix_norm(y)
            side = y.shape[0] <= y.shape[1]
            for a, b, c in COEFS:
                # on the smaller side; both sides give the same polynomial of the singular values
                p = torch.mm(y, y.T) if side else torch.mm(y.T, y)
                q = b * p + c * torch.mm(p, p)
                q.diagonal().add_(a)
                y = torch.mm(q, y) if side else torch.mm(y, q)
            outs.append(y * s["scale"])
        return torch.stack(outs)
    beta, lr, wd = (float(torch.tensor(v, dtype=torch.float32)) for v in (MOMENTUM, LR, DECAY))
    if s["op"] == "update":
        if s["lr"] is not None:
            lr = float(s["lr"])
        p = s["master"].double()
        p = p - lr * (s["o"].double() + wd * p)
        return [p, p]
    if s["op"] == "momentum":
        g = s["g"].double() * (1.0 if s["clip"] is None else float(s["clip"]))
        m = beta * s["m"].double() + (1.0 - beta) * g
        return [m, (1.0 - beta) * g + beta * m]
    k = case["shards"]
    g = torch.zeros(case["n"], dtype=torch.float64, device=DEV)
    for x, w in zip(s["x"], s["w"]):
        g.addcmul_(x.double(), torch.tensor(w, dtype=torch.float64, device=DEV))
    g = g.view(k, -1)
    ms, us = [], []
    for i in range(k):
        gi = g[i] + s["acc"][i].double() if s["acc"] is not None else g[i]
        mi = beta * s["m"][i].double() + (1.0 - beta) * gi
        ms.append(mi)
        us.append((1.0 - beta) * gi + beta * mi)
    return [ms, us]
