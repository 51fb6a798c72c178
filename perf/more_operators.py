"""Cases of a layer's gated feed-forward block, forward and backward, and of the
8-bit activation checkpoints that its backward pass reads.

    h = act(x Wg^T) * (x Wu^T),   y = h Wd^T

x: tokens x model, Wg and Wu: hidden x model, Wd: model x hidden.  A checkpoint
holds 8 bits per value and a power of two per 32 neighbours of a row: the least
one with which the largest of them fits (127 as whole numbers, 448 as e4m3).
The backward pass takes x, x Wg^T and x Wu^T from checkpoints.

Each case can run in a plain form (elementary torch operations in FP32, one
rounding at the end) or, with `own` set, through the package's entry points.
"""
import math

import torch

own = False

BLOCK = 32
LIMIT = dict(int8=127.0, e4m3=448.0)   # the largest value of a format
DEV = "cuda"


def listed():
    return [
        # a short piece of FP32 activations of odd width through a checkpoint and back: latency
        dict(name="checkpoint odd f32 77x1301", op="checkpoint", rows=77, cols=1301, dtype="f32", format="int8", pad=0),
        # the hidden activations of a layer of the 8B Llama-like chain, 16384 tokens
        dict(name="checkpoint 16384x14336", op="checkpoint", rows=16384, cols=14336, dtype="bf16", format="int8", pad=0),
        # a checkpoint of ragged size read back into a wider buffer
        dict(name="load odd e4m3 1999x4101", op="load", rows=1999, cols=4101, dtype="bf16", format="e4m3", pad=3),
        # a layer's hidden activations read back
        dict(name="load 16384x14336", op="load", rows=16384, cols=14336, dtype="bf16", format="int8", pad=0),
        # one token through a layer of the chain: the weights' way from memory
        dict(name="forward 1 token chain", op="forward", tokens=1, model=4096, hidden=14336, act="silu", format="", pad=0),
        # a handful of requests' next tokens through the 7B-class layer
        dict(name="forward 24 tokens layer7b", op="forward", tokens=24, model=4096, hidden=11008, act="silu", format="", pad=0),
        # odd sizes throughout, with checkpoints
        dict(name="forward odd 777x1301x1999", op="forward", tokens=777, model=1301, hidden=1999, act="gelu", format="e4m3", pad=5),
        # a rank's micro-batch through a layer of the chain, with checkpoints
        dict(name="forward 8192 tokens chain", op="forward", tokens=8192, model=4096, hidden=14336, act="silu", format="int8", pad=0),
        # a small block, where launches count
        dict(name="backward 256x512x1408", op="backward", tokens=256, model=512, hidden=1408, act="silu", format="int8", pad=0),
        # odd sizes throughout
        dict(name="backward odd 1001x1301x777", op="backward", tokens=1001, model=1301, hidden=777, act="relu", format="e4m3", pad=5),
        # the 7B-class layer, a ragged batch of tokens
        dict(name="backward 3999 tokens layer7b", op="backward", tokens=3999, model=4096, hidden=11008, act="gelu", format="e4m3", pad=0),
        # a rank's micro-batch through a layer of the chain
        dict(name="backward 8192 tokens chain", op="backward", tokens=8192, model=4096, hidden=14336, act="silu", format="int8", pad=0),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm; a third of them odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.random()
    step = 64 if kind < 0.45 else 8
    return min(hi, max(lo, v | 1 if kind > 0.67 else v // step * step))


def draw(rng):
    op = rng.choice(("checkpoint", "load", "forward", "forward", "backward", "backward"))
    format = rng.choice(("int8", "e4m3"))
    if op in ("checkpoint", "load"):
        cols = _spread(rng, 40, 14336)
        rows = min(_spread(rng, 4, 16384), 16384 * 14336 // cols)
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(("bf16", "bf16", "f32")), format=format,
                    pad=rng.choice((0, 0, 3, 64)))
    case = dict(op=op, tokens=_spread(rng, 1 if op == "forward" else 16, 8192), model=_spread(rng, 128, 4096),
                hidden=_spread(rng, 192, 14336), act=rng.choice(("silu", "silu", "gelu", "relu")), format=format,
                pad=rng.choice((0, 0, 5, 64)))
    if op == "forward" and (case["tokens"] < 64 or rng.random() < 0.3):
        case["format"] = ""
    return case


def _held(rows, cols):
    """Bytes of a checkpoint."""
    return rows * (cols + -(-cols // BLOCK))


def work(case):
    if case["op"] in ("checkpoint", "load"):
        r, c = case["rows"], case["cols"]
        size = 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "load":
            return dict(bytes=_held(r, c) + r * c * size, flops=r * c)
        return dict(bytes=2 * r * c * size + 2 * _held(r, c), flops=4 * r * c)
    t, d, f = case["tokens"], case["model"], case["hidden"]
    held = _held(t, d) + 2 * _held(t, f)
    if case["op"] == "backward":
        return dict(bytes=12 * d * f + 4 * t * d + held, flops=12 * t * d * f)
    # checkpoints are written, and read back as BF16 values
    back = 2 * held + 2 * t * (d + 2 * f) if case["format"] else 0
    return dict(bytes=6 * d * f + 4 * t * d + back, flops=6 * t * d * f)


def _normal(gen, shape, sigma):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, sigma, generator=gen)


def _wide(rows, cols, pad, dtype):
    """A matrix inside a wider buffer."""
    return torch.zeros(rows, cols + pad, dtype=dtype, device=DEV)[:, :cols]


def _activations(gen, rows, cols):
    """Values as a norm's output has them: a few channels far stronger than the others."""
    x = _normal(gen, (rows, cols), 1.0)
    strength = _normal(gen, (cols,), 0.4).exp()
    strength[torch.randint(0, cols, (max(1, cols // 256),), device=DEV, generator=gen)] *= 12.0
    return x * strength


def _held_values(gen, rows, cols, format):
    """A checkpoint (codes, scales) of gate-like activations."""
    return _quantise(_activations(gen, rows, cols), format)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] in ("checkpoint", "load"):
        r, c = case["rows"], case["cols"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["out"] = _wide(r, c, case["pad"], dtype)
        if case["op"] == "load":
            s["held"] = _held_values(gen, r, c, case["format"])
        else:
            s["x"] = _wide(r, c, case["pad"], dtype)
            s["x"].copy_(_activations(gen, r, c))
            s["held"] = _space(r, c)
        return s
    t, d, f = case["tokens"], case["model"], case["hidden"]
    s["w"] = [_normal(gen, shape, sigma).to(torch.bfloat16)
              for shape, sigma in (((f, d), 1.0 / math.sqrt(d)), ((f, d), 1.0 / math.sqrt(d)), ((d, f), 1.0 / math.sqrt(f)))]
    x = _activations(gen, t, d)
    if case["op"] == "forward":
        s["x"] = _wide(t, d, case["pad"], torch.bfloat16)
        s["x"].copy_(x)
        s["y"] = _wide(t, d, case["pad"], torch.bfloat16)
        if case["format"]:
            s["held"] = [_space(t, d), _space(t, f), _space(t, f)]
            s["values"] = [torch.empty(t, n, dtype=torch.bfloat16, device=DEV) for n in (d, f, f)]
        return s
    wide = x.to(torch.bfloat16).to(torch.float32)
    s["held"] = [_quantise(v, case["format"])
                 for v in (wide, wide @ s["w"][0].to(torch.float32).T, wide @ s["w"][1].to(torch.float32).T)]
    s["dy"] = _wide(t, d, case["pad"], torch.bfloat16)
    s["dy"].copy_(_normal(gen, (t, d), 1e-3) * _normal(gen, (t, 1), 0.5).exp())
    s["dx"] = _wide(t, d, case["pad"], torch.bfloat16)
    s["dw"] = [torch.empty_like(w) for w in s["w"]]
    return s


# ------------------------------------------------------------------ plain forms
def _space(rows, cols):
    return (torch.zeros(rows, cols, dtype=torch.uint8, device=DEV),
            torch.zeros(rows, -(-cols // BLOCK), dtype=torch.uint8, device=DEV))


def _power(e):
    """2^e as FP32, e a tensor of whole numbers in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _blocks(x):
    rows, cols = x.shape
    fill = -cols % BLOCK
    if fill:
        x = torch.cat((x, x.new_zeros(rows, fill)), dim=1)
    return x.view(rows, -1, BLOCK)


def _quantise(x, format):
    rows, cols = x.shape
    b = _blocks(x.to(torch.float32))
    mantissa, e = torch.frexp(b.abs().amax(dim=2))
    top, shift = math.frexp(LIMIT[format])
    e = (e - shift + (mantissa > top)).to(torch.int32).clamp(min=-126)
    v = b * _power(-e).unsqueeze(2)
    v = v.round().to(torch.int8) if format == "int8" else v.to(torch.float8_e4m3fn)
    return v.view(torch.uint8).view(rows, -1)[:, :cols].contiguous(), (e + 127).to(torch.uint8)


def _values(held, format):
    """FP32 values of a checkpoint."""
    codes, scales = held
    v = codes.view(torch.int8 if format == "int8" else torch.float8_e4m3fn).to(torch.float32)
    s = _power(scales.to(torch.int32) - 127).repeat_interleave(BLOCK, dim=1)
    return v * s[:, :codes.shape[1]]


def _activate(g, act):
    """act(g) and its derivative."""
    if act == "relu":
        slope = (g > 0).to(torch.float32)
        return g * slope, slope
    if act == "silu":
        p = 1.0 / (1.0 + (-g).exp())
        return g * p, p * (1.0 + g * (1.0 - p))
    c = math.sqrt(2.0 / math.pi)
    t = (c * (g + 0.044715 * g * g * g)).tanh()
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _plain(s):
    if s["op"] == "load":
        s["out"].copy_(_values(s["held"], s["format"]))
        return s["out"]
    if s["op"] == "checkpoint":
        s["out"].copy_(_values(_quantise(s["x"], s["format"]), s["format"]))
        return s["out"]
    wg, wu, wd = (w.to(torch.float32) for w in s["w"])
    if s["op"] == "forward":
        x = s["x"].to(torch.float32)
        g, u = x @ wg.T, x @ wu.T
        s["y"].copy_((_activate(g, s["act"])[0] * u) @ wd.T)
        if not s["format"]:
            return [s["y"]]
        return [s["y"], *(_values(_quantise(v, s["format"]), s["format"]).to(torch.bfloat16) for v in (x, g, u))]
    x, g, u = (_values(h, s["format"]) for h in s["held"])
    dy = s["dy"].to(torch.float32)
    a, slope = _activate(g, s["act"])
    dh = dy @ wd
    dg, du = dh * u * slope, dh * a
    s["dx"].copy_(dg @ wg + du @ wu)
    for out, left, right in zip(s["dw"], (dg, du, dy), (x, x, a * u)):
        out.copy_(left.T @ right)
    return [s["dx"], *s["dw"]]


# ------------------------------------------------------------------ the package's entry points
def _package(s):
    import zero_sharded_optimizer_reduce_amd as z
    if s["op"] == "load":
        z.zero_act8_load(*s["held"], s["out"], format=s["format"])
        return s["out"]
    if s["op"] == "checkpoint":
        z.zero_act8_save(s["x"], *s["held"], format=s["format"])
        z.zero_act8_load(*s["held"], s["out"], format=s["format"])
        return s["out"]
    t, d, f = s["tokens"], s["model"], s["hidden"]
    if "workspace" not in s:
        s["workspace"] = z.zero_ffn_workspace(t, d, f, backward=s["op"] == "backward")
        s["checkpoint"] = z.FfnCheckpoint(*s["held"], format=s["format"]) if s["format"] else None
    if s["op"] == "forward":
        z.zero_ffn_forward(s["x"], *s["w"], s["y"], s["workspace"], activation=s["act"], checkpoint=s["checkpoint"])
        if not s["format"]:
            return [s["y"]]
        for held, values in zip(s["held"], s["values"]):
            z.zero_act8_load(*held, values, format=s["format"])
        return [s["y"], *s["values"]]
    z.zero_ffn_backward(s["dy"], s["checkpoint"], *s["w"], s["dx"], *s["dw"], s["workspace"], activation=s["act"])
    return [s["dx"], *s["dw"]]


def run(state):
    return _package(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _nearest(x, format):
    """Each value's nearest among those that its block's checkpoint can hold, ties to even."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x.double(), (0, -cols % BLOCK)).reshape(rows, -1, BLOCK)
    largest = b.abs().max(dim=2, keepdim=True).values
    exponent = torch.log2(largest.clamp(min=2.0 ** -120) / LIMIT[format]).ceil()
    # log2 may be off by a rounding next to a whole number
    exponent = torch.where(largest > LIMIT[format] * torch.exp2(exponent), exponent + 1, exponent)
    exponent = torch.where(largest <= LIMIT[format] * torch.exp2(exponent - 1), exponent - 1, exponent)
    unit = torch.exp2(exponent)
    if format == "e4m3":   # three bits behind the leading one, down to 2^-9
        unit = unit * torch.exp2(torch.floor(torch.log2((b.abs() / unit).clamp(min=2.0 ** -6))) - 3)
    return (torch.round(b / unit) * unit).reshape(rows, -1)[:, :cols]


def _standing_for(held, format):
    codes, scales = held
    if format == "int8":
        v = torch.where(codes > 127, codes.double() - 256.0, codes.double())
    else:
        exponent, mantissa = (codes >> 3) & 15, (codes & 7).double()
        v = torch.where(exponent > 0, (1.0 + mantissa / 8.0) * torch.exp2(exponent.double() - 7.0), mantissa * 2.0 ** -9)
        v = torch.where(codes > 127, -v, v)
    at = torch.arange(codes.shape[1], device=DEV) // BLOCK
    return v * torch.exp2(scales.double() - 127.0)[:, at]


def _act64(g, act):
    g = g.detach().requires_grad_(True)
    if act == "relu":
        a = torch.nn.functional.relu(g)
    elif act == "silu":
        a = torch.nn.functional.silu(g)
    else:
        a = torch.nn.functional.gelu(g, approximate="tanh")
    slope, = torch.autograd.grad(a.sum(), g)
    return a.detach(), slope


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "load":
        return _standing_for(s["held"], case["format"])
    if case["op"] == "checkpoint":
        return _nearest(s["x"], case["format"])
    gate, up, down = (w.double() for w in s["w"])
    if case["op"] == "forward":
        x = s["x"].double()
        g, u = torch.mm(x, gate.t()), torch.mm(x, up.t())
        y = torch.mm(_act64(g, case["act"])[0] * u, down.t())
        return [y, *(_nearest(v, case["format"]) for v in (x, g, u))] if case["format"] else [y]
    x, g, u = (_standing_for(h, case["format"]) for h in s["held"])
    dy = s["dy"].double()
    a, slope = _act64(g, case["act"])
    dh = torch.mm(dy, down)
    dg, du = dh.mul(u).mul(slope), dh.mul(a)
    return [torch.mm(dg, gate) + torch.mm(du, up), torch.mm(dg.t(), x), torch.mm(du.t(), x), torch.mm(dy.t(), a * u)]
