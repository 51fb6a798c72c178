"""Plain 64-bit implementations of the feed-forward block and of the 8-bit
activations, and inputs whose results are exact: test infrastructure."""
import math

import torch

BLOCK = 32
LIMIT = {"int8": 127.0, "e4m3": 448.0}


def power(e):
    """2^e in FP64 of whole numbers in [-400, 400], from a table: torch.ldexp's powers
    on the GPU are not all exact."""
    table = torch.tensor([math.ldexp(1.0, k) for k in range(-400, 401)], dtype=torch.float64, device=e.device)
    return table[e.to(torch.int64) + 400]


def e4m3_values():
    """The value of each of the 256 codes."""
    v = []
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        x = math.ldexp(f, -9) if e == 0 else math.ldexp(1 + f / 8, e - 7)
        v.append(math.nan if e == 15 and f == 7 else -x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64)


def scale_exponents(x, fmt):
    """e of each block of 32 columns of x (FP64, finite), by search among whole numbers."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    pad = torch.zeros(rows, nb * BLOCK, dtype=torch.float64, device=x.device)
    pad[:, :cols] = x
    top = pad.view(rows, nb, BLOCK).abs().amax(dim=2)
    e = torch.full_like(top, -126, dtype=torch.int64)
    # the least e >= -126 with top <= limit * 2^e
    for k in range(-126, 122):
        e = torch.where(top > LIMIT[fmt] * math.ldexp(1.0, k), torch.full_like(e, k + 1), e)
    return e


def quantised(x, fmt):
    """(values that the checkpoint of x stands for, scale bytes); FP64, from x in FP64 without NaN or infinity."""
    rows, cols = x.shape
    e = scale_exponents(x, fmt)
    s = power(e).repeat_interleave(BLOCK, dim=1)[:, :cols]
    v = x / s
    if fmt == "int8":
        q = torch.round(v)
    else:
        m, k = torch.frexp(v.abs())   # v = m 2^k, m in [1/2, 1): a step is 2^(k - 4), at least 2^-9
        step = power(torch.clamp(k - 4, min=-9))
        q = torch.round(v / step) * step
    return q * s, (e + 127).to(torch.uint8)


def held_values(codes, scales, fmt):
    """FP64 values of a checkpoint."""
    table = (torch.arange(256, dtype=torch.float64) if fmt == "int8" else e4m3_values()).to(codes.device)
    if fmt == "int8":
        table = torch.where(table > 127, table - 256, table)
    v = table[codes.long()]
    s = power(scales.to(torch.int64) - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return v * s.repeat_interleave(BLOCK, dim=1)[:, :codes.shape[1]]


def act64(g, act):
    """act(g) and its derivative in 64 bits."""
    if act == "relu":
        return torch.clamp(g, min=0), (g > 0).to(g.dtype)
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def forward64(x, wg, wu, wd, act):
    g, u = x @ wg.T, x @ wu.T
    h = act64(g, act)[0] * u
    return g, u, h, h @ wd.T


def backward64(dy, x, g, u, wg, wu, wd, act):
    """dx, d_gate, d_up, d_down from the checkpoint's values."""
    a, slope = act64(g, act)
    dh = dy @ wd
    dg, du = dh * u * slope, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ (a * u)


def sparse_signs(gen, rows, cols, most, device="cuda"):
    """A matrix of 0 and +-1 (BF16) with at most `most` nonzeros in a row: sums of
    products of such matrices are whole numbers, exact in every order."""
    m = torch.zeros(rows, cols)
    if rows and cols:
        at = torch.randint(0, cols, (rows, min(most, cols)), generator=gen)
        m.scatter_(1, at, torch.randint(0, 2, at.shape, generator=gen).float() * 2 - 1)
    return m.to(torch.bfloat16).to(device)


def signs(gen, rows, cols, device="cuda"):
    return (torch.randint(0, 2, (rows, cols), generator=gen).float() * 2 - 1).to(torch.bfloat16).to(device)


def small_checkpoint(gen, rows, cols, top, device="cuda"):
    """Whole numbers in [-top, top] (top <= 8) as (codes, scales, FP64 values) of an int8 checkpoint with scale 1."""
    v = torch.randint(-top, top + 1, (rows, cols), generator=gen)
    codes = v.to(torch.int8).view(torch.uint8).contiguous()
    scales = torch.full((rows, -(-cols // BLOCK)), 127, dtype=torch.uint8)
    return codes.to(device), scales.to(device), v.to(torch.float64).to(device)
