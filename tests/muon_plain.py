"""Plain forms of the Muon step's operators for the tests: binary32 arrays, one
operation rounded at a time, and float64 definitions."""
from __future__ import annotations

import numpy as np
import torch

F = np.float32
COEFS = ((3.4445, -4.7750, 2.0315),) * 5


def to_bf16(x: np.ndarray) -> np.ndarray:
    """float32 -> bfloat16 bit patterns (round to nearest even)."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=F)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def from_bf16(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(F)


def reduce_ranks(bits, weights, acc=None):
    red = F(weights[0]) * from_bf16(bits[0])
    for b, w in zip(bits[1:], weights[1:]):
        red = red + F(w) * from_bf16(b)
    return red if acc is None else acc + red


def momentum_f32(m, g, beta, nesterov, scale=None):
    """(m', direction bits), every operation one binary32 rounding."""
    b = F(beta)
    rest = F(1.0) - b
    if scale is not None:
        g = g * F(scale)
    fresh = rest * g
    m1 = b * m + fresh
    u = fresh + b * m1 if nesterov else m1
    return m1, to_bf16(u)


def momentum_f64(m, g, beta, nesterov, scale=None):
    b = np.float64(F(beta))
    g = g.astype(np.float64) * (1.0 if scale is None else np.float64(F(scale)))
    m1 = b * m.astype(np.float64) + (1.0 - b) * g
    return m1, (1.0 - b) * g + b * m1 if nesterov else m1


def update_f32(p, o_bits, lr, wd):
    u = from_bf16(o_bits)
    if wd != 0.0:
        u = u + F(wd) * p
    p1 = p - F(lr) * u
    return p1, to_bf16(p1)


def update_f64(p, o_bits, lr, wd):
    p = p.astype(np.float64)
    return p - np.float64(F(lr)) * (from_bf16(o_bits).astype(np.float64) + np.float64(F(wd)) * p)


def newton_schulz_f64(g: torch.Tensor, coefs=COEFS, scale: float = 1.0) -> torch.Tensor:
    """The definition in float64 on the CPU, one matrix [rows, cols]."""
    x = g.double().cpu()
    norm = torch.linalg.matrix_norm(x)
    if norm == 0:
        return torch.zeros_like(x)
    x = x / norm
    for a, b, c in coefs:
        a, b, c = (float(F(v)) for v in (a, b, c))
        if x.shape[0] <= x.shape[1]:
            s = x @ x.T
            x = a * x + (b * s + c * (s @ s)) @ x
        else:
            s = x.T @ x
            x = a * x + x @ (b * s + c * (s @ s))
    return x * float(F(scale))
