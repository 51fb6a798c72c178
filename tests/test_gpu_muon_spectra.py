"""Newton-Schulz on matrices whose singular values lie far apart, at shapes of the
general path: BF16 and FP32 inputs, against the definition in 64 bits.

Tolerances, in the Frobenius norm, for five quintic steps.  r = 2^-10/sqrt(12) =
2.8e-4 is an FP16 operand's rms rounding, and 1.66e-3 the BF16 rounding's of the
result.
* Falling spectra: as for Gaussian matrices, 5.5e-3.
* A few strong directions and nothing, or next to nothing, in the others: the
  roundings of X lie in those others and are raised by the gains of the steps that
  follow, those after the third step by 3.44^2 = 11.9 (11.9 r = 3.3e-3); of those
  that are carried the image is short by up to 0.4 of itself where half of the
  directions are strong (0.4 * 41 r = 4.7e-3); the factor of two steps is about
  11.9 there, where FP16 steps are 2^-7 (2.3e-3 rms), in two of the products.
  sqrt(3.3^2 + 4.7^2 + 2 * 2.3^2 + 1.7^2) = 6.8e-3; FP32 inputs add what their own
  FP16 remainder leaves (484 * 2^-11 r < 1e-4).  1.1e-2 leaves room for the draw.
* Entries that are all alike round alike, so that the roundings add up: the factor
  of two steps by half a step of its diagonal, 2^-8, and 11.2 * 2^-11 off it, 9.4e-3
  in two places, the first raised by up to 1.61 (the polynomial's steepest slope
  between 0.68 and 1.13) in each of three steps: 3.9e-2 + 9.4e-3 + 3.4 * 2^-11 *
  (1.61^2 + 1.61) and 2^-8 for the result: 5.9e-2."""
import math

import numpy as np
import pytest
import torch

import muon_plain as plain
import zero_sharded_optimizer_reduce_amd as z

pytestmark = pytest.mark.gpu

TOL = dict(pow=5.5e-3, decades=5.5e-3, rank1=1.1e-2, rank6=1.1e-2, half=1.1e-2, spike=1.1e-2, ones=5.9e-2,
           blocks=5.9e-2, two=5.9e-2)
SHAPES = [(128, 320), (300, 300), (97, 1000), (1000, 97), (515, 530), (1290, 1999)]


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _matrix(kind, rows, cols, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "ones":
        return torch.full((rows, cols), 0.375, device="cuda")
    if kind == "two":
        g = torch.ones(rows, cols, device="cuda")
        g[:rows // 2, :cols // 3] = -0.5
        return g
    if kind == "blocks":
        i, j = torch.arange(rows, device="cuda") * 8 // rows, torch.arange(cols, device="cuda") * 8 // cols
        return (i[:, None] == j[None, :]).float()
    if kind in ("rank1", "rank6"):
        r = int(kind[4:])
        return _randn(gen, rows, r) @ _randn(gen, r, cols)
    k = min(rows, cols)
    u = torch.linalg.qr(_randn(gen, rows, k).double())[0]
    v = torch.linalg.qr(_randn(gen, cols, k).double())[0]
    i = torch.arange(k, device="cuda", dtype=torch.float64)
    s = {"pow": (i + 1) ** -1.5, "decades": 10.0 ** (-3 * i / (k - 1)),
         "half": torch.where(i < k // 2, 1.0, 1e-5).double(), "spike": torch.where(i < 1, 1.0, 1e-3).double()}[kind]
    return torch.mm(u * s, v.T.contiguous()).float()


def ns_f64(g, coefs=plain.COEFS, scale=1.0):
    """The definition in float64 on the device."""
    x = g.double()
    x = x / torch.linalg.matrix_norm(x)
    tall = x.shape[0] > x.shape[1]
    for a, b, c in coefs:
        a, b, c = (float(np.float32(v)) for v in (a, b, c))
        s = torch.mm(x.T, x) if tall else torch.mm(x, x.T)
        q = b * s + c * torch.mm(s, s)
        x = a * x + (torch.mm(x, q) if tall else torch.mm(q, x))
    return x * float(np.float32(scale))


@pytest.mark.parametrize("kind", list(TOL))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_spectra(kind, dtype, rows, cols):
    print(f"newton_schulz {kind} {rows}x{cols} {dtype}", flush=True)
    g = _matrix(kind, rows, cols, rows + cols).to(dtype)
    out = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = z.zero_newton_schulz_workspace(g)
    ws.fill_(0xFF)
    z.zero_newton_schulz(g, out, ws)
    ref = ns_f64(g)
    off = float((out.double() - ref).norm() / ref.norm())
    print(f"  off by {off:.2e}", flush=True)
    assert off <= TOL[kind], off


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6])
@pytest.mark.parametrize("rows,cols", [(128, 320), (320, 128), (130, 200)])
def test_fp32_matrices_of_rank_one_in_other_numbers_of_steps(steps, rows, cols):
    print(f"newton_schulz rank one FP32 {rows}x{cols} {steps} steps", flush=True)
    g = _matrix("rank1", rows, cols, steps)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    coefs = plain.COEFS[:1] * steps
    z.zero_newton_schulz(g, out, z.zero_newton_schulz_workspace(g), coefs=coefs)
    ref = ns_f64(g, coefs)
    off = float((out.double() - ref).norm() / ref.norm())
    print(f"  off by {off:.2e}", flush=True)
    # a step more raises what lies in the other directions by up to 3.44
    assert off <= TOL["rank1"] * max(1.0, math.sqrt(3.44) ** (steps - 5)), off


def test_fp32_stack_with_neighbours():
    # every matrix of a stack keeps its own low bits
    g = torch.stack([_matrix("rank1", 130, 200, i) * 10.0 ** (3 * i) for i in range(3)])
    out = torch.empty(3, 130, 200, dtype=torch.bfloat16, device="cuda")
    z.zero_newton_schulz(g, out, z.zero_newton_schulz_workspace(g), scale=0.5)
    for i in range(3):
        ref = ns_f64(g[i], scale=0.5)
        assert float((out[i].double() - ref).norm() / ref.norm()) <= TOL["rank1"], i


# the wider tiles, and a long sum
@pytest.mark.parametrize("mats,rows,cols", [(1, 2900, 2910), (1, 4090, 4097), (1, 4300, 3990), (3, 1025, 3001), (1, 100, 9000)])
@pytest.mark.parametrize("kind", ["rank1", "rank6"])
def test_fp32_matrices_in_wide_tiles(mats, rows, cols, kind):
    print(f"newton_schulz {kind} FP32 {mats}x{rows}x{cols}", flush=True)
    g = torch.stack([_matrix(kind, rows, cols, i) for i in range(mats)])
    out = torch.full(g.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    z.zero_newton_schulz(g, out, z.zero_newton_schulz_workspace(g))
    for i in {0, mats - 1}:
        ref = ns_f64(g[i])
        off = float((out[i].double() - ref).norm() / ref.norm())
        print(f"  off by {off:.2e}", flush=True)
        assert off <= TOL[kind], (i, off)
