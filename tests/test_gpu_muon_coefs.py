"""Newton-Schulz with step coefficients of several kinds at shapes of the general
path: sets whose steps differ, so that each step is known by its result, and sets
that raise roundings further than FP16 operands bear."""
import pytest
import torch

import zero_sharded_optimizer_reduce_amd as z
from test_gpu_muon_spectra import _matrix, ns_f64

pytestmark = pytest.mark.gpu

NS_TOL = 5.5e-3
# Five steps, each the best quintic for the range that the last one leaves, divided
# by a factor: the results reach 1.98 and the next polynomial is steep there.
MINIMAX = ((8.28721201814563, -23.595886519098837, 17.300387312530933),
           (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
           (3.9486908534822946, -2.908902115962949, 0.5518191394370137),
           (3.3184196573706015, -2.488488024314874, 0.51004894012372),
           (2.300652019954817, -1.6689039845749493, 0.4188073119525673))
QUINTIC = (3.4445, -4.7750, 2.0315)


def _divided(coefs, by):
    return tuple((a / by, b / by ** 3, c / by ** 5) for a, b, c in coefs)


SETS = {"minimax/1.01": _divided(MINIMAX, 1.01), "minimax/1.02": _divided(MINIMAX, 1.02),
        "quintic x 8": (QUINTIC,) * 8, "cubic x 16": ((1.5, -0.5, 0.0),) * 16,
        "minimax/1.02 + cubic x 2": _divided(MINIMAX, 1.02) + ((1.5, -0.5, 0.0),) * 2, "1.9 s": ((1.9, 0.0, 0.0),)}


def _off(g, coefs, scale=1.0):
    out = torch.full(g.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = z.zero_newton_schulz_workspace(g)
    ws.fill_(0xFF)
    z.zero_newton_schulz(g, out, ws, coefs=coefs, scale=scale)
    ref = ns_f64(g, coefs, scale)
    return float((out.double() - ref).norm() / ref.norm())


# These sets may run with no fewer than 22 bits: with the sum of the gains after
# the first two steps up to 700 and the steepest slopes' product times the
# coefficients' size about 1300, 2^-22 of either stays under 4e-4, next to the result's
# own BF16 rounding, at most 2^-8 of it.
@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("kind", ["gauss", "rank1", "rank6", "half", "ones", "decades"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(128, 320), (320, 128), (300, 300), (97, 1000)])
def test_sets_that_raise_roundings(name, kind, dtype, rows, cols):
    print(f"newton_schulz {name} {kind} {rows}x{cols} {dtype}", flush=True)
    if kind == "gauss":
        g = torch.randn(rows, cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(rows))
    else:
        g = _matrix(kind, rows, cols, rows)
    off = _off(g.to(dtype), SETS[name])
    print(f"  off by {off:.2e}", flush=True)
    assert off <= 2.0 ** -8 + 4e-4, off


# matrices that one compute unit holds
@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("kind", ["rank1", "half", "ones"])
@pytest.mark.parametrize("rows,cols", [(64, 256), (32, 40), (96, 200), (200, 50)])
def test_sets_that_raise_roundings_of_small_matrices(name, kind, rows, cols):
    print(f"newton_schulz {name} {kind} {rows}x{cols} small", flush=True)
    for dtype in (torch.bfloat16, torch.float32):
        off = _off(_matrix(kind, rows, cols, rows).to(dtype), SETS[name])
        print(f"  off by {off:.2e}", flush=True)
        assert off <= 2.0 ** -8 + 4e-4, off


# every tile width: 64 (short and long sums), 128, 192, 256; stacks, odd sides, tall
@pytest.mark.parametrize("mats,rows,cols", [(2, 515, 530), (7, 517, 650), (1, 300, 2500), (3, 777, 1301), (1, 1290, 4099),
                                            (1, 2900, 2910), (1, 4090, 4097), (1, 4300, 3990)])
def test_sets_that_raise_roundings_in_every_tile(mats, rows, cols):
    print(f"newton_schulz minimax/1.01 {mats}x{rows}x{cols}", flush=True)
    g = torch.stack([_matrix("rank6", rows, cols, i) for i in range(mats)])
    out = torch.full_like(g, 7.0, dtype=torch.bfloat16)
    ws = z.zero_newton_schulz_workspace(g)
    ws.fill_(0xFF)
    z.zero_newton_schulz(g, out, ws, coefs=SETS["minimax/1.01"], scale=0.3)
    for i in {0, mats - 1}:
        ref = ns_f64(g[i], SETS["minimax/1.01"], 0.3)
        off = float((out[i].double() - ref).norm() / ref.norm())
        print(f"  off by {off:.2e}", flush=True)
        assert off <= 2.0 ** -8 + 4e-4, (i, off)


def test_special_matrices_with_a_steep_set():
    g = torch.stack([_matrix("rank6", 130, 200, i) for i in range(5)])
    g[1] = 0
    g[2, 65, 66] = float("nan")
    g[3, 1, 2] = float("inf")
    out = torch.full_like(g, 7.0, dtype=torch.bfloat16)
    z.zero_newton_schulz(g, out, z.zero_newton_schulz_workspace(g), coefs=SETS["minimax/1.01"])
    assert bool((out[1] == 0).all())
    assert bool(torch.isnan(out[2]).all()) and bool(torch.isnan(out[3]).all())
    for i in (0, 4):
        ref = ns_f64(g[i], SETS["minimax/1.01"])
        assert float((out[i].double() - ref).norm() / ref.norm()) <= 2.0 ** -8 + 4e-4


def test_a_steep_set_in_a_replayed_graph():
    x = torch.zeros(2, 130, 200, device="cuda")
    out, eager = (torch.empty(2, 130, 200, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws, ws2 = z.zero_newton_schulz_workspace(x), z.zero_newton_schulz_workspace(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        z.zero_newton_schulz(x, out, ws, coefs=SETS["minimax/1.02"])
    for t in range(4):
        x.copy_(torch.stack([_matrix("rank1", 130, 200, 2 * t + i) for i in range(2)]))
        z.zero_newton_schulz(x, eager, ws2, coefs=SETS["minimax/1.02"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), t


# Steps that differ, none of them flattening what the ones before it did: on a
# spectrum that falls from 0.6, two neighbouring steps exchanged move the result by 9e-3
# to 0.9 of its norm.
STEPS = ((3.4445, -4.7750, 2.0315), (1.5, -0.8, 0.0), (0.7, 0.4, -0.1), (1.4, -0.5, 0.15), (0.8, 0.3, -0.2),
         (1.25, -0.4, 0.1))


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(130, 200), (200, 130), (130, 400), (400, 130), (80, 200)])
def test_steps_that_differ(steps, dtype, rows, cols):
    print(f"newton_schulz {steps} different steps {rows}x{cols} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(steps)
    k = min(rows, cols)
    u = torch.linalg.qr(torch.randn(rows, k, device="cuda", generator=gen).double())[0]
    v = torch.linalg.qr(torch.randn(cols, k, device="cuda", generator=gen).double())[0]
    g = torch.mm(u * 10.0 ** (-torch.arange(k, device="cuda").double() / 8), v.T.contiguous()).to(dtype)
    off = _off(g, STEPS[:steps])
    print(f"  off by {off:.2e}", flush=True)
    assert off <= NS_TOL, off


@pytest.mark.parametrize("rows,cols", [(130, 200), (97, 1000)])
def test_cubic_steps(rows, cols):
    g = torch.randn(rows, cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    assert _off(g, ((1.5, -0.5, 0.0),) * 8, 0.25) <= NS_TOL * 1.3


# Sets whose operands stay single FP16 values: a singular vector is turned by up to
# 55 roundings of half a step, 55 * 2^-11 (five steps whose first slopes' product is 493),
# six quintics raise X's roundings (2^-10/sqrt(12) rms) 56-fold in half of the
# directions, 1.6e-2 / sqrt(2); and the result's own rounding.
@pytest.mark.parametrize("name,coefs", [
    ("five from 4.1 s", ((4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037),
                         (2.8769, -3.1427, 1.2046), (2.8366, -3.0525, 1.2012))),
    ("quintic x 6", (QUINTIC,) * 6), ("cubic x 10", ((1.5, -0.5, 0.0),) * 10)])
@pytest.mark.parametrize("kind", ["rank1", "rank6", "half", "decades"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(128, 320), (320, 128), (300, 300), (97, 1000)])
def test_sets_near_the_default(name, coefs, kind, dtype, rows, cols):
    print(f"newton_schulz {name} {kind} {rows}x{cols} {dtype}", flush=True)
    off = _off(_matrix(kind, rows, cols, rows).to(dtype), coefs)
    print(f"  off by {off:.2e}", flush=True)
    assert off <= 55 * 2.0 ** -11 + 2.0 ** -8, off
