"""The Muon step driver on the GPU: every stage of a step against its plain form,
clipped and graph-captured steps, and matrices of every tile the Newton-Schulz
products choose.

Elementwise stages are bit-exact against binary32 arithmetic.  Newton-Schulz is
held to the relative error derived for it (the final BF16 rounding's 1.7e-3 and
FP16 roundings of the operands, 5.5e-3 in all) in the Frobenius norm."""
import math

import numpy as np
import pytest
import torch

import muon_plain as plain
import zero_sharded_optimizer_reduce_amd as z
from gpu_helpers import bf16_to_dev, bf16_to_host, f32_to_dev, f32_to_host
from zero_sharded_optimizer_reduce_amd.drivers import MuonStep

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-2, momentum=0.95, weight_decay=0.1, nesterov=True)
NS_TOL = 5.5e-3
SHAPES = [(48, 80), (48, 80), (130, 70), (257, 300), (257, 300), (257, 300), (16, 1)]


def _normal(rng, n, sigma):
    return (rng.standard_normal(n) * sigma).astype(np.float32)


def _contributions(rng, st, n_ranks):
    x = [plain.to_bf16(_normal(rng, st.psi_pad, 1e-3)) for _ in range(n_ranks)]
    for v in x:
        v[st.psi:] = 0
    return x


def _same(a, b):
    return np.array_equal(a.view(np.uint8), b.view(np.uint8))


def _check_update_and_gather(st, before, lr):
    off = 0
    u = bf16_to_host(st.update_flat)
    d = bf16_to_host(st.directions)
    for rows, cols in st.shapes:
        sl = slice(off, off + rows * cols)
        g = torch.from_numpy(plain.from_bf16(d[sl])).view(rows, cols)
        ref = plain.newton_schulz_f64(g, scale=math.sqrt(max(1.0, rows / cols)))
        got = torch.from_numpy(plain.from_bf16(u[sl])).view(rows, cols).double()
        assert (got - ref).norm() <= NS_TOL * ref.norm(), (rows, cols)
        off = sl.stop
    assert not u[off:].any()
    view = bf16_to_host(st.view)
    for k in range(st.n):
        sl = slice(k * st.shard, (k + 1) * st.shard)
        p1, b1 = plain.update_f32(before[sl], u[sl], lr, HP["weight_decay"])
        assert _same(f32_to_host(st.master[k]), p1) and _same(view[sl], b1), k


@pytest.mark.parametrize("n_ranks", [1, 3, 4])
@pytest.mark.parametrize("acc", [False, True])
def test_steps(n_ranks, acc):
    rng = np.random.default_rng(n_ranks)
    st = MuonStep(SHAPES, n_ranks)
    assert [tuple(d.shape) for d, _, _ in st.stacks] == [(2, 48, 80), (1, 130, 70), (3, 257, 300), (1, 16, 1)]
    before = _normal(rng, st.psi_pad, 0.02)
    st.load_master(f32_to_dev(before))
    w = z.zero_rank_weights(list(range(5, 5 + n_ranks)), n_ranks)
    m = [np.zeros(st.shard, np.float32) for _ in range(n_ranks)]
    for t in range(2):
        x = _contributions(rng, st, n_ranks)
        ga = [_normal(rng, st.shard, 1e-3) for _ in range(n_ranks)] if acc else None
        out = st.step([bf16_to_dev(v) for v in x], w, HP, grad_acc=[f32_to_dev(v) for v in ga] if acc else None)
        torch.cuda.synchronize()
        assert out.numel() == st.psi
        for k in range(n_ranks):
            sl = slice(k * st.shard, (k + 1) * st.shard)
            g = plain.reduce_ranks([v[sl] for v in x], w, ga[k] if acc else None)
            m[k], u = plain.momentum_f32(m[k], g, HP["momentum"], True)
            assert _same(f32_to_host(st.momentum[k]), m[k]), (t, k)
            assert _same(bf16_to_host(st.directions[sl]), u), (t, k)
        _check_update_and_gather(st, before, HP["lr"])
        before = np.concatenate([f32_to_host(p) for p in st.master])


@pytest.mark.parametrize("max_norm", [1e-2, 1e3])
def test_a_clipped_step(max_norm):
    rng = np.random.default_rng(7)
    st = MuonStep(SHAPES, 2)
    before = _normal(rng, st.psi_pad, 0.02)
    st.load_master(f32_to_dev(before))
    x = _contributions(rng, st, 2)
    st.step([bf16_to_dev(v) for v in x], [0.5, 0.5], HP, max_norm=max_norm)
    torch.cuda.synchronize()
    g = plain.reduce_ranks(x, [0.5, 0.5])
    clip = float(st.clip)
    want = min(1.0, max_norm / (np.linalg.norm(g.astype(np.float64)) + 1e-6))
    assert abs(clip - want) <= 4 * 2.0 ** -24 * want
    m, u = plain.momentum_f32(np.zeros_like(g), g, HP["momentum"], True, scale=clip)
    assert _same(np.concatenate([f32_to_host(v) for v in st.momentum]), m)
    assert _same(bf16_to_host(st.directions), u)
    _check_update_and_gather(st, before, HP["lr"])


def test_clipping_and_accumulated_gradients_together_are_refused():
    st = MuonStep([(8, 8)], 1)
    with pytest.raises(ValueError, match="not supported"):
        st.step([torch.zeros(st.psi_pad, dtype=torch.bfloat16, device="cuda")], [1.0], HP,
                grad_acc=[torch.zeros(st.shard, device="cuda")], max_norm=1.0)


@pytest.mark.parametrize("max_norm", [None, 0.05])
def test_a_captured_step_follows_the_eager_one(max_norm):
    rng = np.random.default_rng(11)
    a, b = MuonStep(SHAPES, 2), MuonStep(SHAPES, 2)
    start = f32_to_dev(_normal(rng, a.psi_pad, 0.02))
    x = [torch.zeros(a.psi_pad, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lr = torch.full((1,), 1e-2, device="cuda")
    args = dict(max_norm=max_norm, lr_dev=lr)
    if max_norm is not None:   # allocates the clipped step's buffers
        b.reduce_momentum_clipped(x, [0.5, 0.5], HP, max_norm)
    for st in (a, b):
        st.load_master(start)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.step(x, [0.5, 0.5], HP, **args)
    for t in range(4):
        lr.fill_(1e-2 / (t + 1))
        for v, bits in zip(x, _contributions(rng, a, 2)):
            v.copy_(bf16_to_dev(bits))
        a.step(x, [0.5, 0.5], HP, **args)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(a.momentum[k], b.momentum[k]) and torch.equal(a.master[k], b.master[k]), (t, k)
        assert torch.equal(a.update_flat, b.update_flat) and torch.equal(a.view, b.view), t


def _ns_f64(g, scale):
    """The definition in float64 on the device."""
    x = g.double()
    x = x / torch.linalg.matrix_norm(x)
    tall = x.shape[0] > x.shape[1]
    for a, b, c in plain.COEFS:
        a, b, c = (float(np.float32(v)) for v in (a, b, c))
        s = torch.mm(x.T, x) if tall else torch.mm(x, x.T)
        q = b * s + c * torch.mm(s, s)
        x = a * x + (torch.mm(x, q) if tall else torch.mm(q, x))
    return x * float(np.float32(scale))


# 64-wide tiles: few, more than one per compute unit, their diagonals riding, and
# with a long summed index; 128; 192 and 256.  Odd sides, so that tiles end inside.
@pytest.mark.parametrize("mats,rows,cols", [(2, 515, 530), (7, 517, 650), (7, 650, 517), (7, 513, 1110), (1, 1030, 1027),
                                            (33, 511, 1021), (3, 777, 1301), (1, 1290, 4099), (1, 2047, 2050),
                                            (1, 2900, 2910),
                                            (1, 4090, 4097), (1, 4300, 3990), (12, 1025, 3001),
                                            (12, 3001, 1025)])
def test_newton_schulz_tiles(mats, rows, cols):
    print(f"newton_schulz {mats}x{rows}x{cols}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(mats * rows + cols)
    g = (torch.randn(mats, rows, cols, device="cuda", generator=gen) * 1e-3).to(torch.bfloat16)
    out = torch.full_like(g, float("nan"))
    z.zero_newton_schulz(g, out, z.zero_newton_schulz_workspace(g), scale=0.3)
    for i in {0, mats // 2, mats - 1}:
        ref = _ns_f64(g[i], 0.3)
        off = float((out[i].double() - ref).norm() / ref.norm())
        assert off <= NS_TOL, (i, off)
    assert bool(torch.isfinite(out).all())
