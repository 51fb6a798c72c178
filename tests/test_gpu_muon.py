"""The Muon step's operators on the GPU: the momentum step (alone and fused with
the reduce-scatter) and the owner update bit for bit against binary32 arrays
and against float64 within their roundings, the Newton-Schulz
orthogonalisation against float64, each at odd sizes, unaligned views, special
values, on side streams and in replayed graphs."""
import numpy as np
import pytest
import torch

import muon_plain as plain
from gpu_helpers import bf16_to_dev, bf16_to_host, f32_to_dev, f32_to_host

pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_reduce_amd as z  # noqa: E402

HP = dict(lr=1e-3, momentum=0.95, weight_decay=0.1, nesterov=True)
SIZES = [0, 1, 3, 4, 5, 255, 256, 257, 1023, 4096 + 3, 257 * 1024 + 1]


def _rng(seed):
    return np.random.default_rng(seed)


def _normal(rng, n, sigma):
    return (rng.standard_normal(n) * sigma).astype(np.float32)


def _same(a, b):
    """Equal bits, or both NaN."""
    t = np.uint32 if a.dtype == np.float32 else np.uint16
    if a.dtype == np.float32:
        nan = np.isnan(a) & np.isnan(b)
    else:
        nan = np.isnan(plain.from_bf16(a)) & np.isnan(plain.from_bf16(b))
    return bool(np.all((a.view(t) == b.view(t)) | nan))


def _sentinel(n, dtype, offset=0):
    """A view of n elements inside a larger buffer, offset elements past a
    64-element margin, and a check that the margins are untouched."""
    fill = 7.0
    buf = torch.full((n + 128 + offset,), fill, dtype=dtype, device="cuda")
    view = buf[64 + offset:64 + offset + n]

    def check():
        assert bool((buf[:64 + offset] == fill).all()) and bool((buf[64 + offset + n:] == fill).all()), "margin written"
    return view, check


# ------------------------------------------------------------ momentum step
@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("scale", [None, 0.37])
def test_momentum(n, nesterov, scale):
    rng = _rng(n + 1)
    m, g = _normal(rng, n, 3e-4), _normal(rng, n, 1e-3)
    mv, check_m = _sentinel(n, torch.float32)
    uv, check_u = _sentinel(n, torch.bfloat16)
    mv.copy_(f32_to_dev(m))
    gs = None if scale is None else torch.full((1,), scale, device="cuda")
    z.zero_muon_momentum(mv, uv, f32_to_dev(g), dict(HP, nesterov=nesterov), grad_scale=gs)
    torch.cuda.synchronize()
    m1, u1 = plain.momentum_f32(m, g, HP["momentum"], nesterov, scale)
    assert _same(f32_to_host(mv), m1) and _same(bf16_to_host(uv), u1)
    check_m()
    check_u()
    # float64: the clip product, two products and a sum round in m, each by at
    # most 2^-24 of a term; u has three more roundings and the one to BF16
    m64, u64 = plain.momentum_f64(m, g, HP["momentum"], nesterov, scale)
    size = np.abs(m).astype(np.float64) + np.abs(g)
    assert np.all(np.abs(f32_to_host(mv) - m64) <= 4 * 2.0 ** -24 * size)
    assert np.all(np.abs(plain.from_bf16(bf16_to_host(uv)) - u64) <= 2.0 ** -8 * np.abs(u64) + 8 * 2.0 ** -24 * size)


@pytest.mark.parametrize("off_m,off_u,off_g", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 2, 0), (4, 4, 4), (3, 1, 2)])
def test_momentum_unaligned_views(off_m, off_u, off_g):
    n = 4099
    rng = _rng(5)
    m, g = _normal(rng, n, 3e-4), _normal(rng, n, 1e-3)
    mv, check_m = _sentinel(n, torch.float32, off_m)
    uv, check_u = _sentinel(n, torch.bfloat16, off_u)
    gv, _ = _sentinel(n, torch.float32, off_g)
    mv.copy_(f32_to_dev(m))
    gv.copy_(f32_to_dev(g))
    z.zero_muon_momentum(mv, uv, gv, HP)
    assert z.zero_last_path_vectorized() == int(off_m % 4 == 0 and off_g % 4 == 0 and off_u % 4 == 0)
    torch.cuda.synchronize()
    m1, u1 = plain.momentum_f32(m, g, HP["momentum"], True)
    assert _same(f32_to_host(mv), m1) and _same(bf16_to_host(uv), u1)
    check_m()
    check_u()


SPECIAL = np.array([0.0, -0.0, np.inf, -np.inf, np.nan, 1e-40, -1e-40, 3e38, -3e38, 1.0, 2.0 ** -133], np.float32)


def test_momentum_special_values():
    rng = _rng(6)
    m, g = rng.choice(SPECIAL, 4099).astype(np.float32), rng.choice(SPECIAL, 4099).astype(np.float32)
    md, u = f32_to_dev(m), torch.empty(4099, dtype=torch.bfloat16, device="cuda")
    z.zero_muon_momentum(md, u, f32_to_dev(g), HP)
    with np.errstate(all="ignore"):
        m1, u1 = plain.momentum_f32(m, g, HP["momentum"], True)
    assert _same(f32_to_host(md), m1) and _same(bf16_to_host(u), u1)


# ------------------------------------------------- reduce-scatter + momentum
@pytest.mark.parametrize("n_ranks", [1, 2, 3, 4, 5, 8, 16])
@pytest.mark.parametrize("n_shards,shard", [(1, 1), (1, 4099), (2, 1025), (3, 256), (4, 4 * 257), (2, 0)])
@pytest.mark.parametrize("acc", [False, True])
def test_reduce_scatter_momentum(n_ranks, n_shards, shard, acc):
    print(f"reduce_scatter_muon ranks={n_ranks} shards={n_shards} shard={shard} acc={acc}", flush=True)
    rng = _rng(1000 * n_ranks + shard)
    numel = n_shards * shard
    x = [plain.to_bf16(_normal(rng, numel, 1e-3)) for _ in range(n_ranks)]
    w = z.zero_rank_weights(list(range(7, 7 + n_ranks)), n_ranks)
    m = [_normal(rng, shard, 3e-4) for _ in range(n_shards)]
    ga = [_normal(rng, shard, 1e-3) for _ in range(n_shards)] if acc else None
    md = [f32_to_dev(v) for v in m]
    us = [_sentinel(shard, torch.bfloat16) for _ in range(n_shards)]
    z.zero_reduce_scatter_muon([bf16_to_dev(v) for v in x], w, md, [u for u, _ in us], HP,
                               grad_acc=[f32_to_dev(v) for v in ga] if acc else None)
    torch.cuda.synchronize()
    for k in range(n_shards):
        sl = slice(k * shard, (k + 1) * shard)
        g = plain.reduce_ranks([v[sl] for v in x], w, ga[k] if acc else None)
        m1, u1 = plain.momentum_f32(m[k], g, HP["momentum"], True)
        assert _same(f32_to_host(md[k]), m1) and _same(bf16_to_host(us[k][0]), u1), k
        us[k][1]()


def test_reduce_scatter_momentum_equals_the_two_calls():
    n_ranks, n_shards, shard = 4, 4, 6 * 1024
    rng = _rng(9)
    x = [bf16_to_dev(plain.to_bf16(_normal(rng, n_shards * shard, 1e-3))) for _ in range(n_ranks)]
    w = z.zero_rank_weights(None, n_ranks)
    m = [f32_to_dev(_normal(rng, shard, 3e-4)) for _ in range(n_shards)]
    m2 = [t.clone() for t in m]
    u, u2 = ([torch.empty(shard, dtype=torch.bfloat16, device="cuda") for _ in range(n_shards)] for _ in range(2))
    g = [torch.empty(shard, device="cuda") for _ in range(n_shards)]
    z.zero_reduce_scatter_muon(x, w, m, u, HP)
    z.zero_reduce_scatter(x, w, g)
    for k in range(n_shards):
        z.zero_muon_momentum(m2[k], u2[k], g[k], HP)
    for a, b in zip(m + u, m2 + u2):
        assert torch.equal(a, b)


def test_reduce_scatter_momentum_unaligned_contributions():
    # contributions that start one BF16 element in, and an unaligned momentum
    n = 4 * 1025
    rng = _rng(10)
    x = [plain.to_bf16(_normal(rng, n + 1, 1e-3)) for _ in range(3)]
    w = z.zero_rank_weights(None, 3)
    for off in (0, 1):
        m = _normal(rng, n, 3e-4)
        mv, check = _sentinel(n, torch.float32, off)
        mv.copy_(f32_to_dev(m))
        u = torch.empty(n, dtype=torch.bfloat16, device="cuda")
        z.zero_reduce_scatter_muon([bf16_to_dev(v)[1:] for v in x], w, [mv], [u], HP)
        assert z.zero_last_path_vectorized() == (1 if off == 0 else 0)
        m1, u1 = plain.momentum_f32(m, plain.reduce_ranks([v[1:] for v in x], w), HP["momentum"], True)
        assert _same(f32_to_host(mv), m1) and _same(bf16_to_host(u), u1)
        check()


# -------------------------------------------------------------- owner update
@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("wd", [0.0, 0.1])
@pytest.mark.parametrize("lr_dev", [None, 3e-4])
def test_update(n, wd, lr_dev):
    rng = _rng(n + 7)
    p, o = _normal(rng, n, 0.02), plain.to_bf16(_normal(rng, n, 0.2))
    pv, check_p = _sentinel(n, torch.float32)
    bv, check_b = _sentinel(n, torch.bfloat16)
    pv.copy_(f32_to_dev(p))
    lr = None if lr_dev is None else torch.full((1,), lr_dev, device="cuda")
    z.zero_muon_shard_step(pv, bv, bf16_to_dev(o), dict(HP, weight_decay=wd), lr_dev=lr)
    torch.cuda.synchronize()
    used = HP["lr"] if lr_dev is None else lr_dev
    p1, b1 = plain.update_f32(p, o, used, wd)
    assert _same(f32_to_host(pv), p1) and _same(bf16_to_host(bv), b1)
    check_p()
    check_b()
    # float64: the last sum rounds by 2^-24 of p', the step lr*u by three roundings
    p64 = plain.update_f64(p, o, used, wd)
    step = np.abs(p64 - p)
    assert np.all(np.abs(f32_to_host(pv) - p64) <= 2.0 ** -24 * np.abs(p64) + 4 * 2.0 ** -24 * (step + 1e-3 * np.abs(p)))


@pytest.mark.parametrize("off_p,off_b,off_o", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 3), (4, 4, 1)])
def test_update_unaligned_views(off_p, off_b, off_o):
    n = 4099
    rng = _rng(15)
    p, o = _normal(rng, n, 0.02), plain.to_bf16(_normal(rng, n, 0.2))
    pv, check_p = _sentinel(n, torch.float32, off_p)
    bv, check_b = _sentinel(n, torch.bfloat16, off_b)
    ov, _ = _sentinel(n, torch.bfloat16, off_o)
    pv.copy_(f32_to_dev(p))
    ov.copy_(bf16_to_dev(o))
    z.zero_muon_shard_step(pv, bv, ov, HP)
    assert z.zero_last_path_vectorized() == int(off_p % 4 == 0 and off_b % 4 == 0)
    torch.cuda.synchronize()
    p1, b1 = plain.update_f32(p, o, HP["lr"], HP["weight_decay"])
    assert _same(f32_to_host(pv), p1) and _same(bf16_to_host(bv), b1)
    check_p()
    check_b()


def test_update_special_values():
    rng = _rng(16)
    p = rng.choice(SPECIAL, 4099).astype(np.float32)
    o = plain.to_bf16(rng.choice(SPECIAL, 4099).astype(np.float32))
    pd, b = f32_to_dev(p), torch.empty(4099, dtype=torch.bfloat16, device="cuda")
    z.zero_muon_shard_step(pd, b, bf16_to_dev(o), HP)
    with np.errstate(all="ignore"):
        p1, b1 = plain.update_f32(p, o, HP["lr"], HP["weight_decay"])
    assert _same(f32_to_host(pd), p1) and _same(bf16_to_host(b), b1)


def test_elementwise_offsets_past_32_bits():
    # more than 2^31 elements: the last ones are reached through 64-bit offsets
    n = (1 << 31) + 5
    p = torch.zeros(n, device="cuda")
    o = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    b = torch.full((n,), 9.0, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, (1 << 31) - 1, 1 << 31, n - 4, n - 1], device="cuda")
    p[at] = 1.0
    o[at] = 2.0
    z.zero_muon_shard_step(p, b, o, dict(HP, lr=0.25, weight_decay=0.0))
    assert bool((p[at] == 0.5).all()) and bool((b[at] == 0.5).all())
    assert int(torch.count_nonzero(p)) == 5 and int(torch.count_nonzero(b)) == 5
    z.zero_muon_momentum(p, b, torch.zeros_like(p), dict(HP, momentum=0.5, nesterov=False))
    assert bool((p[at] == 0.25).all()) and bool((b[at] == 0.25).all())


# ------------------------------------------------------------- Newton-Schulz
# A value rounded to BF16 is off by at most 2^-8 of itself, with an rms of at
# most 2^-7/sqrt(12) = 2.3e-3 of the values.  An FP16 operand's rms is r =
# 2^-10/sqrt(12) = 2.8e-4.  Each step rounds X (gain 1), A (at most |b| + 2|c| -
# 2... taken as 6) and C (3.44 over the 0.7 it leaves at singular value 1: 5):
# sqrt(1 + 36 + 25) r = 2.2e-3 a step, 5.0e-3 over five independent steps; with
# the BF16 rounding 5.5e-3 of the result's norm.  An element is off by
# at most six such deviations and its own BF16 rounding.  BF16 operands
# would be eight times as far off.
NS_TOL = 5.5e-3


def _gauss(seed, *shape, dtype=torch.bfloat16, sigma=1e-3):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * sigma).to(dtype)


def _ns(g, out=None, **kw):
    gd = g.cuda()
    if out is None:
        out = torch.full(gd.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = z.zero_newton_schulz_workspace(gd)
    ws.fill_(0xFF)      # NaNs everywhere: nothing may be read before it is written
    z.zero_newton_schulz(gd, out, ws, **kw)
    torch.cuda.synchronize()
    return out


def _assert_close(got, ref, tol=NS_TOL):
    got, rms = got.double().cpu(), ref.square().mean().sqrt()
    off = (got - ref).norm() / ref.norm()
    assert off <= tol, f"relative error {off:.3g}"
    worst = ((got - ref).abs() - 2.0 ** -8 * ref.abs()).max() / rms
    assert worst <= 6 * tol, f"an element is {worst:.3g} of the rms off"
    return float(off)


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 2), (3, 100), (16, 16), (31, 33), (63, 65), (64, 64), (64, 256), (65, 63),
          (100, 64), (127, 129), (128, 128), (129, 300), (192, 96), (200, 1000), (255, 257), (513, 130), (300, 777),
          (257, 515), (700, 640), (1025, 1031)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_newton_schulz(rows, cols, dtype):
    print(f"newton_schulz {rows}x{cols} {dtype}", flush=True)
    g = _gauss(rows * 10000 + cols, rows, cols, dtype=dtype)
    off = _assert_close(_ns(g, scale=0.5), plain.newton_schulz_f64(g, scale=0.5))
    print(f"  off by {off:.2e}", flush=True)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 16])
@pytest.mark.parametrize("rows,cols", [(96, 130), (96, 400), (400, 96)])
def test_newton_schulz_steps(steps, rows, cols):
    g = _gauss(steps, rows, cols)
    c = plain.COEFS[:1] * steps
    _assert_close(_ns(g, coefs=c), plain.newton_schulz_f64(g, c), NS_TOL * max(1.0, (steps / 5) ** 0.5))


def test_newton_schulz_other_coefficients():
    # the cubic step 1.5 s - 0.5 s^3, and steps that differ from each other
    g = _gauss(3, 80, 200)
    for c in (((1.5, -0.5, 0.0),) * 8, ((3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375))):
        _assert_close(_ns(g, coefs=c), plain.newton_schulz_f64(g, c), NS_TOL * 1.3)


@pytest.mark.parametrize("mats,rows,cols", [(2, 64, 64), (3, 100, 260), (5, 260, 100), (33, 17, 40), (4, 300, 310)])
def test_newton_schulz_stacks_and_strides(mats, rows, cols):
    print(f"newton_schulz stack {mats}x{rows}x{cols}", flush=True)
    # input and output inside wider, taller buffers of odd strides
    gb = torch.full((mats, rows + 3, cols + 5), 100.0, dtype=torch.float32)
    gb[:, :rows, :cols] = _gauss(mats, mats, rows, cols, dtype=torch.float32)
    gd = gb.cuda()[:, :rows, :cols]
    ob = torch.full((mats, rows + 1, cols + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    z.zero_newton_schulz(gd, ob[:, :rows, :cols], z.zero_newton_schulz_workspace(gd))
    torch.cuda.synchronize()
    for q in range(mats):
        _assert_close(ob[q, :rows, :cols], plain.newton_schulz_f64(gb[q, :rows, :cols]))
    ob[:, :rows, :cols] = 7.0
    assert bool((ob == 7.0).all()), "written outside the matrices"


@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_newton_schulz_unaligned_output_and_input(off):
    g = _gauss(21, 72, 200)
    src = torch.zeros(72 * 200 + 64, dtype=torch.bfloat16, device="cuda")
    src[off:off + 72 * 200] = g.cuda().flatten()
    dst = torch.full((72 * 200 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    gd, od = src[off:off + 72 * 200].view(72, 200), dst[off:off + 72 * 200].view(72, 200)
    z.zero_newton_schulz(gd, od, z.zero_newton_schulz_workspace(gd))
    assert torch.equal(od, _ns(g))
    assert bool((dst[:off] == 7.0).all()) and bool((dst[off + 72 * 200:] == 7.0).all())


def test_newton_schulz_far_apart_matrices():
    # matrix strides whose offsets pass 32 bits, in elements and in bytes
    far = (1 << 31) + 24
    src = torch.zeros(far + 64 * 96, dtype=torch.bfloat16, device="cuda")
    dst = torch.zeros(far + 64 * 96, dtype=torch.bfloat16, device="cuda")
    g = _gauss(22, 2, 64, 96)
    gd = src.as_strided((2, 64, 96), (far, 96, 1))
    gd.copy_(g.cuda())
    od = dst.as_strided((2, 64, 96), (far, 96, 1))
    z.zero_newton_schulz(gd, od, z.zero_newton_schulz_workspace(gd))
    assert torch.equal(od.contiguous(), _ns(g))


@pytest.mark.parametrize("rows,cols", [(48, 80), (300, 200)])
def test_newton_schulz_does_not_depend_on_the_scale(rows, cols):
    g = _gauss(23, rows, cols, dtype=torch.float32, sigma=1.0)
    want = _ns(g)
    for e in (-100, -40, 40, 100):
        assert torch.equal(_ns(g * 2.0 ** e), want), e      # a power of two changes no bit
    b = _gauss(24, rows, cols, sigma=1.0)
    assert torch.equal(_ns(b * 2.0 ** 100), _ns(b))
    # subnormal BF16 and FP32 inputs are values like others
    tiny = (_gauss(25, rows, cols, dtype=torch.float32, sigma=1.0) * 2.0 ** -130).to(torch.bfloat16)
    _assert_close(_ns(tiny), plain.newton_schulz_f64(tiny))


def test_newton_schulz_zero_nan_and_infinite_matrices():
    for rows, cols in ((40, 70), (300, 260)):
        g = _gauss(26, 5, rows, cols)
        g[1] = 0
        g[2, rows // 2, cols // 3] = float("nan")
        g[3, 1, 2] = float("inf")
        out = _ns(g)
        assert bool((out[1] == 0).all())
        assert bool(torch.isnan(out[2]).all()) and bool(torch.isnan(out[3]).all())
        for q in (0, 4):       # the neighbours are untouched by it
            _assert_close(out[q], plain.newton_schulz_f64(g[q]))


def test_newton_schulz_low_rank_and_spiked_spectra():
    gen = torch.Generator().manual_seed(27)
    k, l = 128, 320
    rank1 = torch.outer(torch.randn(k, generator=gen), torch.randn(l, generator=gen))
    lowrank = torch.randn(k, 6, generator=gen) @ torch.randn(6, l, generator=gen)
    spiked = rank1 + 0.05 * torch.randn(k, l, generator=gen)
    for g in (rank1, lowrank, spiked):
        g = g.to(torch.bfloat16)
        out, ref = _ns(g).double().cpu(), plain.newton_schulz_f64(g)
        # BF16's own rounding of the input leaves small singular values that the
        # steps raise 3.44^5-fold: the error is bounded against all of the
        # result as above, with the raised share of FP16's r added
        assert (out - ref).norm() / ref.norm() <= 2 * NS_TOL


def test_newton_schulz_repeats_bit_for_bit_and_takes_new_inputs():
    a, b = _gauss(28, 2, 200, 260).cuda(), _gauss(29, 2, 200, 260).cuda()
    out = torch.empty_like(a)
    ws = z.zero_newton_schulz_workspace(a)
    z.zero_newton_schulz(a, out, ws)
    first = out.clone()
    z.zero_newton_schulz(b, out, ws)
    assert not torch.equal(out, first)
    z.zero_newton_schulz(a, out, ws)
    assert torch.equal(out, first)


def test_newton_schulz_empty():
    for shape in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        g = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        z.zero_newton_schulz(g, torch.empty_like(g), torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_binding_refuses_what_the_c_abi_cannot_see():
    g = _gauss(30, 8, 16).cuda()
    out = torch.empty_like(g)
    ws = z.zero_newton_schulz_workspace(g)
    with pytest.raises(ValueError):
        z.zero_newton_schulz(g, out[:, :8], ws)
    with pytest.raises(ValueError):
        z.zero_newton_schulz(g.t(), out.t(), ws)                     # rows not contiguous
    with pytest.raises(TypeError):
        z.zero_newton_schulz(g.half(), out, ws)
    with pytest.raises(TypeError):
        z.zero_newton_schulz(g, out.float(), ws)
    with pytest.raises(TypeError):
        z.zero_newton_schulz(g[0], out[0], ws)
    with pytest.raises(ValueError):
        z.zero_newton_schulz(g, out, ws, coefs=(1.0, 2.0, 3.0))
    with pytest.raises(ValueError):
        z.zero_newton_schulz(g.cpu(), out, ws)
    with pytest.raises(z.ZeroError, match="ZERO_ERR_SIZE"):
        z.zero_newton_schulz(g, out, ws[:256])
    with pytest.raises(z.ZeroError, match="overlap"):
        z.zero_newton_schulz(g, g, ws)
    m = torch.zeros(16, device="cuda")
    with pytest.raises(ValueError):
        z.zero_muon_momentum(m, torch.empty(15, dtype=torch.bfloat16, device="cuda"), m.clone(), HP)
    with pytest.raises(TypeError):
        z.zero_muon_shard_step(m, torch.empty(16, dtype=torch.bfloat16, device="cuda"), m.clone(), HP)
    with pytest.raises(z.ZeroError):
        z.zero_muon_momentum(m, torch.empty(16, dtype=torch.bfloat16, device="cuda"), m.clone(), HP, grad_scale=m[3:4])


# ------------------------------------------------------ streams and graphs
def _step_buffers(seed):
    rng = _rng(seed)
    rows, cols = 96, 160
    n = rows * cols
    return dict(x=[bf16_to_dev(plain.to_bf16(_normal(rng, n, 1e-3))) for _ in range(2)],
                m=f32_to_dev(_normal(rng, n, 3e-4)), u=torch.empty(n, dtype=torch.bfloat16, device="cuda"),
                o=torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda"),
                p=f32_to_dev(_normal(rng, n, 0.02)), b=torch.empty(n, dtype=torch.bfloat16, device="cuda"),
                lr=torch.full((1,), 1e-3, device="cuda"), rows=rows, cols=cols,
                ws=z.zero_newton_schulz_workspace(torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")))


def _one_step(s):
    z.zero_reduce_scatter_muon(s["x"], [0.5, 0.5], [s["m"]], [s["u"]], HP)
    z.zero_newton_schulz(s["u"].view(s["rows"], s["cols"]), s["o"], s["ws"], scale=0.2)
    z.zero_muon_shard_step(s["p"], s["b"], s["o"].flatten(), HP, lr_dev=s["lr"])


def test_step_on_a_side_stream():
    a, b = _step_buffers(40), _step_buffers(40)
    _one_step(a)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        _one_step(b)
    st.synchronize()
    for k in ("m", "u", "o", "p", "b"):
        assert torch.equal(a[k], b[k]), k


def test_step_in_a_replayed_graph():
    a, b = _step_buffers(41), _step_buffers(41)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _one_step(b)
    for t in range(4):
        lr = 1e-3 * (t + 1)
        for s in (a, b):
            s["lr"].fill_(lr)
            for i, x in enumerate(s["x"]):
                x.copy_(_gauss(100 * t + i, x.numel()))
        _one_step(a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in ("m", "u", "o", "p", "b"):
            assert torch.equal(a[k], b[k]), (t, k)
