"""The feed-forward block's forward and backward pass: bit for bit on inputs whose
sums are whole numbers (every tile, edge, alignment and layout), and within the
roundings' bounds of a 64-bit implementation on ordinary inputs."""
import math

import pytest
import torch

import ffn_plain as fp

pytestmark = pytest.mark.gpu

z = pytest.importorskip("zero_sharded_optimizer_reduce_amd")

STEP = 2.0 ** -8   # half a BF16 step, relative


def _at(t, off):
    """A copy of a contiguous tensor that starts `off` elements into its buffer."""
    buf = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
    out = buf[off:].view(t.shape)
    out.copy_(t)
    return out


def _wide(rows, cols, pad, off=0, fill=5.0):
    buf = torch.full((off + rows * (cols + pad) + 9,), fill, dtype=torch.bfloat16, device="cuda")
    return buf, buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def _untouched(buf, view, fill=5.0):
    mark = torch.ones_like(buf, dtype=torch.bool)
    mark.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert bool((buf[mark] == fill).all())


# tokens, model, hidden, pad of x and y, offset of the weights
SHAPES = [(1, 64, 64, 0, 0), (1, 1, 1, 0, 0), (2, 33, 65, 1, 0), (5, 72, 136, 0, 0), (16, 128, 192, 0, 0), (17, 128, 192, 8, 0),
          (31, 70, 250, 3, 1), (33, 256, 320, 0, 8), (64, 192, 128, 0, 1), (65, 192, 128, 0, 0), (127, 320, 448, 4, 0),
          (128, 128, 128, 0, 0), (129, 129, 129, 0, 0), (200, 65, 511, 0, 3), (257, 576, 320, 16, 0), (300, 264, 1032, 0, 0),
          (513, 640, 704, 0, 0), (777, 131, 199, 5, 0), (1025, 256, 2048, 0, 0), (2048, 1024, 1152, 0, 0), (2304, 1024, 2176, 0, 0),
          (100, 2048, 2816, 0, 0), (8192, 2048, 4160, 0, 0), (8209, 2050, 4163, 3, 1), (200, 2053, 8300, 5, 0), (256, 1088, 9024, 0, 0),
          (128, 1088, 11000, 0, 0), (64, 512, 8200, 0, 0), (2100, 1024, 200, 0, 0), (1030, 1024, 4100, 0, 1)]


@pytest.mark.parametrize("saved", [False, True], ids=["", "saved"])
@pytest.mark.parametrize("tokens,model,hidden,pad,off", SHAPES)
def test_forward_exact(tokens, model, hidden, pad, off, saved):
    """Rows of x with at most 8 ones: |g|, |u| <= 8 and |h| <= 64 are exact in BF16."""
    print(f"forward {tokens} x {model} x {hidden} pad {pad} off {off} saved {saved}", flush=True)
    gen = torch.Generator().manual_seed(tokens + model)
    _, x = _wide(tokens, model, pad)
    x.copy_(fp.sparse_signs(gen, tokens, model, 8))
    w = [_at(fp.signs(gen, hidden, model), off), _at(fp.signs(gen, hidden, model), off), _at(fp.signs(gen, model, hidden), off)]
    ybuf, y = _wide(tokens, model, pad)
    ws = z.zero_ffn_workspace(tokens, model, hidden, unaligned=off % 8 != 0)
    ws.fill_(0xFF)   # NaN everywhere
    ck = z.FfnCheckpoint.empty(tokens, model, hidden) if saved else None
    z.zero_ffn_forward(x, *w, y, ws, activation="relu", checkpoint=ck)
    g, u, _, want = fp.forward64(x.double(), *(t.double() for t in w), "relu")
    assert torch.equal(y, want.to(torch.bfloat16))
    _untouched(ybuf, y)
    if saved:
        for held, v in ((ck.x, x.double()), (ck.gate, g), (ck.up, u)):
            assert torch.equal(fp.held_values(*held, "int8"), v)
            assert torch.equal(held[1], fp.quantised(v, "int8")[1])


@pytest.mark.parametrize("tokens,model,hidden,pad,off", SHAPES)
def test_backward_exact(tokens, model, hidden, pad, off):
    """Rows of dy with at most 8 ones and checkpoints of small whole numbers: |dh| <= 8,
    |dg|, |du|, |h| <= 64 are exact in BF16, and the sums in FP32."""
    print(f"backward {tokens} x {model} x {hidden} pad {pad} off {off}", flush=True)
    gen = torch.Generator().manual_seed(tokens + hidden)
    _, dy = _wide(tokens, model, pad)
    dy.copy_(fp.sparse_signs(gen, tokens, model, 8))
    w = [_at(fp.signs(gen, hidden, model), off), _at(fp.signs(gen, hidden, model), off), _at(fp.signs(gen, model, hidden), off)]
    held = [fp.small_checkpoint(gen, tokens, n, 8) for n in (model, hidden, hidden)]
    ck = z.FfnCheckpoint(*(h[:2] for h in held))
    dxbuf, dx = _wide(tokens, model, pad)
    flat = torch.full((3 * hidden * model + 3 * off + 11,), 5.0, dtype=torch.bfloat16, device="cuda")
    d, at = [], 3
    for shape in ((hidden, model), (hidden, model), (model, hidden)):
        d.append(flat[at:at + hidden * model].view(shape))
        at += hidden * model + off
    ws = z.zero_ffn_workspace(tokens, model, hidden, backward=True, unaligned=off % 8 != 0)
    ws.fill_(0xFF)
    z.zero_ffn_backward(dy, ck, *w, dx, *d, ws, activation="relu")
    want = fp.backward64(dy.double(), *(h[2] for h in held), *(t.double() for t in w), "relu")
    for got, ref, name in zip((dx, *d), want, ("dx", "d_gate", "d_up", "d_down")):
        assert torch.equal(got, ref.to(torch.bfloat16)), name
    _untouched(dxbuf, dx)
    assert bool((flat[:3] == 5).all()) and bool((flat[at:] == 5).all())
    for t in d:
        t.fill_(5.0)
    assert bool((flat == 5).all())   # nothing between them
    z.zero_ffn_backward(dy, ck, *w, None, *d, ws, activation="relu")
    for got, ref in zip(d, want[1:]):
        assert torch.equal(got, ref.to(torch.bfloat16))


def _inputs(tokens, model, hidden, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x = n(tokens, model).to(torch.bfloat16)
    w = [(n(hidden, model) / math.sqrt(model)).to(torch.bfloat16), (n(hidden, model) / math.sqrt(model)).to(torch.bfloat16),
         (n(model, hidden) / math.sqrt(hidden)).to(torch.bfloat16)]
    dy = (n(tokens, model) * 1e-3).to(torch.bfloat16)
    return x, w, dy


def _gamma(k):
    """FP32 sums of k products, whatever their order and each rounding towards zero at worst."""
    return k * 2.0 ** -23


def _close(got, want, bound, what):
    """Within its bound everywhere, and within the two roundings' in the 2-norm (each at most
    half a step of each value: 2^-8 of the norm, and independent of the other)."""
    off = (got.double() - want).abs()
    worst = (off / bound).max()
    assert worst <= 1, (what, float(worst))
    assert float(off.norm() / want.norm()) <= math.sqrt(2) * STEP, (what, float(off.norm() / want.norm()))


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("tokens,model,hidden", [(1, 512, 1408), (9, 512, 1408), (50, 130, 333), (256, 512, 1408), (999, 448, 1301),
                                                 (2048, 1024, 1152)])
def test_forward_and_checkpoint(tokens, model, hidden, act):
    x, w, _ = _inputs(tokens, model, hidden)
    xd, wd = x.double(), [t.double() for t in w]
    g, u, h, want = fp.forward64(xd, *wd, act)
    y = torch.empty_like(x)
    ws = z.zero_ffn_workspace(tokens, model, hidden)
    # g and u are sums of `model` products; act's slope is at most 1.13, and what it is computed
    # with is off by a few FP32 steps of values up to 2^5
    eg, eu = _gamma(model) * (xd.abs() @ wd[0].abs().T), _gamma(model) * (xd.abs() @ wd[1].abs().T)
    a = fp.act64(g, act)[0]
    eh = 1.13 * eg * u.abs() + a.abs() * eu + 2.0 ** -18 * h.abs() + STEP * h.abs()
    ey = eh @ wd[2].abs().T + _gamma(hidden) * (h.abs() @ wd[2].abs().T) + STEP * want.abs() * 1.01
    z.zero_ffn_forward(x, *w, y, ws, activation=act)
    _close(y, want, ey, "y")
    for fmt in ("int8", "e4m3"):
        ck = z.FfnCheckpoint.empty(tokens, model, hidden, fmt)
        y2 = torch.empty_like(x)
        z.zero_ffn_forward(x, *w, y2, ws, activation=act, checkpoint=ck)
        _close(y2, want, ey, "y with a checkpoint")
        assert torch.equal(fp.held_values(*ck.x, fmt), fp.quantised(xd, fmt)[0])
        for held, v, e in ((ck.gate, g, eg), (ck.up, u, eu)):
            got = fp.held_values(*held, fmt)
            # half a step of the code, of which a block's largest magnitude may be off by e and the scale by one
            unit = fp.power(held[1].to(torch.int64) - 127)
            unit = unit.repeat_interleave(32, dim=1)[:, :hidden]
            half = 0.5 * unit if fmt == "int8" else torch.maximum(2.0 ** -4 * (v.abs() + e), 2.0 ** -10 * unit)
            assert bool(((got - v).abs() <= half * (1 + 2.0 ** -20) + e).all())
            want_e = fp.quantised(v, fmt)[1].to(torch.int64)
            assert float((held[1].to(torch.int64) != want_e).double().mean()) <= 1e-3 or tokens == 1
            assert int((held[1].to(torch.int64) - want_e).abs().max()) <= 1


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("tokens,model,hidden", [(1, 512, 1408), (9, 512, 1408), (50, 130, 333), (256, 512, 1408), (999, 448, 1301),
                                                 (2048, 1024, 1152)])
def test_backward(tokens, model, hidden, act, fmt):
    x, w, dy = _inputs(tokens, model, hidden, seed=1)
    xd, wd, dyd = x.double(), [t.double() for t in w], dy.double()
    ck = z.FfnCheckpoint.empty(tokens, model, hidden, fmt)
    for v, held in ((x.float(), ck.x), (x.float() @ w[0].float().T, ck.gate), (x.float() @ w[1].float().T, ck.up)):
        z.zero_act8_save(v, *held, format=fmt)
    xv, g, u = (fp.held_values(*held, fmt) for held in (ck.x, ck.gate, ck.up))
    dx = torch.empty_like(x)
    d = [torch.empty_like(t) for t in w]
    ws = z.zero_ffn_workspace(tokens, model, hidden, backward=True)
    z.zero_ffn_backward(dy, ck, *w, dx, *d, ws, activation=act)
    want = fp.backward64(dyd, xv, g, u, *wd, act)
    a, slope = fp.act64(g, act)
    dh = dyd @ wd[2]
    edh = _gamma(model) * (dyd.abs() @ wd[2].abs())
    # act and its slope as computed: a few FP32 steps, of 1 + |g| for the slope's 1 + g (1 - s)
    ea, es = 2.0 ** -18 * (a.abs() + 2.0 ** -20), 2.0 ** -18 * (1 + g.abs())
    dg, du, h = dh * u * slope, dh * a, a * u
    edg = edh * (u * slope).abs() + (dh * u).abs() * es + STEP * dg.abs() * 1.01
    edu = edh * a.abs() + dh.abs() * ea + STEP * du.abs() * 1.01
    eh = u.abs() * ea + STEP * h.abs() * 1.01
    sums = ((edg @ wd[0].abs() + edu @ wd[1].abs() + _gamma(2 * hidden) * (dg.abs() @ wd[0].abs() + du.abs() @ wd[1].abs())),
            edg.T @ xv.abs() + _gamma(tokens) * (dg.abs().T @ xv.abs()), edu.T @ xv.abs() + _gamma(tokens) * (du.abs().T @ xv.abs()),
            dyd.abs().T @ eh + _gamma(tokens) * (dyd.abs().T @ h.abs()))
    for got, ref, e, name in zip((dx, *d), want, sums, ("dx", "d_gate", "d_up", "d_down")):
        _close(got, ref, e + STEP * ref.abs() * 1.01 + 2.0 ** -133, name)
