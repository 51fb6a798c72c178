"""Feed-forward calls at the edges of what they take: with and without a checkpoint,
infinities, workspaces of larger batches, the driver's kept passes, matrices side by
side, far rows, weights and gradients that are not finite, activations far
out, gradients against differences of the forward pass."""
import math

import pytest
import torch

import ffn_plain as fp

pytestmark = pytest.mark.gpu

z = pytest.importorskip("zero_sharded_optimizer_reduce_amd")


def _normal(gen, *shape, sigma=1.0):
    return torch.randn(*shape, generator=gen, device="cuda").mul_(sigma).to(torch.bfloat16)


def _weights(gen, model, hidden):
    return [_normal(gen, hidden, model, sigma=1 / math.sqrt(model)), _normal(gen, hidden, model, sigma=1 / math.sqrt(model)),
            _normal(gen, model, hidden, sigma=1 / math.sqrt(hidden))]


def _forward(x, w, act="silu", checkpoint=None, y=None):
    y = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda") if y is None else y
    ws = z.zero_ffn_workspace(x.shape[0], x.shape[1], w[0].shape[0])
    ws.fill_(0xFF)   # NaN everywhere
    z.zero_ffn_forward(x, *w, y, ws, activation=act, checkpoint=checkpoint)
    return y


def _backward(dy, ck, w, act="silu", dx=None):
    dx = torch.empty(dy.shape, dtype=torch.bfloat16, device="cuda") if dx is None else dx
    d = [torch.empty_like(t) for t in w]
    ws = z.zero_ffn_workspace(dy.shape[0], dy.shape[1], w[0].shape[0], backward=True)
    ws.fill_(0xFF)
    z.zero_ffn_backward(dy, ck, *w, dx, *d, ws, activation=act)
    return [dx, *d]


def _bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


# ------------------------------------------------------------------ with and without a checkpoint
@pytest.mark.parametrize("tokens", [1, 7, 16, 17, 32, 33, 200, 700])
@pytest.mark.parametrize("model,hidden", [(4096, 14336), (1024, 7936), (2048, 11008), (1301, 2999), (512, 1408)])
def test_a_checkpoint_changes_no_bit_of_y(model, hidden, tokens):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x, w = _normal(gen, tokens, model), _weights(gen, model, hidden)
    kept = _forward(x, w, checkpoint=z.FfnCheckpoint.empty(tokens, model, hidden))
    assert _bits(_forward(x, w), kept)


# ------------------------------------------------------------------ infinities
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("tokens", [1, 20, 40, 300, 2100])
@pytest.mark.parametrize("model,hidden", [(64, 65), (70, 33), (64, 96), (33, 1), (1024, 2111)])
def test_an_infinity_gives_the_infinite_sum(model, hidden, tokens, act):
    """Positive weights and +inf in x: g, u, h and y are +inf, whatever fills the rows of the
    matrices up to the kernels' tiles."""
    gen = torch.Generator(device="cuda").manual_seed(hidden)
    x = _normal(gen, tokens, model)
    w = [torch.rand(s, generator=gen, device="cuda").add_(0.5).div_(model).to(torch.bfloat16)
         for s in ((hidden, model), (hidden, model), (model, hidden))]
    want = _forward(x, w, act)
    at = tokens // 2
    x[at, model // 3] = math.inf
    ck = z.FfnCheckpoint.empty(tokens, model, hidden)
    y = _forward(x, w, act, ck)
    assert bool((y[at] == math.inf).all())
    others = torch.arange(tokens, device="cuda") != at
    assert _bits(y[others], want[others]) and bool(torch.isfinite(y[others].float()).all())
    assert bool((ck.gate[1][at] == 255).all()) and bool((ck.up[1][at] == 255).all())


# ------------------------------------------------------------------ a workspace for more tokens
@pytest.mark.parametrize("model,hidden,most,tokens", [(4096, 14336, 513, 512), (4096, 14336, 2049, 2048), (2048, 8192, 1500, 1024),
                                                      (1301, 777, 2000, 64)])
def test_a_workspace_serves_fewer_tokens(model, hidden, most, tokens):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x, w, dy = _normal(gen, tokens, model), _weights(gen, model, hidden), _normal(gen, tokens, model, sigma=1e-3)
    rooms = [z.zero_ffn_workspace(most, model, hidden, backward=back) for back in (False, True)]
    ck = z.FfnCheckpoint.empty(tokens, model, hidden)
    y, dx, d = torch.empty_like(x), torch.empty_like(x), [torch.empty_like(t) for t in w]
    z.zero_ffn_forward(x, *w, y, rooms[0], checkpoint=ck)
    z.zero_ffn_backward(dy, ck, *w, dx, *d, rooms[1])
    assert _bits(y, _forward(x, w))
    for a, b in zip((dx, *d), _backward(dy, ck, w)):
        assert _bits(a, b)


# ------------------------------------------------------------------ the driver's kept passes
HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1)


@pytest.mark.parametrize("update", ["backward_unit", "backward_unit_fused", "update_unit"])
def test_an_update_of_a_unit_forgets_its_kept_pass(update):
    """Whichever of the chain's updates: a kept pass is of the weights before it."""
    from zero_sharded_optimizer_reduce_amd.drivers import Zero3FeedForward

    st = Zero3FeedForward([(64, 96), (64, 96)], 2, 20)
    for t in (*st.master, *st.bf16):
        t.zero_()
    xs = [torch.ones(20, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ys = [torch.empty_like(x) for x in xs]
    w = z.zero_rank_weights([20, 20], 2)
    for u in (0, 1):
        st.forward_layer(u, xs, ys)
    st.contribute(1, xs, [None, None])
    if update == "update_unit":
        st.reduce_unit(1, w)
        st.update_unit(1, HP)
    else:
        getattr(st, update)(1, w, HP)
    with pytest.raises(ValueError, match="other tokens"):
        st.contribute(1, xs, [None, None])
    st.contribute(0, xs, [None, None])   # the other unit's is still of its weights
    st.forward_layer(1, xs, ys)
    st.contribute(1, xs, [None, None])


# ------------------------------------------------------------------ matrices side by side
@pytest.mark.parametrize("tokens,model,hidden,gap", [(1, 64, 96, 0), (20, 64, 96, 0), (40, 64, 128, 0), (200, 70, 96, 3), (300, 256, 320, 8),
                                                     (1000, 512, 1408, 0), (2100, 1024, 1100, 0)])
def test_x_and_y_side_by_side_in_one_buffer(tokens, model, hidden, gap):
    """Columns of one buffer: rows alternate in memory and share no element."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    w = _weights(gen, model, hidden)
    for first in (0, 1):   # x before y, and behind it
        buf = torch.full((tokens, 2 * model + 2 * gap), 3.0, dtype=torch.bfloat16, device="cuda")
        halves = [buf[:, :model], buf[:, model + gap:2 * model + gap]]
        a, b = halves[first], halves[1 - first]
        a.copy_(_normal(gen, tokens, model))
        x = a.contiguous()
        ck = z.FfnCheckpoint.empty(tokens, model, hidden)
        _forward(a, w, checkpoint=ck, y=b)
        assert _bits(b, _forward(x, w)) and _bits(a, x)
        _backward_want = _backward(x, ck, w)
        got = _backward(a, ck, w, dx=b)
        for p, q in zip(got, _backward_want):
            assert _bits(p, q)
        assert _bits(a, x) and bool((buf[:, 2 * model + gap:] == 3).all()) and bool((buf[:, model:model + gap] == 3).all())


def test_matrices_that_share_elements_are_refused():
    gen = torch.Generator(device="cuda").manual_seed(0)
    w = _weights(gen, 64, 96)
    buf = torch.zeros(40, 256, dtype=torch.bfloat16, device="cuda")
    for first in (1, 32, 63):
        with pytest.raises(z.ZeroError, match="overlap"):
            _forward(buf[:, :64], w, y=buf[:, first:first + 64])
        with pytest.raises(z.ZeroError, match="overlap"):
            _forward(buf[:, first:first + 64], w, y=buf[:, :64])
    with pytest.raises(z.ZeroError, match="overlap"):   # a row further on
        _forward(buf[1:, :64], w, y=buf[:39, 33:97])
    with pytest.raises(z.ZeroError, match="overlap"):   # round the row's end
        _forward(buf[:39, 200:].as_strided((39, 64), (256, 1)), w, y=buf[:39, :64])


# ------------------------------------------------------------------ far rows
def test_gradients_with_rows_far_apart():
    """Row strides with which the last rows of dy and dx lie over 2^32 bytes behind the first."""
    tokens, model, hidden, stride = 600, 64, 128, 1 << 22
    gen = torch.Generator().manual_seed(2)
    w = [fp.signs(gen, hidden, model), fp.signs(gen, hidden, model), fp.signs(gen, model, hidden)]
    held = [fp.small_checkpoint(gen, tokens, n, 8) for n in (model, hidden, hidden)]
    ck = z.FfnCheckpoint(*(h[:2] for h in held))
    bufs = [torch.zeros((tokens - 1) * stride + 2 * model, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dy, dx = (b.as_strided((tokens, model), (stride, 1)) for b in bufs)
    dy.copy_(fp.sparse_signs(gen, tokens, model, 8))
    got = _backward(dy, ck, w, "relu", dx)
    want = fp.backward64(dy.double(), *(h[2] for h in held), *(t.double() for t in w), "relu")
    for a, b, name in zip(got, want, ("dx", "d_gate", "d_up", "d_down")):
        assert torch.equal(a, b.to(torch.bfloat16)), name
    assert int(bufs[0].count_nonzero()) == int(dy.count_nonzero()) and int(bufs[1].count_nonzero()) == int(dx.count_nonzero())


# ------------------------------------------------------------------ weights and gradients that are not finite
SIZES = [(5, 64, 96), (31, 130, 70), (40, 70, 33), (200, 256, 320), (1000, 512, 1408), (2100, 1024, 2111)]


def _clean(tokens, model, hidden):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x, w, dy = _normal(gen, tokens, model), _weights(gen, model, hidden), _normal(gen, tokens, model, sigma=1e-2)
    ck = z.FfnCheckpoint.empty(tokens, model, hidden, "e4m3")
    y = _forward(x, w, checkpoint=ck)
    return x, w, dy, ck, y, _backward(dy, ck, w)


def _but(n, *without):
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[list(without)] = False
    return keep


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("tokens,model,hidden", SIZES)
def test_a_weight_that_is_not_finite_reaches_only_its_own_results(tokens, model, hidden, bad):
    x, w, dy, ck, y, grads = _clean(tokens, model, hidden)
    for r, c in ((0, 0), (hidden - 1, model - 1)):   # the last one beside what fills the tiles up
        for k in (0, 1):
            v = [t.clone() for t in w]
            v[k][r, c] = bad
            ck2 = z.FfnCheckpoint.empty(tokens, model, hidden, "e4m3")
            y2 = _forward(x, v, checkpoint=ck2)
            if math.isnan(bad):
                assert bool(y2.isnan().all())
            held, other, ref, same = ((ck2.gate, ck2.up, ck.gate, ck.up), (ck2.up, ck2.gate, ck.up, ck.gate))[k]
            assert torch.equal(other[0], same[0]) and torch.equal(other[1], same[1])
            assert bool((held[1][:, r // 32] == 255).all())
            keep = _but(held[1].shape[1], r // 32)
            assert torch.equal(held[1][:, keep], ref[1][:, keep])
            keep = _but(hidden, *range(r // 32 * 32, min(hidden, r // 32 * 32 + 32)))
            assert torch.equal(held[0][:, keep], ref[0][:, keep])
            got = _backward(dy, ck, v)
            assert not bool(got[0][:, c].isfinite().any()) and _bits(got[0][:, _but(model, c)], grads[0][:, _but(model, c)])
            assert all(_bits(a, b) for a, b in zip(got[1:], grads[1:]))
        v = [t.clone() for t in w]
        v[2][c, r] = bad
        y2 = _forward(x, v)
        assert not bool(y2[:, c].isfinite().any()) and _bits(y2[:, _but(model, c)], y[:, _but(model, c)])
        got = _backward(dy, ck, v)
        assert not bool(got[0].isfinite().any())   # through dh[:, r], in every sum
        for k in (1, 2):
            assert not bool(got[k][r].isfinite().any()) and _bits(got[k][_but(hidden, r)], grads[k][_but(hidden, r)])
        assert _bits(got[3], grads[3])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("tokens,model,hidden", SIZES)
def test_a_gradient_that_is_not_finite_reaches_only_its_own_results(tokens, model, hidden, bad):
    x, w, dy, ck, y, grads = _clean(tokens, model, hidden)
    for t, c in ((0, 0), (tokens - 1, model - 1)):
        dy2 = dy.clone()
        dy2[t, c] = bad
        dx, d_gate, d_up, d_down = _backward(dy2, ck, w)
        assert not bool(dx[t].isfinite().any()) and _bits(dx[_but(tokens, t)], grads[0][_but(tokens, t)])
        assert not bool(d_gate.isfinite().any()) and not bool(d_up.isfinite().any())   # sums over the token
        assert not bool(d_down[c].isfinite().any()) and _bits(d_down[_but(model, c)], grads[3][_but(model, c)])


# ------------------------------------------------------------------ activations far out
def _act(g, act):
    """act(g) and its derivative in 64 bits, without the cancellation of 1 + tanh far out."""
    if act == "relu":
        return torch.clamp(g, min=0), (g > 0).double()
    k, c = math.sqrt(2 / math.pi), 0.044715
    inner, turn = (g, torch.ones_like(g)) if act == "silu" else (2 * k * (g + c * g ** 3), 2 * k * (1 + 3 * c * g * g))
    s, t = torch.sigmoid(inner), torch.sigmoid(-inner)
    return g * s, s + torch.where(s * t > 0, g * s * t * turn, torch.zeros_like(g))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("tokens", [29, 64])
def test_activations_and_slopes_far_out(tokens, act, fmt):
    """x picks one gate value per token, up is 1, down hands h through: y is act(g), and from the
    checkpoint's g the gradients of gate's and up's first rows are act'(g) and act(g)."""
    half = [1e-30, 1e-3, 5.0, 8.0, 12.0, 16.0, 17.0, 30.0, 80.0, 88.0, 104.0, 1e4, 1e18, 3e37]
    big = torch.tensor([0.0, *half, *(-v for v in half)], device="cuda")
    n = big.numel()
    x = torch.zeros(tokens, 64, device="cuda")
    x[:n] = torch.eye(n, 64, device="cuda")
    wg, wu, wd = (torch.zeros(64, 64, device="cuda") for _ in range(3))
    wg[0, :n] = big
    wu[0, :n] = 1.0
    wd[0, 0] = 1.0
    x, *w = [t.to(torch.bfloat16) for t in (x, wg, wu, wd)]
    ck = z.FfnCheckpoint.empty(tokens, 64, 64, fmt)
    y = _forward(x, w, act, ck)
    _, d_gate, d_up, _ = _backward(torch.ones_like(x), ck, w, act)
    held = fp.held_values(*ck.gate, fmt)[:n, 0]
    assert bool(((held - w[0][0, :n].double()).abs() <= 2.0 ** -4 * held.abs() + 1e-38).all())
    # One rounding to BF16, and what act is computed with: exponents of size |v| off by 3 |v| steps of FP32, and
    # below 2^-126 zeros; above 0 sigma and its complement are off by a step of 1, times the slope's g (1 + 3 c g^2)
    # where they are not the limits (|g| <= 17 for SiLU, 6 for GELU)
    for got, v, k in ((y[:n, 0], w[0][0, :n].double(), 0), (d_up[0, :n], held, 0), (d_gate[0, :n], held, 1)):
        want = _act(v, act)[k]
        off = (got.double() - want).abs()
        bound = 2.0 ** -8 * 1.02 * want.abs() + torch.where(v > 0, 2.0 ** -16, 1e-36) * (k == 1) + 1e-36
        assert bool(torch.isfinite(got.float()).all()) and bool((off <= bound).all()), (k, v[off > bound], got[off > bound], want[off > bound])


# ------------------------------------------------------------------ gradients against differences
@pytest.mark.parametrize("tokens,model,hidden", [(1, 64, 64), (3, 33, 70), (20, 64, 130), (40, 70, 131), (150, 192, 256)])
def test_gradients_are_differences_of_the_forward_pass(tokens, model, hidden):
    """Gates that stay on their side of ReLU's corner and whole numbers that BF16 and the
    checkpoints hold: y is a polynomial of degree two in each entry, and central differences
    of the kernels' own y are its derivative, to the last bit."""
    gen = torch.Generator().manual_seed(tokens)
    x = torch.zeros(tokens, model)
    for row in x:   # three entries of +-1: g is an odd multiple of 4, u odd
        row[torch.randperm(model, generator=gen)[:3]] = torch.randint(0, 2, (3,), generator=gen).float() * 2 - 1
    x = x.to(torch.bfloat16).cuda()
    w = [fp.signs(gen, hidden, model) * 4, fp.signs(gen, hidden, model), fp.sparse_signs(gen, model, hidden, 2)]
    dy = fp.signs(gen, tokens, model)
    ck = z.FfnCheckpoint.empty(tokens, model, hidden)
    y = _forward(x, w, "relu", ck)
    g, u, h, want = fp.forward64(x.double(), *(t.double() for t in w), "relu")
    assert torch.equal(y.double(), want) and float(h.abs().max()) <= 36
    assert torch.equal(fp.held_values(*ck.gate, "int8"), g) and torch.equal(fp.held_values(*ck.up, "int8"), u)
    grads = _backward(dy, ck, w, "relu")
    for k, (t, grad) in enumerate(zip((x, *w), grads)):
        flat = grad.double().abs().flatten()
        some = torch.randint(0, t.numel(), (6,), generator=gen).tolist()
        for at in {0, t.numel() - 1, int(flat.argmax()), int(flat.gt(0).nonzero()[-1]), *some}:
            ends = []
            for step in (1, -1):
                moved = [v.clone() for v in (x, *w)]
                moved[k].view(-1)[at] += step
                ends.append(_forward(moved[0], moved[1:], "relu").double())
            slope = ((ends[0] - ends[1]) * dy.double()).sum() / 2
            assert grad.reshape(-1)[at] == slope.to(torch.bfloat16), (k, at)
