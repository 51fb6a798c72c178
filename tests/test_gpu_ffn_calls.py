"""How the feed-forward calls behave: values that are not finite, no tokens, far
offsets, repeated, overlapping and captured calls, refusals; and the driver that
runs them between a chain's gathers and reductions."""
import math

import pytest
import torch

import ffn_plain as fp
import zero_sharded_optimizer_reduce_amd as z
from zero_sharded_optimizer_reduce_amd.drivers import Zero3Chain, Zero3FeedForward

pytestmark = pytest.mark.gpu


def _weights(gen, model, hidden):
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    return [(n(hidden, model) / math.sqrt(model)).to(torch.bfloat16), (n(hidden, model) / math.sqrt(model)).to(torch.bfloat16),
            (n(model, hidden) / math.sqrt(hidden)).to(torch.bfloat16)]


def _case(tokens, model, hidden, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, model, generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn(tokens, model, generator=gen, device="cuda").mul_(1e-2).to(torch.bfloat16)
    return x, _weights(gen, model, hidden), dy


class _Pass:
    """A forward and a backward pass with buffers of their own."""

    def __init__(self, x, w, dy, act="silu", fmt="int8"):
        self.x, self.w, self.dy, self.act = x, w, dy, act
        t, m, h = x.shape[0], x.shape[1], w[0].shape[0]
        self.ck = z.FfnCheckpoint.empty(t, m, h, fmt)
        self.y, self.dx = torch.empty_like(x), torch.empty_like(x)
        self.d = [torch.empty_like(v) for v in w]
        self.ws = z.zero_ffn_workspace(t, m, h), z.zero_ffn_workspace(t, m, h, backward=True)

    def run(self, stream=None):
        z.zero_ffn_forward(self.x, *self.w, self.y, self.ws[0], activation=self.act, checkpoint=self.ck, stream=stream)
        z.zero_ffn_backward(self.dy, self.ck, *self.w, self.dx, *self.d, self.ws[1], activation=self.act, stream=stream)

    def results(self):
        return [t.clone() for t in (self.y, *self.ck.x, *self.ck.gate, *self.ck.up, self.dx, *self.d)]


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b, strict=True))


SIZES = [(5, 64, 96), (31, 130, 70), (200, 256, 320), (1000, 512, 1408), (4096, 1024, 4224)]


@pytest.mark.parametrize("tokens,model,hidden", SIZES)
def test_same_bits_on_every_call(tokens, model, hidden):
    p = _Pass(*_case(tokens, model, hidden))
    p.run()
    first = p.results()
    for fill in (0x00, 0xFF, 0x7F):   # nothing is taken from the workspaces or the results
        for t in (*p.ws, *(v.view(torch.uint8) for v in (p.y, p.dx, *p.d)), *p.ck.x, *p.ck.gate, *p.ck.up):
            t.fill_(fill)
        p.run()
        assert _same(first, p.results())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("tokens,model,hidden", SIZES)
def test_a_token_that_is_not_finite_stays_alone(tokens, model, hidden, bad):
    x, w, dy = _case(tokens, model, hidden)
    clean = _Pass(x, w, dy, fmt="e4m3")
    clean.run()
    at = tokens // 2
    p = _Pass(x.clone(), w, dy, fmt="e4m3")
    p.x[at, model // 3] = bad
    z.zero_ffn_forward(p.x, *w, p.y, p.ws[0], checkpoint=p.ck)
    others = [t for t in range(tokens) if t != at]
    assert not bool(torch.isfinite(p.y[at].float()).any()) if math.isnan(bad) else bool(torch.isnan(p.y[at]).any())
    assert torch.equal(p.y[others], clean.y[others])
    for held, ref in ((p.ck.x, clean.ck.x), (p.ck.gate, clean.ck.gate), (p.ck.up, clean.ck.up)):
        assert torch.equal(held[0][others], ref[0][others]) and torch.equal(held[1][others], ref[1][others])
    assert bool((p.ck.gate[1][at] == 255).all())
    assert int(p.ck.x[1][at, model // 3 // 32]) == 255
    z.zero_ffn_backward(dy, p.ck, *w, p.dx, *p.d, p.ws[1])
    assert bool(torch.isnan(p.dx[at]).all()) and torch.equal(p.dx[others], clean.dx[others])
    assert bool(torch.isnan(p.d[0]).any())   # the weights' gradients sum over the token


def test_activations_far_out():
    """Where e^x overflows and the cube of GELU would: the limits, no NaN."""
    big = torch.tensor([0.0, -0.0, 1e-30, 30.0, -30.0, 88.0, -88.0, 1e4, -1e4, 1e18, -1e18], device="cuda")
    n = big.numel()
    for act in ("silu", "gelu", "relu"):
        # x picks one gate value per token; up is 1 and down hands h through
        x = torch.eye(n, 64, device="cuda").to(torch.bfloat16)
        wg = torch.zeros(64, 64, device="cuda")
        wg[0, :n] = big
        wu = torch.zeros(64, 64, device="cuda")
        wu[0, :n] = 1.0
        wd = torch.zeros(64, 64, device="cuda")
        wd[0, 0] = 1.0
        w = [t.to(torch.bfloat16) for t in (wg, wu, wd)]
        p = _Pass(x, w, torch.ones_like(x), act=act, fmt="e4m3")
        p.run()
        g = w[0][0, :n].double()
        a, slope = fp.act64(g.cpu(), act)
        a, slope = torch.nan_to_num(a), torch.nan_to_num(slope)   # inf * 0 of the plain form
        assert bool(torch.isfinite(p.y.float()).all()) and bool(torch.isfinite(p.dx.float()).all())
        far = a.abs() > 1e-20
        assert torch.allclose(p.y[:, 0].double().cpu()[far], a[far], rtol=2 ** -8 * 1.5, atol=0)


@pytest.mark.parametrize("model,hidden", [(64, 96), (33, 65), (256, 2048)])
def test_no_tokens(model, hidden):
    x, w, dy = _case(0, model, hidden)
    p = _Pass(x, w, dy)
    for t in p.d:
        t.fill_(7.0)
    p.run()
    for t in p.d:
        assert int(t.count_nonzero()) == 0


def test_a_long_batch_whose_activations_pass_32_bit_offsets():
    """300,000 tokens through 64 x 8192: 2.46e9 hidden values.  Whole-number inputs; the
    gradients' sums stay below 2^24, rows are checked here and there."""
    tokens, model, hidden = 300_000, 64, 8192
    gen = torch.Generator().manual_seed(11)
    some = fp.sparse_signs(gen, 1024, model, 8)
    x = some.repeat(293, 1)[:tokens].contiguous()
    dy = some.flip(0).repeat(293, 1)[:tokens].contiguous()
    w = [fp.signs(gen, hidden, model), fp.signs(gen, hidden, model), fp.signs(gen, model, hidden)]
    wd = [t.double() for t in w]
    ck = z.FfnCheckpoint.empty(tokens, model, hidden)
    y = torch.empty_like(x)
    z.zero_ffn_forward(x, *w, y, z.zero_ffn_workspace(tokens, model, hidden), activation="relu", checkpoint=ck)
    at = torch.tensor([0, 1, 1023, 131071, 131072, 262143, 262144, 262145, 290000, tokens - 2, tokens - 1], device="cuda")
    g, u, _, want = fp.forward64(x[at].double(), *wd, "relu")
    assert torch.equal(y[at], want.to(torch.bfloat16))
    for held, v in ((ck.gate, g), (ck.up, u)):
        assert torch.equal(fp.held_values(held[0][at], held[1][at], "int8"), v)
    # every 1024 rows are the same
    assert all(torch.equal(y[k:k + 1024], y[:1024]) for k in (1024, 262144, 291 * 1024))
    dx = torch.empty_like(x)
    d = [torch.empty_like(t) for t in w]
    z.zero_ffn_backward(dy, ck, *w, dx, *d, z.zero_ffn_workspace(tokens, model, hidden, backward=True), activation="relu")
    want = fp.backward64(dy[at].double(), x[at].double(), g, u, *wd, "relu")[0]
    assert torch.equal(dx[at], want.to(torch.bfloat16))
    # the gradients: 292 whole repeats of 1024 tokens and 992 more
    def grads(n):
        gg, uu, _, _ = fp.forward64(x[:n].double(), *wd, "relu")
        return fp.backward64(dy[:n].double(), x[:n].double(), gg, uu, *wd, "relu")[1:]
    for got, whole, rest in zip(d, grads(1024), grads(tokens - 292 * 1024)):
        total = whole * 292 + rest
        assert float(total.abs().max()) < 2 ** 24
        assert torch.equal(got, total.to(torch.bfloat16))


def test_rows_far_apart():
    """Row strides with which the last row lies over 2^32 bytes behind the first."""
    tokens, model, hidden, stride = 600, 64, 128, 1 << 22
    gen = torch.Generator().manual_seed(2)
    buf = torch.zeros((tokens - 1) * stride + 2 * model, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((tokens, model), (stride, 1))
    x.copy_(fp.sparse_signs(gen, tokens, model, 8))
    w = [fp.signs(gen, hidden, model), fp.signs(gen, hidden, model), fp.signs(gen, model, hidden)]
    y = torch.empty(tokens, model, dtype=torch.bfloat16, device="cuda")
    z.zero_ffn_forward(x, *w, y, z.zero_ffn_workspace(tokens, model, hidden), activation="relu")
    want = fp.forward64(x.double(), *(t.double() for t in w), "relu")[3]
    assert torch.equal(y, want.to(torch.bfloat16))
    z.zero_ffn_forward(y.clamp(-1, 1), *w, x, z.zero_ffn_workspace(tokens, model, hidden), activation="relu")
    assert int(buf.count_nonzero()) == int(x.count_nonzero())


@pytest.mark.parametrize("tokens,model,hidden", SIZES)
def test_two_streams_at_once(tokens, model, hidden):
    passes = [_Pass(*_case(tokens, model, hidden, seed=k)) for k in range(2)]
    want = []
    for p in passes:
        p.run()
        want.append(p.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in passes]
    for _ in range(3):
        for p, s in zip(passes, streams):
            p.run(stream=s)
            p.run(stream=s.cuda_stream)
    torch.cuda.synchronize()
    for p, ref in zip(passes, want):
        assert _same(p.results(), ref)


@pytest.mark.parametrize("tokens,model,hidden", SIZES)
def test_captured_and_replayed(tokens, model, hidden):
    x, w, dy = _case(tokens, model, hidden)
    p, eager = _Pass(x.clone(), w, dy.clone(), fmt="e4m3"), _Pass(x, w, dy, fmt="e4m3")
    p.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for k in range(3):
        x2, _, dy2 = _case(tokens, model, hidden, seed=20 + k)
        for q in (p, eager):
            q.x.copy_(x2)
            q.dy.copy_(dy2)
        graph.replay()
        eager.run()
        torch.cuda.synchronize()
        assert _same(p.results(), eager.results()), k


def test_refusals():
    x, w, dy = _case(40, 64, 96)
    p = _Pass(x, w, dy)
    small = torch.empty(p.ws[1].numel() - 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(z.ZeroError, match="needed"):
        z.zero_ffn_backward(dy, p.ck, *w, p.dx, *p.d, small)
    with pytest.raises(ValueError, match="w_up"):
        z.zero_ffn_forward(x, w[0], w[1][:-1], w[2], p.y, p.ws[0])
    with pytest.raises(ValueError, match="contiguous"):
        z.zero_ffn_forward(x, w[0], w[1], w[0].t(), p.y, p.ws[0])
    with pytest.raises(ValueError, match="shape"):
        z.zero_ffn_forward(x, *w, p.y[:-1], p.ws[0])
    with pytest.raises(ValueError, match="tanh"):
        z.zero_ffn_forward(x, *w, p.y, p.ws[0], activation="tanh")
    with pytest.raises(TypeError):
        z.zero_ffn_forward(x.float(), *w, p.y, p.ws[0])
    with pytest.raises(ValueError, match="checkpoint"):
        z.zero_ffn_backward(dy[:-1], p.ck, *w, p.dx[:-1], *p.d, p.ws[1])
    with pytest.raises(ValueError, match="d_gate"):
        z.zero_ffn_backward(dy, p.ck, *w, p.dx, p.d[0][:-1], p.d[1][:-1], p.d[2][:, :-1].contiguous(), p.ws[1])
    with pytest.raises(z.ZeroError, match="overlap"):
        z.zero_ffn_forward(x, *w, x, p.ws[0])
    with pytest.raises(z.ZeroError, match="overlap"):
        z.zero_ffn_backward(dy, p.ck, *w, p.dx, p.d[0], p.d[0], p.d[2], p.ws[1])
    with pytest.raises(z.ZeroError, match="stride"):
        z.zero_ffn_forward(x[:1].expand(40, 64), *w, p.y, p.ws[0])
    odd = torch.zeros(96 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(96, 64)
    x, w, dy = _case(40, 64, 128)
    odd = torch.zeros(128 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(128, 64)
    y = torch.empty_like(x)
    with pytest.raises(z.ZeroError, match="UNALIGNED"):
        z.zero_ffn_forward(x, odd, w[1], w[2], y, z.zero_ffn_workspace(40, 64, 128))
    z.zero_ffn_forward(x, odd, w[1], w[2], y, z.zero_ffn_workspace(40, 64, 128, unaligned=True))
    assert int(y.count_nonzero()) == 0


# ------------------------------------------------------------------ the driver
HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1)


def _driver(layers, n, tokens, **k):
    gen = torch.Generator().manual_seed(9)
    st = Zero3FeedForward(layers, n, max(tokens), **k)
    for u, (m, h) in enumerate(layers):
        flat = torch.randn(st.units[u][2], generator=gen).div_(math.sqrt(m)).cuda()
        s = st.units[u][3]
        for r, (p, b) in enumerate(zip(st.owner_slices(u, st.master), st.owner_slices(u, st.bf16))):
            p.copy_(flat[r * s:(r + 1) * s])
            b.copy_(p)
    return st


def _step(st, xs, dys, w, hp, stream=None):
    hs = [[torch.empty_like(x) for x in xs] for _ in st.layers]
    for u in range(len(st.layers)):
        st.forward_layer(u, hs[u - 1] if u else xs, hs[u], stream=stream)
    ds = dys
    for u in reversed(range(len(st.layers))):
        dxs = [torch.empty_like(x) for x in xs]
        st.backward_layer(u, ds, dxs, w, hp, stream=stream)
        ds = dxs
    return hs, ds


def _state(st):
    return [t.clone() for x in (st.master, st.exp_avg, st.exp_avg_sq, st.bf16) for t in x]


@pytest.mark.parametrize("layers,tokens,act,fmt", [([(64, 96), (64, 160)], (50, 0, 33), "silu", "int8"),
                                                   ([(70, 31)], (7, 300), "gelu", "e4m3"),
                                                   ([(256, 704), (256, 640)], (512, 512, 257, 1), "relu", "int8")])
def test_a_step_of_the_driver(layers, tokens, act, fmt):
    n, model = len(tokens), layers[0][0]
    st = _driver(layers, n, tokens, activation=act, format=fmt)
    twin = _driver(layers, n, tokens, activation=act, format=fmt)
    gen = torch.Generator(device="cuda").manual_seed(4)
    xs = [torch.randn(t, model, generator=gen, device="cuda").to(torch.bfloat16) for t in tokens]
    dys = [torch.randn(t, model, generator=gen, device="cuda").mul_(1e-2).to(torch.bfloat16) for t in tokens]
    w = z.zero_rank_weights(list(tokens), n)
    hs = [[torch.empty_like(x) for x in xs] for _ in layers]
    for u in range(len(layers)):
        st.forward_layer(u, hs[u - 1] if u else xs, hs[u])
    ds = dys
    for u in reversed(range(len(layers))):
        m, h = layers[u]
        psi, pad = st.units[u][1:3]
        flat = torch.cat(st.owner_slices(u, st.bf16))
        wts = [flat[k * m * h:(k + 1) * m * h].view(s).double() for k, s in enumerate(((h, m), (h, m), (m, h)))]
        for g in st.grads:
            g.fill_(3.0)
        dxs = [torch.empty_like(x) for x in xs]
        st.contribute(u, ds, dxs)
        for r, t in enumerate(tokens):
            inp = (hs[u - 1] if u else xs)[r].double()
            if t:
                ref = fp.forward64(inp, *wts, act)[3]
                assert float((hs[u][r].double() - ref).norm()) <= math.sqrt(2) * 2 ** -8 * float(ref.norm())
            held = [fp.held_values(c[:t], s[:t], fmt) for c, s in
                    (st.checkpoints[u][r].x, st.checkpoints[u][r].gate, st.checkpoints[u][r].up)]
            want = fp.backward64(ds[r].double(), *held, *wts, act)
            got = [st.grads[r][k * m * h:(k + 1) * m * h].view(s) for k, s in enumerate(((h, m), (h, m), (m, h)))]
            for a, b in zip((dxs[r], *got), want):
                assert float((a.double() - b).norm()) <= math.sqrt(2) * 2 ** -8 * float(b.norm())
            assert int(st.grads[r][psi:pad].count_nonzero()) == 0
            if t == 0:
                assert int(st.grads[r][:psi].count_nonzero()) == 0
        # the reduction and the updates are the chain's own
        for a, b in zip(twin.grads, st.grads):
            a.copy_(b)
        st.backward_unit(u, w, HP)
        Zero3Chain.backward_unit(twin, u, w, HP)
        ds = dxs
    assert _same(_state(st), _state(twin))


def test_driver_on_a_stream_of_its_own_and_captured():
    layers, tokens = [(64, 96), (64, 160)], (50, 34)
    gen = torch.Generator(device="cuda").manual_seed(4)
    xs = [torch.randn(t, 64, generator=gen, device="cuda").to(torch.bfloat16) for t in tokens]
    dys = [torch.randn(t, 64, generator=gen, device="cuda").mul_(1e-2).to(torch.bfloat16) for t in tokens]
    w = z.zero_rank_weights(list(tokens), 2)
    a, b, c = (_driver(layers, 2, tokens) for _ in range(3))
    for t in range(3):
        _step(a, xs, dys, w, HP)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep = [_step(b, xs, dys, w, HP, stream=side) for _ in range(3)]
    side.synchronize()
    assert _same(_state(a), _state(b))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(c, xs, dys, w, HP)
    for t in range(3):
        graph.replay()
        torch.cuda.synchronize()
    assert _same(_state(a), _state(c))
    last = keep[-1]
    assert all(torch.equal(p, q) for p, q in zip(out[1], last[1]))


def test_driver_refusals():
    st = _driver([(64, 96)], 2, (20, 20))
    xs = [torch.zeros(20, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ys = [torch.empty_like(x) for x in xs]
    with pytest.raises(ValueError, match="other tokens"):
        st.contribute(0, xs, [None, None])
    with pytest.raises(ValueError, match="each of the 2 ranks"):
        st.forward_layer(0, xs[:1], ys[:1])
    with pytest.raises(ValueError, match="max_tokens"):
        st.forward_layer(0, [torch.zeros(21, 64, dtype=torch.bfloat16, device="cuda"), xs[1]], ys)
    st.forward_layer(0, xs, ys, keep=False)
    with pytest.raises(ValueError, match="other tokens"):
        st.contribute(0, xs, [None, None])
    st.forward_layer(0, xs, ys)
    st.contribute(0, xs, [None, None])
    with pytest.raises(ValueError, match="activation"):
        Zero3FeedForward([(64, 96)], 2, 20, activation="tanh")


def test_driver_needs_a_whole_forward_pass_for_each_backward_pass():
    st = _driver([(64, 96)], 2, (20, 20))
    xs = [torch.ones(20, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ys = [torch.empty_like(x) for x in xs]
    w = z.zero_rank_weights([20, 20], 2)
    st.forward_layer(0, xs, ys)
    st.backward_layer(0, xs, [None, None], w, HP)
    before = _state(st)
    with pytest.raises(ValueError, match="other tokens"):   # of the weights before the update
        st.backward_layer(0, xs, [None, None], w, HP)
    assert _same(before, _state(st))
    st.forward_layer(0, xs, ys)
    with pytest.raises(ValueError, match="x's shape"):
        st.forward_layer(0, xs, [ys[0], ys[1][:19]])
    with pytest.raises(ValueError, match="other tokens"):   # rank 0's is of another pass than rank 1's
        st.backward_layer(0, xs, [None, None], w, HP)
    st.forward_layer(0, xs, ys)
    st.backward_layer(0, xs, [None, None], w, HP)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("tokens,model", [(1, 1), (3, 70), (31, 1301), (40, 33), (300, 1301), (2100, 1000)])
def test_the_forward_passes_checkpoint_of_x_is_zero_act8_saves(tokens, model, fmt):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, model + 3, generator=gen, device="cuda").to(torch.bfloat16)[:, :model]
    for k, bad in enumerate((float("nan"), float("inf"), -float("inf"), 3e38, 1e-39, -0.0)):
        x[(k * 7) % tokens, (k * 37) % model] = bad
    w = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((40, model), (40, model), (model, 40))]
    ck = z.FfnCheckpoint.empty(tokens, model, 40, fmt)
    want = z.zero_act8_buffers(tokens, model)
    for t in (*ck.x, *want):
        t.fill_(77)
    z.zero_ffn_forward(x, *w, torch.empty(tokens, model, dtype=torch.bfloat16, device="cuda"),
                       z.zero_ffn_workspace(tokens, model, 40), checkpoint=ck)
    z.zero_act8_save(x, *want, format=fmt)
    assert torch.equal(ck.x[0], want[0]) and torch.equal(ck.x[1], want[1])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("tokens,model", [(3, 70), (40, 33), (300, 1301), (2100, 1000)])
def test_the_backward_pass_takes_x_as_zero_act8_load_gives_it(tokens, model, fmt):
    """dW_gate = dg^T x with dg = 1 in one token alone: x's values themselves."""
    gen = torch.Generator(device="cuda").manual_seed(model)
    x = torch.randn(tokens, model, generator=gen, device="cuda").mul_(1e3).to(torch.bfloat16)
    at, hidden = tokens - 1, 8
    x[at, model - 1] = float("inf")   # the last block
    ck = z.FfnCheckpoint.empty(tokens, model, hidden, fmt)
    z.zero_act8_save(x, *ck.x, format=fmt)
    ones = torch.ones(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    z.zero_act8_save(ones, *ck.gate, format=fmt)
    z.zero_act8_save(ones, *ck.up, format=fmt)
    dy = torch.zeros(tokens, model, dtype=torch.bfloat16, device="cuda")
    dy[at, 0] = 1.0
    w = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((hidden, model), (hidden, model), (model, hidden))]
    w[2][0] = 1.0
    d = [torch.full_like(v, 5.0) for v in w]
    z.zero_ffn_backward(dy, ck, *w, None, *d, z.zero_ffn_workspace(tokens, model, hidden, backward=True), activation="relu")
    want = torch.empty_like(x)
    z.zero_act8_load(*ck.x, want, format=fmt)
    last = (model - 1) // 32 * 32
    assert bool(want[at, last:].isnan().all()) and bool(want[at, :last].isfinite().all())
    for k in (0, 1):
        assert torch.equal(d[k][:, :last], want[at, :last].expand(hidden, last))
        assert bool(d[k][:, last:].isnan().all())
