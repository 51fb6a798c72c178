"""Newton-Schulz at shapes of the general path: unaligned views, matrices far apart,
and a workspace full of NaNs in front of every tile width."""
import pytest
import torch

import zero_sharded_optimizer_reduce_amd as z

pytestmark = pytest.mark.gpu


def _gauss(seed, *shape, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=gen) * 1e-3).to(dtype)


def _ns(g, fill=0, **kw):
    out = torch.full(g.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = z.zero_newton_schulz_workspace(g)
    ws.fill_(fill)
    z.zero_newton_schulz(g, out, ws, **kw)
    return out


@pytest.mark.parametrize("off", [1, 2, 4, 8])
@pytest.mark.parametrize("rows,cols", [(200, 260), (120, 500), (260, 200)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_views(off, rows, cols, dtype):
    print(f"newton_schulz {rows}x{cols} {dtype} {off} elements in", flush=True)
    n = rows * cols
    g = _gauss(off, rows, cols, dtype=dtype)
    src = torch.full((n + 64,), 100.0, dtype=dtype, device="cuda")
    src[off:off + n] = g.flatten()
    dst = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    gd, od = src[off:off + n].view(rows, cols), dst[off:off + n].view(rows, cols)
    z.zero_newton_schulz(gd, od, z.zero_newton_schulz_workspace(gd))
    assert torch.equal(od, _ns(g))
    assert bool((dst[:off] == 7.0).all()) and bool((dst[off + n:] == 7.0).all())


@pytest.mark.parametrize("rows,cols", [(200, 260), (260, 200)])
def test_far_apart_matrices(rows, cols):
    # matrix strides whose offsets pass 32 bits, in elements and in bytes
    far = (1 << 31) + 24
    g = _gauss(22, 2, rows, cols)
    src = torch.zeros(far + rows * cols, dtype=torch.bfloat16, device="cuda")
    dst = torch.zeros(far + rows * cols, dtype=torch.bfloat16, device="cuda")
    gd, od = (t.as_strided((2, rows, cols), (far, cols, 1)) for t in (src, dst))
    gd.copy_(g)
    z.zero_newton_schulz(gd, od, z.zero_newton_schulz_workspace(gd))
    assert torch.equal(od.contiguous(), _ns(g))


def test_far_apart_rows():
    # row strides whose offsets pass 32 bits
    rows, cols = 130, 200
    step = (1 << 31) // 128 + 8
    g = _gauss(23, rows, cols)
    src = torch.zeros(step * (rows - 1) + cols, dtype=torch.bfloat16, device="cuda")
    dst = torch.zeros(step * (rows - 1) + cols, dtype=torch.bfloat16, device="cuda")
    gd, od = (t.as_strided((rows, cols), (step, 1)) for t in (src, dst))
    gd.copy_(g)
    z.zero_newton_schulz(gd, od, z.zero_newton_schulz_workspace(gd))
    assert torch.equal(od.contiguous(), _ns(g))


# 64-wide tiles, riding and not, with short and long sums; 128; 192 and 256
@pytest.mark.parametrize("mats,rows,cols", [(1, 97, 1000), (2, 515, 530), (7, 517, 650), (7, 513, 1110), (3, 777, 1301),
                                            (1, 1290, 4099), (1, 2900, 2910), (1, 4090, 4097), (1, 4300, 3990),
                                            (12, 1025, 3001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nothing_of_the_workspace_is_read_before_it_is_written(mats, rows, cols, dtype):
    print(f"newton_schulz {mats}x{rows}x{cols} {dtype}", flush=True)
    g = _gauss(mats + rows, mats, rows, cols, dtype=dtype)
    want = _ns(g)
    assert bool(torch.isfinite(want).all())
    assert torch.equal(_ns(g, fill=0xFF), want)
