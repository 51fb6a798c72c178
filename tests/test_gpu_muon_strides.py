"""Newton-Schulz on matrices that lie side by side in wider buffers."""
import pytest
import torch

import zero_sharded_optimizer_reduce_amd as z

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mats,rows,cols", [(2, 64, 96), (3, 130, 200), (4, 200, 130), (2, 33, 17), (5, 300, 310)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gap", [0, 3])
def test_side_by_side(mats, rows, cols, dtype, gap):
    print(f"newton_schulz {mats} x {rows}x{cols} side by side, gap {gap} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(mats)
    wide = cols + gap
    src = torch.full((rows, mats * wide), 100.0, dtype=dtype, device="cuda")
    g = src.view(rows, mats, wide)[:, :, :cols].permute(1, 0, 2)
    g.copy_(torch.randn(mats, rows, cols, device="cuda", generator=gen))
    dst = torch.full((rows, mats * wide), 7.0, dtype=torch.bfloat16, device="cuda")
    out = dst.view(rows, mats, wide)[:, :, :cols].permute(1, 0, 2)
    z.zero_newton_schulz(g, out, z.zero_newton_schulz_workspace(g))
    want = torch.empty(mats, rows, cols, dtype=torch.bfloat16, device="cuda")
    z.zero_newton_schulz(g.contiguous(), want, z.zero_newton_schulz_workspace(g))
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert bool((dst == 7.0).all()), "written between the matrices"
