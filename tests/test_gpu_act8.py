"""8-bit activations against a 64-bit definition, bit for bit: formats, types, odd
and long rows, strides, borders of the scale, NaN and infinities, untouched
surroundings, refusals."""
import math

import pytest
import torch

import ffn_plain as fp

pytestmark = pytest.mark.gpu

z = pytest.importorskip("zero_sharded_optimizer_reduce_amd")


def _wide(rows, cols, pad, off, dtype, fill):
    """A rows x cols view with row stride cols + pad, `off` elements into its buffer."""
    buf = torch.full((off + rows * (cols + pad) + 7,), fill, dtype=dtype, device="cuda")
    return buf, buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def _outside_untouched(buf, view, fill):
    mark = torch.ones_like(buf, dtype=torch.bool)
    mark.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert bool((buf[mark] == fill).all())


SHAPES = [(1, 1, 0, 0), (1, 31, 0, 1), (3, 32, 0, 0), (5, 33, 2, 1), (2, 40, 0, 0), (7, 64, 64, 0), (77, 1301, 0, 0),
          (19, 4101, 3, 3), (4, 8192, 0, 0), (3, 8225, 1, 0), (130, 96, 0, 0), (2, 40000, 0, 1), (513, 8, 0, 0)]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,off", SHAPES)
def test_round_trip(rows, cols, pad, off, dtype, fmt):
    gen = torch.Generator().manual_seed(rows * 1000 + cols)
    vals = torch.randn(rows, cols, generator=gen) * torch.exp2(torch.randint(-8, 9, (rows, cols), generator=gen).float())
    _, x = _wide(rows, cols, pad, off, dtype, 9.0)
    x.copy_(vals)
    codes_buf = torch.full((rows * cols + 24,), 77, dtype=torch.uint8, device="cuda")
    codes = codes_buf[off:off + rows * cols].view(rows, cols)
    nb = -(-cols // 32)
    scales_buf = torch.full((rows * nb + 24,), 77, dtype=torch.uint8, device="cuda")
    scales = scales_buf[1:1 + rows * nb].view(rows, nb)
    z.zero_act8_save(x, codes, scales, format=fmt)
    want, bytes_ = fp.quantised(x.double(), fmt)
    assert torch.equal(scales, bytes_)
    assert torch.equal(fp.held_values(codes, scales, fmt), want)
    for buf, view in ((codes_buf, codes), (scales_buf, scales)):
        _outside_untouched(buf, view, 77)
    for out_dtype in (torch.bfloat16, torch.float32):
        obuf, out = _wide(rows, cols, pad, off, out_dtype, 9.0)
        z.zero_act8_load(codes, scales, out, format=fmt)
        assert torch.equal(out.double(), want)   # exact in either type
        _outside_untouched(obuf, out, 9.0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_borders_of_the_scale(fmt):
    """The largest magnitude at, next above and next below M * 2^e, subnormal and
    largest blocks, zeros."""
    limit = fp.LIMIT[fmt]
    tops = []
    for e in (-126, -125, -60, 0, 60, 118):
        m = limit * math.ldexp(1.0, e) if e + 9 < 128 else None
        if m is not None and m < 3.3e38:
            t = torch.tensor(m, dtype=torch.float32)
            tops += [float(t), float(torch.nextafter(t, torch.tensor(math.inf))), float(torch.nextafter(t, torch.tensor(0.0)))]
    tops += [0.0, 1e-45, 1.1754944e-38, 2.0 ** -127, math.ldexp(limit, 121 if fmt == "int8" else 119), 1.0, 255.0, 256.0]
    gen = torch.Generator().manual_seed(5)
    x = torch.rand(len(tops), 32, generator=gen, dtype=torch.float64) * 2 - 1
    top = torch.tensor(tops, dtype=torch.float64)
    x = (x * top[:, None]).to(torch.float32)
    x[:, 11] = -top.to(torch.float32)
    x = x.cuda()
    codes, scales = z.zero_act8_buffers(len(tops), 32)
    z.zero_act8_save(x, codes, scales, format=fmt)
    want, bytes_ = fp.quantised(x.double(), fmt)
    assert torch.equal(scales, bytes_)
    assert torch.equal(fp.held_values(codes, scales, fmt), want)
    out = torch.empty_like(x)
    z.zero_act8_load(codes, scales, out, format=fmt)
    assert torch.equal(out.double(), want)


def test_every_code_reads_back():
    """All 256 codes under the smallest, ordinary and largest scales, and scale 0."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(8, 32).repeat(5, 1).contiguous()
    scales = torch.tensor([[b] for b in (0, 1, 100, 127, 240) for _ in range(8)], dtype=torch.uint8, device="cuda")
    for fmt in ("int8", "e4m3"):
        want = fp.held_values(codes, scales, fmt)
        out = torch.empty(40, 32, device="cuda")
        z.zero_act8_load(codes, scales, out, format=fmt)
        assert torch.equal(torch.nan_to_num(out.double(), nan=7.25), torch.nan_to_num(want.to(torch.float32).double(), nan=7.25))
        low = torch.empty(40, 32, dtype=torch.bfloat16, device="cuda")
        z.zero_act8_load(codes, scales, low, format=fmt)
        ref = want.to(torch.float32).to(torch.bfloat16)
        assert torch.equal(torch.nan_to_num(low, nan=7.25), torch.nan_to_num(ref, nan=7.25))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 3.4e38])   # 3.4e38: its nearest codes stand for 2^128
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_block_without_a_finite_scale_reads_as_nan(fmt, bad):
    x = torch.ones(3, 70, device="cuda")
    x[1, 40] = bad
    x[2, 69] = bad
    codes, scales = z.zero_act8_buffers(3, 70)
    out = torch.empty(3, 70, dtype=torch.bfloat16, device="cuda")
    z.zero_act8_save(x, codes, scales, format=fmt)
    z.zero_act8_load(codes, scales, out, format=fmt)
    nan = torch.zeros(3, 70, dtype=torch.bool, device="cuda")
    nan[1, 32:64] = True
    nan[2, 64:] = True
    assert torch.equal(torch.isnan(out), nan) and bool((out[~nan] == 1).all())
    assert bool((scales == 255).sum() == 2) and bool((codes[nan] == 0).all())


def test_offsets_past_32_bits():
    """A row stride with which the last row lies over 2^32 bytes behind the first."""
    rows, cols, stride = 3, 64, 1 << 30
    buf = torch.zeros((rows - 1) * stride + cols, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((rows, cols), (stride, 1))
    x.copy_(torch.randn(rows, cols, generator=torch.Generator().manual_seed(1)))
    codes, scales = z.zero_act8_buffers(rows, cols)
    z.zero_act8_save(x, codes, scales)
    want, _ = fp.quantised(x.double(), "int8")
    assert torch.equal(fp.held_values(codes, scales, "int8"), want)
    x.zero_()
    z.zero_act8_load(codes, scales, x)
    assert torch.equal(x.double(), want)
    assert int(buf.count_nonzero()) == int(want.count_nonzero())


def test_empty_and_refused():
    for shape in ((0, 5), (5, 0)):
        codes, scales = z.zero_act8_buffers(*shape)
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        z.zero_act8_save(x, codes, scales)
        z.zero_act8_load(codes, scales, x)
    x = torch.zeros(4, 40, dtype=torch.bfloat16, device="cuda")
    codes, scales = z.zero_act8_buffers(4, 40)
    with pytest.raises(ValueError):
        z.zero_act8_save(x, codes, scales, format="int4")
    with pytest.raises(ValueError):
        z.zero_act8_save(x, codes, scales[:, :1].contiguous())
    with pytest.raises(ValueError):
        z.zero_act8_save(x.t(), *z.zero_act8_buffers(40, 4))
    with pytest.raises(TypeError):
        z.zero_act8_save(x.half(), codes, scales)
    with pytest.raises(TypeError):
        z.zero_act8_load(codes.view(torch.int8), scales, x)
    with pytest.raises(ValueError):
        z.zero_act8_load(codes.cpu(), scales, x)
    with pytest.raises(z.ZeroError):   # the codes lie on the values
        z.zero_act8_load(x.view(torch.uint8).view(-1)[:160].view(4, 40), scales, x)
