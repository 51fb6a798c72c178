"""The feed-forward block and the 8-bit activations without a GPU: the argument checks
under the host sanitizers, workspace sizes, what the binding and the C ABI refuse, the
machine code of their kernels, and the plain implementations against printed values."""
import ctypes as C
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

import ffn_plain as fp
from test_device_code_cpu import OBJDUMP, _code_objects

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_validation_under_sanitizers(tmp_path):
    exe = tmp_path / "validate_ffn_driver"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "native", "validate_ffn_driver.cpp"),
           os.path.join(ROOT, "zero_sharded_optimizer_reduce_amd", "csrc", "validate.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def _workspace(L, *args):
    n = C.c_int64(-1)
    st = L.zero_ffn_workspace(*args, C.byref(n))
    return st, n.value


def test_workspace_sizes(libzero):
    L = libzero
    assert L.zero_ffn_workspace(1, 64, 64, 0, None) == -1
    assert _workspace(L, -1, 64, 64, 0)[0] == -1
    assert _workspace(L, 1, 0, 64, 0)[0] == -1
    assert _workspace(L, 1, 64, 64, 4)[0] == -1
    assert _workspace(L, 1, 262145, 64, 0)[0] == -3
    assert _workspace(L, (1 << 24) + 1, 64, 64, 0)[0] == -3
    assert _workspace(L, 1 << 24, 4096, 64, 0)[0] == -3       # activations that a checkpoint could not hold
    # h alone for a few tokens; h and x's room for many; the packed weights where sizes or addresses are odd
    assert _workspace(L, 1, 4096, 14336, 0) == (0, 14336 * 2)
    plain = _workspace(L, 8192, 4096, 14336, 0)[1]
    assert plain == 8192 * (14336 + 4096) * 2
    assert _workspace(L, 8192, 4096, 14336, 2)[1] == plain + 3 * 4096 * 14336 * 2
    assert _workspace(L, 8192, 4096, 14336, 1)[1] == 8192 * (3 * 14336 + 2 * 4096) * 2
    assert _workspace(L, 0, 64, 64, 0) == (0, 0)
    # never less for more tokens' activations, whatever the sums in parts take
    for t in range(33, 2000, 61):
        st, n = _workspace(L, t, 1301, 777, 1)
        assert st == 0 and n >= t * (3 * 832 + 2 * 1344) * 2 and n % 256 == 0


@pytest.mark.parametrize("m,h", [(64, 96), (777, 1301), (1024, 8192), (4096, 14336), (8, 28672)])
@pytest.mark.parametrize("most", [1, 33, 130, 1021])
def test_the_drivers_workspace_serves_every_count_of_tokens(libzero, m, h, most):
    from types import SimpleNamespace

    from zero_sharded_optimizer_reduce_amd.drivers import Zero3FeedForward

    room = Zero3FeedForward._workspace_bytes(SimpleNamespace(max_tokens=most), m, h)
    flags = 2 if m * h % 8 else 0
    needs = [_workspace(libzero, t, m, h, flags | back) for t in range(most + 1) for back in (0, 1)]
    assert all(st == 0 for st, _ in needs) and max(n for _, n in needs) == room


def test_the_c_abi_refuses(libzero):
    L = libzero
    act = lambda **k: L.zero_act8_save(*[{**dict(x=1 << 40, dtype=0, row=64, rows=4, cols=64, fmt=0, codes=1 << 41, scales=1 << 42,
                                                 stream=None), **k}[n] for n in ("x", "dtype", "row", "rows", "cols", "fmt", "codes",
                                                                                 "scales", "stream")])
    assert act(rows=0) == 0 and act(cols=0, x=None, codes=None, scales=None) == 0
    assert act(dtype=7) == -1 and act(fmt=9) == -1 and act(rows=-1) == -1 and act(x=None) == -1
    assert act(x=(1 << 40) + 1) == -2 and act(row=63) == -3 and act(scales=(1 << 41) + 255) == -1
    assert b"overlap" in L.zero_last_error()
    # a workspace that is too small is named before anything is launched
    fwd = lambda bytes_, ws=1 << 45: L.zero_ffn_forward(1 << 40, 64, 100, 64, 96, 1 << 41, 1 << 42, 1 << 43, 0, 1 << 44, 64, None, ws,
                                                        bytes_, None)
    need = _workspace(L, 100, 64, 96, 0)[1]
    assert fwd(need - 1) == -3 and b"needed" in L.zero_last_error()
    assert fwd(need, ws=None) == -1 and fwd(need, ws=(1 << 45) + 64) == -2
    assert L.zero_ffn_forward(None, 0, 0, 64, 96, None, None, None, 0, None, 0, None, None, 0, None) == 0   # no tokens
    # weights at odd addresses need the room for aligned copies
    odd = lambda bytes_: L.zero_ffn_forward(1 << 40, 64, 100, 64, 128, (1 << 41) + 2, 1 << 42, 1 << 43, 0, 1 << 44, 64, None, 1 << 45,
                                            bytes_, None)
    assert odd(_workspace(L, 100, 64, 128, 0)[1]) == -3 and b"ZERO_FFN_UNALIGNED" in L.zero_last_error()
    assert L.zero_ffn_backward(1 << 40, 64, 4, 64, 96, None, 1 << 41, 1 << 42, 1 << 43, 0, None, 0, 1 << 46, 1 << 47, 1 << 48, 1 << 45,
                               1 << 40, None) == -1
    assert b"checkpoint" in L.zero_last_error()


def test_the_binding_refuses_host_tensors(libzero):
    import zero_sharded_optimizer_reduce_amd as z
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    codes, scales = z.zero_act8_buffers(4, 64, device="cpu")
    assert codes.shape == (4, 64) and scales.shape == (4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_act8_save(x, codes, scales)
    with pytest.raises(TypeError, match="2-D"):
        z.zero_act8_save(x[0], codes, scales)
    with pytest.raises(ValueError, match="int4"):
        z.FfnCheckpoint((codes, scales), (codes, scales), (codes, scales), format="int4")
    ck = z.FfnCheckpoint.empty(6, 33, 64, "e4m3", device="cpu").first(2)
    assert ck.x[1].shape == (2, 2) and ck.up[0].shape == (2, 64) and ck.format == "e4m3"


# ------------------------------------------------------------ machine code
@pytest.fixture(scope="module")
def kernels(libzero, tmp_path_factory):
    from zero_sharded_optimizer_reduce_amd import _lib
    tool = OBJDUMP if os.path.exists(OBJDUMP) else shutil.which("llvm-objdump")
    if not tool:
        pytest.skip("no llvm-objdump")
    d, out = tmp_path_factory.mktemp("co"), {}
    for i, (triple, blob) in enumerate(_code_objects(_lib.LIB_PATH)):
        path = d / f"co{i}.o"
        path.write_bytes(blob)
        r = subprocess.run([tool, "-d", "--demangle", str(path)], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr[-500:]
        for m in re.finditer(r"^[0-9a-f]+ <(.*)>:\n((?:.+\n?)*)", r.stdout, re.M):
            if "ffn_" in m.group(1) or "act8_" in m.group(1):
                out[m.group(1)] = m.group(2)
    return out


def test_no_packed_fp32_arithmetic_and_no_spills(kernels):
    assert len([n for n in kernels if "ffn_product_kernel" in n]) >= 15
    for name, text in kernels.items():
        assert not re.search(r"\bv_pk_(?:add|mul|fma)_f32\b", text), name
        assert not re.search(r"\bscratch_(?:load|store)", text), name


def test_the_products_use_the_matrix_cores_and_loads_straight_to_lds(kernels):
    for name, text in kernels.items():
        if "ffn_product_kernel" in name:
            assert "v_mfma_f32_16x16x32_bf16" in text and re.search(r"buffer_load_dwordx4 .* lds", text), name
        if "ffn_few_kernel" in name:
            assert "v_mfma_f32_16x16x32_bf16" in text and "global_load_dwordx4" in text, name


# ------------------------------------------------------------ plain implementations
def test_codes_of_printed_values():
    x = torch.zeros(2, 32, dtype=torch.float64)
    x[0, :4] = torch.tensor([127.0, -0.5, 1.5, 2.5])        # scale 1: ties to even
    x[1, :4] = torch.tensor([127.5, 1.0, -3.0, 127.0])      # over 127: scale 2
    v, s = fp.quantised(x, "int8")
    assert v[0, :4].tolist() == [127, 0, 2, 2] and v[1, :4].tolist() == [128, 0, -4, 128] and s[:, 0].tolist() == [127, 128]
    x[0, :5] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])
    v, s = fp.quantised(x, "e4m3")
    assert v[0, :5].tolist() == [448, 16, 20, 0, 2.0 ** -8] and s[0, 0] == 127
    t = fp.e4m3_values()
    assert t[0x7E] == 448 and math.isnan(t[0x7F]) and t[0x38] == 1 and t[0x01] == 2.0 ** -9 and t[0x88] == -2.0 ** -6


def test_gradients_are_the_differences():
    """The formula's gradients against central differences of the 64-bit forward pass."""
    gen = torch.Generator().manual_seed(3)
    tokens, model, hidden = 3, 5, 7
    x, wg, wu, wd, dy = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in
                         ((tokens, model), (hidden, model), (hidden, model), (model, hidden), (tokens, model)))
    for act in ("silu", "gelu", "relu"):
        g, u, _, _ = fp.forward64(x, wg, wu, wd, act)
        grads = fp.backward64(dy, x, g, u, wg, wu, wd, act)
        for k, (t, grad) in enumerate(zip((x, wg, wu, wd), grads)):
            for at in range(0, t.numel(), 4):
                ends = []
                for sign in (1, -1):
                    moved = [v.clone() for v in (x, wg, wu, wd)]
                    moved[k].view(-1)[at] += sign * 1e-6
                    ends.append(float((fp.forward64(*moved, act)[3] * dy).sum()))
                assert abs((ends[0] - ends[1]) / 2e-6 - float(grad.reshape(-1)[at])) < 1e-7
