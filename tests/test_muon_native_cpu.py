"""The Muon step's native parts on the CPU: the argument checks under the host
sanitizers, and the machine code of its kernels (this repository's own build)."""
import os
import re
import shutil
import subprocess

import pytest

from test_device_code_cpu import OBJDUMP, _code_objects

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_muon_validation_under_sanitizers(tmp_path):
    exe = tmp_path / "validate_muon_driver"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"),
           os.path.join(ROOT, "tests", "native", "validate_muon_driver.cpp"),
           os.path.join(ROOT, "zero_sharded_optimizer_reduce_amd", "csrc", "validate.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@pytest.fixture(scope="module")
def kernels(libzero, tmp_path_factory):
    """name -> instructions of every kernel in the code objects that hold the Muon step's."""
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
        if "ns_product_kernel" in r.stdout or "momentum_vec" in r.stdout:
            assert "gfx950" in triple
            for m in re.finditer(r"^[0-9a-f]+ <(.*)>:\n((?:.+\n?)*)", r.stdout, re.M):
                out[m.group(1)] = m.group(2)
    assert any("ns_product" in n for n in out) and any("momentum" in n for n in out)
    return out


def test_no_packed_fp32_arithmetic_and_no_spills(kernels):
    for name, text in kernels.items():
        assert not re.search(r"\bv_pk_(?:add|mul|fma)_f32\b", text), name
        assert not re.search(r"\bscratch_(?:load|store)", text), name


def test_the_products_use_the_matrix_cores_and_loads_straight_to_lds(kernels):
    products = {n: t for n, t in kernels.items() if "ns_product_kernel" in n}
    assert len(products) >= 12
    for name, text in products.items():
        assert "v_mfma_f32_32x32x16_f16" in text, name
        assert re.search(r"buffer_load_dwordx4 .* lds", text), name
    small = [t for n, t in kernels.items() if "ns_small_kernel" in n]
    assert small and all("v_mfma_f32_16x16x32_f16" in t and "ds_read_b64_tr_b16" in t for t in small)
