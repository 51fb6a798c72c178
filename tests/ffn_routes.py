"""Which kernels the feed-forward calls launch at which sizes, found without a GPU
(tests/native/ffn_routes.cpp), and the sizes with which the GPU tests take the launches that
test_gpu_ffn.SHAPES leaves out."""
import os
import re
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC") or shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

# tokens, model, hidden, pad of x and y, offset of the weights
SHAPES = [(1000, 2050, 8200, 0, 0),   # y in parts of 256 x 256
          (1000, 2050, 4160, 3, 1),   # dx in parts of 256 x 256, y in parts of 128 x 128 with two slots
          (2048, 2050, 200, 0, 0),    # y in 128 x 128 with two slots
          (9000, 264, 130, 5, 0),     # gate and up, x larger than an L2: 128 x 128 with four slots
          (2304, 2176, 1024, 0, 0),   # ... 128 x 256
          (1024, 2048, 8192, 0, 0),   # nothing packed: dx in parts of 256 x 256, added up beside the gradients
          (4160, 512, 4224, 0, 0)]    # ... and by a launch of their own
# for every activation: gate and up in 256 x 256 with quarters, dh in 256 x 256 with quarters; 128 x 128 with two slots;
# 17 to 32 tokens
ACTIVATED = [(2048, 512, 8448), (2304, 1024, 2176), (24, 512, 1408)]


def build(folder):
    exe = os.path.join(folder, "ffn_routes")
    cmd = [HIPCC, "-x", "hip", "--offload-host-only", "--offload-arch=gfx950", "-std=c++17", "-O1", "-I",
           os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "native", "ffn_routes.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return exe


def launches(exe, calls):
    """For each call ("f" or "b", tokens, model, hidden, unaligned weights, saved or with dx) its launches
    as (kernel, workgroups of tiles or parts)."""
    r = subprocess.run([exe], input="".join(" ".join(map(str, c)) + "\n" for c in calls), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-500:]
    lines = r.stdout.splitlines()
    assert len(lines) == len(calls)
    return [[tuple(re.fullmatch(r"(.*) (\S+)", k.strip()).groups()) for k in line.split(":", 1)[1].split(";") if k.strip()] for line in lines]
