"""The feed-forward calls' launches at many sizes, without a GPU: every launch stays inside
the workspace that the call asks for and covers its results, and the GPU tests' sizes take
every kernel that any size takes."""
import math
import os
import random
import shutil

import pytest

import ffn_routes as routes
import test_gpu_ffn as whole

pytestmark = pytest.mark.skipif(not (shutil.which("hipcc") or os.path.exists(routes.HIPCC)), reason="no hipcc")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    return routes.build(str(tmp_path_factory.mktemp("routes")))


def _calls(shapes):
    return [(p, t, m, h, int(off % 8 != 0), extra) for t, m, h, _, off in shapes for p, extra in (("f", 0), ("f", 1), ("b", 0), ("b", 1))]


def _random_calls(n):
    rng = random.Random(1)
    spread = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    calls = []
    for _ in range(n):
        t, m, h = spread(1, 30000), spread(1, 16384), spread(1, 32768)
        if rng.random() < 0.4:
            m, h = -(-m // 64) * 64, -(-h // 64) * 64
        calls.append((rng.choice("fb"), t, m, h, rng.randint(0, 1), rng.randint(0, 1)))
    return calls


def _kinds(launches):
    return {kernel for call in launches for kernel, _ in call}


def test_every_launch_stays_inside_its_workspace_and_covers_its_results(exe):
    calls = _random_calls(40000) + _calls(whole.SHAPES + routes.SHAPES)
    calls += [("b", 0, 64, 96, 0, 1), ("f", 1, 262144, 262144, 0, 1), ("b", 1, 262144, 262144, 0, 1), ("f", 131072, 262144, 64, 1, 1),
              ("b", 131072, 64, 262144, 0, 1), ("f", 16777216, 64, 64, 0, 1), ("b", 16777216, 2048, 1, 1, 1)]
    routes.launches(exe, calls)   # which checks them


def test_the_gpu_tests_take_every_kernel(exe):
    taken = _kinds(routes.launches(exe, _calls(whole.SHAPES + routes.SHAPES)))
    missed = {}
    calls = _random_calls(40000)
    for call, launches in zip(calls, routes.launches(exe, calls)):
        for kernel, _ in launches:
            if kernel not in taken:
                missed.setdefault(kernel, call)
    assert not missed, missed


def test_the_gpu_tests_take_every_gated_kernel_with_every_activation(exe):
    shapes = next(m.args[1] for m in whole.test_forward_and_checkpoint.pytestmark if m.args[0] == "tokens,model,hidden")
    assert shapes == next(m.args[1] for m in whole.test_backward.pytestmark if m.args[0] == "tokens,model,hidden")
    taken = _kinds(routes.launches(exe, _calls([(*s, 0, 0) for s in (*shapes, *routes.ACTIVATED)])))
    # whether its tiles begin at different columns says nothing about a kernel's activations
    gated = lambda kinds: {k.replace(",spread", "") for k in kinds if k.startswith(("kGated", "kSlopes", "few"))}
    assert gated(_kinds(routes.launches(exe, _random_calls(40000)))) <= gated(taken)
