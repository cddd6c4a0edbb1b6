"""The schedule arithmetic of the scaled and gated products and the gradients (csrc/ffn_plan.cuh),
compiled for the CPU with checks for undefined arithmetic: every unit of work exactly once, inside
the operands, and the GPU tests' sizes on the plans that they stand for."""
import os
import shutil
import subprocess
from collections import namedtuple

import pytest

import test_gpu_ffn_plans as plans

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gemv_w4a16_w8a8_b200", "csrc")
# widths, parts, rounds of the weights' tiles in place of a missing tile of dX (-1: two launches), and
# the most units of a pair: of the joined launch, of dX, of the weights' gradients
Grad = namedtuple("Grad", "few together bn_x parts_x bn_w parts_w extra most most_x most_w")
Prod = namedtuple("Prod", "few bn units most")
MOST = 2 ** 31 - 4096


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    exe = str(tmp_path_factory.mktemp("plan") / "check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC,
                    os.path.join(HERE, "ffn_plan_check.cpp"), "-o", exe], check=True)

    def run(*lines):
        r = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-2000:])
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


def test_random_sizes(check):
    check("sweep 5000 1")


def test_the_largest_sizes(check):
    check(f"grad {MOST} 1 8", f"grad 8 {MOST} 8", f"grad 8 8 {MOST}", f"grad {MOST} {MOST} 8",
          f"prod {MOST} 1 1 0 1", f"prod 1 {MOST} 1 1 1", f"prod {MOST} 64 1 1 0", "prod 1 8 33554368 1 0")


def test_gradient_sizes_stand_for_their_plans(check):
    got = check(*("grad %d %d %d" % s for s in plans.GRADIENTS.values()))
    by = {name: Grad(*g) for name, g in zip(plans.GRADIENTS, got)}
    for name, g in by.items():
        assert g.few == name.startswith("few"), name
        assert g.together == name.startswith("one launch"), name

    def some(f):
        return any(f(g) for g in by.values())

    few, two, one = ([g for g in by.values() if f(g)] for f in (
        lambda g: g.few, lambda g: not g.few and not g.together, lambda g: g.together))
    assert any(g.most_w >= 3 for g in few) and any(g.parts_w > 1 for g in few)
    assert any(g.parts_x > 1 and g.parts_w == 1 for g in two) and any(g.parts_w > 1 and g.parts_x == 1 for g in two)
    assert any(g.parts_x > 1 and g.parts_w > 1 for g in two) and any(g.most_x >= 3 and g.most_w >= 3 for g in two)
    assert any(g.bn_x == 128 and g.most_x >= 2 for g in two) and any(g.most_x >= 3 and g.most_w == 1 for g in two)
    assert any(g.extra == 0 and g.most >= 3 for g in one) and {0, 1, 2, 3, 6} <= {g.extra for g in one}
    assert any(g.parts_x > 1 and g.extra >= 2 for g in one) and any(g.most_x >= 3 for g in one)
    assert any(g.parts_x > 1 and g.parts_w > 1 and g.most_x >= 2 for g in one)
    assert some(lambda g: g.together and g.most >= 4)


def test_forward_sizes_take_three_waves_of_tiles(check):
    lines = [f"prod {M} {N} {(K + 127) // 128} 0 1" for M, N, K in plans.SCALED]
    lines += [f"prod {M} {F} {(K + 63) // 64} 1 0" for M, F, K in plans.GATED]
    lines += [f"prod {M} {F} {(K + 127) // 128} 1 1" for M, F, K in [(2600, 2999, 272), (1700, 4098, 144), (2304, 4096, 208)]]
    for line, p in zip(lines, check(*lines)):
        assert not Prod(*p).few and Prod(*p).most >= 3, (line, p)


def test_the_largest_training_step_is_two_launches(check):
    """8192 tokens at 11008 x 4096: the plan that several waves of each product stand for above."""
    g = Grad(*check("grad 8192 11008 4096")[0])
    assert not g.few and not g.together and g.parts_x == g.parts_w == 1 and g.most_x >= 3 and g.most_w >= 3
