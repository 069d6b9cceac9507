"""Which tiles the GPU tests of the 8-bit products run: the library's own choice
(csrc/experts_choice.hpp, built by the host compiler) for every shape that they use, and the
paths that must be among them."""
import os
import shutil
import subprocess

import pytest

import test_gpu_experts as base
import test_gpu_experts_tiles as tiles
import test_gpu_int8 as int8
from test_experts_choice import counts_of

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", "int8_choice.cpp")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def seen(tmp_path_factory):
    """{(op, tile, once, what): shapes}, `what` as in test_experts_choice.seen."""
    exe = tmp_path_factory.mktemp("choice") / "choice"
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", SRC, "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    asked = []
    for shape in int8.doubled(base.SHAPES + base.WIDE + tiles.BF16) + int8.LONG:
        R, T, E, K, mode, masked, C, I = shape
        for op, seed in ("gated", 3), ("linear", 4):
            asked.append((op, shape, f"{E} {R * T * K} {C} {I} {int(op == 'gated')}",
                          counts_of(R, T, E, K, mode, masked, seed)))
    r = subprocess.run([str(exe)], input="\n".join(q for _, _, q, _ in asked),
                       capture_output=True, text=True, timeout=60)
    assert r.returncode == 0
    answers = r.stdout.splitlines()
    assert len(answers) == len(asked)
    out = {}
    for (op, shape, _, counts), answer in zip(asked, answers):
        tile, *v = answer.split()
        bn, bm, kb, stages, slots, chains, once = map(int, v)
        C, wide = shape[6], shape[7] * (2 if op == "gated" else 1)
        total = int((-(-counts // bm)).sum()) * -(-wide // bn)
        did = ["once"]
        if total > slots:
            did += ["again"]
            if chains and -(-C // kb) >= stages:
                did += ["chained"]
            if C // kb >= 8:
                did += ["long", "rest" if C % kb else "whole"]
        for d in did:
            out.setdefault((op, tile, bool(once), d), []).append(shape)
    return out


def test_every_tile_and_loop(seen):
    want = []
    for op in "gated", "linear":
        want += [(op, "large", False, d) for d in ("once", "again", "long", "rest", "whole")]
        want += [(op, "wide", False, d) for d in ("again", "long", "rest", "whole")]
        want += [(op, "medium", False, d) for d in ("again", "chained", "long", "rest")]
        want += [(op, "medium", True, d) for d in ("again", "chained", "long", "rest")]
        want += [(op, "small", once, "again") for once in (True, False)]
        want += [(op, "small", True, d) for d in ("chained", "long", "rest")]
        want += [(op, "tiny", True, d) for d in ("again", "chained")]
        want += [(op, "narrow", False, "once"), (op, "narrow", True, "once")]
    missing = [k for k in want if k not in seen]
    assert not missing, "\n".join(map(str, missing))
