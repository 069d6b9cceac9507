"""Which tiles the GPU tests of the experts' products run: the library's own choice
(csrc/experts_choice.hpp, built by the host compiler) for every shape that they use, and
the paths that must be among them, so that a change of the choice cannot leave a kernel
untested."""
import os
import shutil
import subprocess

import numpy as np
import pytest

import test_gpu_experts as base
import test_gpu_experts_tiles as tiles
from combine_ep_get_layout_amd import ep, inputs

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", "experts_choice.cpp")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

WIDE_FP8 = next(m.args[1] for m in base.test_wide_fp8.pytestmark if m.args[0] == "shape")


def counts_of(R, T, E, K, mode, masked, seed):
    """Rows of every expert, as test_gpu_experts.routed makes them."""
    w = inputs.small("experts", R=R, T=T, H=128, E=E, K=K, mode=mode, seed=seed)
    topk = inputs.gen_topk(w)
    if masked:
        topk = inputs.masked_topk(w, topk, masked, 0.0, seed=seed)
    return np.bincount(topk[topk >= 0].ravel(), minlength=E)


def calls():
    """(key, question to the choice, rows of each expert, contraction bytes, result channels)."""
    for shape in base.SHAPES + base.WIDE + tiles.BF16:
        R, T, E, K, mode, masked, C, I = shape
        rows = R * T * K
        for op, seed in ("gated", 3), ("linear", 4):
            wide = 2 * I if op == "gated" else I
            yield (op, "bf16", "bf16"), f"forward {E} {rows} {C} {wide} 0 0", \
                counts_of(R, T, E, K, mode, masked, seed), 2 * C, wide
    for shape in base.SHAPES + base.WIDE + tiles.GRADIENTS:
        R, T, E, K, mode, masked, C, I = shape
        counts = counts_of(R, T, E, K, mode, masked, 5)
        for O in 2 * I, I:
            yield ("dx",), f"dx {E} {R * T * K} {C} {O}", counts, 2 * O, C
            # an expert's rows are the contraction, one tile a workgroup
            yield ("dw",), f"dw {E} {C} {O}", counts, 2 * int(counts.max()), None
        yield ("dbias",), f"dbias {E} {R * T * K} {I}", counts, None, None
    for shape in base.FP8_SHAPES + WIDE_FP8 + tiles.FP8:
        R, T, E, K, mode, C, I = shape
        counts = counts_of(R, T, E, K, mode, 0.0, 8)
        for op, wide in ("gated", 2 * I), ("linear", I):
            for result in "bf16", "fp8":
                yield (op, "fp8", result), \
                    f"forward {E} {R * T * K} {C} {wide} 1 {int(result == 'fp8')}", counts, C, wide


@pytest.fixture(scope="module")
def seen(tmp_path_factory):
    """{path: the calls' questions}: a path is the key, the tile and one thing that a
    call does with it:
    once     at all
    again    some workgroup takes a second tile
    long     again, with eight or more whole stages (the weights' gradient: of its one tile)
    rest     long, and the last stage is a short one
    whole    long, and it is not
    chained  again, the second tile's loads running through the first one's epilogue"""
    exe = tmp_path_factory.mktemp("choice") / "choice"
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", SRC, "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    asked = list(calls())
    r = subprocess.run([str(exe)], input="\n".join(q for _, q, *_ in asked), capture_output=True,
                       text=True, timeout=60)
    assert r.returncode == 0
    answers = r.stdout.splitlines()
    assert len(answers) == len(asked)
    out = {}
    for (key, question, counts, nbytes, channels), answer in zip(asked, answers):
        tile, *v = answer.split()
        did = ["once"]
        if nbytes:
            bn, bm, kb, stages, slots, chains = map(int, v)
            total = int((-(-counts // bm)).sum()) * -(-channels // bn) if channels else 0
            if total > slots:
                did += ["again"]
                if chains and -(-nbytes // kb) >= stages:
                    did += ["chained"]
            if (total > slots or not channels) and nbytes // kb >= 8:
                did += ["long", "rest" if nbytes % kb else "whole"]
        for d in did:
            out.setdefault((*key, tile, d), []).append(question)
    return out


def test_every_forward_tile(seen):
    want = []
    for op in "gated", "linear":
        for kind in "bf16", "fp8":
            # narrow is chosen for tiles that all run at once
            want += [(op, kind, "bf16", tile, "once")
                     for tile in ("large", "medium", "narrow", "small", "tiny")]
            want += [(op, kind, "bf16", tile, "again")
                     for tile in ("large", "medium", "small", "tiny")]
        want += [(op, "fp8", "fp8", tile, d) for tile in ("large", "medium")
                 for d in ("once", "again", "long")]
    assert not [k for k in want if k not in seen]


def test_the_forward_loops(seen):
    """Steady state, short last stages and the chain of tiles in every kernel that has them."""
    want = []
    for op in "gated", "linear":
        for kind in "bf16", "fp8":
            want += [(op, kind, "bf16", "large", "long")]
            want += [(op, kind, "bf16", tile, d) for tile in ("medium", "small")
                     for d in ("long", "chained")]
            want += [(op, kind, "bf16", "tiny", "chained")]
        want += [(op, "bf16", "bf16", tile, "rest") for tile in ("large", "medium", "small")]
        want += [(op, "bf16", "bf16", "large", "whole")]
    assert not [k for k in want if k not in seen]


def test_the_gradients(seen):
    want = [("dx", tile, d) for tile in ("big", "medium", "small")
            for d in ("once", "again", "long", "rest")]
    want += [("dx", tile, "chained") for tile in ("medium", "small")]
    want += [("dx", "big", "whole")]
    want += [("dw", tile, d) for tile in ("big", "square", "pair") for d in ("once", "long")]
    want += [("dbias", tile, "once") for tile in ("32", "64", "256")]
    assert not [k for k in want if k not in seen]
