"""Which kernels the GPU tests of the layer for a few tokens run: the library's own choice
(csrc/layer_choice.hpp, built by the host compiler) for every shape that they use, against all
that any call can take, so that none is left untested."""
import os
import shutil
import subprocess

import pytest

import test_gpu_layer as layer

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", "layer_choice.cpp")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    exe = tmp_path_factory.mktemp("choice") / "choice"
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", SRC, "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(*args, text=""):
        r = subprocess.run([str(exe), *args], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0
        return r.stdout.splitlines()
    return ask


@pytest.fixture(scope="module")
def every(choice):
    """The kernels that calls of any size can take."""
    return set(choice("every"))


def kernels(choice, shapes, kind):
    """{kernel: shapes that run it}."""
    asked = []
    for s in shapes:
        R, T, E, K, H, I, _ = layer.sized(s, kind)
        asked.append(f"{int(kind != 'bf16')} {R * T * K} {E} {H} {I}")
    answers = choice(text="\n".join(asked))
    assert len(answers) == 2 * len(asked)
    seen = {}
    for i, name in enumerate(answers):
        seen.setdefault(name, []).append(shapes[i // 2])
    return seen


@pytest.mark.parametrize("kind", layer.KINDS)
def test_every_kernel(choice, every, kind):
    own = {name for name in every if name.startswith("0 " if kind == "bf16" else "1 ")}
    # gated: four with their own rows and five with rows in common; down: four (in 8 bits three)
    # and five
    assert len(own) == (18 if kind == "bf16" else 17)
    seen = kernels(choice, layer.SHAPES + layer.MANY + layer.FORMS, kind)
    assert set(seen) == own, own ^ set(seen)


@pytest.mark.parametrize("kind", layer.KINDS)
def test_the_skewed_shape_takes_strips_of_a_wave_alone(choice, kind):
    seen = kernels(choice, [(1, 24, 24, 1, 200, 1032, 0.0)], kind)
    assert any(name.endswith("gated few") for name in seen)
