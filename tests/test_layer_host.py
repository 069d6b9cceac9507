"""What the layer for a few tokens refuses on the host, before any launch."""
import pytest
import torch

from combine_ep_get_layout_amd import ep
from test_experts_host import A, ALIGN, MODE, NULL, SHAPE, no_gpu, problem, ref, weights

WS = -5
I = 64


def call(p=None, x=A, idx=A, wt=A, w13="w13", act=2, w2="w2", out=A, err=A, ws=A, ws_bytes=1 << 20,
         fp8=0):
    w13 = weights(128, 2 * I, fp8=fp8) if w13 == "w13" else w13
    w2 = weights(I, 128, fp8=fp8) if w2 == "w2" else w2
    return ep.lib().ep_expert_layer(ref((p or problem()).c()), x, idx, wt, ref(w13), act, ref(w2),
                                    out, err, ws, ws_bytes, None)


def test_workspace():
    def of(inner, **kw):
        return ep.lib().ep_expert_layer_workspace_bytes(ref(problem(**kw).c()), inner)
    assert of(64) == 2 * 8 * 2 * 64 * 4
    assert of(8, T=0) == 256
    assert of(72, R=1, T=1) == 768
    assert of(64, R=1, T=512) == 1024 * (64 * 4 + 128 * 4)  # and the entries' results in fp32
    assert of(64, R=1, T=513) == 0                       # more than 1,024 entries
    assert of(64, E=5) == 0
    for inner in (0, 4, 12, -8, 32776):
        assert of(inner) == 0
    assert ep.layer_workspace(problem(), 64, device="cpu").numel() == of(64)
    with pytest.raises(ep.EPError):
        ep.layer_workspace(problem(T=4096), 64, device="cpu")


@no_gpu
def test_operands():
    assert call(p=problem(E=5)) == SHAPE
    assert call(p=problem(T=257)) == SHAPE               # 1,028 entries
    assert call(act=4) == MODE
    for k in ("w13", "w2"):
        assert call(**{k: None}) == NULL
    for k in ("x", "idx", "wt", "out", "ws"):
        assert call(**{k: None}) == NULL, k
    assert call(w13=weights(128, 2 * I, w=None)) == NULL
    assert call(w2=weights(I, 128, w=None)) == NULL
    for k in ("x", "out", "ws"):
        assert call(**{k: A + 8}) == ALIGN, k
    for k in ("idx", "wt", "err"):
        assert call(**{k: A + 2}) == ALIGN, k
    assert call(w13=weights(128, 2 * I, w=A + 8)) == ALIGN
    assert call(w2=weights(I, 128, w=A + 8)) == ALIGN
    assert call(w13=weights(136, 2 * I)) == SHAPE
    assert call(w13=weights(128, 2 * I + 16)) == SHAPE
    assert call(w2=weights(I, 136)) == SHAPE
    assert call(w2=weights(12, 128), w13=weights(128, 24)) == SHAPE
    assert call(w13=weights(128, 2 * I, bias=A)) == MODE
    assert call(w2=weights(I, 128, bias=A)) == MODE
    assert call(w13=weights(128, 2 * I, reserved=1)) == SHAPE
    assert call(w2=weights(I, 128, fp8=3)) == MODE
    assert call(w2=weights(I, 128, fp8=1)) == MODE       # the two of different types
    assert call(ws_bytes=2 * 8 * 2 * I * 4 - 1) == WS


@no_gpu
def test_types():
    assert call(fp8=ep.WEIGHTS_FP8) == SHAPE             # 64 inner channels
    w13, w2 = dict(in_channels=0), None                  # noqa: F841
    mk = lambda kind, inner, h=128, **kw: dict(           # noqa: E731
        p=problem(H=h), w13=ep.CWeights(A, kw.get("s13", A), None, h, 2 * inner, kind, 0),
        w2=ep.CWeights(A, kw.get("s2", A), None, inner, h, kind, 0))
    assert call(**mk(ep.WEIGHTS_FP8, 128, h=136)) == SHAPE
    assert call(**mk(ep.WEIGHTS_FP8, 128, s13=None)) == NULL
    assert call(**mk(ep.WEIGHTS_FP8, 128, s2=None)) == NULL
    assert call(**mk(ep.WEIGHTS_FP8, 128, s2=A + 2)) == ALIGN
    assert call(**mk(ep.WEIGHTS_INT8, 24)) == SHAPE
    assert call(**mk(ep.WEIGHTS_INT8, 32, h=136)) == SHAPE
    assert call(**mk(ep.WEIGHTS_INT8, 32, s13=A + 4)) == ALIGN
    assert call(**mk(ep.WEIGHTS_INT8, 32, s2=None)) == NULL


def test_the_binding_checks_shapes_and_types():
    p = problem()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8)      # noqa: E731
    f = torch.zeros
    good = dict(x=bf(2, 8, 128), topk_idx=torch.zeros((2, 8, 2), dtype=torch.int32),
                topk_weights=f(2, 8, 2), w13=bf(4, 2 * I, 128), w2=bf(4, 128, I),
                out=bf(2, 8, 128), err=None, ws=torch.zeros(1 << 16, dtype=torch.uint8))
    bad = [
        dict(x=bf(2, 8, 64)), dict(x=f(2, 8, 128)), dict(out=bf(2, 7, 128)),
        dict(topk_idx=good["topk_idx"].long()), dict(topk_idx=good["topk_idx"][:1]),
        dict(topk_weights=f(2, 8, 1)), dict(topk_weights=f(2, 8, 2).double()),
        dict(w13=bf(3, 2 * I, 128)), dict(w13=bf(4, 2 * I, 64)), dict(w13=bf(4, I, 128)),
        dict(w2=bf(4, 64, I)), dict(w2=f(4, 128, I)),
        dict(w13=i8(4, 2 * I, 128), w2=i8(4, 128, I)),
        dict(w13=i8(4, 2 * I, 128), w2=i8(4, 128, I), w13_scales=f(4, 2 * I), w2_scales=f(4, I)),
        dict(w13=torch.zeros((4, 256, 128), dtype=torch.uint8), w2=bf(4, 128, 128)),
        dict(err=f(1)), dict(ws=f(1 << 16)),
        {},  # whole, but on the host
    ]
    for k, change in enumerate(bad):
        with pytest.raises(ValueError):
            ep.expert_layer(p, **{**good, **change})
            pytest.fail(str(k))
