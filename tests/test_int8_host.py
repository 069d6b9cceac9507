"""What the 8-bit integer forms of dispatch and of the experts' products refuse on the host,
before any launch, and the binding's own checks."""
import ctypes

import pytest
import torch

from combine_ep_get_layout_amd import ep
from test_experts_host import (A, ALIGN, CAP, MODE, NULL, SHAPE, gated, gated_bwd, layout, linear,
                               linear_bwd, no_gpu, problem, ref, rows, weights)

WS = -5


def rows8(channels, **kw):
    return rows(channels, quant=ep.QUANT_INT8, **kw)


def weights8(cin, cout, **kw):
    return weights(cin, cout, **{**dict(fp8=ep.WEIGHTS_INT8), **kw})


@pytest.mark.parametrize("kw,ok", [
    (dict(H=16), True),
    (dict(H=24), False),                                # whole 16-byte vectors of codes
    (dict(H=32768), True),
    (dict(H=128, mode=ep.MODE_LOW_LATENCY), True),
    (dict(H=128, mode=ep.MODE_MESSAGES), False),
    (dict(H=128, mode=ep.MODE_RANK_MAJOR), False),
    (dict(H=128, quant=4), False),
])
def test_problem(kw, ok):
    p = problem(**{**dict(quant=ep.QUANT_INT8), **kw})
    assert (ep.workspace_bytes(p) > 0) == ok
    assert (ep.max_recv_rows(p) >= 0) == ok
    if ok:  # no scales are staged: dispatch needs no workspace of its own
        assert ep.workspace_bytes(p) == ep.workspace_bytes(
            problem(**{**kw, "quant": ep.QUANT_NONE}))


@no_gpu
def test_product_operands():
    for call, y in (gated, rows(16)), (linear, rows(32)):
        x, w = rows8(64), weights8(64, 32)
        kw = {"h" if call is gated else "y": y}
        assert call(x=rows(64), w=w, **kw) == MODE                 # bf16 rows, int8 weights
        assert call(x=x, w=weights(64, 32), **kw) == MODE          # and the other way round
        assert call(x=x, w=weights(64, 32, fp8=1), **kw) == MODE
        assert call(x=rows(64, quant=1), w=w, **kw) == SHAPE       # FP8 rows of 64 channels
        assert call(x=x, w=weights8(64, 32, fp8=3), **kw) == MODE
        assert call(x=rows8(72), w=weights8(72, 32), **kw) == SHAPE
        assert call(x=rows8(64, x=None), w=w, **kw) == NULL
        assert call(x=rows8(64, scales=None), w=w, **kw) == NULL
        assert call(x=x, w=weights8(64, 32, scales=None), **kw) == NULL
        assert call(x=x, w=weights8(64, 32, w=None), **kw) == NULL
        assert call(x=rows8(64, x=A + 8), w=w, **kw) == ALIGN
        assert call(x=rows8(64, scales=A + 2), w=w, **kw) == ALIGN
        assert call(x=x, w=weights8(64, 32, scales=A + 4), **kw) == ALIGN
        assert call(x=x, w=weights8(64, 32, w=A + 8), **kw) == ALIGN
        ll = problem(mode=ep.MODE_LOW_LATENCY)
        assert call(p=ll, x=rows8(64, cap=63), w=w, **kw) == CAP
    assert gated(x=rows8(64), w=weights8(64, 32), h=rows8(16)) == MODE   # results are bf16
    assert linear(x=rows8(64), w=weights8(64, 32), y=rows8(32)) == MODE
    assert linear(x=rows8(64), w=weights8(64, 32), res=rows8(32)) == MODE
    assert linear(x=rows8(64), w=weights8(64, 32), pre=rows8(32)) == MODE
    assert linear_bwd(w=weights8(64, 32)) == MODE
    assert linear_bwd(x=rows8(64)) == MODE
    assert gated_bwd(w=weights8(64, 32)) == MODE


@no_gpu
def test_quantize_rows_operands():
    def call(p=None, lay=None, x="x", q="q"):
        x = rows(64) if x == "x" else x
        q = rows8(64) if q == "q" else q
        return ep.lib().ep_quantize_rows(ref((p or problem()).c()), ref(lay or layout()), ref(x),
                                         ref(q), None)
    assert call(p=problem(E=5)) == SHAPE
    assert call(p=problem(mode=ep.MODE_RANK_MAJOR)) == MODE
    assert call(lay=layout(expert_start=None)) == NULL
    assert call(lay=layout(err=None)) == NULL
    assert call(x=None) == NULL
    assert call(q=None) == NULL
    assert call(x=rows8(64)) == MODE
    assert call(x=rows(64, quant=1)) == MODE
    assert call(q=rows(64)) == MODE
    assert call(q=rows(64, quant=1)) == MODE
    assert call(q=rows8(80)) == SHAPE
    assert call(x=rows(72), q=rows8(72)) == SHAPE
    assert call(x=rows(0), q=rows8(0)) == SHAPE
    assert call(x=rows(32784), q=rows8(32784)) == SHAPE
    assert call(x=rows(64, x=None)) == NULL
    assert call(q=rows8(64, x=None)) == NULL
    assert call(q=rows8(64, scales=None)) == NULL
    assert call(x=rows(64, x=A + 8)) == ALIGN
    assert call(q=rows8(64, x=A + 8)) == ALIGN
    assert call(q=rows8(64, scales=A + 2)) == ALIGN
    assert call(q=rows8(64, cap=-1)) == CAP
    assert call(p=problem(mode=ep.MODE_LOW_LATENCY), q=rows8(64, cap=63),
                x=rows(64, cap=64)) == CAP


@no_gpu
def test_dispatch_operands():
    p = problem(quant=ep.QUANT_INT8)

    def call(p=p, **kw):
        recv = ep.CRecv(**{**dict(x=A, scales=A, capacity=32, topk_idx=None, topk_weights=None),
                           **kw})
        return ep.lib().ep_dispatch(ref(p.c()), ref(layout()), A, None, None, ctypes.byref(recv),
                                    None, None, 0, None)
    assert call(x=None) == NULL
    assert call(scales=None) == NULL
    assert call(x=A + 8) == ALIGN
    assert call(scales=A + 2) == ALIGN
    assert call(capacity=-1) == CAP
    assert call(p=problem(quant=ep.QUANT_INT8, mode=ep.MODE_LOW_LATENCY), capacity=63) == CAP


def test_the_binding_checks_shapes_and_types():
    p = problem()
    lay = ep.Layout(p, device="cpu")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8)      # noqa: E731
    f = torch.zeros
    x, w, sx, sw = i8(32, 64), i8(4, 32, 64), f(32), f(4, 32)
    bad = [
        lambda: ep.expert_gated(p, lay, bf(32, 64), w, bf(32, 16), x_scales=sx, w_scales=sw),
        lambda: ep.expert_gated(p, lay, x, bf(4, 32, 64), bf(32, 16), x_scales=sx),
        lambda: ep.expert_gated(p, lay, x.view(torch.uint8), w, bf(32, 16), x_scales=sx,
                                w_scales=sw),
        lambda: ep.expert_gated(p, lay, x, w, bf(32, 16), w_scales=sw),
        lambda: ep.expert_gated(p, lay, x, w, bf(32, 16), x_scales=sx),
        lambda: ep.expert_gated(p, lay, x, w, bf(32, 16), x_scales=f(31), w_scales=sw),
        lambda: ep.expert_gated(p, lay, x, w, bf(32, 16), x_scales=sx.double(), w_scales=sw),
        lambda: ep.expert_gated(p, lay, x, w, bf(32, 16), x_scales=sx, w_scales=f(4, 16)),
        lambda: ep.expert_gated(p, lay, x, w, i8(32, 16), x_scales=sx, w_scales=sw),
        lambda: ep.expert_gated(p, lay, x, w[:3], bf(32, 16), x_scales=sx, w_scales=sw),
        lambda: ep.expert_linear(p, lay, i8(32, 80), w, bf(32, 32), x_scales=sx, w_scales=sw),
        lambda: ep.expert_linear(p, lay, x, w, bf(32, 32), x_scales=sx, w_scales=sw,
                                 bias=f(4, 31)),
        lambda: ep.quantize_rows(p, lay, x, x, sx),
        lambda: ep.quantize_rows(p, lay, bf(32, 64), bf(32, 64), sx),
        lambda: ep.quantize_rows(p, lay, bf(32, 64), i8(32, 80), sx),
        lambda: ep.quantize_rows(p, lay, bf(32, 64), x, f(31)),
        # whole otherwise, but on the host
        lambda: ep.expert_gated(p, lay, x, w, bf(32, 16), x_scales=sx, w_scales=sw),
        lambda: ep.quantize_rows(p, lay, bf(32, 64), x, sx),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(i))
    p8 = problem(quant=ep.QUANT_INT8)
    lay8, recv = ep.Layout(p8, device="cpu"), ep.Recv(p8, 32, device="cpu")
    assert recv.x.dtype == torch.int8 and recv.scales.shape == (32,)
    recv.scales = f(31)
    with pytest.raises(ValueError, match="scales"):
        ep.dispatch(p8, lay8, bf(2, 8, 128), recv=recv)
    recv.scales, recv.x = f(32), recv.x.view(torch.uint8)
    with pytest.raises(ValueError, match="int8"):
        ep.dispatch(p8, lay8, bf(2, 8, 128), recv=recv)
