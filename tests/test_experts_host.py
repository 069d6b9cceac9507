"""What the experts' products and combine's gradient refuse on the host, before
any launch: through the C ABI with host addresses (no GPU needed), and the
binding's own checks."""
import ctypes

import numpy as np
import pytest
import torch

from combine_ep_get_layout_amd import ep

NULL, ALIGN, SHAPE, MODE, CAP = -1, -2, -3, -4, -6
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="host pointers only where no GPU exists")

_buf = np.zeros(1 << 16, np.uint8)
A = (_buf.ctypes.data + 255) // 256 * 256  # an aligned address; never dereferenced


def problem(**kw):
    return ep.Problem(**{**dict(R=2, T=8, H=128, E=4, K=2), **kw})


def layout(**kw):
    c = ep.CLayout(*([A] * 11), 0, A)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rows(channels, cap=32, quant=0, x=A, scales=A):
    return ep.CRows(x, scales, cap, channels, quant)


def weights(cin, cout, **kw):
    return ep.CWeights(**{**dict(w=A, scales=A, bias=None, in_channels=cin, out_channels=cout,
                                 fp8=0, reserved=0), **kw})


def ref(c):
    return None if c is None else ctypes.byref(c)


def gated(p=None, lay=None, x=None, w=None, act=2, h=None, pre=None):
    p, lay = p or problem(), lay or layout()
    x, w, h = x or rows(64), w or weights(64, 32), h or rows(16)
    return ep.lib().ep_expert_gated(ref(p.c()), ref(lay), ref(x), ref(w), act, ref(h), ref(pre),
                                    None)


def linear(p=None, lay=None, x=None, w=None, act=2, res=None, y=None, pre=None):
    p, lay = p or problem(), lay or layout()
    x, w, y = x or rows(64), w or weights(64, 32), y or rows(32)
    return ep.lib().ep_expert_linear(ref(p.c()), ref(lay), ref(x), ref(w), act, ref(res), ref(y),
                                     ref(pre), None)


def linear_bwd(p=None, lay=None, x="x", w=None, act=2, pre="pre", dy=None, dpre="dpre", dx="dx",
               dw=A, dbias=A):
    p, lay = p or problem(), lay or layout()
    one = dict(x=rows(64), pre=rows(32), dpre=rows(32), dx=rows(64))
    get = lambda v: one[v] if isinstance(v, str) else v  # noqa: E731
    return ep.lib().ep_expert_linear_backward(
        ref(p.c()), ref(lay), ref(get(x)), ref(w or weights(64, 32)), act, ref(get(pre)),
        ref(dy or rows(32)), ref(get(dpre)), ref(get(dx)), dw, dbias, None)


def gated_bwd(x="x", w=None, act=2, pre="pre", dh=None, dpre="dpre", dx="dx", dw=A):
    one = dict(x=rows(64), pre=rows(32), dpre=rows(32), dx=rows(64))
    get = lambda v: one[v] if isinstance(v, str) else v  # noqa: E731
    return ep.lib().ep_expert_gated_backward(
        ref(problem().c()), ref(layout()), ref(get(x)), ref(w or weights(64, 32)), act,
        ref(get(pre)), ref(dh or rows(16)), ref(get(dpre)), ref(get(dx)), dw, None)


@no_gpu
@pytest.mark.parametrize("call", [gated, linear, linear_bwd])
def test_problem_and_layout(call):
    assert call(p=problem(E=5)) == SHAPE
    assert call(p=problem(mode=ep.MODE_RANK_MAJOR)) == MODE
    assert call(lay=layout(expert_start=None)) == NULL
    assert call(lay=layout(recv_tokens_per_expert=None)) == NULL
    assert call(lay=layout(err=None)) == NULL
    assert call(lay=layout(err=A + 2)) == ALIGN
    assert call(lay=layout(recv_tokens_per_expert=A + 1)) == ALIGN
    # messages with more blocks than a row index counts
    big = problem(R=8, T=1 << 19, E=1024, mode=ep.MODE_MESSAGES)
    assert call(p=big) == SHAPE
    assert call(act=4) == MODE
    assert call(act=-1) == MODE


@no_gpu
def test_forward_operands():
    assert gated(x=rows(72)) == SHAPE                       # x's channels are not w's
    assert gated(h=rows(32)) == SHAPE                       # h has half of w's
    assert gated(w=weights(64, 33)) == SHAPE
    assert gated(w=weights(64, 24)) == SHAPE                # 12 channels: no whole vectors
    assert gated(w=weights(60, 32), x=rows(60)) == SHAPE
    assert gated(w=weights(32776, 32), x=rows(32776)) == SHAPE
    assert gated(w=weights(0, 32), x=rows(0)) == SHAPE
    assert gated(w=weights(64, 32, reserved=1)) == SHAPE
    assert gated(w=weights(64, 32, fp8=2)) == MODE
    assert gated(w=weights(64, 32, bias=A)) == MODE
    assert gated(w=weights(64, 32, w=None)) == NULL
    assert gated(w=weights(64, 32, w=A + 8)) == ALIGN
    assert gated(x=rows(64, x=None)) == NULL
    assert gated(x=rows(64, x=A + 8)) == ALIGN
    assert gated(x=rows(64, cap=-1)) == CAP
    assert gated(pre=rows(16)) == SHAPE                     # pre holds both projections
    assert gated(pre=rows(32, quant=1)) == MODE
    assert gated(h=rows(16, quant=3)) == MODE
    ll = problem(mode=ep.MODE_LOW_LATENCY)                  # 4 blocks of 16 rows
    assert gated(p=ll, x=rows(64, cap=63), h=rows(16, cap=64)) == CAP
    assert gated(p=ll, x=rows(64, cap=64), h=rows(16, cap=63)) == CAP
    assert linear(res=rows(64)) == SHAPE
    assert linear(res=rows(32, quant=1)) == MODE
    assert linear(w=weights(64, 32, bias=A + 4)) == ALIGN


@no_gpu
def test_fp8_operands():
    x, y = rows(256, quant=1), rows(128)
    w = weights(256, 128, fp8=1)
    assert linear(x=rows(256), w=w, y=y) == MODE            # bf16 rows, FP8 weights
    assert linear(x=x, w=weights(256, 128), y=y) == MODE    # and the other way round
    assert linear(x=rows(192, quant=1), w=weights(192, 128, fp8=1), y=y) == SHAPE
    assert linear(x=x, w=weights(256, 64, fp8=1), y=rows(64)) == SHAPE
    assert linear(x=rows(256, quant=1, scales=None), w=w, y=y) == NULL
    assert linear(x=rows(256, quant=1, scales=A + 2), w=w, y=y) == ALIGN
    assert linear(x=x, w=weights(256, 128, fp8=1, scales=None), y=y) == NULL
    assert linear(x=rows(256), w=weights(256, 128), y=rows(128, quant=1)) == MODE  # bf16 in, FP8 out
    assert gated(x=x, w=weights(256, 128, fp8=1), h=rows(64)) == SHAPE  # 64 channels of each
    assert linear_bwd(w=weights(64, 32, fp8=1)) == MODE


@no_gpu
def test_backward_operands():
    assert linear_bwd(pre=None) == NULL
    assert linear_bwd(dpre=None) == NULL
    assert linear_bwd(dpre=None, dx=None, dw=None, pre=None) == NULL   # dbias needs pre
    assert linear_bwd(x=None) == NULL                                   # dw needs x
    assert linear_bwd(x=rows(32)) == SHAPE
    assert linear_bwd(dx=rows(32)) == SHAPE
    assert linear_bwd(dy=rows(64)) == SHAPE
    assert linear_bwd(dw=A + 8) == ALIGN
    assert linear_bwd(dbias=A + 2) == ALIGN
    assert linear_bwd(w=weights(64, 32, w=None)) == NULL                # dx needs w
    assert gated_bwd(pre=None) == NULL
    assert gated_bwd(dpre=None) == NULL
    assert gated_bwd(dh=rows(32)) == SHAPE
    assert gated_bwd(dpre=rows(16)) == SHAPE
    assert gated_bwd(dx=rows(64, quant=1)) == MODE


@no_gpu
def test_combine_backward_operands():
    def call(p=None, lay=None, dout=A, w=A, y=A, n=32, dy=A, dw=A):
        return ep.lib().ep_combine_backward(ref((p or problem()).c()), ref(lay or layout()), dout,
                                            w, y, n, dy, dw, None)
    assert call(p=problem(mode=ep.MODE_MESSAGES)) == MODE
    assert call(p=problem(mode=ep.MODE_RANK_MAJOR)) == MODE  # with dweights
    assert call(lay=layout(send_pos=None)) == NULL
    assert call(dout=None) == NULL
    assert call(w=None) == NULL
    assert call(y=None) == NULL
    assert call(n=-1) == CAP
    for k in ("dout", "y", "dy"):
        assert call(**{k: A + 8}) == ALIGN
    for k in ("w", "dw"):
        assert call(**{k: A + 2}) == ALIGN


def test_the_binding_checks_shapes_and_types():
    """ValueErrors before the library is reached; host tensors are refused last."""
    p = problem()
    lay = ep.Layout(p, device="cpu")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)     # noqa: E731
    x, w, h = bf(32, 64), bf(4, 32, 64), bf(32, 16)
    bad = [
        lambda: ep.expert_gated(p, lay, x.float(), w, h),
        lambda: ep.expert_gated(p, lay, x[0], w, h),
        lambda: ep.expert_gated(p, lay, x, w[:3], h),
        lambda: ep.expert_gated(p, lay, x, w[:, :31], h),
        lambda: ep.expert_gated(p, lay, x, w, bf(32, 32)),
        lambda: ep.expert_gated(p, lay, x, w, h, pre=bf(32, 16)),
        lambda: ep.expert_gated(p, lay, u8(32, 128), w, h),
        lambda: ep.expert_gated(p, lay, u8(32, 128), u8(4, 256, 128), bf(32, 128),
                                x_scales=torch.zeros(31), w_scales=torch.zeros(4, 2, 1)),
        lambda: ep.expert_gated(p, lay, u8(32, 128), u8(4, 256, 128), bf(32, 128),
                                x_scales=torch.zeros(32), w_scales=torch.zeros(4, 1, 1)),
        lambda: ep.expert_gated(p, lay, u8(32, 128), u8(4, 256, 128), bf(32, 128),
                                x_scales=torch.zeros(32).double(), w_scales=torch.zeros(4, 2, 1)),
        lambda: ep.expert_linear(p, lay, x, w, bf(32, 32), bias=torch.zeros(4, 31)),
        lambda: ep.expert_linear(p, lay, x, w, bf(32, 32), bias=bf(4, 32)),
        lambda: ep.expert_linear(p, lay, x, w, bf(32, 32), residual=bf(32, 64)),
        lambda: ep.expert_linear_backward(p, lay, x, w, bf(32, 32), dw=w.float()),
        lambda: ep.expert_linear_backward(p, lay, x, w, bf(32, 32), dw=bf(4, 64, 32)),
        lambda: ep.expert_linear_backward(p, lay, x, w, bf(32, 32), dbias=torch.zeros(4, 31)),
        lambda: ep.expert_gated_backward(p, lay, x, w, bf(32, 16), h, dpre=bf(32, 32)),
        lambda: ep.combine_backward(p, lay, bf(16, 64), None, None, dy=bf(32, 128)),
        lambda: ep.combine_backward(p, lay, bf(16, 128), torch.zeros(16, 2), None),
        lambda: ep.combine_backward(p, lay, bf(16, 128), torch.zeros(16, 2), None,
                                    dweights=torch.zeros(16, 2)),
        lambda: ep.combine_backward(p, lay, bf(16, 128), torch.zeros(16, 2), bf(31, 128),
                                    dy=bf(32, 128)),
        lambda: ep.expert_gated(p, ep.Layout(problem(E=8), device="cpu"), x, w, h),
        # whole otherwise, but on the host
        lambda: ep.expert_gated(p, lay, x, w, h),
        lambda: ep.expert_linear(p, lay, x, w, bf(32, 32)),
        lambda: ep.combine_backward(p, lay, bf(16, 128), torch.zeros(16, 2), None, dy=bf(32, 128)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(i))


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int8, torch.bool])
def test_codes_of_another_kind_are_refused(dtype):
    """A byte type that is not e4m3 codes would be read as if it were."""
    x, w = torch.zeros((32, 128), dtype=torch.uint8), torch.zeros((4, 256, 128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="e4m3"):
        ep._rows(problem(), x.view(dtype), "x", 128, torch.zeros(32))
    with pytest.raises(ValueError, match="e4m3"):
        ep._weights(problem(), w.view(dtype), torch.zeros(4, 2, 1))
