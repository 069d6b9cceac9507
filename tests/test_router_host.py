"""What the router and its gradient refuse on the host, before any launch."""
import ctypes

import pytest
import torch

from combine_ep_get_layout_amd import ep
from test_experts_host import A, ALIGN, MODE, NULL, SHAPE, no_gpu, problem, ref


def router(**kw):
    return ep.CRouter(**{**dict(score=0, groups=1, groups_kept=1, group_top=1, normalize=1,
                                bf16=0, scale=1.0, reserved=0), **kw})


def route(p=None, r="r", logits=A, bias=None, idx=A, w=A, err=A):
    r = router() if r == "r" else r
    return ep.lib().ep_route(ref((p or problem()).c()), ref(r), logits, bias, idx, w, err, None)


def route_bwd(p=None, r="r", logits=A, idx=A, dw=A, dl=A, err=A):
    r = router() if r == "r" else r
    return ep.lib().ep_route_backward(ref((p or problem()).c()), ref(r), logits, idx, dw, dl, err,
                                      None)


@no_gpu
@pytest.mark.parametrize("call", [route, route_bwd])
def test_router(call):
    assert call(p=problem(E=5)) == SHAPE
    assert call(p=problem(K=65)) == SHAPE
    assert call(r=None) == NULL
    for kw in (dict(score=2), dict(score=-1), dict(normalize=2), dict(bf16=2)):
        assert call(r=router(**kw)) == MODE, kw
    for kw in (dict(reserved=1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(groups=0), dict(groups=3), dict(groups=2, groups_kept=3),
               dict(groups_kept=0), dict(group_top=0), dict(group_top=3),
               dict(groups=4, groups_kept=2, group_top=2)):  # one expert a group
        assert call(r=router(**kw)) == SHAPE, kw
    assert call(p=problem(E=128), r=router(groups=128, groups_kept=2)) == SHAPE
    assert call(logits=None) == NULL
    assert call(idx=None) == NULL
    assert call(logits=A + 8) == ALIGN
    assert call(idx=A + 2) == ALIGN
    assert call(err=A + 2) == ALIGN


@no_gpu
def test_arrays():
    assert route(w=None) == NULL
    assert route(w=A + 2) == ALIGN
    assert route(bias=A + 4) == ALIGN
    assert route_bwd(dw=None) == NULL
    assert route_bwd(dl=None) == NULL
    assert route_bwd(dw=A + 2) == ALIGN
    assert route_bwd(dl=A + 8) == ALIGN


def test_the_binding_checks_shapes_and_types():
    p = problem()
    f, i = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.int32)
    l, idx, w = f(2, 8, 4), i(2, 8, 2), f(2, 8, 2)
    bad = [
        lambda: ep.route(p, l.half(), idx, w),
        lambda: ep.route(p, l[:1], idx, w),
        lambda: ep.route(p, l, idx.long(), w),
        lambda: ep.route(p, l, idx[:1], w),
        lambda: ep.route(p, l, idx, w.double()),
        lambda: ep.route(p, l, idx, w[:1]),
        lambda: ep.route(p, l, idx, w, f(1)),
        lambda: ep.route(p, l, idx, w, bias=f(3)),
        lambda: ep.route(p, l, idx, w, bias=f(4).double()),
        lambda: ep.route_backward(p, l, idx, w[:1], l),
        lambda: ep.route_backward(p, l, idx, w, l.bfloat16()),
        lambda: ep.route_backward(p, l, idx, w, l[:1]),
        lambda: ep.route_backward(p, l, idx[:1], w, l),
        # whole otherwise, but on the host
        lambda: ep.route(p, l, idx, w),
        lambda: ep.route_backward(p, l, idx, w, l),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(k))
    assert ctypes.sizeof(ep.CRouter) == 32
