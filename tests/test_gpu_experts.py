"""The experts' products and their gradients against plain 64-bit forms
(tests/expert_util.py, where the bounds are derived): segment lengths from none
to several tiles, channel counts that no tile divides, both layouts, every
activation, FP8 rows and weights, poisoned rows around the segments, and the
whole expert layer from dispatch to combine and back."""
import numpy as np
import pytest
import torch

from combine_ep_get_layout_amd import ep, inputs
from expert_util import (ACTS, HALF, act64, backward64, codes_of, dz64, forward64, fp8_weights,
                         held, row_scales, segments)
from gpu_util import DEV, gpu_layout, say

pytestmark = pytest.mark.gpu

N, L, M = ep.MODE_NORMAL, ep.MODE_LOW_LATENCY, ep.MODE_MESSAGES
NAN = float("nan")
INF = float("inf")


def routed(R, T, E, K, mode, seed, masked=0.0, only=None, quant=ep.QUANT_NONE, H=128, align=1):
    """Problem and GPU layout of a random routing; `only`: the experts used."""
    w = inputs.small("experts", R=R, T=T, H=H, E=E, K=K, mode=mode, quant=quant, seed=seed)
    topk = inputs.gen_topk(w)
    if masked:
        topk = inputs.masked_topk(w, topk, masked, 0.0, seed=seed)
    if only is not None:
        topk = np.where(np.isin(topk, only), topk, -1).astype(np.int32)
    p = ep.Problem(R, T, H, E, K, align=align, mode=mode, quant=quant)
    lay, ws = gpu_layout(p, topk)
    return p, lay, topk


def capacity(p):
    return max(ep.max_recv_rows(p), 1)


def rand(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(torch.bfloat16)


def rows_for(gen, p, segs, channels, poison=NAN):
    """bf16 [capacity][channels]: N(0, 1) in the segments, poison everywhere else."""
    t = torch.full((capacity(p), channels), poison, dtype=torch.bfloat16)
    for s, c in segs:
        t[s:s + c] = rand(gen, c, channels)
    return t


def untouched(t, segs, poison_bits):
    """Rows outside the segments still hold the poison."""
    v = t.cpu().view(torch.int16)
    keep = torch.ones(v.shape[0], dtype=torch.bool)
    for s, c in segs:
        keep[s:s + c] = False
    assert (v[keep] == poison_bits).all()


def poisoned(rows, channels):
    return torch.full((rows, channels), 0x5A5A, dtype=torch.int16, device=DEV).view(torch.bfloat16)


# R, T, E, K, mode, masked, C, N: rows an expert from one (most have none) to
# several tiles of the largest kind; channels from one vector to odd counts
SHAPES = [
    (1, 1, 8, 2, L, 0.0, 64, 8),
    (1, 1, 8, 8, N, 0.0, 8, 24),
    (2, 3, 4, 2, N, 0.0, 72, 136),
    (1, 16, 2, 1, L, 0.0, 128, 64),
    (3, 11, 6, 2, L, 0.3, 264, 40),
    (2, 40, 4, 2, N, 0.2, 520, 264),
    (1, 65, 1, 1, N, 0.0, 1032, 520),
    (2, 90, 3 * 2, 3, L, 0.1, 200, 312),
    (1, 300, 2, 1, N, 0.0, 328, 264),
    (4, 130, 4, 2, N, 0.1, 136, 520),
    (1, 520, 2, 2, L, 0.0, 72, 72),
    (2, 33, 64, 4, N, 0.0, 96, 48),
]
SHAPE_IDS = ["-".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
@pytest.mark.parametrize("shape", SHAPES, ids=SHAPE_IDS)
def test_gated(shape, act):
    R, T, E, K, mode, masked, C, I = shape
    say("gated", shape, act)
    p, lay, _ = routed(R, T, E, K, mode, seed=3, masked=masked)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(11)
    x, w = rows_for(gen, p, segs, C), rand(gen, E, 2 * I, C, scale=C ** -0.5)
    h, pre = poisoned(capacity(p), I), poisoned(capacity(p), 2 * I)
    xg, wg = x.to(DEV), w.to(DEV)
    ep.expert_gated(p, lay, xg, wg, h, act=ACTS[act], pre=pre)
    h2 = poisoned(capacity(p), I)
    ep.expert_gated(p, lay, xg, wg, h2, act=ACTS[act])
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    for e, (s, c) in enumerate(segs):
        y, ey, z, ez = forward64(x[s:s + c].double(), w[e].double(), act, True)
        held(h[s:s + c], y, ey, ("h", e))
        held(pre[s:s + c], z, ez, ("pre", e))
    untouched(h, segs, 0x5A5A)
    untouched(pre, segs, 0x5A5A)
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))  # saving pre changes nothing


@pytest.mark.parametrize("extras", ["plain", "bias", "residual", "all", "in_place"])
@pytest.mark.parametrize("shape", SHAPES, ids=SHAPE_IDS)
def test_linear(shape, extras):
    R, T, E, K, mode, masked, C, O = shape
    say("linear", shape, extras)
    p, lay, _ = routed(R, T, E, K, mode, seed=4, masked=masked)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(12)
    act = {"plain": "none", "bias": "gelu", "residual": "relu", "all": "silu",
           "in_place": "none"}[extras]
    x, w = rows_for(gen, p, segs, C), rand(gen, E, O, C, scale=C ** -0.5)
    bias = torch.randn((E, O), generator=gen) if extras in ("bias", "all") else None
    res = None
    if extras in ("residual", "all", "in_place"):
        res = rows_for(gen, p, segs, O)
    y = res.to(DEV) if extras == "in_place" else poisoned(capacity(p), O)
    pre = poisoned(capacity(p), O) if extras == "all" else None
    ep.expert_linear(p, lay, x.to(DEV), w.to(DEV), y, act=ACTS[act],
                     bias=None if bias is None else bias.to(DEV),
                     residual=y if extras == "in_place" else None if res is None else res.to(DEV),
                     pre=pre)
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    for e, (s, c) in enumerate(segs):
        want, ey, z, ez = forward64(x[s:s + c].double(), w[e].double(), act, False,
                                    None if bias is None else bias[e].double(),
                                    None if res is None else res[s:s + c].double())
        held(y[s:s + c], want, ey, ("y", e))
        if pre is not None:
            held(pre[s:s + c], z, ez, ("pre", e))
    if extras != "in_place":
        untouched(y, segs, 0x5A5A)


def relative(got, want):
    """2-norm of the error over the 2-norm of the result, over all given pieces."""
    d = sum(float((g.double().cpu() - w).square().sum()) for g, w in zip(got, want))
    return (d / max(sum(float(w.square().sum()) for w in want), 1e-300)) ** 0.5


@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
@pytest.mark.parametrize("op", ["gated", "linear"])
@pytest.mark.parametrize("shape", SHAPES, ids=SHAPE_IDS)
def test_backward(shape, op, act):
    R, T, E, K, mode, masked, C, I = shape
    say("backward", shape, op, act)
    gated = op == "gated"
    p, lay, _ = routed(R, T, E, K, mode, seed=5, masked=masked)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(13)
    O = 2 * I if gated else I
    x, dy = rows_for(gen, p, segs, C), rows_for(gen, p, segs, I)
    pre, w = rows_for(gen, p, segs, O), rand(gen, E, O, C, scale=C ** -0.5)
    dx, dpre = poisoned(capacity(p), C), poisoned(capacity(p), O)
    dw = torch.full((E, O, C), NAN, dtype=torch.bfloat16, device=DEV)
    dbias = None
    if gated:
        ep.expert_gated_backward(p, lay, x.to(DEV), w.to(DEV), pre.to(DEV), dy.to(DEV),
                                 dpre=dpre, dx=dx, dw=dw, act=ACTS[act])
    else:
        dbias = torch.full((E, I), NAN, device=DEV)
        kw = {} if act == "none" else dict(pre=pre.to(DEV), dpre=dpre)
        ep.expert_linear_backward(p, lay, x.to(DEV), w.to(DEV), dy.to(DEV), dx=dx, dw=dw,
                                  dbias=dbias, act=ACTS[act], **kw)
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    got, want = [], []
    for e, (s, c) in enumerate(segs):
        dz, edz = dz64(dy[s:s + c].double(), pre[s:s + c].double(), act, gated)
        wx, ex, ww, ew = backward64(x[s:s + c].double(), w[e].double(), dz, edz)
        held(dx[s:s + c], wx, ex, ("dx", e))
        held(dw[e], ww, ew, ("dw", e))
        if gated or act != "none":
            held(dpre[s:s + c], dz, edz + 1e-300, ("dpre", e))
        if dbias is not None:
            # fp32 terms (relative error as in edz without its rounding to
            # bf16) summed in fp32
            pz = pre[s:s + c].double().abs()
            term = (4 + pz) * (1 + pz) * 2.0 ** -22 * dy[s:s + c].double().abs()
            if act == "none":
                term = term * 0
            b = term.sum(0) + (c + 8) * 2.0 ** -23 * (dz.abs() + term).sum(0) + 1e-30
            held(dbias[e], dz.sum(0), b, ("dbias", e))
        got += [dx[s:s + c], dw[e]]
        want += [wx, ww]
    untouched(dx, segs, 0x5A5A)
    if gated or act != "none":
        untouched(dpre, segs, 0x5A5A)
    # over all values: two roundings, each uniform within half a step, give at
    # most sqrt(2/3) of the worst case; many values keep to it
    if sum(v.numel() for v in want) > 4096:
        assert relative(got, want) <= HALF


@pytest.mark.parametrize("need", ["dx", "dw", "dbias"])
@pytest.mark.parametrize("op", ["gated", "linear"])
def test_backward_of_one_input(op, need):
    """Each gradient alone, its unneeded operands absent, equals the full call's."""
    gated = op == "gated"
    if gated and need == "dbias":
        pytest.skip("the gated block has no bias")
    p, lay, _ = routed(2, 50, 4, 2, N, seed=6)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(14)
    C, I = 136, 72
    O = 2 * I if gated else I
    x, dy = rows_for(gen, p, segs, C).to(DEV), rows_for(gen, p, segs, I).to(DEV)
    pre, w = rows_for(gen, p, segs, O).to(DEV), rand(gen, 4, O, C).to(DEV)
    outs = lambda: dict(dx=poisoned(capacity(p), C),  # noqa: E731
                        dw=torch.zeros((4, O, C), dtype=torch.bfloat16, device=DEV),
                        dbias=torch.zeros((4, I), device=DEV))
    full, one = outs(), outs()
    dpre = poisoned(capacity(p), O)
    if gated:
        ep.expert_gated_backward(p, lay, x, w, pre, dy, dpre=dpre, dx=full["dx"], dw=full["dw"])
        ep.expert_gated_backward(p, lay, x if need == "dw" else None, w, pre, dy, dpre=dpre,
                                 **{need: one[need]})
    else:
        ep.expert_linear_backward(p, lay, x, w, dy, pre=pre, dpre=dpre, act=ep.ACT_SILU, **full)
        ep.expert_linear_backward(p, lay, x if need == "dw" else None, w, dy, pre=pre,
                                  dpre=None if need == "dbias" else dpre, act=ep.ACT_SILU,
                                  **{need: one[need]})
    torch.cuda.synchronize()
    assert torch.equal(full[need].view(torch.uint8), one[need].view(torch.uint8))


def test_gradients_against_differences():
    """<gradient, v> against central differences of the 64-bit forward, for
    v = the gradient's signs: their sum is the 1-norm, so each value's error
    bound (two bf16 roundings, fp32 sums far below) adds up to 2.02 half steps
    of it; the difference's own error is O(step^2) and checked by halving."""
    p, lay, _ = routed(2, 60, 4, 2, N, seed=7, masked=0.1)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(15)
    C, I = 72, 40
    x, w = rows_for(gen, p, segs, C), rand(gen, 4, 2 * I, C, scale=C ** -0.5)
    dh = rows_for(gen, p, segs, I)
    pre = torch.zeros((capacity(p), 2 * I), dtype=torch.float64)

    def loss(x64, w64):
        total = 0.0
        for e, (s, c) in enumerate(segs):
            z = x64[s:s + c] @ w64[e].t()
            total = total + float((act64("silu", z[:, :I])[0] * z[:, I:]
                                   * dh[s:s + c].double()).sum())
        return total

    x64 = torch.nan_to_num(x.double())
    for e, (s, c) in enumerate(segs):
        pre[s:s + c] = x64[s:s + c] @ w[e].double().t()
    dx = torch.zeros((capacity(p), C), dtype=torch.bfloat16, device=DEV)
    dw = torch.zeros((4, 2 * I, C), dtype=torch.bfloat16, device=DEV)
    pre16 = pre.to(torch.bfloat16)
    ep.expert_gated_backward(p, lay, x.to(DEV), w.to(DEV), pre16.to(DEV), dh.to(DEV),
                             dpre=torch.empty_like(pre16, device=DEV), dx=dx, dw=dw)
    torch.cuda.synchronize()
    # the saved pre-activations are rounded as well: |d(dz)/dz| is at most
    # |dh| (1 + |u|) times 1.13, so one more half step of pre per value, which
    # backward64 turns into a bound per gradient value
    slack_x = slack_w = 0.0
    for e, (s, c) in enumerate(segs):
        half = HALF * pre[s:s + c].abs()
        du = dh[s:s + c].double().abs()
        u = pre[s:s + c, I:].abs()
        edz = torch.cat([du * (1.13 * half[:, I:] + u * half[:, :I]), du * 1.13 * half[:, :I]], 1)
        slack_x += float((edz @ w[e].double().abs()).sum())
        slack_w += float((edz.t() @ x64[s:s + c].abs()).sum())
    for grad, which, slack in (dx, 0, slack_x), (dw, 1, slack_w):
        g64 = grad.double().cpu()
        v = g64.sign()
        got = float((g64 * v).sum())
        found = []
        for step in (1e-4, 5e-5):
            a = [x64, w.double()]
            b = [x64, w.double()]
            a[which], b[which] = a[which] + step * v, b[which] - step * v
            found.append((loss(*a) - loss(*b)) / (2 * step))
        assert abs(found[0] - found[1]) <= 1e-4 * abs(found[1])
        # dz's rounding reaches dx through |dz| |w|, at most this sum
        through = 0.0
        for e, (s, c) in enumerate(segs):
            dz, edz = dz64(dh[s:s + c].double(), pre[s:s + c], "silu", True)
            through += float((edz @ w[e].double().abs()).sum() if which == 0
                             else (edz.t() @ x64[s:s + c].abs()).sum())
        assert abs(got - found[1]) <= 1.01 * HALF * got + through + slack + 2e-4 * abs(found[1])


FP8_SHAPES = [  # R, T, E, K, mode, C, N
    (1, 1, 4, 2, L, 128, 128),
    (2, 5, 4, 2, N, 256, 128),
    (2, 30, 4, 2, L, 384, 256),
    (1, 70, 2, 1, N, 640, 384),
    (2, 150, 2, 2, L, 256, 640),
    (1, 300, 1, 1, N, 128, 256),
]


@pytest.mark.parametrize("quant", [ep.QUANT_FP8_F32, ep.QUANT_FP8_UE8M0])
@pytest.mark.parametrize("op", ["gated", "linear"])
@pytest.mark.parametrize("shape", FP8_SHAPES, ids=["-".join(map(str, s)) for s in FP8_SHAPES])
def test_fp8_rows_of_a_dispatch(shape, op, quant):
    """FP8 rows as dispatch writes them, FP8 weights; the result in bf16, and in
    FP8 as dispatch quantises it."""
    R, T, E, K, mode, C, I = shape
    say("fp8", shape, op, quant)
    gated = op == "gated"
    p, lay, topk = routed(R, T, E, K, mode, seed=8, quant=quant, H=C)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(16)
    recv = ep.Recv(p, capacity(p))
    recv.x.fill_(0x7F)  # NaN codes where no row arrives
    recv.scales.view(torch.uint8).fill_(0xFF)
    xt = rand(gen, R * T, C).to(DEV)
    ep.dispatch(p, lay, xt, recv=recv, ws=ep.workspace(p))
    O = 2 * I if gated else I
    wc, ws, w64 = fp8_weights(gen, E, O, C)
    y, pre = poisoned(capacity(p), I), poisoned(capacity(p), O)
    call = ep.expert_gated if gated else ep.expert_linear
    kw = dict(act=ep.ACT_SILU, x_scales=recv.scales, w_scales=ws)
    bias = None
    if not gated:
        bias = torch.randn((E, I), generator=gen)
        kw["bias"] = bias.to(DEV)
    call(p, lay, recv.x, wc, y, pre=pre, **kw)
    groups = I // 128
    out = {}
    for q in (ep.QUANT_FP8_F32, ep.QUANT_FP8_UE8M0):
        codes = torch.full((capacity(p), I), 0x55, dtype=torch.uint8, device=DEV)
        scales = torch.full((groups * capacity(p),), 0x55, dtype=torch.uint8, device=DEV)
        if q == ep.QUANT_FP8_F32:
            scales = torch.full((groups * capacity(p),), -1.0, device=DEV)
        call(p, lay, recv.x, wc, codes, **{("h" if gated else "y") + "_scales": scales}, **kw)
        out[q] = codes.cpu(), scales.cpu()
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    codes64 = codes_of(recv.x)
    for e, (s, c) in enumerate(segs):
        if c == 0:
            continue
        sx = row_scales(p, recv.scales, capacity(p), C // 128, s, c, e)
        x64 = codes64[s:s + c] * sx.repeat_interleave(128, 1)
        want, ey, z, ez = forward64(x64, w64[e], "silu", gated,
                                    None if bias is None else bias[e].double())
        held(y[s:s + c], want, ey, ("y", e))
        held(pre[s:s + c], z, ez, ("pre", e))
        # FP8 results.  The call may sum in another order than the one with the bf16
        # result, so they are held to the formula.  Its bf16 result b is within ey of
        # want, and so is a group's largest |b| of the group's largest |want|, by the
        # group's largest ey; a scale is that over 448, rounded once (2^-24), or the
        # power of two at or above it.  A code is b / scale (rounded once) to e4m3:
        # half a step is 2^-4 of the value, or 2^-10 of a scale among its subnormals.
        for q, (codes, scales) in out.items():
            amax = want.view(c, groups, 128).abs().amax(-1)
            off = ey.expand_as(want).reshape(c, groups, 128).amax(-1)
            low, high = ((amax + d).clamp(min=1e-4) / 448 for d in (-off, off))
            low, high = low * (1 - 2.0 ** -23), high * (1 + 2.0 ** -23)
            if q == ep.QUANT_FP8_UE8M0:
                low, high = torch.exp2(low.log2().ceil()), torch.exp2(high.log2().ceil())
            got = row_scales(p, scales, capacity(p), groups, s, c, e)
            assert ((low <= got) & (got <= high)).all(), ("scales", e)
            code = codes_of(codes[s:s + c]).view(c, groups, 128)
            if q == ep.QUANT_FP8_F32:  # the largest value's code is e4m3's largest
                assert (code.abs().amax(-1) == 448).all()
            step = got.repeat_interleave(128, 1)
            half = torch.maximum((want.abs() + ey) * 2.0 ** -4 * (1 + 2.0 ** -20), step * 2.0 ** -10)
            held(code.view(c, -1) * step, want, ey + half, ("codes", e))
    untouched(y, segs, 0x5A5A)
    for codes, _ in out.values():
        keep = torch.ones(codes.shape[0], dtype=torch.bool)
        for s, c in segs:
            keep[s:s + c] = False
        assert (codes[keep] == 0x55).all()


def test_alignment_padding_rows_stay():
    """Normal mode with expert_alignment: padding rows between the segments are
    neither read nor written, and experts without rows get zero gradients."""
    p, lay, _ = routed(2, 21, 8, 2, N, seed=9, only=[0, 3, 6], align=64)
    segs = segments(p, lay)
    assert sum(c == 0 for _, c in segs) == 5
    gen = torch.Generator().manual_seed(17)
    C, I = 64, 32
    x, w = rows_for(gen, p, segs, C, INF), rand(gen, 8, 2 * I, C, scale=C ** -0.5)
    w[[1, 2, 4, 5, 7]] = NAN  # weights that no row meets
    h, pre = poisoned(capacity(p), I), poisoned(capacity(p), 2 * I)
    ep.expert_gated(p, lay, x.to(DEV), w.to(DEV), h, pre=pre)
    dx, dpre = poisoned(capacity(p), C), poisoned(capacity(p), 2 * I)
    dw = torch.full((8, 2 * I, C), NAN, dtype=torch.bfloat16, device=DEV)
    dh = rows_for(gen, p, segs, I, INF)
    ep.expert_gated_backward(p, lay, x.to(DEV), w.to(DEV), pre, dh.to(DEV), dpre=dpre, dx=dx,
                             dw=dw)
    torch.cuda.synchronize()
    for e, (s, c) in enumerate(segs):
        if c == 0:
            assert (dw[e] == 0).all()
            continue
        y, ey, z, ez = forward64(x[s:s + c].double(), w[e].double(), "silu", True)
        held(h[s:s + c], y, ey, ("h", e))
        assert torch.isfinite(dw[e].float()).all() and torch.isfinite(dx[s:s + c].float()).all()
    for t in (h, pre, dx, dpre):
        untouched(t, segs, 0x5A5A)


@pytest.mark.parametrize("mode", [N, L, M])
def test_no_tokens_and_nothing_routed(mode):
    """No tokens at all, and tokens whose every entry is masked: nothing is
    written but zero weight gradients."""
    for T, masked in ((0, False), (9, True)):
        p = ep.Problem(2, T, 128, 4, 2, mode=mode)
        topk = np.full((2, T, 2), -1, np.int32)
        lay, _ = gpu_layout(p, topk)
        cap = max(p.E * p.R * p.T if mode != N else ep.max_recv_rows(p), 1)
        x = torch.full((cap, 64), NAN, dtype=torch.bfloat16, device=DEV)
        w = torch.full((4, 64, 64), NAN, dtype=torch.bfloat16, device=DEV)
        h, pre, dx, dpre = (poisoned(cap, c) for c in (32, 64, 64, 64))
        dw = torch.full((4, 64, 64), NAN, dtype=torch.bfloat16, device=DEV)
        ep.expert_gated(p, lay, x, w, h, pre=pre)
        ep.expert_gated_backward(p, lay, x, w, pre, h, dpre=dpre, dx=dx, dw=dw)
        torch.cuda.synchronize()
        assert int(lay.err.item()) == 0
        assert (dw == 0).all()
        for t in (h, pre, dx, dpre):
            assert (t.view(torch.int16) == 0x5A5A).all()


def test_special_values_stay_in_their_rows():
    """An infinity or NaN in one row reaches that row's result (and the gradient
    of its expert's weights) and nothing else."""
    p, lay, _ = routed(1, 200, 2, 1, N, seed=10)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(18)
    C, O = 72, 40
    x, w = rows_for(gen, p, segs, C), rand(gen, 2, O, C)
    clean, bad = x.clone(), x.clone()
    r = segs[0][0] + segs[0][1] // 2
    bad[r, 3], bad[r, 5] = INF, NAN
    outs = []
    for t in (clean, bad):
        y = poisoned(capacity(p), O)
        dw = torch.empty((2, O, C), dtype=torch.bfloat16, device=DEV)
        ep.expert_linear(p, lay, t.to(DEV), w.to(DEV), y)
        ep.expert_linear_backward(p, lay, t.to(DEV), w.to(DEV), y, dw=dw)
        outs.append((y.cpu(), dw.cpu()))
    torch.cuda.synchronize()
    (y0, dw0), (y1, dw1) = outs
    assert torch.isnan(y1[r].float()).all()
    y1[r] = y0[r]
    assert torch.equal(y0.view(torch.int16), y1.view(torch.int16))
    assert torch.isnan(dw1[0].float()).any()
    assert torch.equal(dw0[1].view(torch.int16), dw1[1].view(torch.int16))


def test_overflow_to_infinity_and_large_activations():
    """Pre-activations far outside the exponentials' range: silu and gelu of
    +-1e4 are the argument or zero, their slopes one or zero, nothing is NaN."""
    p, lay, _ = routed(1, 40, 1, 1, N, seed=11)
    C = O = 8
    x = torch.zeros((40, C), dtype=torch.bfloat16)
    x[:, 0] = torch.where(torch.arange(40) % 2 == 0, 1e4, -1e4).to(torch.bfloat16)
    w = torch.zeros((1, O, C), dtype=torch.bfloat16)
    w[0, :, 0] = 1
    for act in (ep.ACT_SILU, ep.ACT_GELU):
        y, pre, dpre = (poisoned(40, O) for _ in range(3))
        ep.expert_linear(p, lay, x.to(DEV), w.to(DEV), y, act=act, pre=pre)
        dx = poisoned(40, C)
        ones = torch.ones((40, O), dtype=torch.bfloat16, device=DEV)
        ep.expert_linear_backward(p, lay, None, w.to(DEV), ones, pre=pre, dpre=dpre, dx=dx,
                                  act=act)
        torch.cuda.synchronize()
        assert (y[0::2].float() == x[0, 0].float().item()).all() and (y[1::2] == 0).all()
        assert (dpre[0::2] == 1).all() and (dpre[1::2] == 0).all()


@pytest.mark.parametrize("mode", [N, L])
def test_capacity_is_reported_and_kept(mode):
    """A normal-mode buffer shorter than the segments: the rows inside it are
    right, nothing past it is touched, and the error bit is set.  Low-latency
    buffers must hold every block."""
    p, lay, _ = routed(2, 70, 4, 2, mode, seed=12)
    gen = torch.Generator().manual_seed(19)
    C, O = 72, 40
    w = rand(gen, 4, O, C)
    if mode == L:
        short = capacity(p) - 1
        with pytest.raises(ep.EPError) as err:
            ep.expert_linear(p, lay, torch.zeros((short, C), dtype=torch.bfloat16, device=DEV),
                             w.to(DEV), poisoned(capacity(p), O))
        assert err.value.status == -6
        return
    segs = segments(p, lay)
    x = rows_for(gen, p, segs, C)
    for short in (segs[2][0] + 3, 0):
        lay.err.zero_()
        room = poisoned(capacity(p), O)
        dw = torch.full((4, O, C), NAN, dtype=torch.bfloat16, device=DEV)
        ep.expert_linear(p, lay, x.to(DEV), w.to(DEV), room[:short])
        assert int(lay.err.item()) == ep.DEVERR_CAPACITY
        lay.err.zero_()
        ep.expert_linear_backward(p, lay, x.to(DEV), w.to(DEV),
                                  torch.ones((short, O), dtype=torch.bfloat16, device=DEV), dw=dw)
        assert int(lay.err.item()) == ep.DEVERR_CAPACITY
        torch.cuda.synchronize()
        assert (room[short:].view(torch.int16) == 0x5A5A).all()
        for e, (s, c) in enumerate(segs):
            c = max(0, min(c, short - s))
            want, ey, _, _ = forward64(x[s:s + c].double(), w[e].double(), "none", False)
            held(room[s:s + c], want, ey, ("y", e))
            one = torch.ones((c, O), dtype=torch.float64)
            _, _, ww, ew = backward64(x[s:s + c].double(), w[e].double(), one, one * 0)
            held(dw[e], ww, ew, ("dw", e))


def test_low_latency_overflow_is_cut_at_the_block():
    """Duplicate ids can count past R*T: the block's rows are used, no others."""
    p = ep.Problem(1, 5, 128, 2, 3, mode=L)
    topk = np.zeros((1, 5, 3), np.int32)  # fifteen entries for a block of five
    lay, _ = gpu_layout(p, topk)
    assert int(lay.err.item()) == ep.DEVERR_LL_OVERFLOW
    segs = segments(p, lay)
    assert segs == [(0, 5), (5, 0)]
    gen = torch.Generator().manual_seed(20)
    x, w = rows_for(gen, p, segs, 64), rand(gen, 2, 32, 64)
    y = poisoned(10, 32)
    ep.expert_linear(p, lay, x.to(DEV), w.to(DEV), y)
    torch.cuda.synchronize()
    want, ey, _, _ = forward64(x[:5].double(), w[0].double(), "none", False)
    held(y[:5], want, ey, "y")
    untouched(y, segs, 0x5A5A)


# ---- combine's gradient ------------------------------------------------------

COMBINE = [  # R, T, H, E, K, mode, masked
    (1, 1, 8, 1, 1, N, 0.0),
    (1, 1, 128, 4, 3, L, 0.0),
    (2, 9, 264, 6, 3, N, 0.4),
    (3, 20, 2056, 9, 2, L, 0.3),
    (4, 33, 7168, 8, 8, N, 0.0),
    (2, 5, 32768, 4, 4, N, 0.2),
    (1, 3, 40, 64, 64, N, 0.1),
    (2, 2100, 512, 16, 4, N, 0.1),
]


@pytest.mark.parametrize("case", COMBINE, ids=["-".join(map(str, c)) for c in COMBINE])
def test_combine_backward(case):
    R, T, H, E, K, mode, masked = case
    say("combine_backward", case)
    p, lay, _ = routed(R, T, E, K, mode, seed=13, masked=masked, H=H)
    gen = torch.Generator().manual_seed(21)
    n, cap = R * T, capacity(p)
    dout, y = rand(gen, n, H), rand(gen, cap, H)
    wt = torch.softmax(torch.randn((n, K), generator=gen), -1)
    dy, dw = poisoned(cap, H), torch.full((n, K), NAN, device=DEV)
    ep.combine_backward(p, lay, dout.to(DEV), wt.to(DEV), y.to(DEV), dy=dy, dweights=dw)
    only = [poisoned(cap, H), torch.full((n, K), NAN, device=DEV)]
    ep.combine_backward(p, lay, dout.to(DEV), wt.to(DEV), None, dy=only[0])
    ep.combine_backward(p, lay, dout.to(DEV), None, y.to(DEV), dweights=only[1])
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    pos = lay.send_pos.cpu().view(n, K).long()
    t, k = torch.nonzero(pos >= 0, as_tuple=True)
    rows = pos[t, k]
    want = dout[t].double() * wt[t, k].double()[:, None]
    held(dy[rows.to(DEV)], want, HALF * want.abs() * (1 + HALF) + 2.0 ** -120, "dy")
    left = torch.ones(cap, dtype=torch.bool)
    left[rows] = False
    assert (dy.cpu().view(torch.int16)[left] == 0x5A5A).all()
    terms = dout[t].double() * y[rows].double()
    full = torch.zeros((n, K), dtype=torch.float64)
    bound = torch.full((n, K), 1e-300, dtype=torch.float64)
    full[t, k] = terms.sum(-1)
    bound[t, k] = (H + 8) * 2.0 ** -23 * terms.abs().sum(-1) + 1e-30
    held(dw, full, bound, "dweights")
    assert torch.equal(dy.view(torch.int16), only[0].view(torch.int16))
    assert torch.equal(dw, only[1])


def test_combine_backward_rank_major():
    R, T, H, E, K = 4, 30, 264, 16, 6
    p, lay, _ = routed(R, T, E, K, ep.MODE_RANK_MAJOR, seed=14, masked=0.3, H=H)
    gen = torch.Generator().manual_seed(22)
    dout = rand(gen, R * T, H)
    dy = poisoned(capacity(p), H)
    ep.combine_backward(p, lay, dout.to(DEV), None, None, dy=dy)
    torch.cuda.synchronize()
    pos = lay.send_pos.cpu().view(R * T, K).long()
    t, k = torch.nonzero(pos >= 0, as_tuple=True)
    got = dy.cpu().view(torch.int16)
    assert torch.equal(got[pos[t, k]], dout[t].view(torch.int16))
    left = torch.ones(got.shape[0], dtype=torch.bool)
    left[pos[t, k]] = False
    assert (got[left] == 0x5A5A).all()


def test_combine_backward_capacity():
    p, lay, _ = routed(2, 20, 4, 2, N, seed=15, H=64)
    rows = 50
    gen = torch.Generator().manual_seed(23)
    dout, y = rand(gen, 40, 64).to(DEV), rand(gen, rows, 64).to(DEV)
    wt = torch.ones((40, 2), device=DEV)
    room, dw = poisoned(80, 64), torch.full((40, 2), NAN, device=DEV)
    ep.combine_backward(p, lay, dout, wt, y, dy=room[:rows], dweights=dw)
    torch.cuda.synchronize()
    assert int(lay.err.item()) == ep.DEVERR_CAPACITY
    pos = lay.send_pos.view(40, 2)
    assert (room[rows:].view(torch.int16) == 0x5A5A).all()
    assert (dw[pos >= rows] == 0).all() and torch.isfinite(dw).all()


# ---- together ------------------------------------------------------------------

@pytest.mark.parametrize("mode", [N, L])
def test_whole_layer_forward_and_backward(mode):
    """layout -> dispatch -> gated -> down projection -> combine, and back to the
    tokens, the weights and the routing weights, against autograd in 64 bits.
    Errors accumulate over five bf16 roundings forward and six backward, each
    at most half a step and, over many values, at most sqrt(1/3) of that in
    the 2-norm relative to the value it is made on; the chain's factors pass
    them on with at most its own gain, so sqrt(n / 3) half steps, doubled."""
    R, T, E, K, H, I = 2, 90, 8, 3, 256, 136
    p, lay, topk = routed(R, T, E, K, mode, seed=16, masked=0.1, H=H)
    cap, n = capacity(p), R * T
    gen = torch.Generator().manual_seed(24)
    x, dout = rand(gen, n, H), rand(gen, n, H)
    w1, w2 = rand(gen, E, 2 * I, H, scale=H ** -0.5), rand(gen, E, H, I, scale=I ** -0.5)
    wt = torch.softmax(torch.randn((n, K), generator=gen), -1)
    xg, dg, w1g, w2g, wtg = (v.to(DEV) for v in (x, dout, w1, w2, wt))
    bf = dict(dtype=torch.bfloat16, device=DEV)
    recv = ep.Recv(p, cap)
    h, pre, y = (torch.empty((cap, c), **bf) for c in (I, 2 * I, H))
    out = torch.empty((n, H), **bf)
    ep.dispatch(p, lay, xg, recv=recv, ws=ep.workspace(p))
    ep.expert_gated(p, lay, recv.x, w1g, h, pre=pre)
    ep.expert_linear(p, lay, h, w2g, y)
    ep.combine(p, lay, y, wtg, out)
    dy, dh, dpre, dr = (torch.empty((cap, c), **bf) for c in (H, I, 2 * I, H))
    dw1, dw2, dwt = torch.empty_like(w1g), torch.empty_like(w2g), torch.empty_like(wtg)
    ep.combine_backward(p, lay, dg, wtg, y, dy=dy, dweights=dwt)
    ep.expert_linear_backward(p, lay, h, w2g, dy, dx=dh, dw=dw2)
    ep.expert_gated_backward(p, lay, recv.x, w1g, pre, dh, dpre=dpre, dx=dr, dw=dw1)
    dx = torch.empty((n, H), **bf)
    ep.combine(p, lay, dr, torch.ones_like(wtg), dx)
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0

    leaves = [v.double().requires_grad_() for v in (x, w1, w2, wt)]
    lx, l1, l2, lw = leaves
    ref = torch.zeros((n, H), dtype=torch.float64)
    ids = torch.from_numpy(topk).view(n, K).long()
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        z = lx[t] @ l1[e].t()
        o = (torch.nn.functional.silu(z[:, :I]) * z[:, I:]) @ l2[e].t()
        ref = ref.index_add(0, t, o * lw[t, k][:, None])
    ref.backward(dout.double())
    lim = lambda m: 2 * (m / 3) ** 0.5 * HALF  # noqa: E731
    assert relative([out], [ref.detach()]) <= lim(5)
    for got, leaf, m in (dx, lx, 6), (dw1, l1, 6), (dw2, l2, 5), (dwt, lw, 4):
        assert relative([got], [leaf.grad]) <= lim(m), m


def test_replayed_in_a_graph_on_another_stream():
    """Forward and backward captured together and replayed with new inputs,
    eager work of the same buffers in between: every replay equals an eager run
    bit for bit."""
    p, lay, _ = routed(2, 120, 4, 2, N, seed=17)
    cap = capacity(p)
    C, I = 136, 72
    gen = torch.Generator().manual_seed(25)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    x, w, dh = torch.empty((cap, C), **bf), torch.empty((4, 2 * I, C), **bf), torch.empty((cap, I), **bf)
    names = dict(h=I, pre=2 * I, dpre=2 * I, dx=C)
    bufs = {k: torch.empty((cap, c), **bf) for k, c in names.items()}
    dw = torch.empty_like(w)

    def step():
        ep.expert_gated(p, lay, x, w, bufs["h"], pre=bufs["pre"])
        ep.expert_gated_backward(p, lay, x, w, bufs["pre"], dh, dpre=bufs["dpre"], dx=bufs["dx"],
                                 dw=dw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for rep in range(4):
        for t in (x, w, dh):
            t.copy_(rand(gen, *t.shape, scale=0.3))
        step()
        torch.cuda.synchronize()
        want = {k: v.clone() for k, v in bufs.items()}
        want_dw = dw.clone()
        for t in list(bufs.values()) + [dw]:
            t.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        for k, v in bufs.items():
            assert torch.equal(v[:sum(c for _, c in segments(p, lay))].view(torch.int16),
                               want[k][:sum(c for _, c in segments(p, lay))].view(torch.int16)), k
        assert torch.equal(dw.view(torch.int16), want_dw.view(torch.int16))


def test_two_streams_and_a_prepared_call():
    """The calls of two problems interleaved on two streams, through prepared
    calls, equal each problem's run alone."""
    made = []
    for seed, (T, C, I) in ((1, (300, 264, 136)), (2, (37, 520, 72))):
        p, lay, _ = routed(2, T, 4, 2, N, seed=18 + seed)
        gen = torch.Generator().manual_seed(26 + seed)
        x = torch.randn((capacity(p), C), generator=gen).to(torch.bfloat16).to(DEV)
        w = rand(gen, 4, 2 * I, C, scale=C ** -0.5).to(DEV)
        alone = torch.zeros((capacity(p), I), dtype=torch.bfloat16, device=DEV)
        ep.expert_gated(p, lay, x, w, alone)
        made.append((p, lay, x, w, alone, torch.zeros_like(alone)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    calls = [ep.prepare(ep.expert_gated, p, lay, x, w, out, stream=s)
             for s, (p, lay, x, w, _, out) in zip(streams, made)]
    for _ in range(20):
        for c in calls:
            c()
    torch.cuda.synchronize()
    for _, _, _, _, alone, out in made:
        assert torch.equal(alone.view(torch.int16), out.view(torch.int16))


def test_rows_past_32_bit_offsets():
    """A low-latency buffer of 2.4 G values: the last block's rows lie past 2^31
    elements and 2^32 bytes."""
    T, E, C, O = 16384, 36, 4104, 64
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GiB")
    p = ep.Problem(1, T, 128, E, 1, mode=L)
    topk = np.full((1, T, 1), -1, np.int32)
    topk[0, :700, 0] = E - 1
    topk[0, 700:705, 0] = 0
    lay, _ = gpu_layout(p, topk)
    cap = capacity(p)
    assert (cap - T) * C > 1 << 31
    gen = torch.Generator().manual_seed(27)
    x = torch.zeros((cap, C), dtype=torch.bfloat16, device=DEV)
    segs = segments(p, lay)
    w = rand(gen, E, O, C, scale=C ** -0.5)
    y = poisoned(cap, O)
    rows = {}
    for e, (s, c) in enumerate(segs):
        rows[e] = rand(gen, c, C)
        x[s:s + c] = rows[e].to(DEV)
    ep.expert_linear(p, lay, x, w.to(DEV), y)
    dx = torch.empty((cap, C), dtype=torch.bfloat16, device=DEV)
    dw = torch.empty((E, O, C), dtype=torch.bfloat16, device=DEV)
    ep.expert_linear_backward(p, lay, x, w.to(DEV), y, dx=dx, dw=dw)
    torch.cuda.synchronize()
    for e, (s, c) in enumerate(segs):
        x64 = rows[e].double()
        want, ey, _, _ = forward64(x64, w[e].double(), "none", False)
        held(y[s:s + c], want, ey, ("y", e))
        dz = y[s:s + c].double().cpu()
        wx, ex, ww, ew = backward64(x64, w[e].double(), dz, dz * 0)
        held(dx[s:s + c], wx, ex, ("dx", e))
        held(dw[e], ww, ew, ("dw", e))
    untouched(y, segs, 0x5A5A)


def test_message_problem_after_unpack_layout():
    """EP_MODE_MESSAGES uses the low-latency blocks that ep_messages_unpack fills."""
    pl, lay, _ = routed(2, 30, 4, 2, L, seed=21)
    pm = ep.Problem(2, 30, 128, 4, 2, mode=M)
    gen = torch.Generator().manual_seed(28)
    segs = segments(pl, lay)
    x, w = rows_for(gen, pl, segs, 72), rand(gen, 4, 40, 72)
    a, b = poisoned(capacity(pl), 40), poisoned(capacity(pl), 40)
    ep.expert_linear(pl, lay, x.to(DEV), w.to(DEV), a)
    ep.expert_linear(pm, lay, x.to(DEV), w.to(DEV), b)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    untouched(b, segs, 0x5A5A)


def test_expert_counts_at_the_limit():
    """2,048 experts, most of them empty: the tile plan's whole range."""
    p, lay, _ = routed(1, 300, 2048, 3, N, seed=22)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(29)
    x, w = rows_for(gen, p, segs, 64), rand(gen, 2048, 16, 64, scale=0.125)
    y = poisoned(capacity(p), 16)
    dw = torch.full((2048, 16, 64), NAN, dtype=torch.bfloat16, device=DEV)
    dx = poisoned(capacity(p), 64)
    ep.expert_linear(p, lay, x.to(DEV), w.to(DEV), y)
    ep.expert_linear_backward(p, lay, x.to(DEV), w.to(DEV), y, dx=dx, dw=dw)
    torch.cuda.synchronize()
    yc = y.cpu()
    for e, (s, c) in enumerate(segs):
        if c == 0:
            assert (dw[e] == 0).all()
            continue
        want, ey, _, _ = forward64(x[s:s + c].double(), w[e].double(), "none", False)
        held(yc[s:s + c], want, ey, ("y", e))
        dz = yc[s:s + c].double()
        wx, ex, ww, ew = backward64(x[s:s + c].double(), w[e].double(), dz, dz * 0)
        held(dx[s:s + c], wx, ex, ("dx", e))
        held(dw[e], ww, ew, ("dw", e))


# more tiles than the chip holds at once, of every kind of tile: from one row an
# expert (32 channels x 16 rows) to segments of 256 x 256; short and long
# contractions, with and without a rest
WIDE = [
    (1, 1500, 2, 2, N, 0.1, 200, 1304),
    (1, 1500, 2, 2, N, 0.1, 200, 2600),
    (1, 1500, 2, 2, N, 0.1, 2600, 72),
    (2, 40, 64, 4, N, 0.0, 840, 328),
    (1, 60, 64, 4, L, 0.0, 264, 1032),
    (1, 300, 32, 4, N, 0.1, 328, 1032),
    (1, 260, 4, 2, N, 0.1, 2056, 1032),
    (1, 400, 16, 4, N, 0.1, 2056, 136),
    (1, 900, 4, 2, N, 0.1, 648, 1096),
]
WIDE_IDS = ["-".join(map(str, s)) for s in WIDE]


@pytest.mark.parametrize("shape", WIDE, ids=WIDE_IDS)
def test_wide_products(shape):
    test_gated(shape, "silu")
    test_linear(shape, "all")


@pytest.mark.parametrize("shape", WIDE, ids=WIDE_IDS)
def test_wide_gradients(shape):
    test_backward(shape, "gated", "gelu")
    test_backward(shape, "linear", "silu")


@pytest.mark.parametrize("quant", [ep.QUANT_FP8_F32, ep.QUANT_FP8_UE8M0])
@pytest.mark.parametrize("shape", [
    (1, 1500, 2, 2, N, 256, 1280),
    (2, 300, 8, 2, L, 512, 1152),
    (1, 40, 64, 4, N, 640, 384),
    (1, 256, 16, 4, N, 1664, 640),
    (1, 200, 64, 4, L, 384, 640),
    (1, 10, 64, 2, L, 2688, 256),
    (1, 1500, 1, 1, N, 1664, 1024),
], ids=lambda s: "-".join(map(str, s)))
def test_wide_fp8(shape, quant):
    test_fp8_rows_of_a_dispatch(shape, "gated", quant)
    test_fp8_rows_of_a_dispatch(shape, "linear", quant)
