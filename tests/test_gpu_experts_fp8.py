"""FP8 results that are not finite: a NaN or infinity becomes the NaN code where it
stands, its group's scale is that of the other values, and everything else is as without
it."""
import pytest
import torch

from combine_ep_get_layout_amd import ep
from expert_util import fp8_weights, segments
from gpu_util import DEV, say
from test_gpu_experts import INF, NAN, L, N, capacity, poisoned, rand, routed

pytestmark = pytest.mark.gpu

QUANTS = [ep.QUANT_FP8_F32, ep.QUANT_FP8_UE8M0]
# rows an expert for the 256 x 64 and the 256 x 128 tile, whole and cut
SHAPES = [(2, 9, 4, 2, L, 256, 384), (1, 300, 2, 1, N, 384, 256), (1, 1500, 2, 2, N, 256, 1280)]


def fp8_out(p, groups, quant):
    codes = torch.full((capacity(p), groups * 128), 0x55, dtype=torch.uint8, device=DEV)
    n = groups * capacity(p)
    scales = (torch.zeros(n, device=DEV) if quant == ep.QUANT_FP8_F32
              else torch.zeros(n, dtype=torch.uint8, device=DEV))
    return codes, scales


def made(shape, seed):
    R, T, E, K, mode, C, I = shape
    p, lay, _ = routed(R, T, E, K, mode, seed=seed, quant=ep.QUANT_FP8_F32, H=C)
    gen = torch.Generator().manual_seed(seed)
    recv = ep.Recv(p, capacity(p))
    ep.dispatch(p, lay, rand(gen, R * T, C).to(DEV), recv=recv, ws=ep.workspace(p))
    return p, lay, segments(p, lay), gen, recv


@pytest.mark.parametrize("quant", QUANTS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_single_values(shape, quant):
    """A residual of NaN and +-infinity in single places, the smallest of their groups in
    size, so that the scales of the call without them hold."""
    say("single", shape, quant)
    E, C, I = shape[2], *shape[5:]
    p, lay, segs, gen, recv = made(shape, 41)
    wc, ws, _ = fp8_weights(gen, E, I, C)
    res = rand(gen, capacity(p), I).to(DEV)
    kw = dict(x_scales=recv.scales, w_scales=ws)
    codes0, scales0 = fp8_out(p, I // 128, quant)
    ep.expert_linear(p, lay, recv.x, wc, codes0, residual=res, y_scales=scales0, **kw)
    torch.cuda.synchronize()
    size = (codes0.cpu() & 0x7F).view(-1, I // 128, 128)
    hit = []
    for s, c in segs:
        for r in {s, s + c // 2, s + c - 1} if c else ():
            for g in range(I // 128):
                at = size[r, g].argsort()[:3]  # the group's smallest
                hit += [(r, g * 128 + int(at[i])) for i in range(3)]
    assert len(hit) > 20
    bad = res.clone()
    for i, (r, ch) in enumerate(hit):
        bad[r, ch] = (NAN, INF, -INF)[i % 3]
    codes, scales = fp8_out(p, I // 128, quant)
    ep.expert_linear(p, lay, recv.x, wc, codes, residual=bad, y_scales=scales, **kw)
    torch.cuda.synchronize()
    want = codes0.clone()
    for r, ch in hit:
        want[r, ch] = 0x7F
    assert torch.equal(codes, want)
    assert torch.equal(scales, scales0)


@pytest.mark.parametrize("quant", QUANTS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_a_row_through_two_products(shape, quant):
    """NaN codes in one row of x: the row's FP8 result is all NaN codes with the scale of
    zeros, the next product's row is NaN, and all other rows are as without them."""
    say("row", shape, quant)
    E, C, I = shape[2], *shape[5:]
    p, lay, segs, gen, recv = made(shape, 42)
    w1, s1, _ = fp8_weights(gen, E, 2 * I, C)
    w2, s2, _ = fp8_weights(gen, E, 128, I)
    s, c = max(segs, key=lambda v: v[1])
    row = s + c // 2
    out = []
    for diverged in False, True:
        x = recv.x.clone()
        if diverged:
            x[row, 5] = 0x7F
        h, hs = fp8_out(p, I // 128, quant)
        y = poisoned(capacity(p), 128)
        ep.expert_gated(p, lay, x, w1, h, x_scales=recv.scales, w_scales=s1, h_scales=hs)
        ep.expert_linear(p, lay, h, w2, y, x_scales=hs, w_scales=s2)
        torch.cuda.synchronize()
        out.append((h, hs, y))
    assert int(lay.err.item()) == 0
    (h0, hs0, y0), (h1, hs1, y1) = out
    assert (h1[row] == 0x7F).all() and torch.isnan(y1[row].float()).all()
    if quant == ep.QUANT_FP8_F32:  # 1e-4 / 448, the floor of a group's scale
        floor = (torch.tensor(1e-4) / 448).item()
    else:
        floor = 127 - 22           # the power of two above it: 1e-4 / 448 = 2^-22.1
    if p.mode == ep.MODE_NORMAL:
        a, b = (v.view(I // 128, -1)[:, row] for v in (hs0, hs1))
    else:
        n = p.R * p.T
        a, b = (v.view(E, I // 128, n)[row // n, :, row % n] for v in (hs0, hs1))
    assert (b == floor).all()
    b.copy_(a)
    h1[row], y1[row] = h0[row], y0[row]
    assert torch.equal(h0, h1) and torch.equal(hs0, hs1)
    assert torch.equal(y0.view(torch.int16), y1.view(torch.int16))
