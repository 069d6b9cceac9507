"""8-bit integer rows and products against plain forms: dispatch's and quantize_rows' codes
and scales bit for bit, the products' integer sums exactly in 64 bits.

The bounds.  The kernel's sum of integers is exact; its conversion to fp32 (four parts of
it where four waves share the contraction, and their three additions) and the products with
the two scales are eight roundings of at most 2^-24 of A = sum |q_x q_w| s_x s_w.  What
follows is as in expert_util: activations (4 + |z|) 2^-22 relative and 1.13 times the
argument's error, bias, gate and residual a rounding of 2^-24 each (2^-23 is allowed), one
rounding to bf16 (2^-8).

The lists are those of the bf16 tests with twice the channels, so with the same bytes a row,
and LONG; tests/test_int8_choice.py asks the library's own choice whether they take every tile
through every path of its loop."""
import numpy as np
import pytest
import torch

from combine_ep_get_layout_amd import ep
from expert_util import ACTS, HALF, LIPSCHITZ, TINY, ULP, act64, held, segments
from gpu_util import DEV, gpu_layout, say
import test_gpu_experts as base
import test_gpu_experts_tiles as tiles
from test_gpu_experts import L, M, N, NAN, INF, capacity, poisoned, rand, routed, rows_for, untouched

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -100


def quantised(x):
    """Codes (int8) and scales (fp32) of bf16 rows on the CPU, each step rounded to fp32."""
    v = x.float()
    amax = v.abs().amax(-1)
    fine = torch.isfinite(v).all(-1)
    scale = torch.clamp(amax, min=FLOOR) / torch.tensor(127.0)
    codes = torch.round(v / scale[:, None])
    codes[~fine] = 0
    return codes.to(torch.int8), torch.where(fine, scale, NAN)


def same_bits(got, want, what):
    assert torch.equal(got.cpu().contiguous().view(torch.uint8),
                       want.contiguous().view(torch.uint8)), what


def int8_rows(gen, p, segs, channels):
    """Codes over the whole range with some rows' scales, poison around the segments."""
    codes = torch.full((capacity(p), channels), -128, dtype=torch.int8)
    scales = torch.full((capacity(p),), NAN)
    for s, c in segs:
        codes[s:s + c] = torch.randint(-127, 128, (c, channels), generator=gen, dtype=torch.int8)
        scales[s:s + c] = torch.rand(c, generator=gen) * 0.02 + 1e-3
    return codes, scales


def int8_weights(gen, e, n, c):
    w = torch.randint(-128, 128, (e, n, c), generator=gen, dtype=torch.int8)
    return w, (torch.rand((e, n), generator=gen) + 0.1) * c ** -0.5 * 0.01


def product64(codes, sx, w, sw):
    """z, and the bound on the error of the kernel's fp32 z."""
    f = sx.double()[:, None] * sw.double()
    q, v = codes.double(), w.double()
    return (q @ v.t()) * f, 8 * 2.0 ** -24 * (q.abs() @ v.abs().t()) * f + TINY


def forward8(codes, sx, w, sw, act, gated, bias=None, residual=None):
    z, ez = product64(codes, sx, w, sw)
    if bias is not None:
        z = z + bias
        ez = ez + ULP * (z.abs() + bias.abs())
    epre = ez + HALF * (z.abs() + ez) + TINY
    if gated:
        n = z.shape[1] // 2
        g, u, eg, eu = z[:, :n], z[:, n:], ez[:, :n], ez[:, n:]
        a, _ = act64(act, g)
        ea = LIPSCHITZ * eg + (4 + g.abs()) * 2.0 ** -22 * a.abs()
        y = a * u
        ey = ea * u.abs() + a.abs() * eu + ea * eu + ULP * y.abs()
    else:
        y, _ = act64(act, z)
        ey = LIPSCHITZ * ez + (4 + z.abs()) * 2.0 ** -22 * y.abs()
        if residual is not None:
            y = y + residual
            ey = ey + ULP * (y.abs() + residual.abs())
    return y, ey + HALF * (y.abs() + ey) + TINY, z, epre


# ---- codes ---------------------------------------------------------------------

DISPATCH = [  # R, T, H, E, K, mode, masked, align
    (1, 1, 16, 1, 1, N, 0.0, 1),
    (1, 1, 1024, 8, 8, L, 0.0, 1),
    (2, 9, 1040, 6, 3, N, 0.4, 4),
    (3, 20, 2048, 9, 2, L, 0.3, 1),
    (2, 33, 2064, 8, 8, N, 0.0, 64),
    (2, 5, 4112, 4, 4, N, 0.2, 1),
    (4, 40, 7168, 8, 2, L, 0.0, 1),
    (1, 7, 8208, 3, 2, N, 0.0, 1),
    (1, 6, 16400, 2, 1, L, 0.0, 1),
    (2, 4, 32768, 4, 2, N, 0.1, 1),
    (1, 3, 48, 64, 64, N, 0.1, 1),
    (2, 5200, 176, 16, 4, N, 0.1, 1),
]


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("case", DISPATCH, ids=["-".join(map(str, c)) for c in DISPATCH])
def test_dispatch(case, fused):
    R, T, H, E, K, mode, masked, align = case
    say("dispatch int8", case, fused)
    p, lay, topk = routed(R, T, E, K, mode, seed=31, masked=masked, H=H, quant=ep.QUANT_INT8,
                          align=align)
    gen = torch.Generator().manual_seed(31)
    x = rand(gen, R * T, H, scale=3.0)
    recv = ep.Recv(p, capacity(p))
    recv.x.fill_(0x5A)
    recv.scales.fill_(-7.0)
    if fused:
        lay = ep.Layout(p)
        tk = torch.from_numpy(np.ascontiguousarray(topk)).to(DEV)
        ep.dispatch_fused(p, tk, lay, x.to(DEV), recv, ep.workspace(p))
    else:
        ep.dispatch(p, lay, x.to(DEV), recv=recv)
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    codes, scales = quantised(x)
    want = torch.full((capacity(p), H), 0x5A, dtype=torch.int8)
    want_s = torch.full((capacity(p),), -7.0)
    pos = lay.send_pos.cpu().view(R * T, K).long()
    t, k = torch.nonzero(pos >= 0, as_tuple=True)
    want[pos[t, k]], want_s[pos[t, k]] = codes[t], scales[t]
    same_bits(recv.x, want, "codes")
    same_bits(recv.scales, want_s, "scales")


@pytest.mark.parametrize("mode", [N, L])
def test_dispatch_without_a_workspace(mode):
    R, T, H, E, K = 2, 33, 272, 8, 3
    p, lay, topk = routed(R, T, E, K, mode, seed=32, masked=0.1, H=H, quant=ep.QUANT_INT8)
    x = rand(torch.Generator().manual_seed(32), R * T, H)
    want = ep.Recv(p, capacity(p))
    got = ep.Recv(p, capacity(p))
    for r in (want, got):
        r.x.fill_(0x5A)
        r.scales.fill_(-7.0)
    ep.dispatch(p, lay, x.to(DEV), recv=want)
    lay = ep.Layout(p)
    tk = torch.from_numpy(np.ascontiguousarray(topk)).to(DEV)
    ep.dispatch_fused_noalloc(p, tk, lay, x.to(DEV), got)
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    same_bits(got.x, want.x.cpu(), "codes")
    same_bits(got.scales, want.scales.cpu(), "scales")


def special_rows(H):
    """Rows that quantisation can go wrong at, bf16."""
    x = torch.zeros((14, H), dtype=torch.bfloat16)
    x[1] = 1.0
    x[2, 5] = -0.0
    x[3, 0], x[3, 1] = 3.0e38, -3.0e38
    x[4, 2], x[4, 3] = 1e-38, 1e-40                       # below the floor
    x[5] = torch.arange(H) % 255 - 127                     # every code
    x[6] = torch.arange(H) % 255 / 2 - 63.5                # halves of 127/127 and ties
    x[6, 0] = 127
    x[7, 1] = NAN
    x[8, H - 1] = INF
    x[9, 0] = -INF
    x[10] = torch.linspace(-5, 5, H).to(torch.bfloat16)
    x[11, H - 1] = 2.0 ** -100
    x[12, 0], x[12, 1:] = 254.0, 1.0                       # quotients of one half: ties to even
    x[12, 1:H:2] = 3.0
    x[13] = -x[10]
    return x


@pytest.mark.parametrize("H", [16, 272, 1040, 2064, 4112, 8208, 16400])
def test_special_rows(H):
    """A NaN or infinity gives zeros and a NaN scale; ties go to the even code; rows of
    zeros and of values below the floor stay finite."""
    x = special_rows(H)
    T = x.shape[0]
    p = ep.Problem(1, T, H, 1, 1, quant=ep.QUANT_INT8)
    lay, _ = gpu_layout(p, np.zeros((1, T, 1), np.int32))
    recv = ep.Recv(p, T)
    ep.dispatch(p, lay, x.to(DEV), recv=recv)
    again, scales2 = torch.empty_like(recv.x), torch.empty_like(recv.scales)
    ep.quantize_rows(p, lay, x.to(DEV), again, scales2)
    torch.cuda.synchronize()
    codes, scales = quantised(x)
    assert torch.equal(recv.x.cpu(), codes)
    assert torch.equal(torch.isnan(recv.scales.cpu()), torch.isnan(scales))
    assert torch.equal(torch.nan_to_num(recv.scales.cpu()), torch.nan_to_num(scales))
    same_bits(again, recv.x.cpu(), "quantize_rows")
    same_bits(scales2, recv.scales.cpu(), "quantize_rows")
    # and such a row's products are NaN, its neighbours' are not
    w = torch.ones((1, 8, H), dtype=torch.int8, device=DEV)
    y = poisoned(T, 8)
    ep.expert_linear(p, lay, recv.x, w, y, x_scales=recv.scales,
                     w_scales=torch.ones((1, 8), device=DEV))
    bad = torch.isnan(y.float()).all(1).cpu()
    assert bad.tolist() == torch.isnan(scales).tolist()
    assert torch.isfinite(y[~bad.to(DEV)].float()).all()


@pytest.mark.parametrize("shape", [s for s in base.SHAPES] + [
    (2, 33, 64, 4, N, 0.0, 4104, 8), (1, 9, 3, 1, L, 0.0, 16384, 8),
    (1, 4000, 5, 2, N, 0.1, 1032, 8)], ids=lambda s: "-".join(map(str, s)))
def test_quantize_rows(shape):
    R, T, E, K, mode, masked, C, _ = shape
    C *= 2
    say("quantize_rows", shape)
    p, lay, _ = routed(R, T, E, K, mode, seed=32, masked=masked)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(32)
    x = rows_for(gen, p, segs, C)
    q = torch.full((capacity(p), C), 0x5A, dtype=torch.int8, device=DEV)
    s = torch.full((capacity(p),), -7.0, device=DEV)
    ep.quantize_rows(p, lay, x.to(DEV), q, s)
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    want = torch.full((capacity(p), C), 0x5A, dtype=torch.int8)
    want_s = torch.full((capacity(p),), -7.0)
    for at, c in segs:
        want[at:at + c], want_s[at:at + c] = quantised(x[at:at + c])
    same_bits(q, want, "codes")
    same_bits(s, want_s, "scales")


# ---- products ------------------------------------------------------------------

def doubled(shapes):
    return [(*s[:6], 2 * s[6], s[7]) for s in shapes]


def name(shape):
    return "-".join(map(str, shape))


def check_gated(shape, act, seed=3):
    R, T, E, K, mode, masked, C, I = shape
    p, lay, _ = routed(R, T, E, K, mode, seed=seed, masked=masked)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(33)
    x, sx = int8_rows(gen, p, segs, C)
    w, sw = int8_weights(gen, E, 2 * I, C)
    h, pre = poisoned(capacity(p), I), poisoned(capacity(p), 2 * I)
    kw = dict(act=ACTS[act], x_scales=sx.to(DEV), w_scales=sw.to(DEV))
    ep.expert_gated(p, lay, x.to(DEV), w.to(DEV), h, pre=pre, **kw)
    h2 = poisoned(capacity(p), I)
    ep.expert_gated(p, lay, x.to(DEV), w.to(DEV), h2, **kw)
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    for e, (s, c) in enumerate(segs):
        y, ey, z, ez = forward8(x[s:s + c], sx[s:s + c], w[e], sw[e], act, True)
        held(h[s:s + c], y, ey, ("h", e))
        held(pre[s:s + c], z, ez, ("pre", e))
    untouched(h, segs, 0x5A5A)
    untouched(pre, segs, 0x5A5A)
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))


def check_linear(shape, extras, seed=4):
    R, T, E, K, mode, masked, C, O = shape
    p, lay, _ = routed(R, T, E, K, mode, seed=seed, masked=masked)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(34)
    act = {"plain": "none", "bias": "gelu", "residual": "relu", "all": "silu",
           "in_place": "none"}[extras]
    x, sx = int8_rows(gen, p, segs, C)
    w, sw = int8_weights(gen, E, O, C)
    bias = torch.randn((E, O), generator=gen) if extras in ("bias", "all") else None
    res = rows_for(gen, p, segs, O) if extras in ("residual", "all", "in_place") else None
    y = res.to(DEV) if extras == "in_place" else poisoned(capacity(p), O)
    pre = poisoned(capacity(p), O) if extras == "all" else None
    ep.expert_linear(p, lay, x.to(DEV), w.to(DEV), y, act=ACTS[act], x_scales=sx.to(DEV),
                     w_scales=sw.to(DEV), bias=None if bias is None else bias.to(DEV), pre=pre,
                     residual=y if extras == "in_place" else None if res is None else res.to(DEV))
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    for e, (s, c) in enumerate(segs):
        want, ey, z, ez = forward8(x[s:s + c], sx[s:s + c], w[e], sw[e], act, False,
                                   None if bias is None else bias[e].double(),
                                   None if res is None else res[s:s + c].double())
        held(y[s:s + c], want, ey, ("y", e))
        if pre is not None:
            held(pre[s:s + c], z, ez, ("pre", e))
    if extras != "in_place":
        untouched(y, segs, 0x5A5A)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
@pytest.mark.parametrize("shape", doubled(base.SHAPES), ids=name)
def test_gated(shape, act):
    say("gated int8", shape, act)
    check_gated(shape, act)


@pytest.mark.parametrize("extras", ["plain", "bias", "residual", "all", "in_place"])
@pytest.mark.parametrize("shape", doubled(base.SHAPES), ids=name)
def test_linear(shape, extras):
    say("linear int8", shape, extras)
    check_linear(shape, extras)


# more tiles of the two largest kinds than run at once, of contractions that each is chosen
# for, with and without a rest; and many experts of one tile
LONG = [
    (1, 9000, 28, 4, N, 0.0, 2064, 272),
    (1, 9000, 28, 4, N, 0.0, 2048, 272),
    (1, 9000, 28, 4, N, 0.0, 4112, 272),
    (1, 9000, 28, 4, N, 0.0, 4224, 272),
    (1, 300, 96, 8, N, 0.0, 1296, 1032),
    (1, 40, 96, 2, L, 0.0, 2320, 2056),
    (1, 250, 24, 4, N, 0.0, 1312, 1304),
    (1, 250, 24, 1, N, 0.0, 256, 1760),
    (1, 12, 16, 2, N, 0.0, 1888, 584),
    (1, 64, 64, 2, N, 0.0, 1824, 296),
]


@pytest.mark.parametrize("shape", doubled(base.WIDE + tiles.BF16) + LONG, ids=name)
def test_wide(shape):
    say("wide int8", shape)
    check_gated(shape, "silu")
    check_linear(shape, "all")


def test_channels_of_one_vector():
    """16 channels, and an odd number of 16-byte vectors in every row."""
    for shape in ((1, 5, 2, 1, N, 0.0, 16, 8), (2, 40, 3 * 2, 2, L, 0.1, 48, 40),
                  (1, 700, 2, 1, N, 0.0, 1808, 328)):
        check_gated(shape, "silu")
        check_linear(shape, "residual")


def test_the_largest_sums_are_exact():
    """32,768 channels of -128 times -128: 2^29, and one less in the last place of the row."""
    C = 32768
    p = ep.Problem(1, 3, 128, 1, 1)
    lay, _ = gpu_layout(p, np.zeros((1, 3, 1), np.int32))
    x = torch.full((3, C), -128, dtype=torch.int8)
    x[1] = 127
    x[2, ::2] = 127
    w = torch.full((1, 8, C), -128, dtype=torch.int8)
    y = poisoned(3, 8)
    ep.expert_linear(p, lay, x.to(DEV), w.to(DEV), y, x_scales=torch.ones(3, device=DEV),
                     w_scales=torch.ones((1, 8), device=DEV))
    want = (x.double() @ w[0].double().t()).to(torch.bfloat16)
    assert torch.equal(y.cpu(), want)


# ---- errors, layouts, together --------------------------------------------------

def test_capacity_is_reported_and_kept():
    p, lay, topk = routed(2, 70, 4, 2, N, seed=35, quant=ep.QUANT_INT8, H=64)
    segs = segments(p, lay)
    gen = torch.Generator().manual_seed(35)
    x = rand(gen, 140, 64)
    codes, scales = quantised(x)
    pos = lay.send_pos.cpu().view(140, 2).long()
    for short in (segs[2][0] + 3, 0):
        room = torch.full((capacity(p), 64), 0x5A, dtype=torch.int8, device=DEV)
        s = torch.full((capacity(p),), -7.0, device=DEV)
        recv = ep.Recv(p, short)
        recv.x, recv.scales = room[:short], s[:short]
        lay.err.zero_()
        ep.dispatch(p, lay, x.to(DEV), recv=recv)
        torch.cuda.synchronize()
        assert int(lay.err.item()) == ep.DEVERR_CAPACITY
        assert (room[short:] == 0x5A).all() and (s[short:] == -7.0).all()
        t, k = torch.nonzero(pos < short, as_tuple=True)
        assert torch.equal(room.cpu()[pos[t, k]], codes[t])
        # quantize_rows
        room.fill_(0x5A)
        s.fill_(-7.0)
        rows = rows_for(gen, p, segs, 64)
        lay.err.zero_()
        ep.quantize_rows(p, lay, rows.to(DEV), room[:short], s[:short])
        torch.cuda.synchronize()
        assert int(lay.err.item()) == ep.DEVERR_CAPACITY
        assert (room[short:] == 0x5A).all() and (s[short:] == -7.0).all()
        assert torch.equal(room[:short].cpu(), quantised(rows[:short])[0])


def test_no_tokens():
    for mode in (N, L):
        p = ep.Problem(2, 0, 64, 4, 2, mode=mode, quant=ep.QUANT_INT8)
        lay, _ = gpu_layout(p, np.zeros((2, 0, 2), np.int32))
        recv = ep.Recv(p, 0)
        ep.dispatch(p, lay, torch.zeros((2, 0, 64), dtype=torch.bfloat16, device=DEV), recv=recv)
        y = poisoned(1, 8)
        ep.expert_linear(p, lay, recv.x, torch.zeros((4, 8, 64), dtype=torch.int8, device=DEV),
                         y[:0], x_scales=recv.scales, w_scales=torch.zeros((4, 8), device=DEV))
        torch.cuda.synchronize()
        assert (y.view(torch.int16) == 0x5A5A).all()


def test_message_problem_quantises_the_blocks():
    """EP_MODE_MESSAGES: the low-latency blocks that ep_messages_unpack fills."""
    pl, lay, _ = routed(2, 30, 4, 2, L, seed=36)
    pm = ep.Problem(2, 30, 128, 4, 2, mode=M)
    gen = torch.Generator().manual_seed(36)
    segs = segments(pl, lay)
    x = rows_for(gen, pl, segs, 80).to(DEV)
    outs = []
    for p in (pl, pm):
        q = torch.full((capacity(pl), 80), 0x5A, dtype=torch.int8, device=DEV)
        s = torch.full((capacity(pl),), -7.0, device=DEV)
        ep.quantize_rows(p, lay, x, q, s)
        outs.append((q, s))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_rows_past_32_bit_offsets():
    """A low-latency buffer whose last block lies past 2^32 codes."""
    T, E, C, O = 16384, 36, 8208, 64
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB")
    p = ep.Problem(1, T, C, E, 1, mode=L, quant=ep.QUANT_INT8)
    topk = np.full((1, T, 1), -1, np.int32)
    topk[0, :700, 0] = E - 1
    topk[0, 700:705, 0] = 0
    lay, _ = gpu_layout(p, topk)
    cap = capacity(p)
    assert (cap - T) * C > 1 << 32
    gen = torch.Generator().manual_seed(37)
    x = rand(gen, T, C)
    recv = ep.Recv(p, cap)
    ep.dispatch(p, lay, x.to(DEV), recv=recv)
    w, sw = int8_weights(gen, E, O, C)
    y = poisoned(cap, O)
    ep.expert_linear(p, lay, recv.x, w.to(DEV), y, x_scales=recv.scales, w_scales=sw.to(DEV))
    torch.cuda.synchronize()
    segs = segments(p, lay)
    codes, scales = quantised(x)
    for e, rows in ((E - 1, slice(0, 700)), (0, slice(700, 705))):
        s, c = segs[e]
        assert torch.equal(recv.x[s:s + c].cpu(), codes[rows])
        want, ey, _, _ = forward8(codes[rows], scales[rows], w[e], sw[e], "none", False)
        held(y[s:s + c], want, ey, ("y", e))
    untouched(y, segs, 0x5A5A)


@pytest.mark.parametrize("rows", [3, 40, 600])
@pytest.mark.parametrize("gated", [False, True])
def test_scales_whose_product_is_no_normal_number(gated, rows):
    """A row's and a channel's scale whose product is subnormal, or an infinity: values that are
    normal numbers lose no more than elsewhere, and sums of 0 are 0.  The integer sum is rounded
    once to fp32 (in up to four parts, added) and once with either scale, the gate's likewise,
    their product once, and the result once to bf16."""
    C, I = 32768, 64
    p, lay, _ = routed(1, rows, 1, 1, N, seed=39, H=C, quant=ep.QUANT_INT8)
    x = torch.full((rows, C), 127, dtype=torch.int8)
    low = torch.arange(rows) % 3 != 1
    sx = torch.where(low, 2.0 ** -107, 2.0 ** 120)
    # channels 0 .. 31: times 2^-107 below the smallest subnormal number, or a few of them;
    # sums of 2^29, so values of 2^-119.  From 32 on: sums of 0, times 2^120 an infinity
    w = torch.full((1, I, C), 127, dtype=torch.int8)
    sw = 2.0 ** -41 * (1 + (torch.arange(I) % 32) / 37.0)
    sw[:16] /= 4
    w[0, 32:], sw[32:] = 0, 2.0 ** 12
    z = (x[:1].double() @ w[0].double().t()) * sw.double() * sx.double()[:, None]
    other = torch.ones_like(z)
    y = poisoned(rows, I)
    kw = dict(act=ep.ACT_NONE, x_scales=sx.to(DEV))
    if gated:
        # the other factor near 1 in the rows that each channel is for; gates and ups by turns
        v = torch.full((1, I, C), 127, dtype=torch.int8)
        sv = torch.full((I,), 2.0 ** 78)
        sv[32:] = 2.0 ** -149
        other = (x[:1].double() @ v[0].double().t()) * sv.double() * sx.double()[:, None]
        turn = torch.arange(I) % 2 == 0
        gates, ups = torch.where(turn[:, None], w, v), torch.where(turn[:, None], v, w)
        scales = torch.cat([torch.where(turn, sw, sv), torch.where(turn, sv, sw)])
        ep.expert_gated(p, lay, x.to(DEV), torch.cat([gates, ups], 1).to(DEV), y,
                        w_scales=scales[None].to(DEV), **kw)
    else:
        ep.expert_linear(p, lay, x.to(DEV), w.to(DEV), y, w_scales=sw[None].to(DEV), **kw)
    torch.cuda.synchronize()
    want, got = (z * other)[low, :32], y.double().cpu()
    assert (want.abs() > 2.0 ** -124).all()
    assert ((got[low, :32] - want).abs() <= (HALF * (1 + HALF) + 20 * 2.0 ** -24) * want.abs()).all()
    assert (got[~low, 32:] == 0).all() and (gated or (got[low, 32:] == 0).all())


@pytest.mark.parametrize("mode", [N, L])
def test_whole_layer_and_its_replays(mode):
    """layout -> dispatch -> gated -> quantize_rows -> linear -> combine in 8-bit integers,
    eager and replayed in a graph with fresh inputs, eager work in between.  Against the
    formula on the kernel's own intermediate codes, each step by its bound."""
    R, T, E, K, H, I = 2, 90, 8, 3, 272, 144
    p, lay, topk = routed(R, T, E, K, mode, seed=38, masked=0.1, H=H, quant=ep.QUANT_INT8)
    segs, cap, n = segments(p, lay), capacity(p), R * T
    gen = torch.Generator().manual_seed(38)
    w1, s1 = int8_weights(gen, E, 2 * I, H)
    w2, s2 = int8_weights(gen, E, H, I)
    s1, s2 = s1 * 5, s2 * 5
    dev = [v.to(DEV) for v in (w1, s1, w2, s2)]
    wt = torch.softmax(torch.randn((n, K), generator=gen), -1)
    wtg, x = wt.to(DEV), torch.empty((n, H), dtype=torch.bfloat16, device=DEV)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    recv, ws = ep.Recv(p, cap), ep.workspace(p)
    h, y, out = torch.empty((cap, I), **bf), torch.empty((cap, H), **bf), torch.empty((n, H), **bf)
    q, qs = torch.empty((cap, I), dtype=torch.int8, device=DEV), torch.empty(cap, device=DEV)
    tk = torch.from_numpy(np.ascontiguousarray(topk)).to(DEV)

    def step():
        ep.get_layout(p, tk, lay, ws)
        ep.dispatch(p, lay, x, recv=recv)
        ep.expert_gated(p, lay, recv.x, dev[0], h, x_scales=recv.scales, w_scales=dev[1])
        ep.quantize_rows(p, lay, h, q, qs)
        ep.expert_linear(p, lay, q, dev[2], y, x_scales=qs, w_scales=dev[3])
        ep.combine(p, lay, y, wtg, out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x.copy_(rand(gen, n, H))
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    pos = lay.send_pos.cpu().view(n, K).long()
    for rep in range(4):
        xh = rand(gen, n, H)
        x.copy_(xh)
        step()
        torch.cuda.synchronize()
        eager = out.clone()
        codes, scales = quantised(xh)
        hc, qc, qsc, yc = h.cpu(), q.cpu(), qs.cpu(), y.cpu()
        tok = torch.zeros(cap, dtype=torch.long)
        t, k = torch.nonzero(pos >= 0, as_tuple=True)
        tok[pos[t, k]] = t
        for e, (s, c) in enumerate(segs):
            rows = tok[s:s + c]
            want, ey, _, _ = forward8(codes[rows], scales[rows], w1[e], s1[e], "silu", True)
            held(hc[s:s + c], want, ey, ("h", e))
            cq, cs = quantised(hc[s:s + c])
            assert torch.equal(qc[s:s + c], cq) and torch.equal(qsc[s:s + c], cs)
            want, ey, _, _ = forward8(cq, cs, w2[e], s2[e], "none", False)
            held(yc[s:s + c], want, ey, ("y", e))
        each = torch.where((pos >= 0)[:, :, None], yc[pos.clamp(min=0)].double(), 0.0)
        each = each * wt.double()[:, :, None]
        want = each.sum(1)
        held(out, want, HALF * want.abs() * (1 + HALF) + (K + 1) * ULP * each.abs().sum(1) + TINY,
             "out")
        for v in (out, h, y):
            v.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
