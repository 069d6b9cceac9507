"""The layer for a few tokens against a plain 64-bit form, for every type of weights: one
entry to the largest number, an expert's rows from one to many tiles, contractions with and
without a rest, experts without a row and ids that name none.

The bounds.  h as in expert_util.forward64 (sums of H products in fp32, an FP8 or 8-bit sum's
scale among the eight more, one rounding to bf16).  The second product takes the h that the
call leaves in its workspace: (I + 8) 2^-23 of the magnitudes for the sums and scales, 2^-23
for each of up to K weighted additions, and a rounding of 2^-8."""
import numpy as np
import pytest
import torch

from combine_ep_get_layout_amd import ep, inputs
from expert_util import ACTS, HALF, TINY, ULP, forward64, fp8_weights, held
from gpu_util import DEV, say
from test_gpu_experts import INF, NAN, poisoned, rand, relative

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp8", "int8"]


def weights_of(gen, kind, E, n, c):
    """(tensor on the GPU, scales or None, values in 64 bits)."""
    if kind == "bf16":
        w = rand(gen, E, n, c, scale=c ** -0.5)
        return w.to(DEV), None, w.double()
    if kind == "fp8":
        return fp8_weights(gen, E, n, c)
    w = torch.randint(-128, 128, (E, n, c), generator=gen, dtype=torch.int8)
    s = (torch.rand((E, n), generator=gen) + 0.5) * c ** -0.5 / 74
    return w.to(DEV), s.to(DEV), w.double() * s.double()[:, :, None]


def routing(R, T, E, K, masked, seed, dup=0.0, only=None):
    w = inputs.small("layer", R=R, T=T, H=128, E=E, K=K, seed=seed)
    topk = inputs.gen_topk(w)
    if masked or dup:
        topk = inputs.masked_topk(w, topk, masked, dup, seed=seed)
    if only is not None:
        topk = np.where(np.arange(K) == 0, only, -1).astype(np.int32) * np.ones_like(topk)
    return torch.from_numpy(np.ascontiguousarray(topk, np.int32)).view(R * T, K)


class Made:
    """A layer's operands, and its call."""

    def __init__(self, R, T, E, K, H, I, kind, topk, seed=61, act="silu"):
        gen = torch.Generator().manual_seed(seed)
        self.p, self.act, self.I = ep.Problem(R, T, H, E, K), act, I
        self.n, self.topk = R * T, topk
        self.x = rand(gen, self.n, H)
        self.wt = torch.softmax(torch.randn((self.n, K), generator=gen), -1)
        self.w13, self.s13, self.v13 = weights_of(gen, kind, E, 2 * I, H)
        self.w2, self.s2, self.v2 = weights_of(gen, kind, E, H, I)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = ep.layer_workspace(self.p, I)
        self.ws.fill_(0xFF)  # NaN

    def call(self, x=None, topk=None, wt=None, out=None, **kw):
        out = poisoned(self.n, self.p.H) if out is None else out
        ep.expert_layer(self.p, (self.x if x is None else x).to(DEV),
                        (self.topk if topk is None else topk).to(DEV),
                        (self.wt if wt is None else wt).to(DEV), self.w13, self.w2, out, self.err,
                        self.ws, act=ACTS[self.act], w13_scales=self.s13, w2_scales=self.s2, **kw)
        return out

    def check(self, out, x=None, topk=None, wt=None):
        x, topk, wt = (a if a is not None else b for a, b in
                       ((x, self.x), (topk, self.topk), (wt, self.wt)))
        n, K, H, I, E = self.n, self.p.K, self.p.H, self.I, self.p.E
        h = self.ws[:n * K * I * 4].view(torch.bfloat16).view(n * K, 2, I).cpu().double().sum(1)
        y, ey = torch.zeros((n, K, H), dtype=torch.float64), torch.zeros((n, K, H)).double()
        flat = topk.reshape(-1)
        ok = (flat >= 0) & (flat < E)
        for e in flat[ok].unique().tolist():
            at = torch.nonzero(flat == e).view(-1)
            want, eh, _, _ = forward64(x[at // K].double(), self.v13[e], self.act, True)
            # without its rounding to bf16 (half a step), with that of what it leaves
            eh = (eh - TINY - HALF * want.abs()) / (1 + HALF)
            held(h[at], want, eh + HALF * HALF * (want.abs() + eh) + TINY, ("h", e))
            h64 = h[at]
            y.view(-1, H)[at] = h64 @ self.v2[e].t()
            ey.view(-1, H)[at] = (I + 8) * ULP * (h64.abs() @ self.v2[e].abs().t())
        w = torch.where(ok.view(n, K), wt, 0.0).double()[:, :, None]
        want = (w * y).sum(1)
        bound = (w.abs() * ey).sum(1) + (K + 1) * ULP * (w * y).abs().sum(1)
        held(out, want, bound + HALF * (want.abs() + bound) + TINY, "out")
        return want


# R, T, E, K, H, I, masked: entries a row and a tile; 8 bf16 channels and up
SHAPES = [
    (1, 1, 1, 1, 8, 8, 0.0),
    (1, 1, 8, 8, 64, 24, 0.0),
    (1, 1, 64, 2, 2048, 768, 0.0),
    (2, 2, 4, 2, 72, 40, 0.0),
    (3, 7, 9, 3, 264, 136, 0.1),
    (1, 17, 2, 1, 1032, 72, 0.0),
    (1, 33, 2, 2, 136, 1032, 0.2),
    (2, 20, 64, 6, 328, 200, 0.0),
    (1, 64, 4, 2, 520, 264, 0.0),
    (8, 8, 256, 8, 200, 104, 0.0),
    (1, 128, 8, 8, 96, 64, 0.1),
    (1, 1000, 3, 1, 48, 32, 0.0),
    (4, 4, 2048, 64, 80, 48, 0.3),
]


# many entries an expert, whose rows workgroups share: rows of whole 4 KiB in either product
# (lines then begin at different places), channels that end inside a strip and a group of them,
# chunks of one entry, in tiles of 16 (32) rows and of 64, of one strip a wave and of two
MANY = [
    (1, 130, 2, 1, 4096, 264, 0.0),
    (2, 65, 2, 1, 264, 4096, 0.0),
    (1, 24, 32, 6, 2048, 520, 0.0),
    (1, 129, 1, 1, 72, 40, 0.0),
    (4, 256, 4, 1, 264, 1032, 0.1),
    (1, 96, 16, 2, 200, 1096, 0.0),
    (1, 200, 6, 5, 1032, 520, 0.4),
    (1, 16, 64, 64, 136, 200, 0.0),
]


# few entries of experts with many channels, whose strips waves take alone, several of them one
# after the other; slots of 8 entries in the second product; 8 to 32 entries an expert with rows
# in common and many channels to give (tests/test_layer_choice.py asks the library's own choice
# which kernels all these lists run)
FORMS = [
    (1, 3, 24, 8, 72, 1032, 0.0),
    (1, 3, 24, 8, 1032, 1096, 0.0),
    (1, 2, 16, 8, 200, 4136, 0.0),
    (1, 1, 8, 8, 136, 8200, 0.1),
    (1, 9, 8, 4, 264, 72, 0.0),
    (1, 20, 5, 1, 136, 1032, 0.1),
    (1, 128, 16, 2, 4096, 136, 0.0),
    (1, 100, 12, 3, 2824, 200, 0.2),
]


def sized(shape, kind):
    """The shape with channels that the type has: 128 in FP8, 16 in 8-bit integers."""
    step = {"bf16": 8, "fp8": 128, "int8": 16}[kind]
    *a, H, I, masked = shape
    up = lambda c: -(-c // step) * step  # noqa: E731
    return (*a, up(H), up(I), masked)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES + MANY, ids=lambda s: "-".join(map(str, s)))
def test_layer(shape, kind):
    R, T, E, K, H, I, masked = sized(shape, kind)
    say("layer", shape, kind)
    m = Made(R, T, E, K, H, I, kind, routing(R, T, E, K, masked, 61))
    out = m.call()
    torch.cuda.synchronize()
    want = m.check(out)
    assert int(m.err.item()) == 0
    again = m.call()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    if want.numel() > 4096:
        # against the formula: one rounding, at most half a step and over many values sqrt(1/3)
        # of that, doubled
        ok = m.topk >= 0
        full = torch.zeros_like(want)
        for e in m.topk[ok].unique().tolist():
            t, k = torch.nonzero(m.topk == e, as_tuple=True)
            z = m.x[t].double() @ m.v13[e].t()
            y = (torch.nn.functional.silu(z[:, :I]) * z[:, I:]) @ m.v2[e].t()
            full.index_add_(0, t, y * m.wt[t, k].double()[:, None])
        assert relative([out], [full]) <= 2 * (1 / 3) ** 0.5 * HALF


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", FORMS, ids=lambda s: "-".join(map(str, s)))
def test_every_form(shape, kind):
    test_layer(shape, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_strips_of_a_wave_alone_with_several_slots(kind):
    """Two experts have all entries, more than a slot holds, of a size whose strips waves take
    alone: they go over a strip's weights again for the rest of the entries."""
    R, T, E, K, H, I, _ = sized((1, 24, 24, 1, 200, 1032, 0.0), kind)
    topk = torch.tensor([3, 5, 3, 3, 5, 3] * 4, dtype=torch.int32)[:, None]
    m = Made(R, T, E, K, H, I, kind, topk)
    out = m.call()
    torch.cuda.synchronize()
    m.check(out)
    assert int(m.err.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("act", ["gelu", "relu", "none"])
def test_activations(act, kind):
    R, T, E, K, H, I, masked = sized((3, 7, 9, 3, 264, 136, 0.1), kind)
    m = Made(R, T, E, K, H, I, kind, routing(R, T, E, K, masked, 62), act=act)
    out = m.call()
    torch.cuda.synchronize()
    m.check(out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 15, 16, 17, 32, 33, 48, 49, 64, 65, 129, 512, 1024])
def test_every_token_to_one_expert(n, kind):
    """One expert's rows: every number of tiles, and several rounds of them."""
    R, T, E, K, H, I, _ = sized((1, n, 5, 1, 144, 80, 0.0), kind)
    m = Made(R, T, E, K, H, I, kind, routing(R, T, E, K, 0.0, 63, only=3))
    out = m.call()
    torch.cuda.synchronize()
    m.check(out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("c", [1, 2, 3, 5, 8, 9, 15, 17, 31, 64, 127, 129])
def test_contractions(c, kind):
    """Contractions of every number of lines and every rest: c times the type's step."""
    step = {"bf16": 24, "fp8": 128, "int8": 48}[kind]
    m = Made(2, 3, 6, 2, c * step, 128, kind, routing(2, 3, 6, 2, 0.0, 64))
    out = m.call()
    m2 = Made(2, 3, 6, 2, 128, c * step, kind, routing(2, 3, 6, 2, 0.0, 65))
    out2 = m2.call()
    torch.cuda.synchronize()
    m.check(out)
    m2.check(out2)


@pytest.mark.parametrize("kind", KINDS)
def test_one_expert_twice(kind):
    """An expert that several entries of a token name gives each its weight."""
    R, T, E, K, H, I, _ = sized((1, 18, 3, 5, 136, 72, 0.0), kind)
    gen = torch.Generator().manual_seed(66)
    topk = torch.randint(-1, E, (R * T, K), generator=gen, dtype=torch.int32)
    m = Made(R, T, E, K, H, I, kind, topk)
    out = m.call()
    torch.cuda.synchronize()
    m.check(out)


@pytest.mark.parametrize("kind", KINDS)
def test_ids_of_no_expert(kind):
    """-1 entries with weights that are no numbers, tokens without any, ids out of range."""
    R, T, E, K, H, I, _ = sized((1, 6, 4, 3, 72, 40, 0.0), kind)
    topk = torch.tensor([[-1, -1, -1], [0, -1, 3], [-1, 2, -1], [1, 1, -1], [-1, -1, 0],
                         [3, 2, 1]], dtype=torch.int32)
    m = Made(R, T, E, K, H, I, kind, topk)
    m.wt[topk < 0] = NAN
    out = m.call()
    torch.cuda.synchronize()
    assert int(m.err.item()) == 0
    m.check(out)
    assert (out[0] == 0).all()
    bad = topk.clone()
    bad[0, 1], bad[4, 0], bad[5, 2] = 4, -2, 1 << 30
    out = m.call(topk=bad)
    torch.cuda.synchronize()
    assert int(m.err.item()) == ep.DEVERR_TOPK_RANGE
    bad[(bad < -1) | (bad >= E)] = -1
    m.check(out, topk=bad, wt=torch.where(bad < 0, 0.0, m.wt))
    out = m.call(topk=torch.full_like(topk, -1))
    torch.cuda.synchronize()
    assert (out == 0).all()


def test_no_tokens():
    p = ep.Problem(2, 0, 64, 4, 2)
    e = lambda *s, **k: torch.zeros(s, device=DEV, **k)  # noqa: E731
    b = dict(dtype=torch.bfloat16)
    ep.expert_layer(p, e(2, 0, 64, **b), e(2, 0, 2, dtype=torch.int32), e(2, 0, 2),
                    e(4, 32, 64, **b), e(4, 64, 16, **b), e(2, 0, 64, **b), None,
                    ep.layer_workspace(p, 16))
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", KINDS)
def test_ids_of_no_expert_among_many(kind):
    """The same where workgroups share rows: ids out of range, tokens without any, no token
    with any."""
    R, T, E, K, H, I, masked = sized((1, 150, 9, 2, 72, 40, 0.2), kind)
    topk = routing(R, T, E, K, masked, 76)
    m = Made(R, T, E, K, H, I, kind, topk)
    m.wt[topk < 0] = NAN
    bad = topk.clone()
    bad[3, 1], bad[149, 0], bad[77, 1], bad[78] = E, -2, 1 << 30, -1
    out = m.call(topk=bad)
    torch.cuda.synchronize()
    assert int(m.err.item()) == ep.DEVERR_TOPK_RANGE
    bad[(bad < -1) | (bad >= E)] = -1
    m.check(out, topk=bad, wt=torch.where(bad < 0, 0.0, m.wt))
    assert (out[78] == 0).all()
    out = m.call(topk=torch.full_like(topk, -1))
    torch.cuda.synchronize()
    assert (out == 0).all()


@pytest.mark.parametrize("T", [40, 140])
@pytest.mark.parametrize("kind", KINDS)
def test_special_values_stay_in_their_tokens(kind, T):
    """An infinity or NaN in one token's row, or in the weights of one expert, reaches the
    tokens that have it and no others."""
    R, T, E, K, H, I, _ = sized((1, T, 6, 2, 264, 72, 0.0), kind)
    topk = routing(R, T, E, K, 0.0, 67)
    m = Made(R, T, E, K, H, I, kind, topk)
    clean = m.call()
    x = m.x.clone()
    x[7, 3], x[21, 5] = INF, NAN
    out = m.call(x=x)
    torch.cuda.synchronize()
    assert torch.isnan(out[21].float()).all() and not torch.isfinite(out[7].float()).any()
    keep = torch.ones(T, dtype=torch.bool)
    keep[7] = keep[21] = False
    assert torch.equal(out[keep].view(torch.int16), clean[keep].view(torch.int16))
    has = (topk == 2).any(1)
    if kind == "bf16":
        m.w2[2, 5, 1] = INF
    elif kind == "fp8":
        m.w2[2, 5, 1] = 0x7F
    else:
        m.s2[2, 5] = NAN
    out = m.call()
    torch.cuda.synchronize()
    assert not torch.isfinite(out[has][:, 5].float()).any()
    assert torch.equal(out[~has].view(torch.int16), clean[~has].view(torch.int16))
    other = torch.arange(H) != 5
    assert torch.equal(out[:, other].view(torch.int16), clean[:, other].view(torch.int16))


def test_weights_past_32_bit_offsets():
    """Experts whose weights lie past 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    E, H, I = 96, 7168, 2048
    gen = torch.Generator().manual_seed(68)
    p = ep.Problem(1, 2, H, E, 2)
    topk = torch.tensor([[95, 0], [94, 95]], dtype=torch.int32)
    x, wt = rand(gen, 2, H), torch.rand((2, 2), generator=gen)
    w13 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device=DEV)
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device=DEV)
    v = {}
    for e in (0, 94, 95):
        v[e] = (rand(gen, 2 * I, H, scale=H ** -0.5), rand(gen, H, I, scale=I ** -0.5))
        w13[e], w2[e] = v[e][0].to(DEV), v[e][1].to(DEV)
    assert w13[95].storage_offset() * 2 > 1 << 32 and w2[94].storage_offset() * 2 > 1 << 31
    out = poisoned(2, H)
    ep.expert_layer(p, x.to(DEV), topk.to(DEV), wt.to(DEV), w13, w2, out, None,
                    ep.layer_workspace(p, I))
    torch.cuda.synchronize()
    want = torch.zeros((2, H), dtype=torch.float64)
    for t in range(2):
        for k in range(2):
            a, b = v[int(topk[t, k])]
            z = x[t].double() @ a.double().t()
            h = torch.nn.functional.silu(z[:I]) * z[I:]
            want[t] += float(wt[t, k]) * (h @ b.double().t())
    assert relative([out], [want]) <= 2 * (1 / 3) ** 0.5 * HALF


# ---- together ---------------------------------------------------------------------

@pytest.mark.parametrize("T", [24, 100])
@pytest.mark.parametrize("kind", KINDS)
def test_routed_and_replayed_in_a_graph(kind, T):
    """route and expert_layer captured together, replayed with fresh rows and logits, eager
    work of the same buffers in between; every replay equals the eager run bit for bit."""
    R, T, E, K, H, I, _ = sized((1, T, 16, 4, 256, 128, 0.0), kind)
    m = Made(R, T, E, K, H, I, kind, routing(R, T, E, K, 0.0, 69))
    gen = torch.Generator().manual_seed(69)
    x, l = torch.empty((T, H), dtype=torch.bfloat16, device=DEV), torch.empty((T, E), device=DEV)
    idx, wt = torch.empty((T, K), dtype=torch.int32, device=DEV), torch.empty((T, K), device=DEV)
    out = poisoned(T, H)

    def step():
        ep.route(m.p, l, idx, wt, m.err, score=ep.SCORE_SIGMOID, scale=2.5)
        ep.expert_layer(m.p, x, idx, wt, m.w13, m.w2, out, m.err, m.ws, w13_scales=m.s13,
                        w2_scales=m.s2)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x.zero_()
        l.zero_()
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(4):
        xh = rand(gen, T, H)
        x.copy_(xh)
        l.copy_(torch.randn((T, E), generator=gen))
        step()
        torch.cuda.synchronize()
        eager = out.clone()
        m.check(out, x=xh, topk=idx.cpu(), wt=wt.cpu())
        for v in (out, wt, m.ws.view(torch.bfloat16)):
            v.fill_(NAN)
        idx.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
    assert int(m.err.item()) == 0


def test_two_streams_and_prepared_calls():
    """Two layers interleaved on two streams, a workspace each, equal their runs alone."""
    made = []
    for i, (kind, shape) in enumerate((("bf16", (1, 9, 8, 4, 520, 264, 0.0)),
                                       ("fp8", (1, 3, 8, 2, 512, 256, 0.0)))):
        R, T, E, K, H, I, _ = shape
        m = Made(R, T, E, K, H, I, kind, routing(R, T, E, K, 0.0, 70 + i))
        alone = m.call()
        made.append((m, alone, torch.zeros_like(alone)))
    torch.cuda.synchronize()
    keep, calls = [], []
    for m, _, out in made:
        t = [m.x.to(DEV), m.topk.to(DEV), m.wt.to(DEV)]
        keep.append(t)
        calls.append(ep.prepare(ep.expert_layer, m.p, *t, m.w13, m.w2, out, m.err, m.ws,
                                w13_scales=m.s13, w2_scales=m.s2, stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c in calls:
            c()
    torch.cuda.synchronize()
    for _, alone, out in made:
        assert torch.equal(alone.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("T", [16, 64])
@pytest.mark.parametrize("kind", ["bf16"])
def test_against_the_separate_calls(kind, T):
    """layout, dispatch, the two products and combine of the same tokens: the same layer but
    for the rounding of h and y to bf16, so within four half steps (2-norm, doubled as above)."""
    R, E, K, H, I = 2, 8, 3, 264, 136
    topk = routing(R, T, E, K, 0.1, 72)
    m = Made(R, T, E, K, H, I, kind, topk)
    out = m.call()
    p, lay, ws = m.p, ep.Layout(m.p), ep.workspace(m.p)
    ep.get_layout(p, topk.to(DEV), lay, ws)
    recv = ep.Recv(p, ep.max_recv_rows(p))
    ep.dispatch(p, lay, m.x.to(DEV), recv=recv, ws=ws)
    h, y, other = poisoned(recv.capacity, I), poisoned(recv.capacity, H), poisoned(R * T, H)
    ep.expert_gated(p, lay, recv.x, m.w13, h)
    ep.expert_linear(p, lay, h, m.w2, y)
    ep.combine(p, lay, y, m.wt.to(DEV), other)
    torch.cuda.synchronize()
    assert relative([out], [other.cpu().double()]) <= 2 * (4 / 3) ** 0.5 * HALF
