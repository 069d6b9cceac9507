"""Cases of the operators around the experts' products, with their plain forms.

* route:     top-k expert ids and weights from a router's logits: softmax or sigmoid
             scores, a bias that counts for the choice alone, the best groups of
             experts, weights normalised over the chosen and scaled;
* route_bwd: the gradient of the logits from the gradient of the weights;
* gated8:    tokens to 8-bit integer receive rows with a scale each (dispatch), and
             the gated block h = act(x Wg^T) * (x Wu^T) on them, the weights
             8-bit integers with a scale per output channel;
* linear8:   bf16 receive rows to 8-bit integers, and y = act(x W^T + bias) + residual;
* layer:     a whole layer for a few tokens, from ids and weights to the weighted sum
             of the experts' results; weights bf16, e4m3 or 8-bit integers.

``run`` computes a case in plain torch operations (32 bits; the choice of experts in
64, where scores next to each other decide), or, where ``own`` is true, makes the
library's calls.  Rows that belong to no expert are zero beforehand and stay so.
"""
import math

import torch

own = False

DEV = "cuda"
LEAST = 2.0 ** -100  # of a row's largest magnitude: its scale is a normal number


def listed():
    return [
        # the prefill step's router: 8 x 4096 tokens, 256 experts in 8 groups of which 4 are
        # kept, top-8 by sigmoid scores with a bias
        dict(name="route_prefill", op="route", ranks=8, tokens=4096, experts=256, topk=8,
             score="sigmoid", bias=True, groups=8, kept=4, gtop=2, normalize=True, scale=2.5,
             bf16=False, masked=0.0),
        # one token of a small model: latency
        dict(name="route_token", op="route", ranks=1, tokens=1, experts=64, topk=8,
             score="softmax", bias=False, groups=1, kept=1, gtop=1, normalize=True, scale=1.0,
             bf16=True, masked=0.0),
        # the training step's router, backwards: 16 x 8192 tokens, 128 experts, every logit
        # has a gradient
        dict(name="route_bwd_train", op="route_bwd", ranks=16, tokens=8192, experts=128, topk=8,
             score="softmax", normalize=False, scale=1.0, bf16=True, masked=0.0),
        # a ragged one: 201 tokens, 78 experts, three in ten of them not to be had
        dict(name="route_bwd_odd", op="route_bwd", ranks=3, tokens=67, experts=78, topk=3,
             score="sigmoid", normalize=True, scale=1.5, bf16=False, masked=0.3),
        # prompt processing: one rank's 64 experts, 2,048 rows each on average, hidden 7168
        dict(name="gated8_prefill", op="gated8", mode="normal", ranks=8, tokens=2048, topk=8,
             experts=64, cin=7168, inner=2048, act="silu", skew=0.4, masked=0.0),
        # the low-latency decode step: 8 x 128 tokens over 256 experts, 32 rows each, bound by
        # reading the weights
        dict(name="gated8_decode", op="gated8", mode="ll", ranks=8, tokens=128, topk=8,
             experts=256, cin=7168, inner=2048, act="silu", skew=0.2, masked=0.0),
        # the prefill case's down projection, with the rows themselves added
        dict(name="linear8_prefill", op="linear8", mode="normal", ranks=8, tokens=2048, topk=8,
             experts=64, cin=2048, inner=7168, act="none", bias=False, residual=True, skew=0.4,
             masked=0.0),
        # odd sizes: 549 entries over 6 experts, masked blocks, bias and activation
        dict(name="linear8_odd", op="linear8", mode="ll", ranks=3, tokens=61, topk=3, experts=6,
             cin=336, inner=520, act="silu", bias=True, residual=False, skew=0.5, masked=0.1),
        # a single token through a small model's layer: latency
        dict(name="layer_token", op="layer", kind="bf16", ranks=1, tokens=1, topk=8, experts=64,
             cin=2048, inner=768, act="silu", skew=0.0, masked=0.0),
        # 64 sequences decoded together, 256 experts of the framework's prefill width, FP8
        # weights: nearly every expert has two or three tokens
        dict(name="layer_decode_fp8", op="layer", kind="fp8", ranks=8, tokens=8, topk=8,
             experts=256, cin=7168, inner=2048, act="silu", skew=0.2, masked=0.0),
        # 32 sequences over 16 experts of the training shape's width
        dict(name="layer_few_experts", op="layer", kind="bf16", ranks=1, tokens=32, topk=2,
             experts=16, cin=4096, inner=1408, act="silu", skew=0.3, masked=0.0),
        # odd sizes, some entries masked, 8-bit integer weights
        dict(name="layer_odd_int8", op="layer", kind="int8", ranks=3, tokens=7, topk=3, experts=9,
             cin=656, inner=368, act="gelu", skew=0.5, masked=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "gated8", "linear8", "layer", "layer"])
    c = dict(op=op, ranks=rng.choice([1, 2, 3, 4, 8]))
    c["experts"] = c["ranks"] * _log(rng, 1, 256 // c["ranks"])
    c["topk"] = min(c["experts"], rng.choice([1, 2, 3, 4, 6, 8]))
    if op.startswith("route"):
        if op == "route_bwd":  # enough of both for a gradient that is not all zeros
            c["experts"] = c["ranks"] * _log(rng, -(-16 // c["ranks"]), 256 // c["ranks"])
            c["topk"] = rng.choice([1, 2, 3, 4, 6, 8])
        c["tokens"] = max(1 if op == "route" else 8, _log(rng, 1, 1 << 17) // c["ranks"])
        c["score"] = rng.choice(["softmax", "sigmoid"])
        # one weight alone, normalised, is constant: no gradient
        c["normalize"] = rng.random() < 0.6 and (op == "route" or c["topk"] > 1)
        c["scale"] = rng.choice([1.0, 1.0, round(rng.uniform(0.5, 3.0), 2)])
        c["bf16"] = rng.random() < 0.5
        c["masked"] = rng.choice([0.0, 0.0, 0.1, 0.6])
        if op == "route":
            c["bias"] = rng.random() < 0.5
            of = [g for g in range(1, 17) if c["experts"] % g == 0]
            c["groups"] = rng.choice(of)
            c["kept"] = rng.randint(1, c["groups"])
            c["gtop"] = rng.randint(1, min(2, c["experts"] // c["groups"]))
        return c
    c["skew"] = round(rng.uniform(0.0, 0.6), 2)
    c["masked"] = rng.choice([0.0, 0.0, 0.1, 0.3])
    c["act"] = rng.choice(["silu", "gelu", "relu", "none"])
    if op == "layer":
        c["kind"] = rng.choice(["bf16", "fp8", "int8"])
        step = {"bf16": 8, "fp8": 128, "int8": 16}[c["kind"]]
        c["tokens"] = max(1, _log(rng, 1, 1024 // c["topk"]) // c["ranks"])
    else:
        step = 16
        c["mode"] = rng.choice(["normal", "ll"])
        c["tokens"] = max(1, _log(rng, 1, 16384) // c["ranks"])
        if op == "linear8":
            c["bias"], c["residual"] = rng.random() < 0.5, rng.random() < 0.5
    c["cin"] = step * _log(rng, max(1, 256 // step), 7168 // step)
    c["inner"] = step * _log(rng, max(1, 256 // step), 4096 // step)

    def cost(q):
        n = q["ranks"] * q["tokens"]
        rows = n * q["topk"] if q.get("mode") != "ll" else n * q["experts"]
        weights = 4.0 * 3 * q["experts"] * q["cin"] * q["inner"]
        return max(n * q["topk"] * q["cin"] * q["inner"] / 1.5e12, weights / 6e10,
                   2.0 * rows * (q["cin"] + 3 * q["inner"]) / 6e9)

    for key, least in ("tokens", 1), ("inner", step), ("cin", step):
        unit = 1 if key == "tokens" else step
        while cost(c) > 1 and c[key] // 2 >= least:
            c[key] = max(least, c[key] // 2 // unit * unit)
    return c


# ---- inputs ----------------------------------------------------------------

def _normal(g, shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(scale)


def _fp8_weights(g, e, n, c):
    """e4m3 codes (bytes) and fp32 scales per 128 x 128 block of [e][n][c] weights."""
    codes = torch.empty((e, n, c), dtype=torch.uint8, device=DEV)
    scales = torch.empty((e, n // 128, c // 128), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 29) // (n * c))
    for i in range(0, e, step):
        v = torch.randn((min(step, e - i), n // 128, 128, c // 128, 128), generator=g, device=DEV)
        v.mul_(c ** -0.5)
        s = v.abs().amax((2, 4), keepdim=True).clamp_(min=1e-4) / 448.0
        codes[i:i + step] = (v / s).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, n, c)
        scales[i:i + step] = s.view(-1, n // 128, c // 128)
    return codes, scales


def _int8_weights(g, e, n, c):
    """int8 codes and fp32 scales per output channel of [e][n][c] weights."""
    codes = torch.empty((e, n, c), dtype=torch.int8, device=DEV)
    scales = torch.empty((e, n), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 29) // (n * c))
    for i in range(0, e, step):
        v = torch.randn((min(step, e - i), n, c), generator=g, device=DEV).mul_(c ** -0.5)
        s = v.abs().amax(2) / 127.0
        codes[i:i + step] = torch.round(v / s[:, :, None]).to(torch.int8)
        scales[i:i + step] = s
    return codes, scales


def _routing(g, case):
    """int32 [ranks][tokens][topk] distinct experts (Gumbel top-k over a drawn
    popularity), a share of the entries masked with -1."""
    n, e = case["ranks"] * case["tokens"], case["experts"]
    pop = torch.randn(e, generator=g, device=DEV) * case["skew"]
    u = torch.rand((n, e), generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)
    t = torch.topk(pop - (-u.log()).log(), case["topk"], dim=1).indices.to(torch.int32)
    t[torch.rand(t.shape, generator=g, device=DEV) < case["masked"]] = -1
    return t.view(case["ranks"], case["tokens"], case["topk"])


def _logits(g, case):
    """[tokens][experts] N(0, 1.5), a share of them -inf (experts that a token may not have)."""
    shape = (case["ranks"] * case["tokens"], case["experts"])
    v = _normal(g, shape, 1.5, torch.bfloat16 if case["bf16"] else torch.float32)
    if case["masked"]:
        v[torch.rand(shape, generator=g, device=DEV) < case["masked"]] = -math.inf
    return v


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    e, n, k = case["experts"], case["ranks"] * case["tokens"], case["topk"]
    op = case["op"]
    if op.startswith("route"):
        s = dict(case=case, logits=_logits(g, case))
        if op == "route":
            if case["bias"]:
                s["bias"] = _normal(g, (e,), 0.1, torch.float32)
            outs = dict(topk_idx=torch.zeros((n, k), dtype=torch.int32, device=DEV),
                        topk_weights=torch.zeros((n, k), device=DEV))
        else:
            best, ids = torch.topk(s["logits"].float(), k, dim=1)
            s["topk"] = torch.where(best > -math.inf, ids, -1).to(torch.int32)
            s["dweights"] = _normal(g, (n, k), 1.0, torch.float32)
            outs = dict(dlogits=torch.zeros_like(s["logits"]))
    else:
        s = dict(case=case, topk=_routing(g, case))
        outs = _prepare_experts(s, g)
    if own:
        s["outs"] = outs
        s["calls"] = _calls(s, outs)
    return s


def _prepare_experts(s, g):
    case = s["case"]
    e, n, k = case["experts"], case["ranks"] * case["tokens"], case["topk"]
    op, c, i, flat = case["op"], case["cin"], case["inner"], s["topk"].view(-1).long()
    # the entries by expert, in (rank, token, k) order
    order = torch.argsort(flat, stable=True)
    order = order[int((flat < 0).sum()):]
    counts = torch.bincount(flat[flat >= 0], minlength=e)
    packed = torch.cumsum(counts, 0) - counts
    within = torch.arange(order.numel(), device=DEV) - packed[flat[order]]
    most = max(1, int(counts.max()))
    slot = torch.arange(most, device=DEV)
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    if op == "layer":
        # the experts that are hit, and their tokens as a padded batch
        s["hit"] = torch.nonzero(counts).view(-1)
        at = packed[s["hit"], None] + torch.minimum(slot[None], counts[s["hit"], None] - 1)
        s["entry"] = order[at] if order.numel() else at
        s["valid"] = slot[None] < counts[s["hit"], None]
        s["x"] = _normal(g, (n, c))
        s["weights"] = torch.softmax(_normal(g, (n, k), 1.0, torch.float32), -1)
        for name, wide, deep in ("w13", 2 * i, c), ("w2", c, i):
            if case["kind"] == "bf16":
                s[name] = _normal(g, (e, wide, deep), deep ** -0.5)
            else:
                make = _fp8_weights if case["kind"] == "fp8" else _int8_weights
                s[name], s[name + "_scales"] = make(g, e, wide, deep)
        return dict(out=torch.zeros((n, c), **bf16))
    ll = case["mode"] == "ll"
    starts = torch.arange(e, device=DEV) * n if ll else packed
    cap = e * n if ll else n * k
    s.update(counts=counts, starts=starts, cap=cap)
    # the padded batch: row and entry of slot (expert, i), slot and row of every entry
    near = torch.minimum(slot[None], (counts - 1).clamp_(min=0)[:, None])
    s["pad"] = (starts[:, None] + near).clamp_(max=cap - 1)
    s["valid"] = slot[None] < counts[:, None]
    at = (packed[:, None] + near).clamp_(max=max(order.numel() - 1, 0))
    s["entry"] = order[at] if order.numel() else at
    s["slot"], s["row"] = flat[order] * most + within, starts[flat[order]] + within
    wide = 2 * i if op == "gated8" else i
    s["w"], s["w_scales"] = _int8_weights(g, e, wide, c)
    s["x"] = _normal(g, (n if op == "gated8" else cap, c))
    if case.get("bias"):
        s["bias"] = _normal(g, (e, i), 1.0, torch.float32)
    if case.get("residual"):
        s["residual"] = _normal(g, (cap, i))
    return dict(y=torch.zeros((cap, i), **bf16))


def _calls(s, outs):
    """The library's calls of one pass, on its layout of the routing."""
    from combine_ep_get_layout_amd import ep

    case = s["case"]
    op, c = case["op"], case.get("cin", 128)
    mode = ep.MODE_LOW_LATENCY if case.get("mode") == "ll" else ep.MODE_NORMAL
    quant = ep.QUANT_INT8 if op in ("gated8", "linear8") else ep.QUANT_NONE
    p = ep.Problem(case["ranks"], case["tokens"], c, case["experts"], case["topk"], mode=mode,
                   quant=quant)
    if op.startswith("route"):
        kw = dict(score=getattr(ep, "SCORE_" + case["score"].upper()),
                  normalize=case["normalize"], scale=case["scale"])
        s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if op == "route":
            return [ep.prepare(ep.route, p, s["logits"], outs["topk_idx"], outs["topk_weights"],
                               s["err"], bias=s.get("bias"), groups=case["groups"],
                               groups_kept=case["kept"], group_top=case["gtop"], **kw)]
        return [ep.prepare(ep.route_backward, p, s["logits"], s["topk"], s["dweights"],
                           outs["dlogits"], s["err"], **kw)]
    act = getattr(ep, "ACT_" + case["act"].upper())
    if op == "layer":
        s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["ws"] = ep.layer_workspace(p, case["inner"])
        return [ep.prepare(ep.expert_layer, p, s["x"], s["topk"], s["weights"], s["w13"], s["w2"],
                           outs["out"], s["err"], s["ws"], act=act,
                           w13_scales=s.get("w13_scales"), w2_scales=s.get("w2_scales"))]
    layout = s["layout"] = ep.Layout(p)
    ws = s["ws"] = ep.workspace(p)
    ep.get_layout(p, s["topk"], layout, ws)
    recv = s["recv"] = ep.Recv(p, s["cap"])
    if op == "gated8":
        return [ep.prepare(ep.dispatch, p, layout, s["x"], recv=recv, ws=ws),
                ep.prepare(ep.expert_gated, p, layout, recv.x, s["w"], outs["y"], act=act,
                           x_scales=recv.scales, w_scales=s["w_scales"])]
    return [ep.prepare(ep.quantize_rows, p, layout, s["x"], recv.x, recv.scales),
            ep.prepare(ep.expert_linear, p, layout, recv.x, s["w"], outs["y"], act=act,
                       x_scales=recv.scales, w_scales=s["w_scales"], bias=s.get("bias"),
                       residual=s.get("residual"))]


# ---- the plain forms --------------------------------------------------------

def _act(name, v):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.5 ** 0.5))
    return v.clamp(min=0) if name == "relu" else v


def _scores(name, v):
    if name == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-v))
    most = v.amax(1, keepdim=True)
    part = torch.exp(v - torch.where(most > -math.inf, most, 0.0))
    return part / part.sum(1, keepdim=True).clamp(min=1e-300 if v.dtype == torch.float64 else 1e-30)


def _route(s):
    case = s["case"]
    n, e, k = s["logits"].shape[0], case["experts"], case["topk"]
    v = s["logits"].double()
    scores = _scores(case["score"], v)
    by = scores + s["bias"].double() if case["bias"] else scores
    by = torch.where(v > -math.inf, by, -math.inf)
    # without a bias the logits themselves are in the scores' order
    choice = by if case["bias"] else v
    if case["kept"] < case["groups"]:
        top = by.view(n, case["groups"], -1).sort(dim=2, descending=True).values[:, :, :case["gtop"]]
        total = torch.where(top > -math.inf, top, 0.0).sum(2)
        total = torch.where(top[:, :, 0] > -math.inf, total, -math.inf)
        kept = total.sort(dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        mask = torch.zeros((n, case["groups"]), dtype=torch.bool, device=DEV)
        mask = mask.scatter_(1, kept, True).repeat_interleave(e // case["groups"], 1)
        choice = torch.where(mask, choice, -math.inf)
    best, ids = choice.sort(dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    has = best > -math.inf
    w = torch.where(has, scores.gather(1, ids), 0.0)
    if case["normalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return dict(topk_idx=torch.where(has, ids, -1).to(torch.int32),
                topk_weights=(w * case["scale"]).float())


def _route_bwd(s):
    case = s["case"]
    v, ids = s["logits"].float(), s["topk"].long()
    has = ids >= 0
    at = ids.clamp(min=0)
    scores = _scores(case["score"], v)
    chosen = torch.where(has, scores.gather(1, at), 0.0)
    dw = torch.where(has, s["dweights"], 0.0) * case["scale"]
    if case["normalize"]:
        total = chosen.sum(1, keepdim=True).clamp(min=1e-30)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(v).scatter_add_(1, at, torch.where(has, dw, 0.0))
    if case["score"] == "sigmoid":
        grad = ds * scores * (1.0 - scores)
    else:
        grad = scores * (ds - (ds * scores).sum(1, keepdim=True))
    return dict(dlogits=grad.to(s["logits"].dtype))


def _quantised(x):
    """8-bit integers (as 32-bit numbers) of every row, and the rows' scales."""
    x = x.float()
    scale = x.abs().amax(-1, keepdim=True).clamp(min=LEAST) / 127.0
    return torch.round(x / scale), scale


def _rows(s, padded):
    """A padded batch's rows in a bf16 row buffer, zero where no expert's row is."""
    out = torch.zeros((s["cap"], padded.shape[2]), dtype=torch.bfloat16, device=DEV)
    flat = padded.view(-1, padded.shape[2])
    return out.index_copy_(0, s["row"], flat[s["slot"]].to(torch.bfloat16))


def _product8(s, codes, scales):
    """codes W^T of the padded batch, with both scales."""
    z = torch.bmm(codes, s["w"].float().transpose(1, 2).contiguous())
    return z.mul_(scales).mul_(s["w_scales"][:, None, :])


def _gated8(s):
    case = s["case"]
    codes, scales = _quantised(s["x"])
    token = s["entry"] // case["topk"]
    gate, up = _product8(s, codes[token], scales[token]).chunk(2, dim=2)
    return dict(y=_rows(s, _act(case["act"], gate) * up))


def _linear8(s):
    z = _product8(s, *_quantised(s["x"][s["pad"]]))
    if "bias" in s:
        z = z + s["bias"][:, None, :]
    y = _act(s["case"]["act"], z)
    if "residual" in s:
        y = y + s["residual"][s["pad"]].float()
    return dict(y=_rows(s, y))


def _of_hit(s, name):
    """The hit experts' weights in 32 bits, contraction first."""
    w, kind = s[name][s["hit"]], s["case"]["kind"]
    if kind == "fp8":
        e, n, c = w.shape
        w = w.view(torch.float8_e4m3fn).float().view(e, n // 128, 128, c // 128, 128)
        w = w.mul_(s[name + "_scales"][s["hit"]][:, :, None, :, None]).view(e, n, c)
    elif kind == "int8":
        w = w.float().mul_(s[name + "_scales"][s["hit"]][:, :, None])
    return w.float().transpose(1, 2).contiguous()


def _layer(s):
    case = s["case"]
    out = torch.zeros(s["x"].shape, dtype=torch.float32, device=DEV)
    token = s["entry"] // case["topk"]
    gate, up = torch.bmm(s["x"].float()[token], _of_hit(s, "w13")).chunk(2, dim=2)
    y = torch.bmm((_act(case["act"], gate) * up).contiguous(), _of_hit(s, "w2"))
    y = y * (s["weights"].view(-1)[s["entry"]] * s["valid"])[:, :, None]
    # to (token, k), then summed over k
    each = torch.zeros((s["topk"].numel() + 1, out.shape[1]), device=DEV)
    last = each.shape[0] - 1
    each.index_copy_(0, torch.where(s["valid"], s["entry"], last).view(-1),
                     y.view(-1, out.shape[1]))
    return dict(out=each[:last].view(-1, case["topk"], out.shape[1]).sum(1).to(torch.bfloat16))


def run(s):
    if own:
        for call in s["calls"]:
            call()
        return s["outs"]
    return dict(route=_route, route_bwd=_route_bwd, gated8=_gated8, linear8=_linear8,
                layer=_layer)[s["case"]["op"]](s)


# ---- the definition in 64 bits, a few tokens or an expert at a time -------------

def _gate64(name, v):
    if name == "none":
        return v
    if name == "relu":
        return torch.relu(v)
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    return v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))


def _before(c):
    """[n][m]: how many of a row's values come before each, ties in their order."""
    m = c.shape[1]
    earlier = torch.arange(m, device=DEV)[None, :] < torch.arange(m, device=DEV)[:, None]
    return ((c[:, None, :] > c[:, :, None])
            | ((c[:, None, :] == c[:, :, None]) & earlier[None])).sum(2)


def _exact_route(s, case):
    k, e, groups = case["topk"], case["experts"], case["groups"]
    ids, weights = [], []
    for v in s["logits"].double().split(max(1, (1 << 26) // (e * e))):
        may = v > -math.inf
        if case["score"] == "sigmoid":
            score = torch.special.expit(v)
        else:
            score = torch.exp(v - torch.logsumexp(torch.where(may, v, -1e9), 1, keepdim=True))
        by = torch.where(may, score + (s["bias"].double() if case["bias"] else 0.0), -math.inf)
        choice = by if case["bias"] else torch.where(may, v, -math.inf)
        if case["kept"] < groups:
            of = by.view(-1, e // groups)
            counted = (_before(of) < case["gtop"]) & (of > -math.inf)
            total = torch.where(counted, of, 0.0).sum(1)
            total = torch.where(counted.any(1), total, -math.inf).view(-1, groups)
            stays = (_before(total) < case["kept"]).repeat_interleave(e // groups, 1)
            choice = torch.where(stays, choice, -math.inf)
        place = torch.where(choice > -math.inf, _before(choice), e)
        at = torch.full((v.shape[0], e + 1), -1, dtype=torch.int64, device=DEV)
        at.scatter_(1, place, torch.arange(e, device=DEV).expand_as(place))
        at[:, e] = -1
        at = at[:, :k]
        w = torch.where(at >= 0, score.gather(1, at.clamp(min=0)), 0.0)
        if case["normalize"]:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / total, 0.0)
        ids.append(at.to(torch.int32))
        weights.append(w * case["scale"])
    return dict(topk_idx=torch.cat(ids), topk_weights=torch.cat(weights))


def _exact_route_bwd(s, case):
    """By the weights' derivatives: dl_e = sum_k dw_k dw_k/dl_e."""
    out = []
    for v, ids, dw in zip(*(s[q].split(4096) for q in ("logits", "topk", "dweights"))):
        v, dw = v.double(), dw.double() * case["scale"]
        has = (ids >= 0).double()
        hot = torch.nn.functional.one_hot(ids.long().clamp(min=0), case["experts"]).double()
        hot = hot * has[:, :, None]  # [n][k][experts]
        if case["score"] == "sigmoid":
            score = torch.special.expit(v)
            each = (hot * score[:, None, :]).sum(2)
            jac = hot * (score * torch.special.expit(-v))[:, None, :]
        else:
            lse = torch.logsumexp(torch.where(v > -math.inf, v, -1e9), 1, keepdim=True)
            score = torch.exp(v - lse)
            each = (hot * score[:, None, :]).sum(2)
            jac = each[:, :, None] * (hot - score[:, None, :])
        if case["normalize"]:  # of s_k / S
            total = each.sum(1)[:, None, None].clamp(min=1e-300)
            jac = jac / total - each[:, :, None] / total ** 2 * jac.sum(1, keepdim=True)
        out.append((dw[:, :, None] * jac).sum(1))
    return dict(dlogits=torch.cat(out))


def _exact_codes(x):
    """The integers that rows stand for and their scales, which are 32-bit numbers."""
    scale = torch.maximum(x.abs().max(-1).values, torch.tensor(LEAST, device=DEV).to(x.dtype))
    scale = (scale.double() / 127.0).float().double()[:, None]
    return torch.round(x.double() / scale), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s, case)
    if op == "route_bwd":
        return _exact_route_bwd(s, case)
    i, c, k = case["inner"], case["cin"], case["topk"]
    flat = s["topk"].view(-1).long()
    order = torch.argsort(torch.where(flat < 0, case["experts"], flat), stable=True)
    count = torch.bincount(flat[flat >= 0], minlength=case["experts"]).tolist()
    f64 = dict(dtype=torch.float64, device=DEV)
    layer = op == "layer"
    out = torch.zeros((s["x"].shape[0], c) if layer else (s["cap"], i), **f64)
    done = 0
    for e, rows in enumerate(count):
        entries = order[done:done + rows]
        done += rows
        if rows == 0:
            continue
        if layer:
            w = []
            for name in ("w13", "w2"):
                v = s[name][e]
                if case["kind"] == "fp8":
                    per = s[name + "_scales"][e].double()
                    v = v.view(torch.float8_e4m3fn).double()
                    v = v * per.repeat_interleave(128, 0).repeat_interleave(128, 1)
                elif case["kind"] == "int8":
                    v = v.double() * s[name + "_scales"][e].double()[:, None]
                w.append(v.double())
            z = s["x"][entries // k].double() @ w[0].t()
            y = (_gate64(case["act"], z[:, :i]) * z[:, i:]) @ w[1].t()
            out.index_add_(0, entries // k, y * s["weights"].view(-1)[entries].double()[:, None])
            continue
        first = e * s["topk"].numel() // k if case["mode"] == "ll" else done - rows
        at = slice(first, first + rows)
        codes, scale = _exact_codes(s["x"][entries // k] if op == "gated8" else s["x"][at])
        z = (codes @ s["w"][e].double().t()) * scale * s["w_scales"][e].double()
        if "bias" in s:
            z = z + s["bias"][e].double()
        y = _gate64(case["act"], z[:, :i]) * (z[:, i:] if op == "gated8" else 1.0)
        if "residual" in s:
            y = y + s["residual"][at].double()
        out[at] = y
    return dict(out=out) if layer else dict(y=out)


# ---- what a pass cannot do without --------------------------------------------

def work(case):
    n, e, k = case["ranks"] * case["tokens"], case["experts"], case["topk"]
    op = case["op"]
    if op.startswith("route"):
        size = 2 if case["bf16"] else 4
        passes = 1 if op == "route" else 2
        return dict(bytes=float(passes * n * e * size + 8 * n * k), flops=8.0 * n * e)
    c, i = case["cin"], case["inner"]
    rows = n * k * (1.0 - case["masked"])
    hit = e * (1.0 - (1.0 - (1.0 - case["masked"]) * k / e) ** n)  # experts with a row
    if op == "layer":
        size = 2 if case["kind"] == "bf16" else 1
        return dict(bytes=hit * 3.0 * i * c * size + 4.0 * n * c + 8.0 * n * k,
                    flops=6.0 * rows * i * c)
    wide = 2 * i if op == "gated8" else i
    taken = 2.0 * (n if op == "gated8" else rows) * c
    given = 2.0 * rows * i * (2 if case.get("residual") else 1)
    return dict(bytes=taken + given + hit * wide * c, flops=2.0 * rows * wide * c)
