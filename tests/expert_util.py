"""Plain 64-bit forms of the experts' products, written from the formulas, and
the error bounds the GPU results are held to.

Rounding: a bf16 result is off by at most half a step, 2^-8 of its value.  A
sum of n products in fp32 is off by at most (n + 8) 2^-23 of the sum of the
products' magnitudes (every addition may lose one unit in the last place of a
partial sum, which no partial sum exceeds; 8 covers the scaling of FP8 sums,
the bias and the residual).  The activations are evaluated in fp32 with a
relative error of at most (4 + |z|) 2^-22 of |act(z)| (the exponential's
argument carries |z| 2^-24) and, since |act'| <= 1.13 for all of them, pass on
at most 1.13 times their argument's error.
"""
import math

import torch

from combine_ep_get_layout_amd import ep

HALF = 2.0 ** -8          # half a step of bf16, relative
ULP = 2.0 ** -23
TINY = 2.0 ** -120        # below this, subnormal results may be lost
ACTS = {"none": ep.ACT_NONE, "relu": ep.ACT_RELU, "silu": ep.ACT_SILU, "gelu": ep.ACT_GELU}
LIPSCHITZ = 1.13


def act64(name, z):
    """act(z), act'(z) in 64 bits."""
    if name == "none":
        return z.clone(), torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
    return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def forward64(x, w, act, gated, bias=None, residual=None):
    """One expert: (y, bound on |y - y64|, pre, bound on |pre - pre64|), all fp64."""
    z = x @ w.t()
    ez = (x.shape[1] + 8) * ULP * (x.abs() @ w.abs().t())
    if bias is not None:
        z = z + bias
        ez = ez + ULP * bias.abs()
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


def dz64(dy, pre, act, gated):
    """One expert's gradient of the pre-activations and a bound on the error of
    the bf16 values the kernels use."""
    if gated:
        n = pre.shape[1] // 2
        g, u = pre[:, :n], pre[:, n:]
        a, s = act64(act, g)
        dz = torch.cat([dy * u * s, dy * a], 1)
        big = torch.cat([(dy * u).abs(), (dy * a).abs()], 1)
        z = torch.cat([g, g], 1)
    elif act != "none":
        dz = dy * act64(act, pre)[1]
        big, z = dy.abs(), pre
    else:
        return dy, torch.zeros_like(dy)
    # the slope's own error: its terms are at most 1 + |z| each
    e = (4 + z.abs()) * (1 + z.abs()) * 2.0 ** -22 * big
    return dz, e + HALF * (dz.abs() + e) + TINY


def backward64(x, w, dz, edz):
    """One expert's dx and dw with their bounds."""
    n, r = dz.shape[1], dz.shape[0]
    dx, dw = dz @ w, dz.t() @ x
    ex = edz @ w.abs() + (n + 8) * ULP * ((dz.abs() + edz) @ w.abs())
    ew = edz.t() @ x.abs() + (r + 8) * ULP * ((dz.abs() + edz).t() @ x.abs())
    return (dx, ex + HALF * (dx.abs() + ex) + TINY, dw, ew + HALF * (dw.abs() + ew) + TINY)


def segments(p, lay):
    """[(first row, rows)] of every expert, read back from the layout."""
    count = lay.recv_tokens_per_expert.cpu().tolist()
    if p.mode == ep.MODE_NORMAL:
        return list(zip(lay.expert_start.cpu().tolist(), count))
    n = p.R * p.T
    return [(e * n, min(c, n)) for e, c in enumerate(count)]


def held(got, want, bound, what):
    """Every value of got (any float type) within `bound` of want."""
    d = (got.detach().double().cpu() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(d[bad].max()),
                           float((d / bound.clamp(min=1e-300)).max()))


def scales_of(s):
    """Scale values, fp64: fp32 as they are, UE8M0 bytes as powers of two."""
    return s.double() if s.dtype == torch.float32 else torch.exp2(s.double() - 127)


def codes_of(c):
    return c.cpu().view(torch.float8_e4m3fn).double()


def row_scales(p, scales, cap, groups, start, count, e):
    """fp64 [count][groups] scales of a segment, from the column-major array."""
    s = scales.cpu()
    if p.mode == ep.MODE_NORMAL:
        s = s[:groups * cap].view(groups, cap)[:, start:start + count]
    else:
        n = p.R * p.T
        s = s[:p.E * groups * n].view(p.E, groups, n)[e, :, :count]
    return scales_of(s).t()


def fp8_weights(gen, e, n, c, device="cuda"):
    """Random e4m3 codes (bytes) and 128 x 128 block scales, and their fp64 values."""
    codes = (torch.randn((e, n, c), generator=gen) * 60).clamp(-448, 448)
    codes = codes.to(torch.float8_e4m3fn)
    scales = torch.rand((e, n // 128, c // 128), generator=gen) * 2e-3 + 1e-4
    full = scales.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    return (codes.view(torch.uint8).to(device), scales.to(device), codes.double() * full)
