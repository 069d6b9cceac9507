"""Plain 64-bit forms of the router and its gradient, written from the formulas, a token
at a time, and the bounds that the fp32 results are held to.

A score: the exponential's argument l - max is rounded (|l - max| 2^-24 relative in the
exponential), the exponential to 2^-23, one plus it and the quotient to 2^-24 each; sums of
up to 2,048 scores are taken in at most 64 steps one after another (32 values of a lane, and
six steps between lanes, or 64 entries), each 2^-24; then a quotient and the scale.  All
relative, so a weight is off by less than (64 + |l - max|) 2^-23 of itself."""
import itertools

import numpy as np

ULP = 2.0 ** -23
TINY = 2.0 ** -120


def scores64(l, sigmoid):
    with np.errstate(over="ignore"):
        if sigmoid:
            return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))),
                            np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
        m = l.max()
        if m == -np.inf:
            return np.zeros_like(l)
        z = np.exp(l - m)
        return z / z.sum()


def weights64(l, ids, sigmoid, normalize, scale):
    """Weights of the entries ids (some -1) of one token, and their bound."""
    ok = ids >= 0
    w, e = np.zeros(len(ids)), np.full(len(ids), TINY)
    if ok.any():
        chosen = l[ids[ok]]
        if normalize and sigmoid:  # in logarithms: nothing vanishes
            log = np.minimum(chosen, 0) - np.log1p(np.exp(-np.abs(chosen)))
            s = np.exp(log - log.max())
        elif normalize:
            s = np.exp(chosen - chosen.max())
        else:
            s = scores64(l, sigmoid)[ids[ok]]
        top = chosen.max() if normalize else l.max()
        far = np.abs(chosen - top) if not sigmoid or (normalize and top < -30) else 0.0
        w[ok] = s / s.sum() * scale if normalize else s * scale
        e[ok] += (64 + far) * ULP * np.abs(w[ok])
    return w, e


def choices64(l, bias, sigmoid, groups, kept, top, K):
    """The ids of one token, in a list; none where it has a logit, or choice, that is no
    number.

    More than one answer where groups' sums of choices are nearer to each other than 64 bits
    tell: with choices s + b, two groups may have the same sum by the formula and their
    computed sums differ in the last places.  A score is computed to (E + 8) 2^-53 (the
    exponential, up to E additions, the quotient), bias and sum add 2^-53 of |c| each, so a
    sum is off by at most (E + 16) 2^-53 of the magnitudes in it, on either side."""
    if np.isnan(l).any() or (not sigmoid and (l == np.inf).any()):
        return []
    s = scores64(l, sigmoid)
    by = np.where(l > -np.inf, s + (0 if bias is None else bias), -np.inf)
    if bias is not None and np.isnan(by).any():
        return []
    choice = by if bias is not None else l.copy()
    masks = [np.ones(groups, bool)]
    if kept < groups:
        of = (by if top > 1 else choice).reshape(groups, -1)
        score, off = np.empty(groups), np.zeros(groups)
        for g in range(groups):
            best = np.sort(of[g])[::-1][:top]
            best = best[best > -np.inf]
            score[g] = best.sum() if len(best) else -np.inf
            if len(best) > 1:
                mass = np.abs(best) + 2 * s.max()
                off[g] = (len(l) + 16) * 2.0 ** -53 * mass.sum()
        order = np.argsort(-score, kind="stable")
        border = score[order[kept - 1]]
        near = np.zeros(groups, bool)
        if np.isfinite(border):
            near = np.abs(score - border) <= off + off[order[kept - 1]]
        exact = [g for g in range(groups) if near[g] and off[g] > 0]
        masks = []
        # groups of the very same choices stay in the order of their index
        sure = [g for g in order[:kept] if not near[g] or not exact]
        for more in itertools.combinations(np.flatnonzero(near) if exact else [],
                                           kept - len(sure)):
            mask = np.zeros(groups, bool)
            mask[list(sure) + list(more)] = True
            if all(mask[a] or not mask[b] for a in range(groups) for b in range(a + 1, groups)
                   if near[a] and near[b]
                   and np.array_equal(np.sort(of[a])[::-1][:top], np.sort(of[b])[::-1][:top])):
                masks.append(mask)
    out = []
    for mask in masks:
        c = np.where(np.repeat(mask, len(l) // groups), choice, -np.inf)
        order = np.argsort(-c, kind="stable")[:K]
        ids = np.full(K, -1)
        order = order[c[order] > -np.inf]
        ids[:len(order)] = order
        out.append(ids)
    return out


def grad64(l, ids, dw, sigmoid, normalize, scale):
    """dl of one token, and the bound on the fp32 computation of it (before its rounding to
    the logits' type)."""
    E = len(l)
    ok = ids >= 0
    count, d = np.zeros(E), np.zeros(E)
    np.add.at(count, ids[ok], 1)
    np.add.at(d, ids[ok], dw[ok])
    size = np.zeros(E)
    np.add.at(size, ids[ok], np.abs(dw[ok]))
    if not ok.any():
        return np.zeros(E), np.full(E, TINY)
    rest = 1 - scores64(l, True) if not sigmoid else scores64(-l, True)
    if not sigmoid:
        rest = np.ones(E)
    if normalize:
        m = l[count > 0].max()
        if m == -np.inf:  # nothing that a weight could move to: no gradient
            return np.zeros(E), np.full(E, TINY)
        if sigmoid:
            s = scores64(l, True) if m > -30 else np.exp(np.minimum(l - m, 0))
        else:
            s = np.where(count > 0, np.exp(np.minimum(l - m, 0)), 0)
        s = np.where(count > 0, s, 0)
        s = s / (count * s).sum()
        mean, far = (d * s).sum(), m - l[(count > 0) & (l > -np.inf)].min()
        dl = scale * s * (d - count * mean) * rest
        mass = (size * s).sum()
        bound = np.abs(scale) * s * (size + count * mass) * rest
    elif sigmoid:
        s, far = scores64(l, True), 0.0
        dl = scale * d * s * rest
        bound = np.abs(scale) * size * s * rest
    else:
        s, fine = scores64(l, False), l[l > -np.inf]
        far = fine.max() - fine.min() if len(fine) else 0.0
        dl = scale * s * (d - (d * s).sum())
        bound = np.abs(scale) * s * (size + (size * s).sum())
    # s, the sums of d s and of s, the difference and three products, twice over
    return dl, 2 * (64 + far) * ULP * bound + TINY
