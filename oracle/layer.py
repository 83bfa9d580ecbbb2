"""What stands around a layer's expert products, in float64: the norm before them, the choice and the order of each
token's experts, the rows' way out and back, and their gradients.  Arrays are float64 values (of bf16 or fp32
tensors), plain loops over tokens where that says most clearly what is meant.
"""
from __future__ import annotations

import numpy as np

from .mx import mx_quantize_rowwise_values
from .plain import int8_quantize_rows


def rmsnorm(h, w, eps):
    """(y, r): r = 1 / sqrt(mean(h^2) + eps) of each row, y = h r w."""
    r = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * r[:, None] * w, r


def rmsnorm_int8(h, w, eps):
    """(codes, scales): the codes are those of h w, since a row's r divides out; the scale is amax r / 127."""
    v = h * w
    q, _ = int8_quantize_rows(v)
    amax = np.abs(v).max(axis=1)
    return q, np.where(amax > 0, amax * rmsnorm(h, w, eps)[1] / 127.0, 1.0)


def rmsnorm_mx(h, w, eps):
    return mx_quantize_rowwise_values(rmsnorm(h, w, eps)[0])


def rmsnorm_bwd(dy, h, w, eps, dres=None):
    """(dx, dw): dx = r (g - h r^2 mean(g h)) + dres with g = dy w; dw = sum over rows of dy h r."""
    r = rmsnorm(h, w, eps)[1][:, None]
    g = dy * w
    dx = r * (g - h * r * r * (g * h).mean(axis=1, keepdims=True))
    return (dx if dres is None else dx + dres), (dy * h * r).sum(axis=0)


def route_scores(logits, score):
    """p [T, E]; an expert with a logit of -infinity has 0, and so have all where every logit is that."""
    p = np.zeros_like(logits)
    for t, row in enumerate(logits):
        if score == "sigmoid":
            e = np.exp(-np.abs(row))
            p[t] = np.where(row >= 0, 1.0, e) / (1.0 + e)
        else:
            m = row.max()
            if m > -np.inf:
                with np.errstate(invalid="ignore"):
                    e = np.where(row == m, 1.0, np.exp(row - m))
                p[t] = e / e.sum()
    return p


def _chosen_scores(row, p, ids, score, renorm):
    """Scores of a token's chosen experts; renormalised softmax scores are a softmax over the chosen, since e^x / sum over
    all cancels to it."""
    return route_scores(row[None, ids], score)[0] if renorm and score == "softmax" else p[ids]


def route(logits, top, score="softmax", bias=None, groups=1, keep=None, group_top=1, renorm=True, scale=1.0, valid=None):
    """(ids int32 [T, top], weights float64 [T, top])."""
    T, E = logits.shape
    size = E // groups
    p = route_scores(logits, score)
    ids, w = np.full((T, top), -1, np.int32), np.zeros((T, top))
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        c = logits[t] if bias is None else p[t] + bias
        allowed = range(E)
        if groups > 1:
            with np.errstate(invalid="ignore"):
                best = [sum(sorted(c[g * size:(g + 1) * size])[-group_top:]) for g in range(groups)]
            best = [-np.inf if v != v else v for v in best]
            order = sorted(range(groups), key=lambda g: (-best[g], g))[:groups if keep is None else keep]
            allowed = [e for g in order for e in range(g * size, (g + 1) * size)]
        ids[t] = sorted(allowed, key=lambda e: (-c[e], e))[:top]
        sel = _chosen_scores(logits[t], p[t], ids[t], score, renorm)
        total = sel.sum() if renorm else 1.0
        w[t] = scale * sel / total if total > 0 else 0.0
    return ids, w


def route_bwd(dweights, ids, logits, score="softmax", renorm=True, scale=1.0):
    """dlogits [T, E]: the chain from the weights over the scores to the logits; the choice is constant."""
    T, E = logits.shape
    p = route_scores(logits, score)
    out = np.zeros((T, E))
    for t in range(T):
        here = [k for k in range(ids.shape[1]) if 0 <= ids[t, k] < E]
        if not here:
            continue
        sel, dw = _chosen_scores(logits[t], p[t], ids[t, here], score, renorm), dweights[t, here]
        total = sel.sum() if renorm else 1.0
        if total == 0:
            continue
        ds = scale * dw / total
        if renorm:
            ds = ds - (scale * dw * (sel / total)).sum() / total
        if score == "softmax" and renorm:              # (a softmax over the chosen: the others' gradient is 0, not a rounding)
            np.add.at(out[t], ids[t, here], ds * sel)
            continue
        dp = np.zeros(E)
        np.add.at(dp, ids[t, here], ds)
        # (1 - p by its own formula: near 1 the difference keeps few bits)
        out[t] = dp * p[t] * route_scores(-logits[t:t + 1], score)[0] if score == "sigmoid" else p[t] * (dp - (dp * p[t]).sum())
    return out


def sort_pairs(ids, G, first=0):
    """(offs, row_idx, pos): pairs of the experts first .. first + G - 1 in the order of expert, token, choice."""
    T, top = ids.shape
    flat = ids.reshape(-1).astype(np.int64) - first
    rows = [i for g in range(G) for i in range(T * top) if ids.reshape(-1)[i] >= 0 and flat[i] == g]
    offs = np.array([0] + [int(((flat >= 0) & (flat <= g) & (ids.reshape(-1) >= 0)).sum()) for g in range(G)], np.int32)
    row_idx, pos = np.full(T * top, -1, np.int32), np.full(T * top, -1, np.int32)
    for r, i in enumerate(rows):
        row_idx[r], pos[i] = i // top, r
    return offs, row_idx, pos.reshape(T, top)


def combine(y, pos, weights=None, residual=None):
    """(out [T, C], sum of magnitudes): residual + sum_k w y[pos]."""
    T, top = pos.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.copy()
    mag = np.abs(out)
    for t in range(T):
        for k in range(top):
            if 0 <= pos[t, k] < y.shape[0]:
                term = y[pos[t, k]] * (1.0 if weights is None else weights[t, k])
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def combine_bwd(dout, pos, weights, y, dy):
    """(dy with the named rows replaced, dweights [T, top], sum of magnitudes of the latter)."""
    T, top = pos.shape
    dy, dw, mag = dy.copy(), np.zeros((T, top)), np.zeros((T, top))
    for t in range(T):
        for k in range(top):
            if 0 <= pos[t, k] < y.shape[0]:
                dy[pos[t, k]] = dout[t] * (1.0 if weights is None else weights[t, k])
                dw[t, k] = dout[t] @ y[pos[t, k]]
                mag[t, k] = np.abs(dout[t]) @ np.abs(y[pos[t, k]])
    return dy, dw, mag
