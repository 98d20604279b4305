"""Plain fp64 implementations of the routing to experts, of its gradient, of the
order by expert and of the tokens' sums (CPU, numpy; test infrastructure only,
no code shared with the library)."""

import numpy as np


def scores(z, score):
    z = np.asarray(z, dtype=np.float64)
    if score == "softmax":
        top = z.max(axis=-1, keepdims=True)
        e = np.exp(z - np.where(np.isfinite(top), top, 0.0))
        total = e.sum(axis=-1, keepdims=True)
        return np.divide(e, total, out=np.zeros_like(e), where=total > 0)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


def route_token(z, k, bias=None, score="softmax", groups=1, top_groups=1, group_best=2, renormalize=True, scale=1.0):
    """(chosen experts, weights) of one token, each of length k."""
    n = len(z)
    if np.isnan(z).any() or (bias is not None and np.isnan(bias).any()) or (score == "softmax" and (z == np.inf).any()):
        return [-1] * k, [np.nan] * k
    s = scores(z, score)
    by_score = bias is not None or (groups > 1 and group_best > 1)
    key = s + (0 if bias is None else bias) if by_score else z
    left = [e for e in range(n) if z[e] != -np.inf]
    if groups > 1:
        size = n // groups
        marks = []
        for g in range(groups):
            best = sorted((key[e] for e in left if e // size == g), reverse=True)[:group_best]
            marks.append(sum(best) if best else -np.inf)
        stay = sorted(range(groups), key=lambda g: (-marks[g], g))[:top_groups]
        left = [e for e in left if e // size in stay]
    chosen = sorted(left, key=lambda e: (-key[e], e))[:k]
    picked = np.array([s[e] for e in chosen])
    if renormalize and score == "softmax" and chosen:  # the row's sum falls out (it may be out of range)
        picked = scores(np.array([z[e] for e in chosen]), "softmax")
    total = picked.sum() if renormalize else 1.0
    w = [scale * p / total if total > 0 else 0.0 for p in picked]
    return chosen + [-1] * (k - len(chosen)), w + [0.0] * (k - len(chosen))


def route(z, k, mask=None, **kw):
    """int [tokens, k], float [tokens, k]."""
    chosen, weights = [], []
    for t in range(len(z)):
        c, w = ([-1] * k, [0.0] * k) if mask is not None and not mask[t] else route_token(z[t], k, **kw)
        chosen.append(c)
        weights.append(w)
    return np.array(chosen).reshape(-1, k), np.array(weights).reshape(-1, k)


def order(chosen, experts, align):
    """(slots, pairs, offsets, loads): the pairs by expert, tokens in order."""
    tokens, k = chosen.shape
    slots = np.full((tokens, k), -1)
    offsets, pairs, loads = [0], [], []
    for e in range(experts):
        mine = [t * k + j for t in range(tokens) for j in range(k) if chosen[t, j] == e]
        for i, p in enumerate(mine):
            slots[p // k, p % k] = offsets[e] + i
        loads.append(len(mine))
        pairs += mine + [-1] * (-len(mine) % align)
        offsets.append(len(pairs))
    rows = -(-(tokens * k + experts * (align - 1)) // align) * align
    return slots, np.array(pairs + [-1] * (rows - len(pairs))), np.array(offsets), np.array(loads)


def weights_of(z, chosen, score, renormalize, scale):
    """The weights of a fixed choice, as a function of the logits (for its gradient)."""
    s = scores(z, score)
    out = np.zeros(chosen.shape)
    for t in range(chosen.shape[0]):
        there = chosen[t] >= 0
        p = s[t, chosen[t, there]]
        total = p.sum() if renormalize else 1.0
        out[t, there] = scale * p / total if total > 0 else 0.0
    return out


def route_backward(z, chosen, grad, score, renormalize, scale):
    """Gradient of the logits from that of the weights, by the chain rule through the scores."""
    s = scores(z, score)
    out = np.zeros_like(s)
    for t in range(chosen.shape[0]):
        there = np.flatnonzero(chosen[t] >= 0)
        e = chosen[t, there]
        ds = np.zeros(s.shape[1])
        total = s[t, e].sum() if renormalize else 1.0
        if total > 0:
            g = grad[t, there]
            mean = (g * s[t, e]).sum() / total if renormalize else 0.0
            ds[e] = scale * (g - mean) / total
        if score == "softmax":
            out[t] = s[t] * (ds - (ds * s[t]).sum())
        else:
            out[t] = ds * s[t] * (1 - s[t])
    return out


def balance(bias, loads, rate):
    return bias + rate * np.sign(loads.mean() - loads)


def expert_sum(y, slots, weights=None):
    """(sums, sums of magnitudes)."""
    out = np.zeros((slots.shape[0], y.shape[1]))
    size = np.zeros_like(out)
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            if 0 <= slots[t, j] < y.shape[0]:
                term = y[slots[t, j]] * (1.0 if weights is None else weights[t, j])
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def expert_dot(grad, y, slots):
    """(dots, sums of magnitudes)."""
    out = np.zeros(slots.shape)
    size = np.zeros(slots.shape)
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            if 0 <= slots[t, j] < y.shape[0]:
                out[t, j] = grad[t] @ y[slots[t, j]]
                size[t, j] = np.abs(grad[t]) @ np.abs(y[slots[t, j]])
    return out, size
