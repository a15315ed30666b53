"""Float64 definitions of the operators that pick weights by token: the router of
a mixture of experts and its gradient, the rows in the experts' order and back,
that gradient, and low-rank adapters. Plain loops over numpy arrays; nothing here
is shared with the GPU path."""

import math

import numpy as np


def _rank(x):
    """Where a logit stands in the order of the choice: NaN, then larger ones."""
    return (0, 0.0) if math.isnan(x) else (1, -x)


def _exp(x):
    return 0.0 if x == -math.inf else float(np.exp(np.float64(x)))


def _sigmoid(x):
    return 1.0 / (1.0 + math.exp(-x)) if x > -700 else math.exp(x)


def _log_sigmoid(x):
    return -math.log1p(math.exp(-x)) if x > 0 else x - math.log1p(math.exp(x))


def _scores(row, score):
    """Scores of a row's logits; a row of nothing but -inf has none."""
    if score == "sigmoid":
        return [x if math.isnan(x) else (_sigmoid(x) if x > -math.inf else 0.0) for x in row]
    if any(math.isnan(x) or x == math.inf for x in row):
        return [math.nan] * len(row)
    m = max(row)
    if m == -math.inf:
        return [0.0] * len(row)
    e = [_exp(x - m) for x in row]
    return [v / math.fsum(e) for v in e]


def _shares(chosen, score):
    """Scores of the chosen logits over their sum, also where every score is below the smallest number."""
    if any(math.isnan(x) for x in chosen):
        return [math.nan] * len(chosen)
    if score == "softmax":
        return _scores(chosen, score)
    logs = [_log_sigmoid(x) if x < math.inf else 0.0 for x in chosen]
    m = max(logs)
    e = [_exp(x - m) for x in logs]
    return [v / math.fsum(e) for v in e]


def route(logits, k, score, renormalize, scale):
    """(ids [T, k], weights [T, k])."""
    T, E = logits.shape
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        row = [float(x) for x in logits[t]]
        order = sorted((e for e in range(E) if row[e] != -math.inf), key=lambda e: (_rank(row[e] + 0.0), e))[:k]
        ids[t, :len(order)] = order
        if not order:
            continue
        p = _shares([row[e] for e in order], score) if renormalize else np.array(_scores(row, score))[order]
        weights[t, :len(order)] = scale * np.array(p)
    return ids, weights


def route_grad(logits, ids, dweights, score, renormalize, scale):
    """dlogits [T, E] from the Jacobian of each row's weights, one entry at a time."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        row = [float(x) for x in logits[t]]
        at = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and row[ids[t, j]] != -math.inf]
        es = [int(ids[t, j]) for j in at]
        g = [scale * float(dweights[t, j]) for j in at]
        if renormalize:
            if not es:
                continue
            p = _shares([row[e] for e in es], score)
            for i, e in enumerate(es):
                slope = _sigmoid(-row[e]) if score == "sigmoid" else 1.0
                out[t, e] += slope * math.fsum(g[j] * p[j] * ((i == j) - p[i]) for j in range(len(es)))
        elif score == "sigmoid":
            for e, v in zip(es, g):
                out[t, e] += v * _sigmoid(row[e]) * _sigmoid(-row[e])
        else:
            s = _scores(row, score)
            for e in range(E):
                out[t, e] = math.fsum(v * s[i] * ((i == e) - s[e]) for i, v in zip(es, g))
    return out


def sort(ids, E):
    """(offsets [E + 1], slots like ids, choices without an expert)."""
    flat = ids.reshape(-1)
    slots, at = np.full(flat.shape, -1, np.int32), 0
    offsets = np.zeros(E + 1, np.int32)
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        slots[mine] = at + np.arange(mine.size)
        at += mine.size
        offsets[e + 1] = at
    return offsets, slots.reshape(ids.shape), int(flat.size - at)


def combine(y, slots, weights=None, residual=None):
    """(out [T, D], the sums of the terms' sizes)."""
    T, k = slots.shape
    out, size = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    if residual is not None:
        out += residual
        size += np.abs(residual)
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < y.shape[0]:
                term = y[slots[t, j]] * (1.0 if weights is None else weights[t, j])
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_grad(dout, y, slots, weights, dy):
    """(dy, with the named rows written, dweights [T, k], the sums of the products' sizes)."""
    dy, dw, size = dy.copy(), np.zeros(slots.shape), np.zeros(slots.shape)
    for t, j in np.ndindex(slots.shape):
        s = slots[t, j]
        if 0 <= s < y.shape[0]:
            dy[s] = weights[t, j] * dout[t]
            dw[t, j] = dout[t] @ y[s]
            size[t, j] = np.abs(dout[t]) @ np.abs(y[s])
    return dy, dw, size


def lora(x, A, B, adapter, base, scale=None):
    """(y [M, N], the sums of sizes of the first product's terms carried through the second, of the second's)."""
    n, r, K = A.shape
    y, first, second = base.copy(), np.zeros(base.shape), np.zeros(base.shape)
    for m, a in enumerate(adapter):
        if not 0 <= a < n:
            continue
        s = 1.0 if scale is None else scale[a]
        h = A[a] @ x[m]
        y[m] += s * (B[a] @ h)
        first[m] = abs(s) * (np.abs(B[a]) @ (np.abs(A[a]) @ np.abs(x[m])))
        second[m] = abs(s) * (np.abs(B[a]) @ np.abs(h))
    return y, first, second
