"""CPU oracle of the serving operators (test infrastructure only): plain NumPy
in float64, one sequence, token or row at a time, from the definitions in
include/wq.h. It shares no code with the GPU path.

Caches are float64 arrays [P, 2, Hkv, S, D] of the values that the codes stand
for before their scales.
"""

import math

import numpy as np


def e4m3_values():
    """The 256 values of e4m3 (4 exponent bits of bias 7, 3 fraction bits, one
    NaN per sign and no infinity)."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if e == 15 and f == 7:
            v = math.nan
        out[c] = -v if c & 128 else v
    return out


def e4m3_codes(x):
    """The code of the nearest e4m3 value (ties to the even code), beyond the
    largest the largest; x float64 without NaN."""
    grid = e4m3_values()[:127]  # 0 .. 448, ascending
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(a >= grid[126], 126, pick)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def token_places(table, P, S, seq, pos):
    """(page, slot) of each token, page -1 where the token is left out."""
    out = []
    B, W = table.shape
    for s, p in zip(seq, pos):
        page = -1
        if 0 <= s < B and 0 <= p < W * S:
            page = int(table[s, p // S])
            if not 0 <= page < P:
                page = -1
        out.append((page, int(p) % S))
    return out


def attn_decode(q, kv, table, lens, sm_scale, window=0, k_scale=None, v_scale=None):
    """(out [B, Hq, D], lse [B, Hq], pages left out, score bound): the last is
    the largest sm_scale * sum |q k| met, for error bounds."""
    P, _, H, S, D = kv.shape
    B, Hq, _ = q.shape
    W = table.shape[1]
    G = Hq // H
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    bad, bound = 0, 0.0
    for b in range(B):
        n = min(max(int(lens[b]), 0), W * S)
        first = max(0, n - window) if window else 0
        if n <= first:
            continue
        pages = {j for j in range(first // S, (n - 1) // S + 1)}
        gone = {j for j in pages if not 0 <= table[b, j] < P}
        bad += len(gone)
        t = np.array([i for i in range(first, n) if i // S not in gone], dtype=np.int64)
        if t.size == 0:
            continue
        page, slot = table[b, t // S], t % S
        for h in range(Hq):
            g = h // G
            k = kv[page, 0, g, slot] * (1.0 if k_scale is None else float(k_scale[g]))
            v = kv[page, 1, g, slot] * (1.0 if v_scale is None else float(v_scale[g]))
            with np.errstate(invalid="ignore"):
                x = sm_scale * (k @ q[b, h])
                bound = max(bound, float(np.max(abs(sm_scale) * (np.abs(k) @ np.abs(q[b, h])))))
            m = np.max(x)
            if m == -np.inf:
                continue
            p = np.exp(x - m)
            out[b, h] = p @ v / p.sum()
            lse[b, h] = m + np.log(p.sum())
    return out, lse, bad, bound


def pages_of(n, S, W):
    return min(W, (max(int(n), 0) + S - 1) // S)


def pages_fork(table, lens, ref, S, parent, child):
    """(table, lens, ref, granted, [(from, to)])."""
    B, W = table.shape
    P = len(ref)
    t2, l2, r2 = table.copy(), lens.copy(), ref.copy()
    free = [p for p in range(P) if ref[p] == 0]
    asked, granted, moves = 0, [], []
    for a, c in zip(parent, child):
        ok = 0 <= a < B and 0 <= c < B and a != c
        n = min(max(int(lens[a]), 0), W * S) if ok else 0
        need = int(n % S != 0)
        at = asked
        asked += need
        ok = ok and (need == 0 or asked <= len(free))
        granted.append(int(ok))
        if 0 <= c < B:
            l2[c] = n if ok else 0
        if not ok:
            continue
        for j in range(n // S):
            t2[c, j] = table[a, j]
            if 0 <= table[a, j] < P:
                r2[table[a, j]] += 1
        if need:
            to = free[at]
            t2[c, n // S] = to
            r2[to] = 1
            moves.append((int(table[a, n // S]), to))
    return t2, l2, r2, np.array(granted, dtype=np.int32), moves


def pages_reserve(table, lens, new_lens, ref, S):
    """(table, ref, granted)."""
    B, W = table.shape
    t2, r2 = table.copy(), ref.copy()
    free = [p for p in range(len(ref)) if ref[p] == 0]
    asked, granted = 0, []
    for b in range(B):
        fits = new_lens[b] <= W * S
        have, want = pages_of(lens[b], S, W), pages_of(new_lens[b], S, W)
        need = max(0, want - have) if fits else 0
        at = asked
        asked += need
        ok = fits and (need == 0 or asked <= len(free))
        granted.append(int(ok))
        if ok:
            for j in range(need):
                t2[b, have + j] = free[at + j]
                r2[free[at + j]] = 1
    return t2, r2, np.array(granted, dtype=np.int32)


def pages_free(table, lens, ref, S, seqs):
    """(lens, ref, bad)."""
    B, W = table.shape
    l2, r2, bad = lens.copy(), ref.copy(), 0
    for b in seqs:
        if not 0 <= b < B:
            bad += 1
            continue
        for j in range(pages_of(lens[b], S, W)):
            p = table[b, j]
            if 0 <= p < len(ref) and r2[p] > 0:
                r2[p] -= 1
            else:
                bad += 1
        l2[b] = 0
    return l2, r2, bad


def pages_compact(table, lens, ref, S):
    """(table, ref, remap, n_live, [(from, to)])."""
    B, W = table.shape
    P = len(ref)
    n = int(np.count_nonzero(ref))
    movers = [p for p in range(n, P) if ref[p]]
    holes = [p for p in range(n) if not ref[p]]
    remap = np.array([p if ref[p] else -1 for p in range(P)], dtype=np.int32)
    r2 = ref.copy()
    for s, d in zip(movers, holes):
        remap[s], r2[d], r2[s] = d, ref[s], 0
    t2 = table.copy()
    for b in range(B):
        for j in range(pages_of(lens[b], S, W)):
            p = table[b, j]
            t2[b, j] = remap[p] if 0 <= p < P else -1
    return t2, r2, remap, n, list(zip(movers, holes))


def token_logprobs(logits, ids, top_k, temperature):
    """(logprob, rank, entropy, top_logprobs, top_ids, bad); logits float64 [T, V]."""
    T, V = logits.shape
    lp, rank, ent = np.full(T, -np.inf), np.zeros(T, dtype=np.int32), np.zeros(T)
    top, top_ids, bad = np.empty((T, top_k)), np.empty((T, top_k), dtype=np.int32), 0
    for t in range(T):
        x = logits[t]
        # value down, NaN first, then the id up
        order = np.lexsort((np.arange(V), -np.where(np.isnan(x), 0.0, x), ~np.isnan(x)))
        with np.errstate(invalid="ignore"):
            m = np.max(x)
            if m == -np.inf:
                y = np.full(V, -np.inf)
                ent[t] = 0.0
            else:
                d = (x - m) / temperature
                e = np.exp(d)
                y = d - np.log(e.sum())
                ent[t] = np.log(e.sum()) - np.sum(np.where(d == -np.inf, 0.0, e * d)) / e.sum()
                if np.isnan(e.sum()):
                    y, ent[t] = np.full(V, np.nan), np.nan
        top_ids[t], top[t] = order[:top_k], y[order[:top_k]]
        if 0 <= ids[t] < V:
            lp[t], rank[t] = y[ids[t]], 1 + int(np.nonzero(order == ids[t])[0][0])
        else:
            bad += 1
    return lp, rank, ent, top, top_ids, bad
