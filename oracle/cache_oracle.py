"""fp64 oracle of the cache operators: attention of a drafted tree, attention
that records the weight each slot received, eviction by that weight, and
acceptance of a drafted path.  Plain loops over sequences and heads, written
from the definitions; values that an operator must not look at (cache rows
behind a sequence, padding nodes) are never read here.
"""
import numpy as np


def ancestors(parents, t):
    """Node t and its ancestors, ascending; None where t does not hang on the cache."""
    chain = [t]
    while parents[chain[-1]] >= 0:
        p = int(parents[chain[-1]])
        if p >= chain[-1]:
            return None
        chain.append(p)
    return sorted(chain) if parents[chain[-1]] == -1 else None


def _softmax(s):
    e = np.exp(s - s.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def tree_attention(q, k, v, kv_lens, kn, vn, parents):
    """out [B, T, H, hd]; and per row sum_j p_j |v_j| and the largest
    sum_d |q_d k_jd| / sqrt(hd) over its keys, the scales of its rounding errors."""
    B, T, H, hd = q.shape
    rep = H // k.shape[2]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    dot = np.zeros(q.shape[:3] + (1,))
    for b in range(B):
        for t in range(T):
            chain = ancestors(parents[b], t)
            if chain is None:
                continue
            for h in range(H):
                g = h // rep
                kk = np.concatenate((k[b, :kv_lens[b], g], kn[b, chain, g]))
                vv = np.concatenate((v[b, :kv_lens[b], g], vn[b, chain, g]))
                p = _softmax(kk @ q[b, t, h] / np.sqrt(hd))
                out[b, t, h] = p @ vv
                mag[b, t, h] = p @ np.abs(vv)
                dot[b, t, h] = (np.abs(kk) @ np.abs(q[b, t, h])).max() / np.sqrt(hd)
    return out, mag, dot


def observed_attention(q, k, v, kv_lens, seq_lens, weights_in):
    """out, its error scales as tree_attention gives them, and the weights
    [B, KV, cap] (NaN where the operator writes nothing)."""
    B, S, H, hd = q.shape
    cap, KV = k.shape[1:3]
    rep = H // KV
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    dot = np.zeros(q.shape[:3] + (1,))
    weights = np.full((B, KV, cap), np.nan)
    for b in range(B):
        x, n = int(kv_lens[b]), int(seq_lens[b])
        weights[b, :, :x + n] = 0.0
        if weights_in is not None:
            weights[b, :, :x] = weights_in[b, :, :x]
        if n == 0:
            continue
        hide = np.arange(x + n)[None, :] > x + np.arange(n)[:, None]
        for h in range(H):
            g = h // rep
            kk, vv = k[b, :x + n, g], v[b, :x + n, g]
            p = _softmax(np.where(hide, -np.inf, q[b, :n, h] @ kk.T / np.sqrt(hd)))
            out[b, :n, h] = p @ vv
            mag[b, :n, h] = p @ np.abs(vv)
            dot[b, :n, h, 0] = (np.abs(q[b, :n, h]) @ np.abs(kk).T).max(-1) / np.sqrt(hd)
            weights[b, g, :x + n] += p.sum(0)
    return out, mag, dot, weights


def evict_sources(weights, slot_pos, n, position, budget, recent):
    """The slot that each of the first min(n, budget) slots of one row is filled from."""
    left = min(n, budget)
    rank = []
    for j in range(n):
        w = float(weights[j])
        if slot_pos[j] >= position - recent:
            rank.append((0, 0.0, j))
        elif w != w:
            rank.append((1, 0.0, j))
        else:
            rank.append((2, -w, j))
    kept = sorted(r[2] for r in sorted(rank)[:left])
    spare = [j for j in kept if j >= left]
    return [i if i in set(kept) else spare.pop(0) for i in range(left)]


def accept(draft, target, parents):
    """Accepted nodes of one tree in order, and the token behind the last one (-1 without)."""
    T = len(parents)
    if parents[0] != -1:
        return [], -1
    path = [0]
    while True:
        nxt = [c for c in range(T) if c > path[-1] and parents[c] == path[-1] and draft[c] == target[path[-1]]]
        if not nxt:
            return path, int(target[path[-1]])
        path.append(nxt[0])
