"""Plain 64-bit implementations of the calls on drafted tokens."""
import numpy as np


def ancestors(par):
    """[n, n] bool: j on the path from i to the root."""
    n = len(par)
    a = np.zeros((n, n), bool)
    for i in range(n):
        if par[i] >= 0:
            a[i] = a[par[i]]
        a[i, i] = True
    return a


def random_tree(rng, n, roots=1, spread=4):
    """parent[i] < i; the first `roots` nodes follow the cache directly."""
    par = np.full(n, -1, np.int32)
    for i in range(roots, n):
        par[i] = rng.integers(max(0, i - spread), i)
    return par


def attention(q, k, v, kc, vc, par):
    """q [n, H, D], k, v [n, Hkv, D], kc, vc [Hkv, len, D] (float64): out
    [n, H, D], lse [H, n], the bound sum_j p_j |v_j| of a relative error of the
    probabilities, and the largest sum of |q_d k_d| / sqrt(D)."""
    n, H, D = q.shape
    Hkv, L = kc.shape[:2]
    see = np.concatenate([np.ones((n, L), bool), ancestors(par)], 1)
    out, mag = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, amax = np.zeros((H, n)), 0.0
    for h in range(H):
        g = h // (H // Hkv)
        K = np.concatenate([kc[g], k[:, g]])
        V = np.concatenate([vc[g], v[:, g]])
        for i in range(n):
            s = K[see[i]] @ q[i, h] / np.sqrt(D)
            amax = max(amax, float((np.abs(K[see[i]]) @ np.abs(q[i, h])).max() / np.sqrt(D)))
            m = s.max()
            p = np.exp(s - m)
            z = p.sum()
            out[i, h] = (p / z) @ V[see[i]]
            mag[i, h] = (p / z) @ np.abs(V[see[i]])
            lse[h, i] = m + np.log(z)
    return out, lse, mag, amax


def weights(z, T, top_k, top_p):
    """Integer weights of a row of fp32 logits, as Python-exact int64."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, np.float64))
    V = len(z)
    w = np.zeros(V, np.int64)
    best = int(np.argmax(z))
    if T == 0:
        w[best] = 2 ** 36
        return w
    with np.errstate(invalid="ignore"):
        d = np.where(z == z[best], 0.0, z[best] - z)
    w = np.rint(np.exp(-d / float(np.float32(T))) * 2.0 ** 36).astype(np.int64)
    order = sorted(range(V), key=lambda i: (-z[i], i)) if V < 2000 else \
        np.lexsort((np.arange(V), -z))
    order = np.asarray(order)
    if top_k > 0:
        w[order[top_k:]] = 0
    if top_p < 1:
        goal = float(np.float32(top_p)) * float(w.sum())
        before = np.concatenate([[0], np.cumsum(w[order])[:-1]]).astype(np.float64)
        w[order[before >= goal]] = 0
    return w


def verify(logits, draft, tokens, par, u, T, top_k, top_p):
    """One sequence: (accepted nodes, next token)."""
    n, V = logits.shape
    u = np.clip(np.nan_to_num(u.astype(np.float64), nan=0.0), 0.0, 1.0)
    cur, path = 0, [0]
    while True:
        w = weights(logits[cur], T, top_k, top_p)
        kids = [i for i in range(cur + 1, n) if par[i] == cur]
        x = weights(draft[cur], T, top_k, top_p) if draft is not None and kids else None
        for c in kids:
            t, S = int(tokens[c]), float(w.sum())
            real = 0 <= t < V
            wt = float(w[t]) if real else 0.0
            if x is None:
                ok = u[c] * S < wt
                left = w.copy()
                if real:
                    left[t] = 0
            else:
                f = S / float(x.sum())
                ok = u[c] * ((float(x[t]) if real else 0.0) * f) < wt
                left = np.maximum(w - np.rint(x * f).astype(np.int64), 0)
            if ok:
                cur = c
                path.append(c)
                break
            if left.sum() > 0:
                w = left
        else:
            cum = np.cumsum(w).astype(np.float64)
            over = np.nonzero(cum > u[0] * cum[-1])[0]
            return path, int(over[0] if len(over) else np.nonzero(w)[0][-1])
