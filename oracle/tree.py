"""64-bit CPU definitions of the drafted-tree operators, of sampling and of
distillation (numpy, one row at a time, no code shared with the library)."""
import math

import numpy as np


def tree_mask(parents):
    """Ancestor words [B, N, ceil(N / 32)] uint32 of trees [B, N] (see nc_tree_mask)."""
    B, N = parents.shape
    out = np.zeros((B, N, (N + 31) // 32), np.uint32)
    for b in range(B):
        for i in range(N):
            path, at = [], i
            while at >= 0:
                path.append(at)
                at = parents[b, at] if parents[b, at] < at else -2
            if at == -1:
                for j in path:
                    out[b, i, j // 32] |= np.uint32(1 << (j % 32))
    return out


def _sees(words, i, N):
    return [j for j in range(N) if (int(words[i, j // 32]) >> (j % 32)) & 1]


def tree_attention(q, kv, cache, lens, mask, window):
    """q [B, N, H, D], kv [B, N, 2, Hkv, D], cache [B, T, 2, Hkv, D] float64 -> [B, N, H, D]."""
    B, N, H, D = q.shape
    Hkv = kv.shape[3]
    out = np.zeros_like(q)
    for b in range(B):
        n = int(lens[b])
        path = [_sees(mask[b], i, N) for i in range(N)]
        for i in range(N):
            if i not in path[i]:
                continue
            p = n + len(path[i]) - 1
            ts = [t for t in range(n) if window <= 0 or p - t < window]
            js = [j for j in path[i] if j in path[j] and (window <= 0 or len(path[i]) - len(path[j]) < window)]
            for h in range(H):
                g = h // (H // Hkv)
                k = np.concatenate([cache[b, ts, 0, g], kv[b, js, 0, g]])
                v = np.concatenate([cache[b, ts, 1, g], kv[b, js, 1, g]])
                s = k @ q[b, i, h] / math.sqrt(D)
                e = np.exp(s - s.max())
                out[b, i, h] = e @ v / e.sum()
    return out


def tree_accept(tokens, parents, mask, sampled, lens, T_max):
    """[(path, next)] of every row."""
    B, N = tokens.shape
    res = []
    for b in range(B):
        used = [bool((int(mask[b, j, j // 32]) >> (j % 32)) & 1) for j in range(N)]
        at, path, nxt = (0 if used[0] else None), [], tokens[b, 0]
        while at is not None and lens[b] + len(path) < T_max:
            path.append(at)
            nxt = sampled[b, at]
            at = next((j for j in range(at + 1, N) if used[j] and parents[b, j] == at and tokens[b, j] == nxt), None)
        res.append((path, int(nxt)))
    return res


def sample_row(l, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, slack) of one row of float32 logits: slack is the distance, as a
    share of the kept mass, of u from the nearest border of the token's interval."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    top = l.max()
    if top == -np.inf:
        return -1, -math.inf, 1.0
    if not T > 0:
        return int(np.argmax(l)), 0.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(l == top, 1.0, np.where(l == -np.inf, 0.0, np.exp((l - top) / T)))
    order = np.lexsort((np.arange(len(l)), -l))
    if 0 < top_k < len(l):
        order = order[:top_k]
    if not top_p >= 1:
        z = math.fsum(w[order])
        before = np.cumsum(w[order]) - w[order]
        n = max(1, int((before < (top_p if top_p > 0 else 0.0) * z).sum()))
        order = order[:n]
    if min_p > 0:
        order = order[w[order] >= min(min_p, 1.0)]
    kept = np.sort(order)
    kept = kept[w[kept] > 0]
    cum = np.cumsum(w[kept])
    x = min(max(u, 0.0), 1.0) * cum[-1] if u == u else 0.0
    i = min(int((cum <= x).sum()), len(kept) - 1)
    lo = cum[i - 1] if i else -1.0
    return int(kept[i]), math.log(w[kept[i]] / cum[-1]) if w[kept[i]] else -math.inf, min(x - lo, cum[i] - x) / cum[-1]


def distill_row(z, idx, t, tau, cap, weight=1.0):
    """(loss, dz) of one row."""
    z = z.astype(np.float64)
    V = len(z)
    l = cap * np.tanh(z / cap) if cap > 0 else z
    ok = (idx >= 0) & (idx < V) & (t > -np.inf)
    if not ok.any():
        return 0.0, np.zeros(V)
    i, t = idx[ok], t[ok].astype(np.float64) / tau
    lq = t - t.max()
    lq = lq - math.log(np.exp(lq).sum())
    x = l / tau - (l / tau).max()
    lp = x - math.log(np.exp(x).sum())
    loss = tau * tau * float((np.exp(lq) * (lq - lp[i])).sum())
    d = np.exp(lp)
    np.subtract.at(d, i, np.exp(lq))
    d *= weight * tau
    if cap > 0:
        d *= 1 - (l / cap) ** 2
    return loss, d


def sample_units(l, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob) of one row as nc_sample defines it: weights rounded to units of 2^-sh, sums of
    whole numbers.  u, top_p and min_p as exact fractions; few distinct logits (each costs a 60-digit exponential)."""
    from decimal import Decimal, getcontext
    from fractions import Fraction
    getcontext().prec = 60
    V = len(l)
    sh = min(62 - (V - 1).bit_length(), 51)
    top = l.max()
    vals, which = np.unique(l, return_inverse=True)
    units = [int((((Decimal(float(v)) - Decimal(float(top))) / Decimal(T)).exp() * (1 << sh)).to_integral_value()) for v in vals]
    w = np.array(units, np.int64)[which]  # sums stay under 2^63
    order = np.lexsort((np.arange(V), -l))
    if 0 < top_k < V:
        order = order[:top_k]
    if top_p < 1:
        c = np.cumsum(w[order])
        want = Fraction(max(top_p, 0.0)) * int(c[-1])
        order = order[:max(1, int(np.searchsorted(c - w[order], -(-want.numerator // want.denominator), side="left")))]
    if min_p > 0:
        least = Fraction(min(min_p, 1.0)) * (1 << sh)
        order = order[w[order] >= -(-least.numerator // least.denominator)]
    kept = np.sort(order)
    kept = kept[w[kept] > 0]
    c = np.cumsum(w[kept])
    x = Fraction(min(max(u, 0.0), 1.0)) * int(c[-1])
    i = min(int(np.searchsorted(c, x.numerator // x.denominator, side="right")), len(kept) - 1)
    return int(kept[i]), float(l[kept[i]] - top) / T - math.log(int(c[-1])) + sh * math.log(2)
