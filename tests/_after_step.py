"""Plain 64-bit forms of the calls that follow a step (draft verification,
attention-weight accumulation, eviction), from their definitions."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def dequant(codes, scales):
    """MXFP4 rows -> float64 [rows, n]."""
    codes = np.asarray(codes)
    v = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    v[..., 0::2] = E2M1[codes & 15]
    v[..., 1::2] = E2M1[codes >> 4]
    return v * np.repeat(np.exp2(np.asarray(scales).astype(np.float64) - 127), 32, axis=-1)


def prob(x):
    x = np.asarray(x, np.float64)
    return np.where(x > 0, x, 0.0)


def verify(target, draft, tokens, q_off, u, r):
    """(n_accept, next_tok) of every sequence; probabilities as float64 arrays."""
    V = target.shape[1]
    B = len(q_off) - 1
    n_acc, nxt = np.zeros(B, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        lo, hi = int(q_off[b]), int(q_off[b + 1])
        if hi <= lo:
            continue
        a = 0
        while lo + a + 1 < hi:
            i, x = lo + a, int(tokens[lo + a + 1])
            if not 0 <= x < V:
                break
            q = prob(draft[i, x]) if draft is not None else 1.0
            if not float(u[i]) * q < prob(target[i, x]):
                break
            a += 1
        i = lo + a
        w = prob(target[i])
        if i + 1 < hi:
            x = int(tokens[i + 1])
            if draft is not None:
                less = np.maximum(w - prob(draft[i]), 0)
            else:
                less = w.copy()
                if 0 <= x < V:
                    less[x] = max(w[x] - 1.0, 0.0)
            if less.sum() > 0:
                w = less
        n_acc[b] = a
        if w.sum() > 0:
            c = np.cumsum(w)
            hit = np.nonzero((c > float(r[b]) * c[-1]) & (w > 0))[0]
            nxt[b] = hit[0] if len(hit) else np.nonzero(w > 0)[0][-1]
    return n_acc, nxt


def weights(q, codes, scales, row_of, topk, lse, sm_scale, q_seq, counted):
    """(weights [Q, k], absolute sums A [Q, k]) in float64.  row_of(seq, positions) -> cache rows."""
    Q, k = topk.shape
    w, A = np.zeros((Q, k)), np.zeros((Q, k))
    for i in range(Q):
        if not counted[i]:
            continue
        slot = np.nonzero(topk[i] >= 0)[0]
        if not len(slot):
            continue
        rows = row_of(q_seq[i], topk[i][slot].astype(np.int64))
        key = dequant(codes[rows], scales[rows])
        x = (q[i].astype(np.float64) @ key.T) * sm_scale
        L = lse[i].astype(np.float64)[:, None]
        with np.errstate(invalid="ignore"):
            w[i, slot] = np.where(np.isneginf(L), 0.0, np.exp(x - L)).sum(0)
        A[i, slot] = (np.abs(q[i].astype(np.float64)) @ np.abs(key).T).max(0) * sm_scale
    return w, A


def rank(a):
    """Sort key of accumulated weights: NaN below every number, -0 as +0."""
    a = np.asarray(a, np.float64) + 0.0
    return np.where(np.isnan(a), -np.inf, a), ~np.isnan(a)


def evict_positions(acc, keep, first, last):
    """Kept positions (ascending) of one sequence whose entries carry acc [L]."""
    L = len(acc)
    n = min(max(int(keep), 0), L)
    l = min(last, n)
    f = min(first, n - l)
    mid = np.arange(f, L - l)
    val, num = rank(acc[mid])
    order = np.lexsort((mid, -val, ~num))     # numbers first, value descending, position ascending
    best = np.sort(mid[order[:n - f - l]])
    return np.concatenate([np.arange(f), best, np.arange(L - l, L)]).astype(np.int64)
