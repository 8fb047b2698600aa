"""The training-objective operators in 64 bits, one row at a time, from their
definitions in include/scape.h (test infrastructure: numpy, no code of the
package), and bounds on how far fp32 arithmetic may be from them.

Bounds.  U = 2^-24 is fp32's unit roundoff.  A term exp((x - m) c) of a softmax
sum carries a relative error of about 3U |x - m| c (the difference, the factor,
the product) and 4U of the exponential; weighted by the softmax the first is at
most 3U (ln V + 1), as sum p |log p| <= ln V.  Adding n terms in a tree whose
longest path has V/256 + 64 additions adds U for each.  So log sum exp is off
by at most lse_tol(V) absolutely, and by a rounding of its own size.
"""
import numpy as np

U = 2.0 ** -24
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half a unit in the last place (8, 11, 24 significant bits)
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-38}             # half the least denormal (flushed: least normal)


def lse_tol(V, lse=0.0):
    lse = abs(lse) if np.isfinite(lse) else 0.0
    return U * (V / 256 + 64 + 3 * (np.log(V) + 1) + 4 + 4 * lse)


def lse(x):
    m = np.max(x, initial=-np.inf)
    if not np.isfinite(m):
        return m
    return m + np.log(np.sum(np.exp(x - m)))


def topk(x, k):
    """Indices of the k largest, descending, ties by index, NaN first."""
    key = np.where(np.isnan(x), np.inf, x) + 0.0
    return np.lexsort((np.arange(x.size), -key, ~np.isnan(x)))[:k]


def distill(x, idx, vals, tlse, y, w, tau, kd, ce):
    """(loss, its bound, grad, its bound before rounding) of one row."""
    V = x.size
    if w == 0:
        return 0.0, 0.0, np.zeros(V), np.zeros(V)
    s = x / tau
    L, L1 = lse(s), lse(x)
    smax = np.max(np.abs(s[np.isfinite(s)]), initial=0.0)
    p, p1 = np.exp(s - L), np.exp(x - L1)
    ok = (idx >= 0) & (idx < V)
    at = idx[ok]
    t = vals[ok].astype(np.float64) / tau
    has = bool(np.any(t > -np.inf))
    loss, bound = 0.0, 0.0
    grad, gb = np.zeros(V), np.zeros(V)
    with np.errstate(divide="ignore", invalid="ignore"):
        if has:
            q = np.exp(t - (lse(t) if tlse is None else tlse))
            tmax = np.max(np.abs(t[t > -np.inf]))
            eq = U * (8 + 6 * tmax + 6 * (abs(tlse) if tlse is not None else 0.0) + at.size / 8)  # relative, of a q
            es = lse_tol(V, L) + U * 6 * smax                                                   # relative, of a p
            kl = np.sum(np.where(q > 0, q * (np.log(q) - (s[at] - L)), 0.0))
            size = np.sum(np.where(q > 0, q * (np.abs(np.log(q)) + np.abs(s[at] - L) + 1), 0.0))
            e = np.sum(q) * (eq + es) + eq * size + U * 16 * size
            qr, Q = 0.0, np.sum(q)
            dq = eq * Q + 2 * U  # of q_rest
            if tlse is not None:
                rest = np.ones(V, bool)
                rest[at] = False
                Lr = lse(s[rest])
                if Lr > -np.inf:
                    qr = max(0.0, 1.0 - Q)
                    soft = np.where(rest, np.exp(s - Lr), 0.0)
                    if qr > 0:
                        kl += qr * (np.log(qr) - (Lr - L))
                    # the bucket's value changes by at most this when q_rest is off by dq
                    e += dq * (2 + np.abs(np.log(max(qr, dq))) + np.abs(Lr - L)) + (qr + dq) * 2 * (es + 8 * U)
                    grad -= kd * tau * qr * soft
                    gb += kd * tau * soft * (dq + qr * 4 * es) + kd * tau * 8 * U * soft * (qr + np.exp(Lr - L))
            loss += kd * tau ** 2 * kl
            bound += abs(kd) * tau ** 2 * e
            gk = p * (Q + qr)
            gl = np.zeros(V)
            np.add.at(gl, at, q)
            grad += kd * tau * (gk - gl)
            gb += abs(kd) * tau * (gk * (2 * es + 2 * eq + 16 * U) + p * 2 * dq + gl * (eq + 8 * U))
        if 0 <= y < V:
            e1 = lse_tol(V, L1) + U * 6 * np.max(np.abs(x[np.isfinite(x)]), initial=0.0)
            loss += ce * (L1 - x[y])
            bound += abs(ce) * (e1 + 4 * U * (abs(L1) + abs(x[y]) if np.isfinite(x[y]) else 0.0))
            h = p1.copy()
            h[y] -= 1
            grad += ce * h
            gb += abs(ce) * (p1 * (2 * e1 + 16 * U) + 2 * U * (np.arange(V) == y))
    w = float(w)
    return w * loss, abs(w) * (bound + 8 * U * abs(loss)), w * grad, abs(w) * gb + 8 * U * abs(w) * np.abs(grad)


def route(x, k, cu, valid, renorm):
    """Forward over all tokens: idx, weights, counts, live, balance, z."""
    T, E = x.shape
    G = len(cu) - 1
    idx, wts = np.full((T, k), -1), np.zeros((T, k))
    counts, P, live = np.zeros((G, E), np.int64), np.zeros((G, E)), np.zeros(G, np.int64)
    z = 0.0
    for g in range(G):
        for t in range(cu[g], cu[g + 1]):
            if not valid[t] or not np.any(x[t] > -np.inf):
                continue
            L = lse(x[t])
            p = np.exp(x[t] - L)
            at = topk(x[t], k)
            idx[t] = at
            wts[t] = np.exp(x[t][at] - (lse(x[t][at]) if renorm else L))
            counts[g][at] += 1
            P[g] += p
            live[g] += 1
            z += L * L
    used = live > 0
    tg = np.maximum(live, 1)[:, None]
    bal = np.sum(E * counts / (k * tg) * P / tg) / max(1, used.sum())
    return idx, wts, counts, np.concatenate([live, [live.sum(), used.sum()]]), bal, z / max(1, live.sum())


def route_grad(x, idx, counts, live, cu, dw, dl, renorm):
    T, E = x.shape
    G, k = len(cu) - 1, idx.shape[1]
    g_of = np.searchsorted(np.asarray(cu[1:]), np.arange(T), side="right")
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if idx[t, 0] < 0:
            continue
        L = lse(x[t])
        p = np.exp(x[t] - L)
        g = g_of[t]
        d = dl[0] / max(1, live[G + 1]) * E * counts[g] / (k * float(live[g]) ** 2)
        zt = 2 * dl[1] / max(1, live[G]) * L
        out[t] = p * (d - p @ d) + zt * p
        size[t] = p * (np.abs(d) + p @ np.abs(d) + abs(zt))
        at = idx[t]
        w = np.exp(x[t][at] - (lse(x[t][at]) if renorm else L))
        dot, adot = w @ dw[t], w @ np.abs(dw[t])
        if renorm:
            out[t][at] += w * (dw[t] - dot)
        else:
            out[t][at] += w * dw[t]
            out[t] -= p * dot
            size[t] += p * adot
        size[t][at] += w * (np.abs(dw[t]) + adot)
    return out, size
