"""The vocabulary-wide post-training operators in 64 bits, written out from their definitions, and how far
a kernel that works in fp32 may be from them.

Error model, with u = 2^-24 (half a step of fp32) and D = max_v |c z_v - m| log2-units of a row's spread:
  - an exponential 2^(c z - m): the argument is rounded once (D u, times ln 2), its constant c once
    (u |d|), and the unit's result is within 2^-22 = 4 u relative;
  - a sum of V positive terms by at least 256 threads in sequence, then a tree: (V / 256 + 40) u relative
    (partial sums are rescaled at each new maximum, counted in the 40);
  - so S, and with it every probability of the row, is within EPS = (V / 256 + 60 + 3 D) u relative, a
    log-prob within EPS + 4 u |logp| + 2 u log2(V) absolute;
  - results are rounded once to their type: half a step, finfo.eps / 2.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def half_step(dtype: str) -> float:
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


class Rows:
    """Softmax quantities of every row in 64 bits, and their fp32 error bounds."""

    def __init__(self, z: np.ndarray, inv_tau: float = 1.0):
        self.z = z.astype(np.float64) * inv_tau
        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
            m = self.z.max(1, keepdims=True)
            d = np.where(np.isneginf(self.z), -np.inf, self.z - m)
            e = np.exp(d)
            s = e.sum(1, keepdims=True)
            self.p = e / s
            self.lp = d - np.log(s)
            fin = np.where(np.isfinite(d), d, 0.0)
            self.spread = np.minimum(-fin.min(1), 126.0) / np.log(2)
            self.entropy = -np.where(self.p > 0, self.p * np.where(self.p > 0, self.lp, 0), 0).sum(1)
            self.mean_d = (self.p * np.abs(fin)).sum(1) / np.log(2)
        V = z.shape[1]
        self.V = V
        self.eps = (V / 256 + 60 + 3 * self.spread) * U

    def logp_tol(self, lp):
        return self.eps + 4 * U * np.abs(np.where(np.isfinite(lp), lp, 0)) + 2 * U * np.log2(self.V + 1)


def token_logp(z, y, mask):
    r = Rows(z)
    ok = (y >= 0) & (y < z.shape[1])
    lp = np.where(ok, r.lp[np.arange(len(y)), np.where(ok, y, 0)], np.nan)
    on = mask != 0
    logp = np.where(on, lp, 0.0)
    ent = np.where(on, r.entropy, 0.0)
    ent_tol = r.eps * (1 + 2 * r.mean_d) + 4 * U * np.log2(r.V + 1)
    return r, logp, ent, r.logp_tol(lp), ent_tol


def weights(mask, cu, per_token):
    S = len(cu) - 1
    n = np.array([int((mask[a:b] != 0).sum()) for a, b in zip(cu, cu[1:])])
    w = np.zeros(len(mask))
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        if n[i]:
            w[a:b] = 1.0 / n.sum() if per_token else 1.0 / (S * n[i])
    return w * (mask != 0), n


def onehot_grad(r: Rows, g, y, dg, logp_tol, dtype):
    """g (1[v = y] - p_v) and its tolerance, for coefficients g known to dg absolute."""
    T, V = r.p.shape
    d = -g[:, None] * r.p
    live = (g != 0) & (y >= 0) & (y < V)
    d[~live] = 0.0
    at = np.where(live, y, 0)
    rows = np.arange(T)
    one = np.where(live, g * -np.expm1(np.where(live, r.lp[rows, at], -1.0)), d[rows, at])
    d[rows, at] = one
    p_y = r.p[rows, at]
    tol = half_step(dtype) * np.abs(d) + (np.abs(g) * (r.eps + 8 * U) + dg)[:, None] * r.p + 1e-37
    tol[rows, at] += np.abs(g) * p_y * logp_tol + dg + 4 * U * np.abs(one)
    return d, tol


# ---------------------------------------------------------------- the loss with a KL term

def kl_terms(kind, d):
    if kind == "k1":
        return d, np.ones_like(d)
    if kind == "k2":
        return d * d / 2, d
    return np.expm1(-d) + d, -np.expm1(-d)


def kl_loss_part(logp, logp_ref, mask, w, kind, coef):
    """coef sum_t w_t k_t, the estimates and the coefficients they add to dL/dlogp."""
    d = np.where(mask != 0, logp, 0.0) - np.where(mask != 0, logp_ref, 0.0)
    k, dk = kl_terms(kind, d)
    on = mask != 0
    return coef * (w * np.where(on, k, 0)).sum(), np.where(on, k, 0.0), np.where(on, coef * w * dk, 0.0)


# ---------------------------------------------------------------- distillation

def distill_row(z, ids, vals, mode, reverse, inv_tau, floor):
    """One row: KL and dKL/dz, by the definition over a vocabulary of outcomes."""
    z = z.astype(np.float64) * inv_tau
    V = len(z)
    m = z.max()
    lz = m + np.log(np.exp(z - m).sum())
    lp = z - lz
    p = np.exp(lp)
    sel = ids >= 0
    at, v = ids[sel], vals[sel].astype(np.float64)
    if len(at) == 0 or (mode == "renorm" and np.all(np.isneginf(v))):
        return 0.0, np.zeros(V)
    if mode == "renorm":
        mm = v.max()
        lq = v - (mm + np.log(np.exp(v - mm).sum()))
        qo = 0.0
    else:
        lq = v
        qo = max(1.0 - np.exp(v).sum(), floor)
    q = np.exp(lq)
    out = np.ones(V, bool)
    out[at] = False
    rest = out.any() and mode == "tail"
    po = p[out].sum()
    kl, d = 0.0, np.zeros(V)
    with np.errstate(divide="ignore", invalid="ignore"):
        if not reverse:
            kl = np.where(q > 0, q * (lq - lp[at]), 0.0).sum()
            d = p * (q.sum() + qo)
            d[at] -= q
            if rest:
                kl += qo * (np.log(qo) - np.log(po)) if qo > 0 else 0.0
                d[out] -= (p[out] * qo / po) if po > 0 else 0.0
                if po == 0:
                    d[out] = 0.0
        else:
            a = np.zeros(V)
            a[at] = np.where(p[at] > 0, lp[at] - lq, 0.0)
            kl = np.where(p[at] > 0, p[at] * a[at], 0.0).sum()
            if rest and po > 0:
                a[out] = np.log(po / qo)
                kl += po * np.log(po / qo)
            d = p * (a - kl)
    return kl, d * inv_tau


def distill(z, ids, vals, mask, cu, mode, reverse, tau, scale, floor, per_token):
    T, V = z.shape
    w, _ = weights(mask, cu, per_token)
    kl, d = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        if mask[t]:
            kl[t], row = distill_row(z[t], ids[t], vals[t], mode, reverse, 1.0 / tau, floor)
            d[t] = scale * w[t] * row
    return scale * (w * kl).sum(), kl, d


def distill_tol(z, ids, vals, mask, cu, mode, reverse, tau, scale, floor, per_token, dtype, kl, d):
    """Bounds from the error model: every log-prob of the student within lt, the teacher's q within
    (4 + 2 |ln q|) u relative (q_o within u relative: it is taken in 64 bits), K terms summed with at most
    K / 32 + 8 roundings of their magnitudes."""
    T, V = z.shape
    r = Rows(np.where(np.isfinite(z) | np.isneginf(z), z, 0), 1.0 / tau)
    w, _ = weights(mask, cu, per_token)
    K = ids.shape[1]
    kt, dt = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        if not mask[t] or not (ids[t] >= 0).any():
            continue
        sel = ids[t] >= 0
        at, v = ids[t][sel], vals[t][sel].astype(np.float64)
        if mode == "renorm":
            mm = v.max()
            if np.isneginf(mm):
                continue
            lq = v - (mm + np.log(np.exp(v - mm).sum()))
            qo = 0.0
        else:
            lq, qo = v, max(1.0 - np.exp(v).sum(), floor)
        q, p, lp = np.exp(lq), r.p[t], r.lp[t]
        lqf = np.where(np.isfinite(lq), lq, 0.0)
        lpf = np.where(np.isfinite(lp), lp, 0.0)
        out = np.ones(V, bool)
        out[at] = False
        po = p[out].sum()
        lt = r.logp_tol(np.abs(lpf).max())[t]
        num = (K / 32 + 8) * U
        val_err = 4 * U * (1 + (np.abs(v[np.isfinite(v)]).max() if np.isfinite(v).any() else 0))
        head = p[at] if reverse else q
        terms = head * (np.abs(lqf) + np.abs(lpf[at]))
        ko = 0.0
        if mode == "tail" and out.any():
            mo = po if reverse else qo
            lo = abs(np.log(max(po, 1e-300))) + abs(np.log(max(qo, 1e-300))) if mo > 0 else 0.0
            ko = mo * (2 * lt + (6 * U + r.eps[t]) * (1 + lo))
            terms = np.append(terms, mo * lo)
        kt[t] = (head * (lt + val_err + 8 * U * (1 + np.abs(lqf) + np.abs(lpf[at])))).sum() + num * terms.sum() + ko \
            + (r.eps[t] * terms.sum() if reverse else 0.0)
        coef = abs(scale) * w[t] / tau
        e = r.eps[t] + 8 * U
        dt[t] = half_step(dtype) * np.abs(d[t]) + coef * p * e * (2 + qo) + 1e-37
        if reverse:
            a = np.zeros(V)
            a[at] = np.where(p[at] > 0, lpf[at] - lqf, 0.0)
            if mode == "tail" and po > 0 and qo > 0:
                a[out] = np.log(po / qo)
            dt[t] += coef * p * (kt[t] + lt + val_err + (e + 8 * U) * (np.abs(a) + abs(kl[t]) + np.abs(lpf)))
        else:
            dt[t][at] += coef * q * (val_err + (4 + 2 * np.abs(lqf)) * U)
            if mode == "tail" and po > 0:
                dt[t][out] += coef * p[out] * (qo / po) * e
    loss_tol = (abs(scale) * w * kt).sum() + 2 * U * (abs(scale) * w * np.abs(np.where(np.isfinite(kl), kl, 0))).sum()
    return loss_tol, kt + U * np.abs(np.where(np.isfinite(kl), kl, 0)), dt


# ---------------------------------------------------------------- preference

def preference(z, y, ref, mask, cu, kind, mean, beta, margin, smoothing, nll, logp=None):
    r = Rows(z) if logp is None else None
    T, V = z.shape
    ok = (y >= 0) & (y < V)
    lp = r.lp[np.arange(T), np.where(ok, y, 0)] if logp is None else logp
    on = (mask != 0) & ok
    S = len(cu) - 1
    P = S // 2
    ref = np.zeros(T) if ref is None else ref.astype(np.float64)
    n = np.array([int((mask[a:b] != 0).sum()) for a, b in zip(cu, cu[1:])])
    s, like = np.zeros(S), np.zeros(S)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        o = on[a:b]
        s[i] = lp[a:b][o].sum() - ref[a:b][o].sum()
        like[i] = -lp[a:b][o].sum() / n[i] if n[i] else 0.0
        if mean:
            s[i] = s[i] / n[i] if n[i] else 0.0
    D = s[0::2] - s[1::2]
    h = beta * D - margin
    if kind == "sigmoid":
        lose, win = np.logaddexp(0, -h), np.logaddexp(0, h)
        pair = (1 - smoothing) * lose + smoothing * win
        slope = beta * (smoothing / (1 + np.exp(-h)) - (1 - smoothing) / (1 + np.exp(h)))
    elif kind == "hinge":
        pair, slope = np.maximum(0, 1 - h), np.where(h < 1, -beta, 0.0)
    else:
        pair, slope = (D - 0.5 / beta) ** 2, 2 * (D - 0.5 / beta)
    pair = pair + nll * like[0::2]
    g = np.zeros(T)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        if n[i]:
            per = 1.0 / n[i] if mean else 1.0
            gi = slope[i // 2] * per * (1 if i % 2 == 0 else -1) - (nll / n[i] if i % 2 == 0 else 0.0)
            g[a:b] = np.where(on[a:b], gi / P, 0.0)
    return dict(rows=r, logp=np.where(mask != 0, np.where(ok, lp, np.nan), 0.0), s=s, pair=pair, loss=pair.mean(), g=g,
                slope=slope, n=n)
