"""fp64 numpy oracle of differential attention and of rotary positions with
several axes, with elementwise bounds on what 16-bit roundings may do to them.

Layouts as the library's: q [B, Sq, H, 2, D], k [B, Sk, Hk, 2, D],
v [B, Sk, Hk, Dv], lam broadcastable to [B, Sq, H], lse [2, B, H, Sq].

Formulas, per head: P_c = softmax(scale q_c k_c^T + mask), W = P_1 - lam P_2,
O = W V, O_2 = P_2 V; with G = dO: dV = W^T G, dP = G V^T, Delta_c =
rowsum(P_c dP), dS_1 = P_1 (dP - Delta_1), dS_2 = -lam P_2 (dP - Delta_2),
dq_c = scale dS_c k_c, dk_c = scale dS_c^T q_c, dlam = -Delta_2.

Bounds. u is the largest relative rounding error of the 16-bit type (half a
step) and t half its smallest subnormal step (0 for bf16, whose range is
fp32's). The kernels round P_c (or W) once before a product, every dS_c once,
O and O_2 once (both are read again by the backward), every output once; EXP
covers the fp32 part: a polynomial exp2 of relative error 7.5e-5 in numerator
and denominator, the logsumexp, and fp32 sums.
"""
from __future__ import annotations

import numpy as np

EXP = 5e-4


def visible(Sq, Sk, causal, n_keys=None):
    """bool [Sq, Sk]: which keys each row sees; n_keys limits the keys and moves the causal diagonal."""
    n = Sk if n_keys is None else int(n_keys)
    j, i = np.arange(Sk)[None, :], np.arange(Sq)[:, None]
    see = np.broadcast_to(j < n, (Sq, Sk))
    return see & (j <= i + (n - Sq)) if causal else see


def softmax_rows(x, see):
    """(P, LSE) of one map; rows that see nothing give P = 0 and LSE = -inf."""
    x = np.where(see, x, -np.inf)
    top = x.max(axis=1, initial=-np.inf)
    e = np.exp(x - np.where(np.isfinite(top), top, 0.0)[:, None])
    total = e.sum(axis=1)
    some = total > 0
    lse = np.full(total.shape, -np.inf)
    lse[some] = top[some] + np.log(total[some])
    return e / np.where(some, total, 1.0)[:, None], lse


def differential(q, k, v, lam, scale, causal, do=None, n_keys=None, u=0.0, t=0.0):
    """Dict of o, o2, lse (and with do: dq, dk, dv, dlam in [B, Sq, H]) and, under
    the same names with "_bound", the elementwise bounds for roundings u, t."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, Sq, H, _, D = q.shape
    Sk, Hk, Dv = v.shape[1:]
    lam = np.broadcast_to(np.asarray(lam, np.float64), (B, Sq, H))
    z = {n: np.zeros((B, Sq, H, Dv)) for n in ("o", "o2", "o_bound", "o2_bound")}
    z["lse"] = np.full((2, B, H, Sq), -np.inf)
    if do is not None:
        do = np.asarray(do, np.float64)
        for n, like in (("dq", q), ("dk", k), ("dv", v), ("dlam", lam)):
            z[n], z[n + "_bound"] = np.zeros(like.shape), np.zeros(like.shape)
    for b in range(B):
        see = visible(Sq, Sk, causal, None if n_keys is None else n_keys[b])
        for h in range(H):
            g = h // (H // Hk)
            vals = np.where(see.any(axis=0)[:, None], v[b, :, g], 0.0) if n_keys is not None else v[b, :, g]
            p = []
            for c in (0, 1):
                keys = np.where(see.any(axis=0)[:, None], k[b, :, g, c], 0.0) if n_keys is not None else k[b, :, g, c]
                pc, z["lse"][c, b, h] = softmax_rows(scale * (q[b, :, h, c] @ keys.T), see)
                p.append(pc)
            w8 = lam[b, :, h][:, None]
            o2 = p[1] @ vals
            o = p[0] @ vals - w8 * o2
            z["o"][b, :, h], z["o2"][b, :, h] = o, o2
            av = np.abs(vals)
            sub = t * (see @ av)  # entries below the type's normal range
            e1, e2 = (u + EXP) * (p[0] @ av) + sub, (u + EXP) * (p[1] @ av) + sub
            bo = (1 + u) * (e1 + np.abs(w8) * e2) + u * np.abs(o) + t
            bo2 = (1 + u) * e2 + u * np.abs(o2) + t
            z["o_bound"][b, :, h], z["o2_bound"][b, :, h] = bo, bo2
            if do is None:
                continue
            G = do[b, :, h]
            ag = np.abs(G)
            W = p[0] - w8 * p[1]
            A = p[0] + np.abs(w8) * p[1]
            dP = G @ vals.T
            delta = [(p[c] * dP).sum(1) for c in (0, 1)]
            z["dv"][b, :, g] += W.T @ G
            z["dv_bound"][b, :, g] += (u * np.abs(W) + EXP * A + t * see).T @ ag
            z["dlam"][b, :, h] = -delta[1]
            b2 = (ag * bo2).sum(1) + 1e-5 * (ag * np.abs(o2)).sum(1)
            b1 = (ag * (bo + np.abs(w8) * bo2)).sum(1) + 1e-5 * (ag * (np.abs(o) + np.abs(w8 * o2))).sum(1)
            z["dlam_bound"][b, :, h] = b2
            for c, weight, bd in ((0, 1.0, b1), (1, -w8, b2)):
                dS = weight * p[c] * (dP - delta[c][:, None])
                aS = np.abs(weight) * p[c]
                e = (u + EXP) * np.abs(dS) + aS * (bd[:, None] + 1e-5 * (ag @ av.T)) * (1 + u) + t * see
                z["dq"][b, :, h, c] = scale * dS @ k[b, :, g, c]
                z["dq_bound"][b, :, h, c] = scale * e @ np.abs(k[b, :, g, c])
                z["dk"][b, :, g, c] += scale * dS.T @ q[b, :, h, c]
                z["dk_bound"][b, :, g, c] += scale * e.T @ np.abs(q[b, :, h, c])
    if do is not None:
        for n in ("dq", "dk", "dv"):  # 1e-5: fp32 accumulation; then the output's own rounding
            z[n + "_bound"] = (1 + u) * z[n + "_bound"] + (u + 1e-5) * np.abs(z[n]) + t + 1e-30
    return z


def rotary(x, positions, inv_freq, sections, interleaved=False, inverse=False):
    """x [B, S, heads, D] turned by positions [axes, B, S] times inv_freq [R]."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    R = len(inv_freq)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for j in range(R):
        th = np.asarray(positions[axis[j]], np.float64) * float(inv_freq[j])
        c, s = np.cos(th)[..., None], np.sin(th)[..., None] * (-1.0 if inverse else 1.0)
        ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + R)
        y[..., ia] = x[..., ia] * c - x[..., ib] * s
        y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y
