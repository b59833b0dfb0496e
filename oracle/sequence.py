"""The prompt scan, the single-token step and the paged cache's attention, in
fp64. TEST INFRASTRUCTURE ONLY: imported by tests/ alone.

Everything is computed from its definition, token by token and row by row:

    H <- exp(dt A) H + dt x (outer) B,    y = H C + D x
    o_i = sum_j softmax_j(scale q_i . k_j) v_j

``scan`` and ``attend`` also return the same sums of absolute values, from which
the tests derive elementwise error bounds.
"""
from __future__ import annotations

import numpy as np

F8_MAX = 448.0


def scan(x, dt, A, B, C, D, h):
    """One sequence: x [L,H,P], dt [L,H], B, C [L,G,N], h [H,P,N] (float64).
    (y, h, |y| summed, |h| summed)."""
    L, H, P = x.shape
    rep = H // B.shape[1] if L else 1
    h, ha = h.copy(), np.abs(h)
    y, ya = np.zeros((L, H, P)), np.zeros((L, H, P))
    for t in range(L):
        Bt, Ct = np.repeat(B[t], rep, 0), np.repeat(C[t], rep, 0)
        a = np.exp(dt[t] * A)[:, None, None]
        add = (dt[t][:, None] * x[t])[:, :, None] * Bt[:, None, :]
        h = a * h + add
        ha = a * ha + np.abs(add)
        y[t] = np.einsum("hpn,hn->hp", h, Ct) + D[:, None] * x[t]
        ya[t] = np.einsum("hpn,hn->hp", ha, np.abs(Ct)) + np.abs(D[:, None] * x[t])
    return y, h, ya, ha


def root_path(par, i):
    p = []
    while i >= 0:
        p.append(int(i))
        i = par[i]
    return p[::-1]


def attend(q, k, v, par, kc, vc, scale):
    """One item: q [T,H,D], k, v [T,Hk,D], kc, vc [L,Hk,D] (float64), par [T].
    (o, sum of p |v|, the largest scale * sum |q k|)."""
    T, H, D = q.shape
    g = H // k.shape[1]
    o, oa, top = np.zeros((T, H, D)), np.zeros((T, H, D)), 0.0
    for i in range(T):
        path = root_path(par, i)
        K, V = np.concatenate([kc, k[path]]), np.concatenate([vc, v[path]])
        for h in range(H):
            s = K[:, h // g] @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h] = p @ V[:, h // g]
            oa[i, h] = p @ np.abs(V[:, h // g])
            top = max(top, float((np.abs(K[:, h // g]) @ np.abs(q[i, h])).max() * abs(scale)))
    return o, oa, top


def cache_rows(cache, scale, table, n, page):
    """The first n positions of an item's cache, as float64: [n,Hk,D]."""
    pos = np.arange(n)
    pg, off = table[pos // page], pos % page
    rows = cache[pg, :, off].astype(np.float64)
    return rows if scale is None else rows * scale[pg, :, off].astype(np.float64)[..., None]
