"""The short causal convolution, the heads' norms with the position rotation, and the attention of packed rows over a
cache, in fp64. TEST INFRASTRUCTURE ONLY: imported by tests/ alone.

Everything is computed from its definition, token by token and row by row:

    y_t = act(bias + sum_k w[W-1-k] u_{t-k})
    z = w x / sqrt(mean x^2 + eps),   (z_a + i z_b) <- (z_a + i z_b) e^{i position inv_freq}
    o_i = sum_j softmax_j(scale q_i . k_j) v_j over the positions that row i sees

and comes with the sums of absolute values from which the tests derive elementwise error bounds.
"""
from __future__ import annotations

import math

import numpy as np


def silu(y):
    return y / (1.0 + np.exp(np.minimum(-y, 700.0)))


def conv_token(past, u, weight, bias, act):
    """One token: past [W-1,C] oldest first, u [C], weight [C,W]. (y, sum of |terms|, the sum before act)."""
    W = weight.shape[1]
    y, ya = bias.copy(), np.abs(bias)
    taps = np.concatenate([past, u[None]])
    for k in range(W):
        y = y + weight[:, W - 1 - k] * taps[W - 1 - k]
        ya = ya + np.abs(weight[:, W - 1 - k] * taps[W - 1 - k])
    return (silu(y) if act else y), ya, y


def conv(u, state, weight, bias, act):
    """One sequence: u [L,C], state [W-1,C]. (y [L,C], sums of |terms|, sums before act, the state after)."""
    out, past = [], state.copy()
    for t in range(len(u)):
        out.append(conv_token(past, u[t], weight, bias, act))
        past = np.concatenate([past, u[t:t + 1]])[1:]
    shape = (0, u.shape[1])
    y, ya, raw = (np.stack([o[i] for o in out]) if out else np.zeros(shape) for i in range(3))
    return y, ya, raw, past


def rope(x, position, inv_freq, weight, eps, interleaved):
    """One row: x [H,D]. (out, sum of absolute terms of each element)."""
    z = x.copy()
    if weight is not None:
        z = np.stack([h / math.sqrt(float(np.mean(h * h)) + eps) * weight for h in x])
    out, mag = z.copy(), np.abs(z)
    R = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        t = float(position) * float(f)
        c, s = math.cos(t), math.sin(t)
        out[:, a] = z[:, a] * c - z[:, b] * s
        out[:, b] = z[:, b] * c + z[:, a] * s
        mag[:, a] = mag[:, b] = np.abs(z[:, a]) + np.abs(z[:, b])
    return out, mag


def sees(p, j, window, sinks):
    """Whether the row at position p sees position j."""
    return j <= p and (window == 0 or j > p - window or j < sinks)


def attend(q, old, kc, vc, scale, window=0, sinks=0):
    """Rows q [n,H,D] at positions old, old + 1, ... over kc, vc [old+n,Hk,D].
    (o, sum of p |v|, the largest scale * sum |q k|)."""
    n, H, D = q.shape
    g = H // kc.shape[1]
    o, oa, top = np.zeros((n, H, D)), np.zeros((n, H, D)), 0.0
    for i in range(n):
        see = [j for j in range(old + i + 1) if sees(old + i, j, window, sinks)]
        K, V = kc[see], vc[see]
        for h in range(H):
            s = K[:, h // g] @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h] = p @ V[:, h // g]
            oa[i, h] = p @ np.abs(V[:, h // g])
            top = max(top, float((np.abs(K[:, h // g]) @ np.abs(q[i, h])).max() * abs(scale)))
    return o, oa, top
