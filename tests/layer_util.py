"""Inputs and bounds of the tests of the convolution, the rotation and the attention of packed rows."""
import numpy as np
import torch

from oracle import layer as Y
from oracle import sequence as S
from tests import seq_util as U

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def starts(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def wide(seed, *shape, dtype, lead=0, tail=0, device="cuda"):
    """Rows that are slices of wider ones."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(*shape[:-1], lead + shape[-1] + tail, generator=g).to(dtype).to(device)
    return t[..., lead:lead + shape[-1]]


def conv_bound(y, ya, raw, W, dtype, act):
    """A sum of W products and the bias: (W + 1) half steps of the absolute terms; SiLU's slope is at most 1.1; its
    exponential is off by half steps of its argument and, with the sum, the quotient and the product, by some more
    relatively; -88 and below its exponential is infinite, and the result 0 instead of at most 1e-36; bf16 rounds once."""
    e = (W + 1) * 2.0 ** -24 * ya
    b = 1.1 * e + ((np.abs(raw) + 12) * 2.0 ** -24) * np.abs(y) + 1e-35 if act else e
    return b + (2.0 ** -8 * (np.abs(y) + b) if dtype == BF else 0)


def rope_bound(out, mag, D, normed, dtype):
    """The norm's sum has D half steps, its root halves them, and a few more follow; an angle is rounded at half a
    turn (2^-26 turns, 2^-23.3), its sine and cosine are off by 2^-23 more, and the two products and their sum by
    three half steps."""
    e = ((D / 2 + 8 if normed else 0) * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -24) * mag + 1e-37
    return e + (2.0 ** -8 * (np.abs(out) + e) if dtype == BF else 0)


def attend_bound(r, oa, top, D, L, dtype):
    """A score is off by at most (D + 8) 2^-24 top, a weight by twice that relatively, the sums over L keys by
    (L + 64) 2^-24; bf16 adds half a step of o, and half a step of each weighted value."""
    b = (2 * (D + 8) * top + L + 64) * 2.0 ** -24 * oa + 1e-30
    return b + (2.0 ** -8 * (np.abs(r) + 1.02 * oa) if dtype == BF else 0)


def cached(c, b, n):
    """The first n positions of item b: (keys, values), float64."""
    t, page = c["page_table"][b].cpu().numpy(), c["k_cache"].shape[2]
    return [S.cache_rows(U.np8(c[m + "_cache"]), U.np8(c[m + "_scale"]), t, n, page) for m in "kv"]
