"""Inputs of the tests of the prompt scan, the step and the paged attention."""
import numpy as np
import torch


def ssd(seed, rows, n, H, P, N, G, dtype, dt_bias=-2.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    d = {"x": rnd(rows, H, P).to(dtype), "dt": torch.nn.functional.softplus(rnd(rows, H) + dt_bias).to(dtype),
         "A": -torch.exp(2.7 * torch.rand(H, generator=g)), "B": rnd(rows, G, N).to(dtype),
         "C": rnd(rows, G, N).to(dtype), "D": rnd(H), "h": 0.1 * rnd(n, H, P, N)}
    return {k: v.to(device) for k, v in d.items()}


def f64(t):
    return t.detach().cpu().double().numpy()


def trees(seed, n, T, kind="random"):
    if kind == "chain":
        return torch.arange(-1, T - 1, dtype=torch.int32).repeat(n, 1)
    if kind == "star":
        p = torch.zeros(n, T, dtype=torch.int32)
    else:
        p = (torch.rand(n, T, generator=torch.Generator().manual_seed(seed)) * torch.arange(T)).floor().to(torch.int32)
    p[:, 0] = -1
    return p


def quantise(v):
    """fp32 rows [..., D] -> (e4m3 rows, scales), as the header defines them."""
    top = v.abs().amax(-1)
    scale = (top / torch.full_like(top, 448.0)).clamp_min(2.0 ** -126)
    return (v / scale[..., None]).to(torch.float8_e4m3fn), scale


def cache(seed, n, lens, Hk, D, page, dtype, cache_dtype, room=0, device="cuda"):
    """Pages in a random order; the unused rows of the pool hold NaN where the type has it."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-(int(L) + room) // page) for L in lens]
    pages, most = sum(per) + 2, max(1, max(per)) + 1
    order = torch.randperm(pages, generator=g)
    table = torch.full((n, most), -5, dtype=torch.int32)  # entries no call may use
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = order[at:at + k].to(torch.int32)
        at += k
    c = {"page_table": table, "cache_len": torch.tensor(lens, dtype=torch.int32), "k_scale": None, "v_scale": None}
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, L in enumerate(lens):
        for p in range(int(L)):
            used[int(table[b, p // page]), p % page] = True
    for m in "kv":
        val = torch.randn(pages, Hk, page, D, generator=g)
        if cache_dtype == torch.float8_e4m3fn:
            by, sc = quantise(val)
            by = torch.where(used[:, None, :, None], by.view(torch.uint8), torch.tensor(0x7f, dtype=torch.uint8))
            c[m + "_cache"] = by.view(torch.float8_e4m3fn)
            c[m + "_scale"] = torch.where(used[:, None, :], sc, torch.tensor(float("nan")))
        else:
            c[m + "_cache"] = torch.where(used[:, None, :, None], val, torch.tensor(float("nan"))).to(dtype)
    return {k: v if v is None else v.to(device) for k, v in c.items()}


def cache_args(c):
    return (c["k_cache"], c["v_cache"], c["page_table"], c["cache_len"]), {"k_scale": c["k_scale"], "v_scale": c["v_scale"]}


def np8(t):
    return None if t is None else t.detach().cpu().float().numpy()


def within(got, want, bound, what):
    """Elementwise |got - want| <= bound; the worst ratio is part of the message."""
    assert np.isfinite(got).all(), f"{what}: not finite"
    r = np.abs(got - want) / np.maximum(bound, 1e-300)
    worst = float(r.max()) if r.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound at {np.unravel_index(int(r.argmax()), r.shape)}"
    return worst
