"""Measured cases of what a hybrid model's layers do between their projections and the packed-tree pass: the short
causal convolution in front of an SSM layer (prompts, single tokens, tree nodes, accepted paths), the heads' norms
with the position rotation, the same on the way into the paged cache, and the attention of a chunk of new tokens
over that cache, whole or in a window with a few first tokens.

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs on the GPU, ``run()`` one pass: in plain
torch operations in 32 bits where ``own`` is false, through the library's binding where it is true. ``exact()``
computes the same outputs in 64 bits, step by step from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"
KINDS = ("conv", "conv_step", "conv_tree", "conv_commit", "rope", "append", "attend", "attend")
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases
def listed():
    hyb = dict(heads=64, P=64, N=64, groups=8, width=4)
    ssd = dict(heads=80, P=64, N=128, groups=1, width=4)
    att = dict(heads=32, kv_heads=8, D=128, page=16)
    rot = dict(rot=128, pairs="halves", norm=True)
    return [
        # the convolution of a batch of prompts of very different lengths, packed, at an 8B hybrid's sizes
        dict(name="conv-packed-32", kind="conv", n=32, lo=1, hi=1531, dtype="bf16", **hyb),
        # the convolution of a batch's draft trees in front of a Mamba2-2.7B-shaped layer
        dict(name="conv-tree31-16", kind="conv_tree", n=16, T=31, dtype="bf16", **ssd),
        # fp32 inputs (the precision the library's parity runs use): a few ragged prompts, narrow and two groups
        dict(name="conv-f32", kind="conv", n=3, lo=130, hi=777, dtype="f32", heads=24, P=64, N=128, groups=2, width=4),
        # queries and keys of the nodes of a batch's 63-node trees
        dict(name="rope-tree63-32", kind="rope", n=32, T=63, lo=300, hi=4099, dtype="bf16", **att, **rot),
        # one new token far into a conversation, half of each head rotated, in neighbouring pairs, no norm: latency
        dict(name="rope-1", kind="rope", n=1, T=1, lo=65533, hi=65533, dtype="f32", **att, rot=64, pairs="neighbours", norm=False),
        # the prompts of a batch enter a cache in 8 bits, rotated and quantised as they are written
        dict(name="append-packed-e4m3", kind="append", n=16, lo=1, hi=2047, old=1000, dtype="bf16", cache="e4m3", **att, **rot),
        # one new token of each request of a batch enters the cache
        dict(name="append-64", kind="append", n=64, lo=1, hi=1, old=8190, dtype="bf16", cache="bf16", **att, **rot),
        # a long prompt from its start
        dict(name="attend-4096", kind="attend", n=1, lo=4096, hi=4096, old_lo=0, old=0, window=0, sinks=0, dtype="bf16", cache="bf16", **att),
        # a chunk of a much longer prompt: few rows over a long cache
        dict(name="attend-509-of-33258", kind="attend", n=1, lo=509, hi=509, old_lo=32749, old=32749, window=0, sinks=0, dtype="bf16", cache="bf16", **att),
        # chunks and single tokens of one batch, caches in 8 bits
        dict(name="attend-mixed-16-e4m3", kind="attend", n=16, lo=1, hi=701, old_lo=0, old=4099, window=0, sinks=0, dtype="bf16", cache="e4m3", **att),
        # a layer with a window: one new token of each request of a batch of long conversations
        dict(name="attend-window-64", kind="attend", n=64, lo=1, hi=1, old_lo=17, old=8190, window=1021, sinks=4, dtype="bf16", cache="bf16", **att),
        # fp32 inputs in a window, a few ragged prompts, one key head for eight query heads
        dict(name="attend-window-f32", kind="attend", n=3, lo=130, hi=777, old_lo=0, old=333, window=255, sinks=4, dtype="f32", cache="f32", heads=24, kv_heads=3, D=64, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(KINDS)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if kind.startswith("conv"):
        heads, P, N, groups = rng.choice([(80, 64, 128, 1), (64, 64, 64, 8), (24, 64, 128, 2), (5, 64, 128, 1), (3, 40, 16, 1)])
        case = dict(kind=kind, dtype=dtype, heads=heads, P=P, N=N, groups=groups, width=rng.choice([4, 4, 4, 3, 2]))
        n = _log(rng, 1, 64)
        if kind == "conv":
            hi = _log(rng, 2, min(8192, (18000 if dtype == "bf16" else 9000) // n))
            return dict(case, n=n, lo=rng.randint(0, hi // 2), hi=hi)
        if kind == "conv_step":
            return dict(case, n=n)
        case = dict(case, n=n, T=rng.choice([1, 7, 15, 31, 63, 255]))
        return dict(case, path=rng.randint(1, 9)) if kind == "conv_commit" else case
    heads, kv_heads, D = rng.choice([(32, 8, 128), (32, 8, 64), (16, 16, 128), (20, 4, 128)])
    att = dict(heads=heads, kv_heads=kv_heads, D=D, page=rng.choice([16, 16, 32, 64, 24]), dtype=dtype)
    rot = dict(rot=rng.choice([D, D, D // 2]), pairs=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.6)
    n = _log(rng, 1, 48)
    if kind == "rope":
        hi = _log(rng, 16, 131072)
        return dict(kind=kind, n=n, T=rng.choice([1, 1, 7, 15, 31, 63, 255]), lo=rng.randint(0, hi // 2), hi=hi, **att, **rot)
    att["cache"] = rng.choice([dtype, "e4m3"])
    if kind == "append":
        hi = _log(rng, 1, 16384 // n)
        return dict(kind=kind, n=n, lo=rng.randint(0, hi // 2) if n > 1 else hi, hi=hi, old=_log(rng, 1, 2000), **att, **rot)
    hi, old = _log(rng, 1, min(4096, 8192 // n)), _log(rng, 1, min(65536, 90000 // n))
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    case = dict(kind=kind, n=n, lo=rng.randint(1, max(1, hi // 2)) if n > 1 else hi, hi=hi, old_lo=rng.randint(0, old // 2), old=old,
                window=window, sinks=rng.choice([0, 1, 4, 9]) if window else 0, **att)
    most = 2.5e11 if dtype == "bf16" else 2e10
    while work(case)["flops"] > most:  # shorter until it costs no more than the longest listed one
        case["old"] //= 2
        case["old_lo"] //= 2
        case["hi"] = max(1, case["hi"] * 3 // 4)
        case["lo"] = min(case["lo"], case["hi"]) if n > 1 else case["hi"]
    return case


def _spread(n, lo, hi, by):
    """n lengths over lo..hi in a mixed order."""
    if n == 1:
        return [hi]
    by = by if math.gcd(by, n) == 1 else 1
    return [lo + (hi - lo) * ((by * b + 3) % n) // (n - 1) for b in range(n)]


def _lens(case):
    return _spread(case["n"], case["lo"], case["hi"], 7)


def _olds(case):
    return _spread(case["n"], case.get("old_lo", 0), case["old"], 11)


_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def _channels(case):
    return case["heads"] * case["P"] + 2 * case["groups"] * case["N"]


def work(case):
    io, kind, n = _BYTES[case["dtype"]], case["kind"], case["n"]
    if kind.startswith("conv"):
        C, W = _channels(case), case["width"]
        if kind == "conv_commit":
            rows = n * min(W - 1, case["path"])
            return {"bytes": io * C * (rows + n * (W - 1)), "flops": n * C}
        rows = {"conv": lambda: sum(_lens(case)), "conv_step": lambda: n, "conv_tree": lambda: n * case["T"]}[kind]()
        states = n * (W - 1) * (1 if kind == "conv_tree" else 2)
        # a multiply-add per tap, the bias, and the activation's exponential, sum, quotient and product
        return {"bytes": io * C * (2 * rows + states) + 4 * C * (W + 1), "flops": rows * C * (2 * W + 5)}
    H, Hk, D = case["heads"], case["kv_heads"], case["D"]
    if kind in ("rope", "append"):
        rows = n * case["T"] if kind == "rope" else sum(_lens(case))
        b = io * rows * 2 * H * D + 4 * rows
        if kind == "rope":
            b += io * rows * 2 * Hk * D
        else:
            c = case["cache"]
            b += rows * Hk * 2 * (io * D + _BYTES[c] * D + (4 if c == "e4m3" else 0))
        return {"bytes": b, "flops": rows * (H + Hk) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    c, window, sinks = case["cache"], case["window"], case["sinks"]
    row = 2 * Hk * (_BYTES[c] * D + (4 if c == "e4m3" else 0))
    pairs = seen = 0
    for new, old in zip(_lens(case), _olds(case)):
        if not window:
            pairs += new * old + new * (new + 1) // 2
            seen += (old + new) if new else 0
            continue
        # the first `low` rows see all positions up to their own, the others the window and the sinks before it
        low = min(new, max(0, window + sinks - old))
        pairs += low * old + low * (low + 1) // 2 + (new - low) * (window + sinks)
        seen += min(old + new, window + new - 1 + sinks) if new else 0
    return {"bytes": seen * row + 2 * io * sum(_lens(case)) * H * D, "flops": 4 * H * D * pairs}


# ---------------------------------------------------------------------------------------------- inputs
def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _quantised(v):
    """A cache in 8 bits: each row by its own scale, the largest value at 448."""
    top = v.abs().amax(-1)
    scale = (top / torch.full_like(top, 448.0)).clamp_min(2.0 ** -126)  # a true division, not a product with 1/448
    return (v / scale[..., None]).to(torch.float8_e4m3fn), scale


def _starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def _trees(n, T, seed):
    """Random recursive trees: each node hangs on one of those before it."""
    u = torch.rand(n, T, generator=torch.Generator().manual_seed(seed))
    parent = (u * torch.arange(T)).floor().to(torch.int32)
    parent[:, 0] = -1
    return parent


def _depths(parent):
    depth = torch.zeros_like(parent)
    for i in range(1, parent.shape[1]):
        depth[:, i] = depth.gather(1, parent[:, i : i + 1].long())[:, 0] + 1
    return depth


def _conv_inputs(case, g, seed):
    """A projection's output, whose first columns are the gate's and the last ones the steps', as in a layer."""
    kind, n, C, W, t = case["kind"], case["n"], _channels(case), case["width"], _dtype(case["dtype"])
    H, P, N, G = case["heads"], case["P"], case["N"], case["groups"]
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    st = {"weight": 0.5 * rnd(C, W), "bias": 0.1 * rnd(C), "state": rnd(n, W - 1, C).to(t)}
    if kind == "conv":
        st["lens"] = _lens(case)
        st["seq_start"] = _starts(st["lens"])
        rows = (sum(st["lens"]) + 5,)  # five rows behind the last sequence, as a padded batch has them
    else:
        rows = (n,) if kind == "conv_step" else (n, case["T"])
    wide = rnd(*rows, H * P + C + H).to(t)
    st["xbc"] = wide[..., H * P : H * P + C]
    if kind in ("conv_tree", "conv_commit"):
        parent = _trees(n, case["T"], seed)
        st["parent"] = parent.to(DEV)
    if kind == "conv_commit":
        # root paths of random nodes, cut after `path` nodes
        acc, count = torch.full((n, case["path"]), -1, dtype=torch.int32), []
        ends = torch.randint(0, case["T"], (n,), generator=torch.Generator().manual_seed(seed + 1)).tolist()
        for b, (up, j) in enumerate(zip(parent.tolist(), ends)):
            p = []
            while j >= 0:
                p.append(j)
                j = up[j]
            p = p[::-1][: case["path"]]
            acc[b, : len(p)] = torch.tensor(p, dtype=torch.int32)
            count.append(len(p))
        st.update(accepted=acc.to(DEV), accepted_len=torch.tensor(count, dtype=torch.int32, device=DEV))
    else:
        st["out"] = tuple(torch.zeros(*rows, *s, dtype=t, device=DEV) for s in ((H, P), (G, N), (G, N)))
    return st


def _cache_inputs(case, g, room):
    """Pages in a random order, `room` positions for each sequence, some pages of the pool in nobody's table."""
    page, Hk, D, n = case["page"], case["kv_heads"], case["D"], case["n"]
    per = [-(-r // page) for r in room]
    most, pages = max(1, max(per)), sum(per) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(g.initial_seed()))
    table, at = torch.zeros(n, most, dtype=torch.int32), 0
    for b, k in enumerate(per):
        table[b, :k] = order[at : at + k].to(torch.int32)
        at += k
    st = {"page_table": table.to(DEV), "k_scale": None, "v_scale": None}
    for name in ("k", "v"):
        v = torch.randn(pages, Hk, page, D, generator=g, device=DEV)
        if case["cache"] == "e4m3":
            st[name + "_cache"], st[name + "_scale"] = _quantised(v)
        else:
            st[name + "_cache"] = v.to(_dtype(case["cache"]))
    return st


def _rope_inputs(case, g):
    D, R = case["D"], case["rot"]
    st = {"inv_freq": (10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) * 2 / R)).float().to(DEV), "q_weight": None, "k_weight": None}
    if case["norm"]:
        for m in "qk":
            st[m + "_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
    return st


def _heads(case, g, *rows):
    """q, k, v as slices of a projection's output."""
    H, Hk, D = case["heads"], case["kv_heads"], case["D"]
    wide = torch.randn(*rows, H + 2 * Hk, D, generator=g, device=DEV).to(_dtype(case["dtype"]))
    return dict(zip("qkv", wide.split([H, Hk, Hk], -2)))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kind, n = case["kind"], case["n"]
    if kind.startswith("conv"):
        return {"case": case, **_conv_inputs(case, g, seed)}
    if kind == "rope":
        T = case["T"]
        at = torch.tensor(_lens(case), dtype=torch.int32)[:, None] + _depths(_trees(n, T, seed))
        st = _heads(case, g, n, T)
        del st["v"]
        return {"case": case, **_rope_inputs(case, g), **st, "position": at.to(DEV)}
    lens, olds = _lens(case), _olds(case)
    st = _cache_inputs(case, g, [a + b for a, b in zip(lens, olds)])
    st.update(lens=lens, olds=olds, seq_start=_starts(lens), cache_len=torch.tensor(olds, dtype=torch.int32, device=DEV))
    if kind == "append":
        rows = sum(lens) + 5
        st.update(_heads(case, g, rows), **_rope_inputs(case, g))
        st["q_out"] = torch.zeros(rows, case["heads"], case["D"], dtype=_dtype(case["dtype"]), device=DEV)
    else:
        st["q"] = torch.randn(sum(lens), case["heads"], case["D"], generator=g, device=DEV).to(_dtype(case["dtype"]))
    return {"case": case, **st}


# ---------------------------------------------------------------------------------------------- plain forms
def _taps(s, rows):
    """rows(k): the inputs k tokens before each, in 32 bits -> the convolution's sum with bias and activation."""
    W = s["weight"].shape[1]
    y = s["bias"]
    for k in range(W):
        y = y + rows(k).float() * s["weight"][:, W - 1 - k]
    return y / (1 + (-y).exp())


def _split(s, y, where=None):
    """Columns to x, B and C, at rows `where` of them."""
    at = 0
    for o in s["out"]:
        width = o.shape[-2] * o.shape[-1]
        part = y[..., at : at + width].reshape(*y.shape[:-1], *o.shape[-2:]).to(o.dtype)
        if where is None:
            o.copy_(part)
        else:
            o[where] = part
        at += width
    return s["out"]


def _plain_conv(s):
    xbc, state, start = s["xbc"], s["state"], s["seq_start"]
    n, back, C = state.shape
    rows = sum(s["lens"])
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), start.diff(), output_size=rows)
    at = torch.arange(rows, device=DEV) - start[seq]
    both = torch.cat([state.reshape(-1, C), xbc])  # the states' rows, then the inputs'
    first = n * back

    def rows_before(seq, at, k):
        t = at - k
        return torch.where(t < 0, seq * back + back + t, first + start[seq] + t)

    y = _taps(s, lambda k: both[rows_before(seq, at, k)])
    _split(s, y, torch.arange(rows, device=DEV))
    every = torch.arange(n, device=DEV)
    state.copy_(torch.stack([both[rows_before(every, start.diff(), back - m)] for m in range(back)], 1))
    return (*s["out"], state)


def _plain_conv_step(s):
    state, xbc = s["state"], s["xbc"]
    both = torch.cat([state, xbc[:, None]], 1)
    back = state.shape[1]
    _split(s, _taps(s, lambda k: both[:, back - k]))
    state.copy_(both[:, 1:])
    return (*s["out"], state)


def _plain_conv_tree(s):
    state, xbc, parent = s["state"], s["xbc"], s["parent"].long()
    n, back, C = state.shape
    both = torch.cat([state, xbc], 1)
    # node t is row back + t; its k-th ancestor, and past the root the state's rows from the last one on
    up = torch.cat([torch.arange(back, device=DEV).expand(n, back) - 1, parent + back], 1).clamp_min(0)
    at = torch.arange(xbc.shape[1], device=DEV).expand(n, -1) + back
    rows = []
    for _ in range(back + 1):
        rows.append(at)
        at = up.gather(1, at)
    return _split(s, _taps(s, lambda k: both.gather(1, rows[k][..., None].expand(-1, -1, C))))


def _plain_conv_commit(s):
    state, xbc, acc = s["state"], s["xbc"], s["accepted"].long().clamp_min(0)
    n, back, C = state.shape
    both = torch.cat([state, xbc.gather(1, acc[..., None].expand(-1, -1, C))], 1)
    at = s["accepted_len"].long()[:, None] + torch.arange(back, device=DEV)
    state.copy_(both.gather(1, at[..., None].expand(-1, -1, C)))
    return state


def _plain_rotated(s, name, position, bits=torch.float32):
    """Norm and rotation of rows [..., H, D] at positions [...], in 32 bits (the angles in 64)."""
    v, R = s[name].to(bits), 2 * s["inv_freq"].numel()
    if s[name + "_weight"] is not None:
        v = v * (v.square().mean(-1, keepdim=True) + EPS).rsqrt() * s[name + "_weight"]
    angle = position[..., None].double() * s["inv_freq"].double()
    cos, sin = angle.cos().to(bits)[..., None, :], angle.sin().to(bits)[..., None, :]
    out = v.clone()
    if s["case"]["pairs"] == "halves":
        a, b = slice(0, R // 2), slice(R // 2, R)
    else:
        a, b = slice(0, R, 2), slice(1, R, 2)
    out[..., a] = v[..., a] * cos - v[..., b] * sin
    out[..., b] = v[..., b] * cos + v[..., a] * sin
    return out


def _plain_rope(s):
    return {m: _plain_rotated(s, m, s["position"]).to(s[m].dtype) for m in "qk"}


def _appended(s):
    out = {m: s[m] for m in ("k_cache", "v_cache", "k_scale", "v_scale") if s[m] is not None}
    return {"q": s["q_out"], **out}


def _plain_append(s):
    n, page, rows = len(s["lens"]), s["case"]["page"], sum(s["lens"])
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), s["seq_start"].diff(), output_size=rows)
    at = torch.arange(rows, device=DEV) - s["seq_start"][seq] + s["cache_len"][seq]
    cut = {**s, "q": s["q"][:rows], "k": s["k"][:rows]}
    s["q_out"][:rows] = _plain_rotated(cut, "q", at).to(s["q"].dtype)
    pages, slot = s["page_table"][seq, at // page].long(), at % page
    # in 8 bits a row's values lie next to the borders between two of them: in 64 up to that rounding
    bits = torch.float32 if s["k_scale"] is None else torch.float64
    for name, v in (("k", _plain_rotated(cut, "k", at, bits)), ("v", s["v"][:rows].to(bits))):
        if s[name + "_scale"] is None:
            s[name + "_cache"][pages, :, slot] = v.to(s[name + "_cache"].dtype)
        else:
            w, scale = _quantised(v)
            s[name + "_cache"].view(torch.uint8)[pages, :, slot] = w.view(torch.uint8)
            s[name + "_scale"][pages, :, slot] = scale.float()
    return _appended(s)


def _plain_attend(s):
    case, q, out = s["case"], s["q"], torch.empty_like(s["q"])
    page, window, sinks, Hk = case["page"], case["window"], case["sinks"], case["kv_heads"]
    H, D = q.shape[1:]
    row = 0
    for b, (new, old) in enumerate(zip(s["lens"], s["olds"])):
        if new == 0:
            continue
        L = old + new
        pos = torch.arange(L, device=DEV)
        p = pos[old:, None]
        seen = pos <= p
        if window:  # the positions that some row sees, in their order
            keep = torch.cat([pos[: min(sinks, max(0, old - window + 1))], pos[max(0, old - window + 1) :]])
            pos = keep
            seen = (pos <= p) & ((pos > p - window) | (pos < sinks))
        at = (s["page_table"][b].long()[pos // page], slice(None), pos % page)
        k, v = (s[m + "_cache"][at].float() if s[m + "_scale"] is None else s[m + "_cache"][at].float() * s[m + "_scale"][at][..., None] for m in "kv")
        k, v = k.permute(1, 2, 0).contiguous(), v.transpose(0, 1).contiguous()  # [Hk, D, L], [Hk, L, D]
        rows = q[row : row + new].float().view(new, Hk, H // Hk, D).permute(1, 2, 0, 3).reshape(Hk, -1, D)
        score = (rows @ k * D ** -0.5).view(Hk, H // Hk, new, -1).masked_fill(~seen, -math.inf)
        w = (score - score.amax(-1, keepdim=True)).exp()
        w = (w / w.sum(-1, keepdim=True)).view(Hk, (H // Hk) * new, -1)
        out[row : row + new] = (w @ v).view(Hk, H // Hk, new, D).permute(2, 0, 1, 3).reshape(new, H, D).to(q.dtype)
        row += new
    return out


def run(state):
    case, s = state["case"], state
    kind = case["kind"]
    if not own:
        plain = {"conv": _plain_conv, "conv_step": _plain_conv_step, "conv_tree": _plain_conv_tree, "conv_commit": _plain_conv_commit,
                 "rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}
        return plain[kind](s)
    from speculative_tree_verification_amd import binding as tsv

    if kind == "conv_commit":
        tsv.conv_commit(s["xbc"], s["state"], s["parent"], s["accepted"], s["accepted_len"], case["heads"], case["P"], case["groups"], case["N"])
        return s["state"]
    if kind.startswith("conv"):
        taps = (s["xbc"], s["weight"], s["bias"], s["state"])
        if kind == "conv":
            tsv.conv_prefill(*taps, s["seq_start"], *s["out"])
        elif kind == "conv_step":
            tsv.conv_step(*taps, *s["out"])
        else:
            tsv.conv_verify(*taps, s["parent"], *s["out"])
            return s["out"]
        return (*s["out"], s["state"])
    cache = [s[m] for m in ("k_cache", "v_cache", "page_table", "cache_len")] if kind != "rope" else None
    how = {"interleaved": case["pairs"] == "neighbours", "q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": EPS} if kind != "attend" else None
    if kind == "rope":
        return dict(zip("qk", tsv.attn_rope(s["q"], s["k"], s["position"], s["inv_freq"], **how)))
    scales = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if kind == "append":
        tsv.attn_append_rope(s["q"], s["k"], s["v"], s["seq_start"], s["inv_freq"], *cache, **scales, **how, q_out=s["q_out"])
        return _appended(s)
    return tsv.attn_prefill(s["q"], s["seq_start"], *cache, **scales, window=case["window"], sinks=case["sinks"])


# ---------------------------------------------------------------------------------------------- 64 bits
def _exact_conv(s, case):
    kind, state, xbc = case["kind"], s["state"].double(), s["xbc"].double()
    n, back, C = state.shape
    w, bias = s["weight"].double(), s["bias"].double()
    if kind == "conv_commit":
        out = []
        for b, (path, count) in enumerate(zip(s["accepted"].tolist(), s["accepted_len"].tolist())):
            out.append(torch.cat([state[b], xbc[b, path[:count]]])[-back:] if count else state[b])
        return torch.stack(out)

    def output(window):  # [..., W, C], oldest first
        y = (window * w.T).sum(-2) + bias
        return y * torch.sigmoid(y)

    def split(y):
        H, P, N, G = case["heads"], case["P"], case["N"], case["groups"]
        x, B, Cm = y.split([H * P, G * N, G * N], -1)
        return x.unflatten(-1, (H, P)), B.unflatten(-1, (G, N)), Cm.unflatten(-1, (G, N))

    if kind == "conv_step":
        both = torch.cat([state, xbc[:, None]], 1)
        return (*split(output(both)), both[:, 1:])
    if kind == "conv_tree":
        y = torch.zeros_like(xbc)
        for b, up in enumerate(s["parent"].tolist()):
            for i in range(len(up)):
                path, j = [], i
                while j >= 0 and len(path) <= back:
                    path.append(j)
                    j = up[j]
                y[b, i] = output(torch.cat([state[b], xbc[b, path[::-1]]])[-back - 1 :])
        return split(y)
    y, row = torch.zeros_like(xbc), 0
    for b, count in enumerate(s["lens"]):
        both = torch.cat([state[b], xbc[row : row + count]])
        if count:
            y[row : row + count] = output(both.unfold(0, back + 1, 1).transpose(1, 2))
        state[b] = both[-back:]
        row += count
    return (*split(y), state)


def _exact_rotated(s, name, position):
    v, R, case = s[name].double(), 2 * s["inv_freq"].numel(), s["case"]
    if s[name + "_weight"] is not None:
        v = v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + EPS) * s[name + "_weight"].double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), position.double()[..., None] * s["inv_freq"].double())[..., None, :]
    if case["pairs"] == "halves":
        z = torch.complex(v[..., : R // 2].contiguous(), v[..., R // 2 : R].contiguous()) * turn
        return torch.cat([z.real, z.imag, v[..., R:]], -1)
    z = torch.view_as_complex(v[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), v[..., R:]], -1)


def _exact_append(s, case):
    at = [old + i for new, old in zip(s["lens"], s["olds"]) for i in range(new)]
    seq = [b for b, new in enumerate(s["lens"]) for _ in range(new)]
    at, seq = torch.tensor(at, device=DEV), torch.tensor(seq, device=DEV)
    rows = len(at)
    cut = {**s, "q": s["q"][:rows], "k": s["k"][:rows]}
    q = s["q_out"].double()
    q[:rows] = _exact_rotated(cut, "q", at)
    got = {"q": q}
    pages, slot = s["page_table"].long()[seq, at // case["page"]], at % case["page"]
    for m, new in (("k", _exact_rotated(cut, "k", at)), ("v", s["v"][:rows].double())):
        cache, scales = s[m + "_cache"].double(), s[m + "_scale"]
        if scales is not None:
            scales = scales.double()
            by = torch.clamp(new.abs().max(-1).values / 448, min=2.0 ** -126)
            new = new / by[..., None]  # before its rounding to 8 bits, as everything here
            scales[pages, :, slot] = by
            got[m + "_scale"] = scales
        cache[pages, :, slot] = new
        got[m + "_cache"] = cache
    order = [m for m in ("q", "k_cache", "v_cache", "k_scale", "v_scale") if m in got]
    return {m: got[m] for m in order}


def _exact_attend(s, case):
    H, D = s["q"].shape[1:]
    group, page, window, sinks, out, row = H // case["kv_heads"], case["page"], case["window"], case["sinks"], [], 0
    for b, (new, old) in enumerate(zip(s["lens"], s["olds"])):
        if new == 0:
            continue
        pos = torch.arange(old + new, device=DEV)
        pages, slot = s["page_table"][b].long()[pos // page], pos % page
        p = old + torch.arange(new, device=DEV)[:, None]
        gone = pos > p
        if window:
            gone = gone | ((pos <= p - window) & (pos >= sinks))
        heads = []
        for h in range(H):
            k, v = (s[m + "_cache"][pages, h // group, slot].double() for m in "kv")
            if s["k_scale"] is not None:
                k, v = (t * s[m + "_scale"][pages, h // group, slot].double()[:, None] for t, m in ((k, "k"), (v, "v")))
            score = s["q"][row : row + new, h].double() @ k.T.contiguous() / math.sqrt(D)
            heads.append(torch.softmax(score.masked_fill(gone, -math.inf), -1) @ v)
        out.append(torch.stack(heads, 1))
        row += new
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind.startswith("conv"):
        return _exact_conv(s, case)
    if kind == "rope":
        return {m: _exact_rotated(s, m, s["position"]) for m in "qk"}
    return (_exact_append if kind == "append" else _exact_attend)(s, case)
