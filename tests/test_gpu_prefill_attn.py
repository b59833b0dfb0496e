"""GPU: attention of packed rows over the paged cache (tree_attn_prefill) against the fp64 definition; the layers'
run of rotation, append and attention, and of the convolution with the SSM calls (the bounds are in layer_util)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import layer as Y
from tests import layer_util as V
from tests import seq_util as U
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF, F32, E4 = V.BF, V.F32, V.E4


@pytest.fixture(scope="module")
def bnd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from speculative_tree_verification_amd import binding
    return binding


def case(seed, lens, old, Hk, D, page, dtype, cdtype):
    """A cache that holds old + new positions of each item, cache_len the old ones."""
    c = U.cache(seed, len(lens), [a + b for a, b in zip(lens, old)], Hk, D, page, dtype, cdtype)
    c["cache_len"] = torch.tensor(old, dtype=torch.int32, device="cuda")
    return c


def check(bnd, q, lens, old, c, what, window=0, sinks=0, scale=None, rows=None, first=0, items=None, **kw):
    """rows(n): the rows of a sequence to compare (default: all)."""
    L, H, D = q.shape
    n, dtype = len(lens), q.dtype
    o, st = torch.full_like(q, 7.0), torch.full((n,), -3, dtype=torch.int32, device="cuda")
    args, scales = U.cache_args(c)
    say(f"[chunk] {what}")
    bnd.attn_prefill(q, V.starts(lens, first), *args, **scales, window=window, sinks=sinks, scale=scale, o=o, seq_status=st, **kw)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * n
    og, at, worst = U.f64(o), first, 0.0
    for b, new in enumerate(lens):
        if new and (items is None or b in items):
            kc, vc = V.cached(c, b, old[b] + new)
            pick = sorted(set(rows(new))) if rows else range(new)
            for i in pick:
                p = old[b] + i
                r, oa, top = Y.attend(U.f64(q[at + i:at + i + 1]), p, kc[:p + 1], vc[:p + 1], D ** -0.5 if scale is None else scale, window, sinks)
                bound = V.attend_bound(r, oa, top, D, p + 1, dtype)
                worst = max(worst, U.within(og[at + i:at + i + 1], r, bound, f"{what}, row {i} of {b}"))
        at += new
    assert (o[:first] == 7).all() and (o[at:] == 7).all(), "rows of no sequence"
    say(f"[chunk] {what}: {worst:.3f} of the bound")
    return o


def queries(seed, L, H, D, dtype):
    return torch.randn(L, H, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def some(n):
    return {i for i in (0, 1, 2, 15, 16, 31, 32, 63, 64, 65, 127, 128, n // 2, n - 2, n - 1) if 0 <= i < n}


TYPES = [(BF, BF), (BF, E4), (F32, F32), (F32, E4)]
HEADS = [(8, 2, 128), (4, 4, 64), (6, 1, 128), (16, 1, 64), (3, 1, 40), (2, 2, 256), (2, 1, 1), (20, 1, 64)]


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("H,Hk,D", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_heads_and_types(bnd, dtype, cdtype, H, Hk, D, window, sinks):
    lens, old = [5, 0, 1, 70, 33], [0, 4, 63, 130, 31]
    c = case(D, lens, old, Hk, D, 16, dtype, cdtype)
    check(bnd, queries(D, sum(lens) + 3, H, D, dtype), lens, old, c, f"{dtype} {cdtype} H={H}/{Hk} D={D} window {window}", window, sinks, rows=some, first=1)


@pytest.mark.parametrize("cdtype", [BF, E4])
@pytest.mark.parametrize("page", [1, 7, 24, 64, 1000])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 9)])
def test_pages(bnd, cdtype, page, window, sinks):
    lens, old = [90, 1], [243, 64]
    c = case(page, lens, old, 2, 64, page, BF, cdtype)
    check(bnd, queries(page, 91, 4, 64, BF), lens, old, c, f"page {page} {cdtype} window {window}", window, sinks, rows=some)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 4), (1, 0), (64, 64)])
def test_mixed_lengths(bnd, dtype, cdtype, window, sinks):
    """Single tokens over long caches, short and long chunks in one call, cut into parts that are joined."""
    lens, old = [1, 300, 1, 40, 2, 64, 1], [5000, 0, 17, 2100, 700, 64, 0]
    c = case(3, lens, old, 2, 128, 16, dtype, cdtype)
    assert bnd.attn_prefill_workspace_bytes(7, sum(lens), 8, 2, 128, 16, c["page_table"].shape[1], dtype, cdtype) > 0
    check(bnd, queries(4, sum(lens), 8, 128, dtype), lens, old, c, f"mixed {dtype} {cdtype} window {window}+{sinks}", window, sinks, rows=some)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (16, 16, 64), (5, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 4)])
def test_single_tokens(bnd, dtype, cdtype, H, Hk, D, window, sinks):
    """One row of each item, with caches of very different lengths."""
    old = [3000, 0, 1, 63, 64, 65, 900, 255, 256, 257, 1024, 31]
    c = case(5, [1] * 12, old, Hk, D, 16, dtype, cdtype)
    check(bnd, queries(6, 12, H, D, dtype), [1] * 12, old, c, f"tokens {dtype} {cdtype} H={H}/{Hk} D={D} window {window}", window, sinks)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (4, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_short_chains(bnd, dtype, cdtype, H, Hk, D, window, sinks):
    """A few tokens of some items beside single tokens of the others: sequences of several of the smallest blocks."""
    lens, old = [7, 1, 1, 0, 1, 13, 1, 2, 1, 1, 1, 1], [0, 700, 31, 5, 64, 1100, 1, 63, 255, 2000, 17, 9]
    c = case(17, lens, old, Hk, D, 16, dtype, cdtype)
    check(bnd, queries(18, sum(lens) + 2, H, D, dtype), lens, old, c, f"chains {dtype} {cdtype} H={H}/{Hk} D={D} window {window}", window, sinks, first=1)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D", [128, 40])
def test_windows_past_everything(bnd, dtype, cdtype, D):
    """The largest window, and the most first positions, leave nothing out."""
    lens, old = [70, 1, 300], [40, 900, 0]
    c = case(19, lens, old, 2, D, 16, dtype, cdtype)
    q = queries(20, sum(lens), 4, D, dtype)
    whole = check(bnd, q, lens, old, c, f"whole {dtype} {cdtype} D={D}", rows=some)
    most = 2 ** 31 - 1
    for window, sinks in ((most, 0), (most, most), (most - 1, 7), (1, most), (64, 1300)):
        o = torch.full_like(q, 7.0)
        args, scales = U.cache_args(c)
        bnd.attn_prefill(q, V.starts(lens), *args, **scales, window=window, sinks=sinks, o=o)
        torch.cuda.synchronize()
        err = (o.double() - whole.double()).abs().max().item()
        # two computations of the same sums, each within its bound: outputs of unit size differ by four roundings of
        # the type at most in what the matrix kernels' weights and outputs lose (bf16), or by the sums' own (fp32)
        assert err <= (4 * 2.0 ** -8 if dtype == BF else 1e-4) * max(1.0, whole.double().abs().max().item()), (window, sinks, err)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk,D", [(4, 1, 128), (2, 2, 64)])
@pytest.mark.parametrize("n,old", [(1, 0), (63, 1), (129, 63), (520, 0), (777, 333)])
def test_prompts(bnd, dtype, H, Hk, D, n, old):
    """One sequence: blocks of rows, tiles of keys, and their ends."""
    c = case(n, [n], [old], Hk, D, 16, dtype, dtype)
    check(bnd, queries(n, n, H, D, dtype), [n], [old], c, f"prompt {dtype} {n} after {old} H={H}/{Hk} D={D}", rows=some)


@pytest.mark.parametrize("cdtype", [BF, E4])
@pytest.mark.parametrize("window,sinks", [(0, 0), (513, 2)])
def test_many_rows(bnd, cdtype, window, sinks):
    """Enough rows for the largest blocks."""
    lens, old = [1500, 700, 3], [10, 900, 2000]
    c = case(8, lens, old, 4, 128, 16, BF, cdtype)
    check(bnd, queries(9, sum(lens), 16, 128, BF), lens, old, c, f"many rows {cdtype} window {window}", window, sinks,
          rows=lambda n: {i for i in (0, 1, 63, 64, 255, 256, n // 2, n - 1) if i < n})


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [64, 65, 200])
def test_many_items(bnd, dtype, n):
    """More sequences than lanes, some of them long enough to be cut."""
    lens, old = [(7 * b) % 5 for b in range(n)], [(37 * b) % 90 for b in range(n)]
    old[1], lens[n - 2], lens[2] = 3000, 150, 1
    c = case(n, lens, old, 1, 64, 16, dtype, dtype)
    check(bnd, queries(n, sum(lens), 2, 64, dtype), lens, old, c, f"{n} items {dtype}", rows=some, items={0, 1, 2, 3, n // 2, n - 2, n - 1})


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_plain_kernel(bnd, dtype, cdtype, D):
    """The plain kernel where another would be taken."""
    lens, old = [40, 1, 9], [600, 2500, 0]
    c = case(11, lens, old, 2, D, 16, dtype, cdtype)
    check(bnd, queries(12, 50, 6, D, dtype), lens, old, c, f"plain {dtype} {cdtype} D={D}", 1000, 2, force_generic=True, rows=some)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unaligned(bnd, dtype):
    lens, old = [30, 1], [100, 9]
    c = case(13, lens, old, 2, 64, 16, dtype, dtype)
    q = queries(14, 31, 4, 64, dtype)
    u = torch.empty(q.numel() + 1, dtype=dtype, device="cuda")[1:].view(q.shape).copy_(q)
    assert u.data_ptr() % 16
    check(bnd, u, lens, old, c, f"unaligned {dtype}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 4.0])
def test_factor_of_the_scores(bnd, dtype, scale):
    lens, old = [50, 1], [200, 700]
    c = case(15, lens, old, 2, 64, 16, dtype, dtype)
    check(bnd, queries(16, 51, 4, 64, dtype), lens, old, c, f"scale {scale} {dtype}", scale=scale, rows=some)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n,window,sinks", [(150, 0, 0), (150, 50, 3), (9, 0, 0), (700, 100, 1)])
def test_values_that_are_not_finite(bnd, dtype, value, n, window, sinks):
    """A position's key or value reaches the rows that see it and no others, bit for bit."""
    old, at = 40, 52
    c = case(17, [n], [old], 2, 64, 16, dtype, dtype)
    if n == 9:
        at = 44
    q = queries(18, n, 8, 64, dtype)
    args, _ = U.cache_args(c)
    clean = bnd.attn_prefill(q, V.starts([n]), *args, window=window, sinks=sinks)
    see = [i for i in range(n) if Y.sees(old + i, at, window, sinks)]
    others = [i for i in range(n) if i not in set(see)]
    assert see and others
    page, slot = int(c["page_table"][0, at // 16]), at % 16
    for m in ("v_cache", "k_cache"):
        keep = c[m].clone()
        c[m][page, 1, slot, 5] = value
        o = bnd.attn_prefill(q, V.starts([n]), *args, window=window, sinks=sinks)
        assert torch.equal(o[others], clean[others]), m
        assert torch.equal(o[:, :4], clean[:, :4]), "the other key head"
        if m == "v_cache":
            assert not torch.isfinite(o[see][:, 4:, 5].float()).any()
            rest = [d for d in range(64) if d != 5]
            assert torch.equal(o[..., rest], clean[..., rest])
        elif value != value:
            assert torch.isnan(o[see][:, 4:].float()).all()
        c[m].copy_(keep)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("n,window,sinks", [(150, 0, 0), (150, 50, 3), (3, 0, 0), (700, 100, 1)])
def test_scales_that_are_not_finite(bnd, dtype, value, n, window, sinks):
    """A row of an 8-bit cache whose scale, or one of whose bytes, is a NaN: as a value that is not finite."""
    old, at = 40, 41
    c = case(35, [n], [old], 2, 64, 16, dtype, E4)
    q = queries(36, n, 8, 64, dtype)
    args, scales = U.cache_args(c)
    clean = bnd.attn_prefill(q, V.starts([n]), *args, **scales, window=window, sinks=sinks)
    see = [i for i in range(n) if Y.sees(old + i, at, window, sinks)]
    others = [i for i in range(n) if i not in set(see)]
    assert see and others
    page, slot = int(c["page_table"][0, at // 16]), at % 16
    for m in ("k_scale", "v_scale", "v_cache"):
        t = c[m] if m != "v_cache" else c[m].view(torch.uint8)
        keep = t.clone()
        if m == "v_cache":
            t[page, 1, slot, 7] = 0x7f
        else:
            t[page, 1, slot] = value
        o = bnd.attn_prefill(q, V.starts([n]), *args, **scales, window=window, sinks=sinks)
        assert torch.equal(o[others], clean[others]), m
        assert torch.equal(o[:, :4], clean[:, :4]), "the other key head"
        if m == "v_cache":
            assert torch.isnan(o[see][:, 4:, 7].float()).all()
        elif m == "v_scale":
            assert not torch.isfinite(o[see][:, 4:].float()).any()
        elif value != value:
            assert torch.isnan(o[see][:, 4:].float()).all()
        t.copy_(keep)


def test_pages_outside_the_window_are_not_looked_at(bnd):
    """Entries of the table behind the window's start may hold anything."""
    lens, old, window, sinks = [20, 1], [500, 300], 60, 5
    c = case(19, lens, old, 2, 64, 16, BF, BF)
    q = queries(20, 21, 4, 64, BF)
    args, _ = U.cache_args(c)
    want = bnd.attn_prefill(q, V.starts(lens), *args, window=window, sinks=sinks)
    for b in range(2):
        c["page_table"][b, 1:(old[b] - window + 1) // 16] = 2 ** 30
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert torch.equal(bnd.attn_prefill(q, V.starts(lens), *args, window=window, sinks=sinks, seq_status=st), want) and st.tolist() == [0, 0]
    o = torch.full_like(q, 7.0)
    bnd.attn_prefill(q, V.starts(lens), *args, window=window, sinks=17, seq_status=st, o=o)
    assert st.tolist() == [64, 64] and (o == 7).all()


def test_invalid_items_are_left_whole(bnd):
    lens, old = [200, 1, 0, 30, 3], [3000, 9, 5, 40, 7]
    c = case(21, lens, old, 2, 64, 16, BF, BF)
    q = queries(22, sum(lens), 8, 64, BF)
    args, _ = U.cache_args(c)
    want = bnd.attn_prefill(q, V.starts(lens), *args)
    c["page_table"][0, 190] = -1      # a page of the first item's middle: all of its rows are left
    c["page_table"][3, 4] = 10 ** 6   # the last page of the fourth
    c["cache_len"][2] = 10 ** 6       # an empty sequence past its pages
    c["cache_len"][4] = -7
    o, st = torch.full_like(q, 7.0), torch.zeros(5, dtype=torch.int32, device="cuda")
    bnd.attn_prefill(q, V.starts(lens), *args, o=o, seq_status=st)
    assert st.tolist() == [64, 0, 64, 64, 64]
    assert (o[:200] == 7).all() and torch.equal(o[200], want[200]) and (o[201:] == 7).all()
    for bad in ([0, 300, 200, 201, 231, 234], [0, 1, 2, 3, 4, 999], [-1, 1, 2, 3, 4, 5]):
        o.fill_(7)
        bnd.attn_prefill(q, torch.tensor(bad, dtype=torch.int32, device="cuda"), *args, o=o, seq_status=st)
        assert st.tolist() == [32] * 5 and (o == 7).all()


def test_empty_calls(bnd):
    c = case(23, [0, 0], [5, 0], 2, 64, 16, BF, BF)
    args, _ = U.cache_args(c)
    st = torch.full((2,), -3, dtype=torch.int32, device="cuda")
    bnd.attn_prefill(torch.empty(0, 4, 64, dtype=BF, device="cuda"), V.starts([0, 0]), *args, seq_status=st)
    assert st.tolist() == [0, 0]


def test_graph_of_other_lengths(bnd):
    """Captured once, replayed with other lengths and inputs."""
    lens, old = [60, 1, 20], [400, 1500, 3]
    c = case(24, [70, 70, 70], [1800, 1800, 1800], 2, 64, 16, BF, BF)
    q = queries(25, 120, 8, 64, BF)
    start, o = V.starts(lens), torch.zeros_like(q)
    c["cache_len"].copy_(torch.tensor(old))
    args, _ = U.cache_args(c)
    run = lambda: bnd.attn_prefill(q, start, *args, o=o, window=900, sinks=2)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lens, old in (([60, 1, 20], [400, 1500, 3]), ([1, 1, 1], [1700, 30, 1000]), ([0, 70, 50], [5, 0, 1750]), ([60, 1, 20], [400, 1500, 3])):
        start.copy_(V.starts(lens))
        c["cache_len"].copy_(torch.tensor(old))
        o.fill_(7)
        run()
        want = o.clone()
        o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), lens


@pytest.mark.parametrize("cdtype", [BF, E4])
def test_attention_layer_from_prompt_to_tree(bnd, cdtype):
    """Chunks of a prompt, then a draft tree and its accepted path, then a token: rotated, appended and attended to as
    a layer does, each against the item's own token sequence."""
    H, Hk, D, page, n, T = 4, 2, 64, 16, 3, 9
    f = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)).float().cuda()
    g = torch.Generator().manual_seed(26)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    c = U.cache(27, n, [0] * n, Hk, D, page, BF, cdtype, room=200)
    args, scales = U.cache_args(c)
    wide = lambda *s: torch.randn(*s, H + 2 * Hk, D, generator=g).to(BF).cuda().split([H, Hk, Hk], -2)

    def verify_rows(q, o, at, lens, what):
        for b, new in enumerate(lens):
            done = int(c["cache_len"][b])
            kc, vc = V.cached(c, b, done + new)
            for i in range(new):
                p = done + i
                r, oa, top = Y.attend(U.f64(q[at + i:at + i + 1]), p, kc[:p + 1], vc[:p + 1], D ** -0.5)
                U.within(U.f64(o[at + i:at + i + 1]), r, V.attend_bound(r, oa, top, D, p + 1, BF), f"{what} {b} {i}")
            at += new

    for lens in ([33, 0, 64], [20, 50, 1]):
        q, k, v = wide(sum(lens))
        qo = bnd.attn_append_rope(q, k, v, V.starts(lens), f, *args, **scales, q_weight=wq, k_weight=wk)
        o = bnd.attn_prefill(qo, V.starts(lens), *args, **scales)
        verify_rows(qo, o, 0, lens, "chunk")
        c["cache_len"] += torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = wide(n, T)
    par = U.trees(28, n, T)
    depth = bnd.tree_info(par.cuda())[0]
    qo, ko = bnd.attn_rope(q, k, c["cache_len"][:, None] + depth, f, wq, wk)
    v = v.contiguous()
    o = bnd.attn_verify(qo, ko, v, par.cuda(), *args, **scales)
    from oracle import sequence as S
    acc, count = torch.full((n, 4), -1, dtype=torch.int32), []
    for b in range(n):
        kc, vc = V.cached(c, b, int(c["cache_len"][b]))
        r, oa, top = S.attend(U.f64(qo[b]), U.f64(ko[b]), U.f64(v[b]), par[b].numpy(), kc, vc, D ** -0.5)
        U.within(U.f64(o[b]), r, V.attend_bound(r, oa, top, D, 200, BF), f"tree {b}")
        path = S.root_path(par[b].numpy(), T - 1)[:4]
        acc[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        count.append(len(path))
    count = torch.tensor(count, dtype=torch.int32, device="cuda")
    bnd.attn_commit(ko, v, par.cuda(), acc.cuda(), count, *args, **scales)
    c["cache_len"] += count
    q, k, v = wide(n)
    qo = bnd.attn_append_rope(q, k, v, V.starts([1] * n), f, *args, **scales, q_weight=wq, k_weight=wk)
    o = bnd.attn_prefill(qo, V.starts([1] * n), *args, **scales)
    verify_rows(qo, o, 0, [1] * n, "token")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ssm_layer_from_projection_to_token(bnd, dtype):
    """Convolution and scan over a prompt, a tree verified and committed, one token: the states and outputs are those of
    the accepted sequence as one prompt."""
    H, P, N, G, W, T, lens = 2, 64, 64, 1, 4, 7, [10, 3]
    C, n = H * P + 2 * G * N, 2
    g = torch.Generator().manual_seed(29)
    rnd = lambda *s: torch.randn(*s, generator=g)
    w, bias = (0.5 * rnd(C, W)).cuda(), (0.1 * rnd(C)).cuda()
    A, D = -torch.exp(rnd(H)).cuda(), rnd(H).cuda()
    io = lambda *rows: tuple(torch.zeros(*rows, *s, dtype=dtype, device="cuda") for s in ((H, P), (G, N), (G, N)))
    dts = lambda *rows: torch.nn.functional.softplus(rnd(*rows, H) - 3).to(dtype).cuda()
    xbc, dt = rnd(sum(lens), C).to(dtype).cuda(), dts(sum(lens))
    conv, h = torch.zeros(n, W - 1, C, dtype=dtype, device="cuda"), torch.zeros(n, H, P, N, device="cuda")
    x, B, Cc = io(sum(lens))
    bnd.conv_prefill(xbc, w, bias, conv, V.starts(lens), x, B, Cc)
    bnd.prefill(x, dt, A, B, Cc, D, h, V.starts(lens))
    txbc, tdt, par = rnd(n, T, C).to(dtype).cuda(), dts(n, T), U.trees(30, n, T)
    tx, tB, tC = io(n, T)
    bnd.conv_verify(txbc, w, bias, conv, par.cuda(), tx, tB, tC)
    ty = bnd.verify(tx, tdt, A, tB, tC, D, h, par.cuda())
    from oracle import sequence as S
    paths = [S.root_path(par[b].numpy(), T - 1 - b) for b in range(n)]
    acc = torch.full((n, T), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        acc[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    count = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    bnd.conv_commit(txbc, conv, par.cuda(), acc.cuda(), count, H, P, G, N)
    bnd.commit(tx, tdt, A, tB, h, par.cuda(), acc.cuda(), count)
    sxbc, sdt = rnd(n, C).to(dtype).cuda(), dts(n)
    sx, sB, sC = io(n)
    bnd.conv_step(sxbc, w, bias, conv, sx, sB, sC)
    sy = bnd.step(sx, sdt, A, sB, sC, D, h)
    # the same as one prompt
    at, seqs, sdts = 0, [], []
    for b, L in enumerate(lens):
        seqs.append(torch.cat([xbc[at:at + L], txbc[b, paths[b]], sxbc[b:b + 1]]))
        sdts.append(torch.cat([dt[at:at + L], tdt[b, paths[b]], sdt[b:b + 1]]))
        at += L
    total = [len(s) for s in seqs]
    conv2, h2 = torch.zeros_like(conv), torch.zeros_like(h)
    x2, B2, C2 = io(sum(total))
    bnd.conv_prefill(torch.cat(seqs), w, bias, conv2, V.starts(total), x2, B2, C2)
    y2 = bnd.prefill(x2, torch.cat(sdts), A, B2, C2, D, h2, V.starts(total))
    assert torch.equal(conv, conv2)
    ends = np.cumsum(total) - 1
    assert all(torch.equal(a, b[ends]) for a, b in ((sx, x2), (sB, B2), (sC, C2)))
    tol = 2e-2 if dtype == BF else 1e-4
    err = lambda a, b: float((a.float() - b.float()).abs().max() / b.float().abs().max())
    assert err(h, h2) <= 1e-4 and err(sy, y2[ends]) <= tol
    for b in range(n):
        assert err(ty[b, paths[b][-1]], y2[ends[b] - 1]) <= tol


def test_calls_on_two_streams(bnd):
    """Calls on two streams share nothing but their read-only inputs."""
    lens, old = [60, 1, 20], [400, 1500, 3]
    c = case(31, lens, old, 2, 64, 16, BF, BF)
    q = queries(32, 81, 8, 64, BF)
    args, _ = U.cache_args(c)
    start, f = V.starts(lens), torch.ones(32, device="cuda")
    pos = torch.arange(81, dtype=torch.int32, device="cuda")
    xbc, w = V.wide(33, 81, 192, dtype=BF, lead=8), torch.ones(192, 4, device="cuda")
    s0 = V.wide(34, 3, 3, 192, dtype=BF).contiguous()

    def once(stream=None):
        state = s0.clone()
        out = tuple(torch.zeros(81, 1, 64, dtype=BF, device="cuda") for _ in range(3))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        bnd.conv_prefill(xbc, w, None, state, start, *out, stream=stream)
        return (*out, state, bnd.attn_prefill(q, start, *args, stream=stream), bnd.attn_rope(q, None, pos, f, stream=stream)[0])

    want = once()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        got += [once(s) for s in streams]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_cache_past_32_bits(bnd):
    """Pages whose bytes lie past 2^32: written by the rotated append, read by each kernel."""
    Hk, D, page, pages = 8, 128, 64, 35000  # 4.6 GB a cache
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    kc, vc = (torch.empty(pages, Hk, page, D, dtype=BF, device="cuda") for _ in range(2))
    table = torch.tensor([[pages - 1, 5, pages - 3, pages - 2], [pages - 7, 0, 0, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(37)
    q, k, v = (torch.randn(203, h, D, generator=g).to(BF).cuda() for h in (16, Hk, Hk))
    f = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    qo = bnd.attn_append_rope(q, k, v, V.starts([200, 3]), f, kc, vc, table, lens)
    c = {"k_cache": kc[[pages - 1, 5, pages - 3, pages - 2, pages - 7]], "v_cache": vc[[pages - 1, 5, pages - 3, pages - 2, pages - 7]],
         "page_table": torch.tensor([[0, 1, 2, 3], [4, 0, 0, 0]], dtype=torch.int32), "cache_len": lens, "k_scale": None, "v_scale": None}
    pos = torch.tensor([*range(200), *range(3)], dtype=torch.int32, device="cuda")
    want = bnd.attn_rope(None, k, pos, f)[1]
    rows = torch.arange(200)
    assert torch.equal(c["k_cache"][(rows // page).cuda(), :, (rows % page).cuda()], want[:200])
    for generic in (False, True):
        o = bnd.attn_prefill(qo, V.starts([200, 3]), kc, vc, table, lens, force_generic=generic)
        for b, i, at in ((0, 0, 0), (0, 199, 199), (0, 77, 77), (1, 2, 202)):
            kk, vv = V.cached(c, b, i + 1)
            r, oa, top = Y.attend(U.f64(qo[at:at + 1]), i, kk, vv, D ** -0.5)
            U.within(U.f64(o[at:at + 1]), r, V.attend_bound(r, oa, top, D, i + 1, BF), f"row {i} of {b}")
    lens.copy_(torch.tensor([199, 2]))
    one = bnd.attn_prefill(qo[[199, 202]], V.starts([1, 1]), kc, vc, table, lens)  # the few rows' kernel
    for x, (b, i, at) in zip(one, ((0, 199, 199), (1, 2, 202))):
        kk, vv = V.cached(c, b, i + 1)
        r, oa, top = Y.attend(U.f64(qo[at:at + 1]), i, kk, vv, D ** -0.5)
        U.within(U.f64(x[None]), r, V.attend_bound(r, oa, top, D, i + 1, BF), f"token {i} of {b}")


def test_layer_calls_in_a_graph(bnd):
    """Rotation, append, attention, convolution and their tree forms, captured once and replayed with other lengths and
    inputs, with eager work between the replays."""
    H, Hk, D, n, T = 4, 2, 64, 3, 5
    c = U.cache(38, n, [0] * n, Hk, D, 16, BF, E4, room=120)
    args, scales = U.cache_args(c)
    g = torch.Generator().manual_seed(39)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()
    wide, f = rnd(40, H + 2 * Hk, D), torch.rand(D // 2, generator=g).cuda()
    q, k, v = wide.split([H, Hk, Hk], -2)
    start, pos, par = V.starts([20, 0, 13]), torch.zeros(n, T, dtype=torch.int32, device="cuda"), U.trees(40, n, T, "chain").cuda()
    tq, tk = rnd(n, T, H, D), rnd(n, T, Hk, D)
    xbc, w, state0 = rnd(40, 192), torch.rand(192, 4, generator=g).cuda(), rnd(n, 3, 192)
    txbc, acc, count = rnd(n, T, 192), torch.arange(T, dtype=torch.int32).repeat(n, 1).cuda(), torch.tensor([2, 0, 5], dtype=torch.int32, device="cuda")
    out = [torch.zeros(*s, 1, 64, dtype=BF, device="cuda") for s in ((40,), (n, T), (n,)) for _ in range(3)]
    qo, o, state = torch.zeros(40, H, D, dtype=BF, device="cuda"), torch.zeros(40, H, D, dtype=BF, device="cuda"), state0.clone()
    tqo, tko = torch.zeros_like(tq), torch.zeros_like(tk)

    def once():
        bnd.attn_append_rope(q, k, v, start, f, *args, **scales, q_out=qo)
        bnd.attn_prefill(qo, start, *args, **scales, o=o)
        bnd.attn_rope(tq, tk, pos, f, q_out=tqo, k_out=tko)
        bnd.conv_prefill(xbc, w, None, state, start, *out[:3])
        bnd.conv_verify(txbc, w, None, state, par, *out[3:6])
        bnd.conv_commit(txbc, state, par, acc, count, 1, 64, 1, 64)
        bnd.conv_step(txbc[:, 0], w, None, state, *out[6:])

    everything = [qo, o, tqo, tko, state, *out, c["k_scale"], c["v_scale"]]
    caches = [c["k_cache"].view(torch.uint8), c["v_cache"].view(torch.uint8)]
    first = [t.clone() for t in everything + caches]

    def fresh(lens, old):
        for t, t0 in zip(everything + caches, first):
            t.copy_(t0)
        start.copy_(V.starts(lens))
        c["cache_len"].copy_(torch.tensor(old))
        pos.copy_(torch.tensor(old)[:, None] + torch.arange(T))

    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for lens, old in (([20, 0, 13], [0, 5, 90]), ([1, 1, 1], [100, 0, 17]), ([0, 30, 10], [3, 70, 0]), ([20, 0, 13], [0, 5, 90])):
        fresh(lens, old)
        once()
        want = [t.clone() for t in everything + caches]
        fresh(lens, old)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(everything + caches, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), lens


def few_rows(bnd, lens, H, Hk, D, dtype, cdtype=None):
    """Whether the call's blocks are those of few rows (16; 64 or 128 otherwise): by what a table that is cut needs."""
    need = bnd.attn_prefill_workspace_bytes(len(lens), sum(lens), H, Hk, D, 16, 4096, dtype, cdtype)
    return need / (2 * 512 * 4 * (D + 2)) < 32


# kernel, new tokens of the one item: blocks of few rows, of many, and the plain kernel
KERNELS = [("few", 1), ("few", 4), ("many", 21), ("many", 150), ("plain", 4), ("plain", 21)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("old", [0, 38, 1210])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 2)])
def test_last_scale_that_is_not_finite(bnd, dtype, value, kernel, n, old, window, sinks):
    """The newest position's scale or byte is a NaN, as appended from a row that is not finite: it reaches the last
    token's rows alone, and positions behind it (whose rows of the pool are finite here, and pages of the pool) none."""
    c = case(41, [n], [old], 2, 64, 16, dtype, E4)
    c["page_table"].clamp_(min=0)
    for m in ("k_scale", "v_scale"):
        c[m].nan_to_num_(nan=1.0)
    for m in ("k_cache", "v_cache"):
        u = c[m].view(torch.uint8)
        u[u == 0x7f] = 0x30
    q = queries(42, n, 8, 64, dtype)
    assert kernel == "plain" or few_rows(bnd, [n], 8, 2, 64, dtype, E4) == (kernel == "few")
    args, scales = U.cache_args(c)
    run = lambda: bnd.attn_prefill(q, V.starts([n]), *args, **scales, window=window, sinks=sinks, force_generic=kernel == "plain")
    clean = run()
    p = old + n - 1
    page, slot = int(c["page_table"][0, p // 16]), p % 16
    for m in ("k_scale", "v_scale", "v_cache"):
        t = c[m] if m != "v_cache" else c[m].view(torch.uint8)
        keep = t.clone()
        if m == "v_cache":
            t[page, 1, slot, 7] = 0x7f
        else:
            t[page, 1, slot] = value
        say(f"[last] {m} {value} {kernel} {dtype} {n} after {old} window {window}+{sinks}")
        o = run()
        assert torch.equal(o[:-1], clean[:-1]), m
        assert torch.equal(o[:, :4], clean[:, :4]), "the other key head"
        if m == "v_cache":
            assert torch.isnan(o[-1, 4:, 7].float()).all()
        elif m == "v_scale":
            assert not torch.isfinite(o[-1, 4:].float()).any()
        elif value != value:
            assert torch.isnan(o[-1, 4:].float()).all()
        t.copy_(keep)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("n", [4, 20])
@pytest.mark.parametrize("size", [8.0, 2.0 ** 18 + 2.0 ** 16])
def test_rows_do_not_depend_on_their_neighbours(bnd, dtype, cdtype, n, size):
    """Rows with the same score at every position, beside rows whose maximum moves at every step: an output is the mean of
    the values whatever the neighbours do, to the bit."""
    items, H, Hk, D, old = 6, 8, 2, 64, 490
    lens, olds = [n] * items, [old] * items
    c = case(45, lens, olds, Hk, D, 16, dtype, cdtype)
    ramp = torch.zeros(old + n, D)
    ramp[:, 0], ramp[:, 1] = 1, torch.arange(old + n) // 16
    rows = torch.arange(old + n)
    for b in range(items):
        pages = c["page_table"][b].cpu()[rows // 16]
        c["k_cache"][pages.cuda(), :, (rows % 16).cuda()] = ramp.cuda()[:, None].expand(-1, Hk, -1).to(c["k_cache"].dtype)
        if cdtype == E4:
            c["k_scale"][pages.cuda(), :, (rows % 16).cuda()] = 1.0
    assert few_rows(bnd, lens, H, Hk, D, dtype, cdtype) == (n == 4)
    q = torch.zeros(items, n, H, D, dtype=dtype, device="cuda")
    q[..., 0] = size
    args, scales = U.cache_args(c)
    run = lambda x: bnd.attn_prefill(x.view(-1, H, D), V.starts(lens), *args, **scales).view(items, n, H, D)
    want = run(q)
    for b in range(items):
        _, vc = V.cached(c, b, old + n)
        for i in (0, 1, n - 1):
            v = vc[:old + i + 1]
            mean, oa = v.mean(0), np.abs(v).mean(0)
            # all scores are one number, so the weights are equal: the sums round, in bf16 the output, and in blocks of many
            # rows the weight beside its sum
            half = 2.0 ** -8 if dtype == BF else 0.0
            bound = (old + 64) * 2.0 ** -24 * oa + half * (np.abs(mean) * 1.01 + (oa if n > 4 else 0)) + 1e-30
            U.within(U.f64(want[b, i]).reshape(Hk, 4, D), mean[:, None], bound[:, None], f"mean {b} {i}")
    x = q.clone()
    x[:, :, 1::2, 1] = 4.0
    x[:, :2, :, 1] = 2.0
    got = run(x)
    assert torch.equal(got[:, 2:, ::2], want[:, 2:, ::2])
    assert not torch.equal(got[:, :2], want[:, :2])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("kernel,n", KERNELS[1:])
@pytest.mark.parametrize("old,back,window,sinks", [(40, -1, 0, 0), (40, 0, 0, 0), (700, -1, 0, 0), (700, 299, 300, 2), (700, 0, 300, 2), (700, 699, 300, 2)])
def test_positions_that_are_not_finite_in_each_kernel(bnd, dtype, value, kernel, n, old, back, window, sinks):
    """A key or a value that is not finite, at the newest position (back -1) or `back` before the first new one, in bits: the
    rows that see it have it, an infinite value as an infinity, the others are as they were."""
    c = case(48, [n], [old], 2, 64, 16, dtype, dtype)
    q = queries(49, n, 8, 64, dtype)
    assert kernel == "plain" or few_rows(bnd, [n], 8, 2, 64, dtype) == (kernel == "few")
    args, _ = U.cache_args(c)
    run = lambda: bnd.attn_prefill(q, V.starts([n]), *args, window=window, sinks=sinks, force_generic=kernel == "plain")
    clean, at = run(), old + n - 1 if back < 0 else old - back
    see = [i for i in range(n) if Y.sees(old + i, at, window, sinks)]
    others = [i for i in range(n) if i not in set(see)]
    assert see
    page, slot = int(c["page_table"][0, at // 16]), at % 16
    rest = [d for d in range(64) if d != 5]
    for m in ("v_cache", "k_cache"):
        keep = c[m].clone()
        c[m][page, 1, slot, 5] = value
        o = run()
        assert torch.equal(o[others], clean[others]), m
        assert torch.equal(o[:, :4], clean[:, :4]), "the other key head"
        if m == "v_cache":
            hit = o[see][:, 4:, 5]
            assert torch.isnan(hit.float()).all() if value != value else (hit == value).all(), hit
            assert torch.equal(o[..., rest], clean[..., rest])
        elif value != value:
            assert torch.isnan(o[see][:, 4:].float()).all()
        else:  # an infinite score: its weight is the only one (NaN), or none
            up = (q[see][:, 4:, 5].double() * value > 0)[..., None].expand(-1, -1, 64)
            got = o[see][:, 4:]
            assert torch.isnan(got[up].float()).all() and torch.isfinite(got[~up].float()).all()
        c[m].copy_(keep)
