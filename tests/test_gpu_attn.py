"""GPU: tree attention over the paged cache (tree_attn_verify) and the cache's
writes (tree_attn_commit, tree_attn_append) against the fp64 definitions.

Bounds of an output, elementwise, with oa = sum_j p_j |v_j| and top the largest
scale sum_d |q_d k_d|: a score is off by at most (D + 8) 2^-24 top, a weight by
twice that relatively, the sums over L keys by (L + 64) 2^-24; bf16 adds half a
step (2^-8) of o, and half a step of each weighted value: 2^-8 oa.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import sequence as S
from tests import seq_util as U
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bnd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from speculative_tree_verification_amd import binding
    return binding


def nodes(seed, n, T, H, Hk, D, dtype):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    return rnd(n, T, H, D), rnd(n, T, Hk, D), rnd(n, T, Hk, D)


def check(bnd, q, k, v, par, c, dtype, what, scale=None, only=None, **kw):
    """`only`: the items to compare (the others are checked by the caller)."""
    n, T, H, D = q.shape
    o = torch.full_like(q, 7.0)
    st = torch.full((n,), -3, dtype=torch.int32, device="cuda")
    args, scales = U.cache_args(c)
    say(f"[attn] {what}")
    bnd.attn_verify(q, k, v, par.cuda(), *args, **scales, scale=scale, o=o, tree_status=st, **kw)
    torch.cuda.synchronize()
    og, worst = U.f64(o), 0.0
    page = c["k_cache"].shape[2]
    for b in range(n) if only is None else only:
        assert int(st[b]) == 0
        L = int(c["cache_len"][b])
        t = c["page_table"][b].cpu().numpy()
        kc, vc = (S.cache_rows(U.np8(c[m + "_cache"]), U.np8(c[m + "_scale"]), t, L, page) for m in "kv")
        r, oa, top = S.attend(U.f64(q[b]), U.f64(k[b]), U.f64(v[b]), par[b].numpy(), kc, vc, D ** -0.5 if scale is None else scale)
        f = (2 * (D + 8) * top + L + T + 64) * 2.0 ** -24
        bound = f * oa + 1e-30
        if dtype == BF:
            bound = bound + 2.0 ** -8 * (np.abs(r) + 1.02 * oa)
        worst = max(worst, U.within(og[b], r, bound, f"{what}, item {b}"))
    say(f"[attn] {what}: {worst:.3f} of the bound")
    return o, st


TYPES = [(BF, BF), (BF, E4), (F32, F32), (F32, E4)]
HEADS = [(8, 2, 128), (4, 4, 64), (6, 1, 128), (16, 1, 64), (3, 1, 40), (2, 2, 256), (2, 1, 1)]


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("H,Hk,D", HEADS)
@pytest.mark.parametrize("T", [1, 15])
def test_heads_and_types(bnd, dtype, cdtype, H, Hk, D, T):
    lens = [0, 1, 63, 130]
    c = U.cache(D + T, 4, lens, Hk, D, 16, dtype, cdtype)
    check(bnd, *nodes(D, 4, T, H, Hk, D, dtype), U.trees(T, 4, T), c, dtype, f"{dtype} {cdtype} H={H}/{Hk} D={D} T={T}")


@pytest.mark.parametrize("cdtype", [BF, E4])
@pytest.mark.parametrize("page", [1, 7, 16, 24, 64, 1000])
@pytest.mark.parametrize("T", [1, 40])
def test_pages(bnd, cdtype, page, T):
    """Pages that end inside a tile, hold many tiles, or hold one position."""
    c = U.cache(page, 2, [333, 64], 2, 64, page, BF, cdtype)
    check(bnd, *nodes(page, 2, T, 4, 2, 64, BF), U.trees(T, 2, T), c, BF, f"page {page} T={T} {cdtype}")


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("T", [1, 33])
def test_split_lengths(bnd, dtype, cdtype, T):
    """Caches of very different lengths, cut into parts that are joined."""
    lens = [5000, 0, 17, 256, 257, 1025]
    c = U.cache(3, 6, lens, 2, 128, 16, dtype, cdtype)
    assert bnd.attn_verify_workspace_bytes(6, T, 8, 2, 128, 16, c["page_table"].shape[1], dtype, cdtype) > 0
    check(bnd, *nodes(T, 6, T, 8, 2, 128, dtype), U.trees(T, 6, T), c, dtype, f"split {dtype} {cdtype} T={T}")


@pytest.mark.parametrize("T,kind", [(2, "chain"), (16, "star"), (17, "random"), (63, "random"), (64, "chain"), (65, "random"),
                                    (130, "random"), (257, "chain")])
@pytest.mark.parametrize("H,Hk", [(4, 1), (2, 2)])
def test_trees(bnd, T, kind, H, Hk):
    c = U.cache(T, 2, [37, 0], Hk, 64, 16, BF, BF)
    check(bnd, *nodes(T, 2, T, H, Hk, 64, BF), U.trees(T, 2, T, kind), c, BF, f"tree {kind} T={T} H={H}/{Hk}")


@pytest.mark.parametrize("T,kind", [(2, "chain"), (16, "star"), (17, "random"), (63, "random"), (65, "random"), (130, "chain")])
@pytest.mark.parametrize("H,Hk,D,cdtype", [(4, 1, 64, F32), (2, 2, 64, E4), (8, 2, 128, F32), (5, 1, 128, E4)])
def test_trees_f32(bnd, T, kind, H, Hk, D, cdtype):
    """The fp32 kernels' trees: blocks of rows, nodes past a tile, an empty cache."""
    c = U.cache(T, 2, [37, 0], Hk, D, 16, F32, cdtype)
    check(bnd, *nodes(T, 2, T, H, Hk, D, F32), U.trees(T, 2, T, kind), c, F32, f"fp32 tree {kind} T={T} H={H}/{Hk} D={D} {cdtype}")


def test_largest_tree_f32(bnd):
    c = U.cache(4, 1, [90], 1, 64, 16, F32, F32)
    check(bnd, *nodes(4, 1, 1024, 2, 1, 64, F32), U.trees(4, 1, 1024), c, F32, "1024 nodes, fp32")


@pytest.mark.parametrize("cdtype", [F32, E4])
@pytest.mark.parametrize("page", [1, 7, 24, 1000])
@pytest.mark.parametrize("T", [1, 40])
def test_pages_f32(bnd, cdtype, page, T):
    c = U.cache(page, 2, [333, 64], 2, 128, page, F32, cdtype)
    check(bnd, *nodes(page, 2, T, 4, 2, 128, F32), U.trees(T, 2, T), c, F32, f"fp32 page {page} T={T} {cdtype}")


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 21])
def test_plain_kernel(bnd, dtype, cdtype, D, T):
    """The plain kernel where the matrix kernels would be taken, with a split."""
    c = U.cache(14, 3, [2600, 0, 90], 2, D, 16, dtype, cdtype)
    check(bnd, *nodes(14, 3, T, 6, 2, D, dtype), U.trees(14, 3, T), c, dtype, f"plain {dtype} {cdtype} D={D} T={T}",
          force_generic=True)


@pytest.mark.parametrize("T", [1, 21])
def test_unaligned_f32(bnd, T):
    """fp32 tensors that are not 16-byte aligned take the plain kernel."""
    c = U.cache(15, 2, [150, 9], 2, 64, 16, F32, F32)
    q, k, v = nodes(15, 2, T, 4, 2, 64, F32)
    u = torch.empty(q.numel() + 1, device="cuda")[1:].view(q.shape).copy_(q)
    assert u.data_ptr() % 16 != 0
    check(bnd, u, k, v, U.trees(15, 2, T), c, F32, f"unaligned fp32 T={T}")


MANY = [(9, 32, 8, 31, "random"), (17, 8, 4, 63, "random"), (66, 2, 1, 255, "chain"), (33, 6, 2, 41, "star"), (10, 8, 8, 128, "random")]


@pytest.mark.parametrize("n,H,Hk,T,kind", MANY)
@pytest.mark.parametrize("D,cdtype", [(64, BF), (128, BF), (64, E4), (128, E4)])
def test_trees_of_many_items(bnd, n, H, Hk, T, kind, D, cdtype):
    """Enough items and rows for the largest blocks of rows; caches that are empty, end inside a tile, or are cut."""
    lens = [(41 * b) % 130 for b in range(n)]
    lens[1], lens[2], lens[3] = 2600, 64, 700
    c = U.cache(n, n, lens, Hk, D, 16, BF, cdtype)
    check(bnd, *nodes(n, n, T, H, Hk, D, BF), U.trees(n, n, T, kind), c, BF, f"{n} items T={T} {kind} H={H}/{Hk} D={D} {cdtype}",
          only=[0, 1, 3, n - 1] if T < 100 else [1, n - 1])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_masked_nodes_of_many_items(bnd, value):
    """A node's value reaches its descendants in its own item only."""
    n, T, bad = 9, 33, 5
    par = U.trees(18, n, T)
    c = U.cache(18, n, [50 + b for b in range(n)], 8, 64, 16, BF, BF)
    q, k, v = nodes(18, n, T, 32, 8, 64, BF)
    args, _ = U.cache_args(c)
    clean = bnd.attn_verify(q, k, v, par.cuda(), *args)
    below = [i for i in range(T) if bad in S.root_path(par[4].numpy(), i)]
    others = [i for i in range(T) if i not in below]
    vv = v.clone()
    vv[4, bad] = value
    o = bnd.attn_verify(q, k, vv, par.cuda(), *args)
    assert torch.equal(o[4, others], clean[4, others]) and not torch.isfinite(o[4, below].float()).any()
    keep = [b for b in range(n) if b != 4]
    assert torch.equal(o[keep], clean[keep])


def test_largest_tree(bnd):
    c = U.cache(4, 1, [90], 1, 64, 16, BF, BF)
    check(bnd, *nodes(4, 1, 1024, 2, 1, 64, BF), U.trees(4, 1, 1024), c, BF, "1024 nodes")


def test_many_items(bnd):
    """More items than threads of the search for a part."""
    lens = [(37 * b) % 90 for b in range(300)]
    c = U.cache(6, 300, lens, 1, 64, 16, BF, BF)
    q, k, v = nodes(6, 300, 1, 2, 1, 64, BF)
    par = U.trees(6, 300, 1)
    check(bnd, q, k, v, par, c, BF, "300 items", only=range(0, 300, 13))


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("n", [64, 65, 300])
def test_many_items_split(bnd, n, T):
    """Items on both sides of the search's one-wave form, some of them cut into parts."""
    lens = [(11 * b) % 20 for b in range(n)]
    lens[1], lens[n - 2] = 3000, 900
    c = U.cache(7, n, lens, 1, 64, 16, BF, BF)
    q, k, v = nodes(7, n, T, 2, 1, 64, BF)
    check(bnd, q, k, v, U.trees(7, n, T), c, BF, f"{n} items, T={T}", only=[0, 1, 2, n // 2, n - 2, n - 1])


@pytest.mark.parametrize("dtype,cdtype", TYPES)
def test_large_scores(bnd, dtype, cdtype):
    """Scores far apart: the running maximum moves, weights underflow."""
    c = U.cache(8, 2, [700, 90], 1, 64, 16, dtype, cdtype)
    q, k, v = nodes(8, 2, 9, 4, 1, 64, dtype)
    check(bnd, q * 8, k, v, U.trees(8, 2, 9), c, dtype, f"large scores {dtype} {cdtype}")
    check(bnd, q, k, v, U.trees(8, 2, 9), c, dtype, "negative scale", scale=-0.3)
    check(bnd, q, k, v, U.trees(8, 2, 9), c, dtype, "scale 0", scale=0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_masked_nodes_that_are_not_finite(bnd, dtype, value):
    """A node's key or value reaches its descendants only."""
    T, bad = 21, 4
    par = U.trees(10, 1, T)
    c = U.cache(10, 1, [50], 1, 64, 16, dtype, dtype)
    q, k, v = nodes(10, 1, T, 4, 1, 64, dtype)
    args, _ = U.cache_args(c)
    clean = bnd.attn_verify(q, k, v, par.cuda(), *args)
    below = [i for i in range(T) if bad in S.root_path(par[0].numpy(), i)]
    others = [i for i in range(T) if i not in below]
    assert len(others) > 2 and len(below) > 0
    for name in "kv":
        kk, vv = k.clone(), v.clone()
        (kk if name == "k" else vv)[0, bad] = value
        o = bnd.attn_verify(q, kk, vv, par.cuda(), *args)
        assert torch.equal(o[0, others], clean[0, others]), name
        if name == "v" or value != value:
            assert not torch.isfinite(o[0, below].float()).any(), name


def test_bad_pages_f32(bnd):
    """A page out of range stops its own item only, whatever part it is in."""
    for T in (1, 30):
        c = U.cache(16, 3, [2000, 1500, 20], 2, 64, 16, F32, F32)
        q, k, v = nodes(16, 3, T, 4, 2, 64, F32)
        par = U.trees(16, 3, T).cuda()
        args, _ = U.cache_args(c)
        want = bnd.attn_verify(q, k, v, par, *args)
        c["page_table"][1, 70] = c["k_cache"].shape[0]
        o, st = torch.full_like(q, 5.0), torch.zeros(3, dtype=torch.int32, device="cuda")
        bnd.attn_verify(q, k, v, par, *args, o=o, tree_status=st)
        assert st.tolist() == [0, 64, 0]
        assert (o[1] == 5.0).all() and torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])


def test_bad_items_keep_their_output(bnd):
    """Status bits, and the items beside a bad one."""
    n, T = 7, 9
    lens = [300, 20, 40, 60, 300, 50, 10]
    for room in (0, 2000):  # without and with a split
        c = U.cache(12, n, lens, 2, 64, 16, BF, BF, room=room)
        q, k, v = nodes(12, n, T, 4, 2, 64, BF)
        par = U.trees(12, n, T)
        par[0, 0], par[1, 5] = 0, 5
        cap = c["page_table"].shape[1] * 16
        c["cache_len"][2], c["cache_len"][3] = -1, cap + 1
        c["page_table"][4, 3] = c["k_cache"].shape[0]
        c["page_table"][5, 0] = -1
        o, st = check(bnd, q, k, v, par, c, BF, f"bad items, room {room}", only=[6])
        assert st.tolist() == [1, 2, 64, 64, 64, 64, 0]
        assert (o[:6] == 7.0).all()
        par[1, 0] = 3
        _, st = check(bnd, q, k, v, par, c, BF, "two bits", only=[6])
        assert int(st[1]) == 3


def test_empty_pool(bnd):
    """No page at all: the tree alone."""
    q, k, v = nodes(14, 2, 5, 2, 1, 64, BF)
    par = U.trees(14, 2, 5)
    c = {"k_cache": torch.zeros(0, 1, 16, 64, dtype=BF, device="cuda"), "v_cache": torch.zeros(0, 1, 16, 64, dtype=BF, device="cuda"),
         "page_table": torch.zeros(2, 0, dtype=torch.int32, device="cuda"), "cache_len": torch.zeros(2, dtype=torch.int32, device="cuda"),
         "k_scale": None, "v_scale": None}
    check(bnd, q, k, v, par, c, BF, "no pages")


def test_far_pages(bnd):
    """Rows whose element offset passes 32 bits (a pool of 2^31 + elements per cache)."""
    page, Hk, D = 64, 8, 128
    pages = 2 ** 31 // (page * Hk * D) + 9
    pool = {m: torch.zeros(pages, Hk, page, D, dtype=BF, device="cuda") for m in "kv"}
    table = torch.arange(pages - 1, pages - 9, -1, dtype=torch.int32, device="cuda")[None]
    lens, g = 500, torch.Generator(device="cuda").manual_seed(3)
    for m in "kv":
        pool[m][table[0].long()] = torch.randn(8, Hk, page, D, generator=g, device="cuda").to(BF)
    c = {"k_cache": pool["k"], "v_cache": pool["v"], "page_table": table, "k_scale": None, "v_scale": None,
         "cache_len": torch.tensor([lens], dtype=torch.int32, device="cuda")}
    near = dict(c, k_cache=pool["k"][pages - 9:].clone(), v_cache=pool["v"][pages - 9:].clone(), page_table=table - (pages - 9))
    for T in (1, 20):
        q, k, v = nodes(16 + T, 1, T, 16, Hk, D, BF)
        par = U.trees(16, 1, T).cuda()
        a = bnd.attn_verify(q, k, v, par, *U.cache_args(c)[0])
        b = bnd.attn_verify(q, k, v, par, *U.cache_args(near)[0])
        assert torch.equal(a, b)
    start = torch.tensor([0, 12], dtype=torch.int32, device="cuda")
    rows = torch.randn(12, Hk, D, device="cuda", generator=g).to(BF)
    bnd.attn_append(rows, -rows, start, *U.cache_args(c)[0])
    for i in range(12):
        p = lens + i
        at = int(table[0, p // page])
        assert torch.equal(pool["k"][at, :, p % page], rows[i]) and torch.equal(pool["v"][at, :, p % page], -rows[i])


def test_verify_on_a_side_stream_and_in_a_graph(bnd):
    c = U.cache(18, 3, [2000, 100, 700], 2, 128, 16, BF, E4)
    q, k, v = nodes(18, 3, 15, 8, 2, 128, BF)
    par = U.trees(18, 3, 15).cuda()
    args, scales = U.cache_args(c)
    want = bnd.attn_verify(q, k, v, par, *args, **scales)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # the current stream is busy
    o = bnd.attn_verify(q, k, v, par, *args, **scales, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    o = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bnd.attn_verify(q, k, v, par, *args, **scales, o=o)
    old = c["cache_len"].clone()
    for lens in ([2000, 100, 700], [1, 1900 % 112, 300], [2000, 100, 700]):  # the split follows the lengths on replay
        c["cache_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        want = bnd.attn_verify(q, k, v, par, *args, **scales)
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        # bit for bit: 108 of item 1's positions reach rows that were never written and hold NaN
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)), lens
    c["cache_len"].copy_(old)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 3, 33])
@pytest.mark.parametrize("L", [64, 128, 1000])
def test_scores_of_few_channels(bnd, dtype, cdtype, D, T, L):
    """Four channels alone carry scores of several hundred, of either sign: those that the fp32 products of 4
    channels a step take in the last one. A maximum that lacks them lets the weights overflow or vanish."""
    q, k, v = nodes(D + T, 1, T, 4, 1, D, dtype)
    c = U.cache(L, 1, [L], 1, D, 16, dtype, F32 if cdtype == E4 else cdtype)
    big = [D - 13, D - 9, D - 5, D - 1]
    for t, by in ((q, 16.0), (k, 5.0), (c["k_cache"], 5.0)):
        kept = t[..., big] * by
        t *= 0.01
        t[..., big] = kept
    if cdtype == E4:
        for m in "kv":
            by, sc = U.quantise(torch.nan_to_num(c[m + "_cache"].cpu().float()))
            c[m + "_cache"], c[m + "_scale"] = by.cuda(), sc.cuda()
    check(bnd, q, k, v, U.trees(T, 1, T), c, dtype, f"few channels {dtype} {cdtype} D={D} T={T} L={L}", scale=1.0)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 3])
def test_large_scores_of_few_rows(bnd, dtype, cdtype, D, T):
    """At most 16 rows a key head: their own kernels' maxima, factors and join of the waves."""
    c = U.cache(40 + D, 3, [700, 90, 3000], 1, D, 16, dtype, cdtype)
    q, k, v = nodes(41 + T, 3, T, 4, 1, D, dtype)
    par = U.trees(42, 3, T, "chain")
    what = f"few rows {dtype} {cdtype} D={D} T={T}"
    check(bnd, q * 64, k, v, par, c, dtype, f"{what} large")
    check(bnd, q * 8, k, v, par, c, dtype, f"{what} negative", scale=-0.3)
    check(bnd, q, k, v, par, c, dtype, f"{what} 0", scale=0.0)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_masked_nodes_of_few_rows(bnd, dtype, cdtype, D, value):
    """A node that is not finite reaches its descendants only, 16 rows a key head."""
    par = torch.tensor([[-1, 0, 1, 0]], dtype=torch.int32)
    c = U.cache(43, 1, [130], 2, D, 16, dtype, cdtype)
    q, k, v = nodes(44, 1, 4, 8, 2, D, dtype)
    args, scales = U.cache_args(c)
    clean = bnd.attn_verify(q, k, v, par.cuda(), *args, **scales)
    for name in "kv":
        kk, vv = k.clone(), v.clone()
        (kk if name == "k" else vv)[0, 1] = value
        o = bnd.attn_verify(q, kk, vv, par.cuda(), *args, **scales)
        assert torch.equal(o[0, [0, 3]], clean[0, [0, 3]]), name
        if name == "v":
            assert ((o[0, [1, 2]] == value) | (torch.isnan(o[0, [1, 2]]) & (value != value))).all()
        elif value != value:
            assert torch.isnan(o[0, [1, 2]]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 3, 33])
@pytest.mark.parametrize("L", [1, 63, 64, 130, 1000])
@pytest.mark.parametrize("generic", [False, True])
def test_infinite_values_of_the_cache(bnd, dtype, D, T, L, generic):
    """One infinite element of the last position, or of the first: that element of every output is the infinity, in
    every kernel and at every length; the others do not change."""
    c = U.cache(45, 1, [L], 1, D, 16, dtype, dtype)
    q, k, v = nodes(46, 1, T, 4, 1, D, dtype)
    par = U.trees(47, 1, T).cuda()
    args, _ = U.cache_args(c)
    clean = bnd.attn_verify(q, k, v, par, *args, force_generic=generic)
    for pos, d, value in ((L - 1, 5, float("inf")), (0, D - 1, -float("inf"))):
        at = int(c["page_table"][0, pos // 16]), 0, pos % 16, d
        kept = float(c["v_cache"][at])
        c["v_cache"][at] = value
        o = bnd.attn_verify(q, k, v, par, *args, force_generic=generic)
        c["v_cache"][at] = kept
        assert (o[..., d] == value).all(), (pos, o[..., d])
        rest = [x for x in range(D) if x != d]
        assert torch.equal(o[..., rest], clean[..., rest])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_largest_tree_of_one_head_each(bnd, dtype):
    """1024 nodes, a query head a key head: the largest tables of ancestors, beside the largest tiles."""
    c = U.cache(48, 1, [70], 2, 128, 16, dtype, dtype)
    check(bnd, *nodes(48, 1, 1024, 2, 2, 128, dtype), U.trees(48, 1, 1024), c, dtype, f"1024 nodes, one head each, {dtype}")


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("H,T", [(64, 1), (300, 1), (200, 3)])
def test_many_heads_of_one_key_head(bnd, dtype, cdtype, H, T):
    """More query heads than a block of rows holds."""
    c = U.cache(49, 2, [77, 600], 1, 64, 16, dtype, cdtype)
    check(bnd, *nodes(49, 2, T, H, 1, 64, dtype), U.trees(49, 2, T), c, dtype, f"{H} heads T={T} {dtype} {cdtype}")


@pytest.mark.parametrize("T", [1, 21])
def test_shared_pages(bnd, T):
    """Items that share the pages of a prefix read the same keys."""
    c = U.cache(50, 3, [500, 9, 40], 2, 64, 16, BF, BF)
    c["page_table"][1, :31], c["cache_len"][1] = c["page_table"][0, :31], 491
    c["page_table"][2, :2], c["cache_len"][2] = c["page_table"][0, :2], 32
    check(bnd, *nodes(50, 3, T, 4, 2, 64, BF), U.trees(50, 3, T), c, BF, f"shared pages T={T}")


def test_two_graphs_of_one_pool_replayed_in_turn(bnd):
    """The workspaces of two captured calls may lie in the same memory of the graphs' pool."""
    calls, pool = [], None
    for seed, T in ((51, 1), (52, 30)):
        c = U.cache(seed, 2, [3000, 40], 2, 64, 16, BF, BF)
        q, k, v = nodes(seed, 2, T, 4, 2, 64, BF)
        par, (args, _) = U.trees(seed, 2, T).cuda(), U.cache_args(c)
        want, o = bnd.attn_verify(q, k, v, par, *args), torch.zeros_like(q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            bnd.attn_verify(q, k, v, par, *args, o=o)
        pool = g.pool()
        calls.append((g, o, want, (q, k, v, par, args)))
    for _ in range(3):
        for g, o, want, (q, k, v, par, args) in calls:
            o.zero_()
            g.replay()
            assert torch.equal(o, want)
            assert torch.equal(bnd.attn_verify(q, k, v, par, *args), want)


# ---------------------------------------------------------------- writes
def expect(c, rows, at, what):
    """The cache with rows ([m,Hk,D] k, v) written at (item, position)s, as header and torch's types define it."""
    page = c["k_cache"].shape[2]
    want = {m: None if c[m] is None else c[m].clone().cpu() for m in ("k_cache", "v_cache", "k_scale", "v_scale")}
    table = c["page_table"].cpu()
    for i, (b, p) in enumerate(at):
        pg, off = int(table[b, p // page]), p % page
        for m, r in zip("kv", rows):
            r = r[i].cpu()
            if want[m + "_scale"] is None:
                want[m + "_cache"][pg, :, off] = r
            else:
                by, sc = U.quantise(r.float())
                want[m + "_cache"].view(torch.uint8)[pg, :, off] = by.view(torch.uint8)
                want[m + "_scale"][pg, :, off] = sc
    return want


def same(c, want):
    for m, w in want.items():
        if w is None:
            continue
        a, b = c[m].cpu().contiguous().view(torch.uint8), w.contiguous().view(torch.uint8)
        assert torch.equal(a, b), m


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("Hk,D,page", [(2, 128, 16), (3, 64, 24), (1, 40, 7), (2, 256, 1), (5, 1, 16), (1, 97, 3)])
def test_commit(bnd, dtype, cdtype, Hk, D, page):
    n, T = 6, 30
    lens = [0, 5, 16, 47, 100, 33]
    c = U.cache(D, n, lens, Hk, D, page, dtype, cdtype, room=32)
    _, k, v = nodes(D + 1, n, T, Hk, Hk, D, dtype)
    k[:, 3] *= 1e-30
    v[:, 4] = 0
    par = U.trees(D, n, T)
    par[4:] = U.trees(0, 2, T, "chain")
    paths = [S.root_path(par[b].numpy(), i) for b, i in enumerate([29, 11, 0, 17, 29, 19])]
    paths[2] = []
    acc, count = torch.full((n, 30), -1, dtype=torch.int32), torch.tensor([len(p) for p in paths], dtype=torch.int32)
    for b, p in enumerate(paths):
        acc[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    at = [(b, lens[b] + i) for b, p in enumerate(paths) for i in range(len(p))]
    src = [(b, j) for b, p in enumerate(paths) for j in p]
    rows = [torch.stack([t[b, j] for b, j in src]) for t in (k, v)]
    want = expect(c, rows, at, "commit")
    st = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    args, scales = U.cache_args(c)
    bnd.attn_commit(k, v, par.cuda(), acc.cuda(), count.cuda(), *args, **scales, tree_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * n
    same(c, want)


def test_commit_bad_items_are_not_written(bnd):
    n, T, page = 10, 8, 16
    lens = [10] * n
    c = U.cache(20, n, lens, 2, 64, page, BF, E4, room=8)
    _, k, v = nodes(20, n, T, 2, 2, 64, BF)
    par = U.trees(0, n, T, "chain")
    acc = torch.arange(T, dtype=torch.int32).repeat(n, 1)
    count = torch.full((n,), 8, dtype=torch.int32)
    par[0, 0], par[1, 3] = 0, 7
    count[2], count[3] = 9, -1
    acc[4, 0], acc[5, 2], acc[6, 7] = 1, 3, 8
    cap = c["page_table"].shape[1] * page
    c["cache_len"][7], c["cache_len"][8] = cap - 7, -1
    c["page_table"][9, 1] = 10 ** 6
    want = expect(c, [k[:0, 0], v[:0, 0]], [], "none")
    st = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    args, scales = U.cache_args(c)
    bnd.attn_commit(k, v, par.cuda(), acc.cuda(), count.cuda(), *args, **scales, tree_status=st)
    torch.cuda.synchronize()
    got = st.tolist()
    assert got[0] & 1 and got[1] & 2 and got[2:7] == [4] * 5 and got[7:] == [64] * 3
    same(c, want)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("Hk,D,page", [(2, 128, 16), (8, 64, 24), (1, 40, 7), (2, 256, 1)])
@pytest.mark.parametrize("lens", [[1], [0, 37, 0, 16, 1, 0], [130, 3]])
def test_append(bnd, dtype, cdtype, Hk, D, page, lens):
    n = len(lens)
    old = [(5 * b) % 19 for b in range(n)]
    c = U.cache(D + n, n, old, Hk, D, page, dtype, cdtype, room=max(lens))
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(sum(lens) + 5, Hk, D, generator=g).to(dtype).cuda() for _ in range(2))  # 2 rows before, 3 behind
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + 2, dtype=torch.int32, device="cuda")
    at = [(b, old[b] + i) for b in range(n) for i in range(lens[b])]
    want = expect(c, [k[2:2 + sum(lens)], v[2:2 + sum(lens)]], at, "append")
    st = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    args, scales = U.cache_args(c)
    bnd.attn_append(k, v, starts, *args, **scales, seq_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * n
    same(c, want)
    bnd.attn_append(k, v, starts, *args, **scales)  # without a status
    torch.cuda.synchronize()
    same(c, want)


def test_append_bad_items_are_not_written(bnd):
    lens, n, page = [20, 5, 7, 0, 30], 5, 16
    c = U.cache(22, n, [3] * n, 2, 64, page, BF, BF, room=40)
    k, v = nodes(22, 1, sum(lens), 2, 2, 64, BF)[1:]
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    cap = c["page_table"].shape[1] * page
    c["page_table"][0, 1] = -1
    c["cache_len"][1] = cap - 4
    c["cache_len"][3] = -2
    want = expect(c, [t[0][torch.tensor(list(range(25, 32)) + list(range(32, 62)))] for t in (k, v)],
                  [(2, 3 + i) for i in range(7)] + [(4, 3 + i) for i in range(30)], "append")
    st = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    args, _ = U.cache_args(c)
    bnd.attn_append(k[0], v[0], starts, *args, seq_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [64, 64, 0, 64, 0]
    same(c, want)
    for bad in ([0, 9, 8, 8, 8, 8], [-1, 2, 3, 4, 5, 6], [0, 1, 2, 3, 4, 63]):
        bnd.attn_append(k[0], v[0], torch.tensor(bad, dtype=torch.int32, device="cuda"), *args, seq_status=st)
        torch.cuda.synchronize()
        assert st.tolist() == [32] * 5
        same(c, want)


def test_append_many_short_sequences_and_a_long_one(bnd):
    """Rows of many sequences in one work-group, some of them bad; and a sequence of 150 pages, a late one bad."""
    lens = [(3 * b) % 4 for b in range(60)] + [150, 150, 2]
    n, bad = len(lens), {3, 17, 18, 42, 61}
    c = U.cache(26, n, [5] * n, 2, 64, 1, BF, E4, room=160)
    k, v = nodes(26, 1, sum(lens), 2, 2, 64, BF)[1:]
    for b in bad - {61}:
        c["page_table"][b, 5] = -1
    c["page_table"][61, 5 + 140] = c["k_cache"].shape[0]
    starts = np.concatenate([[0], np.cumsum(lens)])
    rows = [(b, i) for b in range(n) if b not in bad for i in range(lens[b])]
    src = torch.tensor([starts[b] + i for b, i in rows])
    want = expect(c, [t[0][src] for t in (k, v)], [(b, 5 + i) for b, i in rows], "append")
    st = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    args, scales = U.cache_args(c)
    bnd.attn_append(k[0], v[0], torch.tensor(starts, dtype=torch.int32, device="cuda"), *args, **scales, seq_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [64 if b in bad and lens[b] else 0 for b in range(n)]
    same(c, want)


def test_rows_that_are_not_finite_read_back_as_nan(bnd):
    c = U.cache(24, 1, [0], 1, 64, 16, BF, E4, room=4)
    k = torch.ones(4, 1, 64, dtype=BF, device="cuda")
    k[1, 0, 5], k[2, 0, 63] = float("nan"), -float("inf")
    args, scales = U.cache_args(c)
    bnd.attn_append(k, k, torch.tensor([0, 4], dtype=torch.int32, device="cuda"), *args, **scales)
    page = int(c["page_table"][0, 0])
    back = c["k_cache"][page, 0, :4].float() * c["k_scale"][page, 0, :4, None]
    assert torch.isnan(back[1:3]).all() and ((back[[0, 3]] - 1).abs() <= 2.0 ** -23).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bytes_of_zeros_and_small_values(bnd, dtype):
    """Zeros of either sign, values far below the row's largest, and rows near the ends of the types' range: the
    bytes of the rounded quotients."""
    c = U.cache(25, 1, [0], 1, 64, 16, dtype, E4, room=12)
    g = torch.Generator().manual_seed(27)
    k = torch.randn(12, 1, 64, generator=g)
    k[0, 0, ::2] = -0.0
    k[1], k[2, 0, 1:] = -0.0, -0.0
    k[3] *= torch.logspace(-38, 0, 64)
    k[4:] *= torch.logspace(-40, 37, 8)[:, None, None]
    k = k.to(dtype).cuda()
    want = expect(c, [k, -k], [(0, i) for i in range(12)], "append")
    args, scales = U.cache_args(c)
    bnd.attn_append(k, -k, torch.tensor([0, 12], dtype=torch.int32, device="cuda"), *args, **scales)
    torch.cuda.synchronize()
    same(c, want)


def test_prompt_trees_and_tokens_together(bnd):
    """A layer's life: prompts enter the cache, trees are verified over it and their accepted paths committed,
    then single tokens follow; every output is that of the tokens' own sequence."""
    n, H, Hk, D, page, T = 3, 4, 2, 64, 16, 9
    lens = [20, 0, 35]
    for dtype, cdtype in TYPES:
        c = U.cache(30, n, [0] * n, Hk, D, page, dtype, cdtype, room=64)
        args, scales = U.cache_args(c)
        g = torch.Generator().manual_seed(31)
        k, v = (torch.randn(sum(lens), Hk, D, generator=g).to(dtype).cuda() for _ in range(2))
        starts = torch.tensor([0, 20, 20, 55], dtype=torch.int32, device="cuda")
        bnd.attn_append(k, v, starts, *args, **scales)
        c["cache_len"].add_(torch.tensor(lens, dtype=torch.int32, device="cuda"))
        for step in range(3):
            q, k, v = nodes(32 + step, n, T, H, Hk, D, dtype)
            par = U.trees(33 + step, n, T)
            check(bnd, q, k, v, par, c, dtype, f"tree {step} {dtype} {cdtype}")
            draft, target = (torch.randint(0, 2, (n, T), generator=g, dtype=torch.int32).cuda() for _ in range(2))
            acc, count, _, st = bnd.accept_greedy(par.cuda(), draft, target, 6)
            bnd.attn_commit(k, v, par.cuda(), acc, count, *args, **scales)
            c["cache_len"].add_(count)
        q, k, v = nodes(40, n, 1, H, Hk, D, dtype)
        check(bnd, q, k, v, U.trees(0, n, 1), c, dtype, f"token {dtype} {cdtype}")
