"""GPU: the heads' norms with the position rotation (tree_attn_rope), and on the way into the paged cache
(tree_attn_append_rope), against the fp64 definition.

An e4m3 row stands for byte * scale: its scale is off by two half steps of fp32 beside the row's own bound, an element
by half a step of e4m3 (2^-4 of it, or 2^-10 of the scale where it is subnormal) beside the row's bound.
"""
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


def freqs(R, base=10000.0):
    return (base ** (-torch.arange(R // 2, dtype=torch.float64) * 2 / max(R, 1))).float().cuda()


def weights(seed, D, normed):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(D, generator=g)).cuda() if normed else None for _ in range(2)]


def expect(x, pos, f, w, inter, dtype):
    """x [rows,H,D] -> values and bounds."""
    ref, bound = np.zeros(x.shape), np.zeros(x.shape)
    for r in range(len(x)):
        ref[r], mag = Y.rope(x[r], pos[r], f, w, 1e-6, inter)
        bound[r] = V.rope_bound(ref[r], mag, x.shape[-1], w is not None, dtype)
    return ref, bound


HEADS = [(8, 2, 128, 128), (4, 4, 64, 64), (6, 1, 128, 64), (2, 2, 256, 256), (3, 1, 80, 32), (3, 1, 96, 96), (2, 1, 40, 20), (2, 2, 256, 32),
         (1, 1, 2, 2), (2, 1, 33, 6), (2, 1, 64, 0), (40, 8, 16, 16)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk,D,R", HEADS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_rows(bnd, dtype, H, Hk, D, R, inter, normed):
    rows = 11
    x = V.wide(D + R, rows, (H + 2 * Hk) * D, dtype=dtype).view(rows, H + 2 * Hk, D)
    q, k = x[:, :H], x[:, H:H + Hk]
    pos = [0, 1, 2, 77, 4095, 65533, 1048575, -1, 5, 6, 131071]
    f, (wq, wk) = freqs(R), weights(D, D, normed)
    qo, ko = (torch.full(t.shape, 7.0, dtype=dtype, device="cuda") for t in (q, k))
    what = f"rope {dtype} H={H}/{Hk} D={D} R={R} {'pairs' if inter else 'halves'} norm={normed}"
    say(f"[rope] {what}")
    bnd.attn_rope(q, k, torch.tensor(pos, dtype=torch.int32, device="cuda"), f, wq, wk, interleaved=inter, q_out=qo, k_out=ko)
    keep, worst = [i for i, p in enumerate(pos) if p >= 0], 0.0
    for t, o, w, name in ((q, qo, wq, "q"), (k, ko, wk, "k")):
        ref, bound = expect(U.f64(t)[keep], np.array(pos)[keep], U.f64(f), None if w is None else U.f64(w), inter, dtype)
        worst = max(worst, U.within(U.f64(o)[keep], ref, bound, f"{what}, {name}"))
        assert (o[7] == 7).all()
    say(f"[rope] {what}: {worst:.3f} of the bound")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows_and_in_place(bnd, dtype):
    """Enough rows for several in a work-group; outputs in place of contiguous inputs; one of q and k alone."""
    n, T, H, Hk, D = 37, 63, 5, 1, 64
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(n, T, h, D, generator=g).to(dtype).cuda() for h in (H, Hk))
    pos = torch.randint(0, 5000, (n, T), generator=g, dtype=torch.int32).cuda()
    f, (wq, wk) = freqs(D), weights(2, D, True)
    qo, ko = bnd.attn_rope(q, k, pos, f, wq, wk)
    pick = [0, 1, 2, 3, 4, 1000, n * T - 1]
    for t, o, w in ((q, qo, wq), (k, ko, wk)):
        flat = lambda v: U.f64(v.reshape(-1, *v.shape[2:])[pick])
        ref, bound = expect(flat(t), pos.view(-1)[pick].cpu().numpy(), U.f64(f), U.f64(w), False, dtype)
        U.within(flat(o), ref, bound, "many rows")
    assert torch.equal(bnd.attn_rope(q, None, pos, f, wq)[0], qo) and torch.equal(bnd.attn_rope(None, k, pos, f, k_weight=wk)[1], ko)
    q2, k2 = q.clone(), k.clone()
    bnd.attn_rope(q2, k2, pos, f, wq, wk, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_heads_of_zeros_and_not_finite(bnd):
    """A head of zeros stays one; a head that is not finite touches no other."""
    g = torch.Generator().manual_seed(3)
    q = torch.randn(6, 4, 64, generator=g).to(BF).cuda()
    pos, f, (w, _) = torch.arange(6, dtype=torch.int32, device="cuda"), freqs(64), weights(4, 64, True)
    clean = bnd.attn_rope(q, None, pos, f, w)[0]
    bad = q.clone()
    bad[1, 2], bad[3, 0, 5], bad[4, 3, 60] = 0, float("nan"), float("inf")
    o = bnd.attn_rope(bad, None, pos, f, w)[0]
    assert (o[1, 2] == 0).all() and not torch.isfinite(o[3, 0].float()).any()
    assert not torch.isfinite(o[4, 3, 60].float())
    hit = torch.zeros(6, 4, dtype=torch.bool)
    hit[1, 2] = hit[3, 0] = hit[4, 3] = True
    assert torch.equal(o[~hit], clean[~hit])


def check_append(bnd, q, k, v, lens, c, f, wq, wk, inter, what, first=1, **kw):
    """Packed rows behind `first` that belong to nobody."""
    L, dtype, Hk, D = k.shape[0], k.dtype, k.shape[1], k.shape[2]
    n, page = len(lens), c["k_cache"].shape[2]
    args, scales = U.cache_args(c)
    before = {m: c[m].clone() for m in ("k_cache", "v_cache", "k_scale", "v_scale") if c[m] is not None}
    qo = None if q is None else torch.full((L, q.shape[1], D), 7.0, dtype=dtype, device="cuda")
    st = torch.full((n,), -3, dtype=torch.int32, device="cuda")
    say(f"[append] {what}")
    bnd.attn_append_rope(q, k, v, V.starts(lens, first), f, *args, **scales, q_weight=wq, k_weight=wk, interleaved=inter, q_out=qo,
                         seq_status=st, **kw)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * n
    old, table = c["cache_len"].tolist(), c["page_table"].cpu().numpy()
    touched = torch.zeros(c["k_cache"].shape[0], page, dtype=torch.bool)
    at, worst, W = first, 0.0, [None if w is None else U.f64(w) for w in (wq, wk)]
    caches = {m: U.np8(c[m]) for m in before}
    for b, new in enumerate(lens):
        rows, pos = slice(at, at + new), old[b] + np.arange(new)
        at += new
        if not new:
            continue
        pages, slot = table[b, pos // page], pos % page
        touched[pages, slot] = True
        if q is not None:
            ref, bound = expect(U.f64(q[rows]), pos, U.f64(f), W[0], inter, dtype)
            worst = max(worst, U.within(U.f64(qo[rows]), ref, bound, f"{what}, q of {b}"))
        kr, kb = expect(U.f64(k[rows]), pos, U.f64(f), W[1], inter, F32)
        for m, ref, bound in (("k", kr, kb), ("v", U.f64(v[rows]), np.zeros((new, Hk, D)))):
            got = caches[m + "_cache"][pages, :, slot].astype(np.float64)
            if c[m + "_scale"] is None:
                lim = bound + 2.0 ** -8 * (np.abs(ref) + bound) if dtype == BF and m == "k" else bound
                worst = max(worst, U.within(got, ref, lim + 1e-300, f"{what}, {m} of {b}"))
                continue
            sc = caches[m + "_scale"][pages, :, slot].astype(np.float64)
            top = np.abs(ref).max(-1)
            U.within(sc, np.maximum(top / 448, 2.0 ** -126), (bound.max(-1) + 2 * 2.0 ** -24 * top) / 448 + 1e-44, f"{what}, {m}_scale of {b}")
            lim = 2.0 ** -4 * (np.abs(ref) + bound) + bound + sc[..., None] * (2.0 ** -10 + 448 * 2.0 ** -22)
            U.within(got * sc[..., None], ref, lim, f"{what}, {m} of {b}")
    # everything else as it was
    if q is not None:
        assert (qo[:first] == 7).all() and (qo[at:] == 7).all()
    for m, t in before.items():
        a, o = (x.view(torch.uint8).cpu() if x.dtype == E4 else x.view(torch.int16 if x.dtype == BF else torch.int32).cpu() for x in (c[m], t))
        same = ~touched[:, None, :].expand(a.shape[:3])
        assert torch.equal(a[same], o[same]), f"{what}: {m} elsewhere"
    say(f"[append] {what}: {worst:.3f} of the bound")


def rows_of(seed, L, H, Hk, D, dtype):
    x = V.wide(seed, L, (H + 2 * Hk) * D, dtype=dtype).view(L, H + 2 * Hk, D)
    return x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]


TYPES = [(BF, BF), (BF, E4), (F32, F32), (F32, E4)]


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("H,Hk,D,R,inter,normed", [(8, 2, 128, 128, False, True), (4, 4, 64, 32, True, True), (3, 1, 40, 20, False, False),
                                                   (2, 2, 256, 256, True, False), (6, 2, 80, 80, False, True), (5, 1, 33, 6, True, True)])
def test_append(bnd, dtype, cdtype, H, Hk, D, R, inter, normed):
    lens, old = [5, 0, 1, 40, 17], [3, 9, 64, 0, 31]
    c = U.cache(D, 5, old, Hk, D, 16, dtype, cdtype, room=50)
    q, k, v = rows_of(D + 1, sum(lens) + 3, H, Hk, D, dtype)
    check_append(bnd, q, k, v, lens, c, freqs(R), *weights(D, D, normed), inter, f"append {dtype} {cdtype} H={H}/{Hk} D={D} R={R}")


@pytest.mark.parametrize("cdtype", [BF, E4])
@pytest.mark.parametrize("page", [1, 7, 64, 1000])
def test_append_pages(bnd, cdtype, page):
    lens, old = [70, 130, 1], [0, 63, 999]
    c = U.cache(page, 3, old, 2, 64, page, BF, cdtype, room=140)
    q, k, v = rows_of(page, sum(lens) + 2, 2, 2, 64, BF)
    check_append(bnd, None if page == 7 else q, k, v, lens, c, freqs(64), *weights(page, 64, True), False, f"append page {page} {cdtype}")


@pytest.mark.parametrize("cdtype", [BF, E4])
def test_append_many_rows(bnd, cdtype):
    """Several rows a work-group, of sequences that begin and end inside one; far positions."""
    lens = [3, 1, 0, 1300, 2, 2, 1, 0, 0, 77]
    old = [40000, 5, 7, 100, 65000, 0, 1, 2, 3, 4]
    c = U.cache(9, 10, old, 1, 64, 64, BF, cdtype, room=1400)
    q, k, v = rows_of(10, sum(lens) + 2, 2, 1, 64, BF)
    check_append(bnd, q, k, v, lens, c, freqs(64), *weights(9, 64, True), False, f"append many rows {cdtype}")


def test_append_single_tokens(bnd):
    """One row of each of 100 items."""
    old = [(37 * b) % 300 for b in range(100)]
    c = U.cache(11, 100, old, 2, 64, 16, BF, E4, room=1)
    q, k, v = rows_of(12, 101, 4, 2, 64, BF)
    check_append(bnd, q, k, v, [1] * 100, c, freqs(64), *weights(13, 64, True), False, "append of 100 tokens", first=0)


def test_append_equals_its_parts(bnd):
    """Rotated rows appended as they are give the same bf16 cache."""
    lens, old = [33, 4], [10, 0]
    c, d = (U.cache(14, 2, old, 2, 128, 16, BF, BF, room=40) for _ in range(2))
    q, k, v = rows_of(15, 37, 4, 2, 128, BF)
    f, (wq, wk) = freqs(128), weights(16, 128, True)
    args, _ = U.cache_args(c)
    qo = bnd.attn_append_rope(q, k, v, V.starts(lens), f, *args, q_weight=wq, k_weight=wk)
    pos = torch.tensor([o + i for n, o in zip(lens, old) for i in range(n)], dtype=torch.int32, device="cuda")
    q2, k2 = bnd.attn_rope(q, k, pos, f, wq, wk)
    args, _ = U.cache_args(d)
    bnd.attn_append(k2, v.contiguous(), V.starts(lens), *args)
    assert torch.equal(qo, q2)
    for m in ("k_cache", "v_cache"):
        assert torch.equal(c[m].view(torch.int16), d[m].view(torch.int16))


def test_invalid_items_are_left_whole(bnd):
    lens, old = [3, 20, 2, 4], [5, 6, 7, 8]
    c = U.cache(17, 4, old, 2, 64, 8, BF, BF, room=24)
    c["page_table"][1, 2] = 10 ** 6  # a page past the pool, of a row in the middle
    c["cache_len"][2] = -1
    q, k, v = rows_of(18, sum(lens), 2, 2, 64, BF)
    f = freqs(64)
    args, _ = U.cache_args(c)
    kc = c["k_cache"].clone()
    qo, st = torch.full(q.shape, 7.0, dtype=BF, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    bnd.attn_append_rope(q, k, v, V.starts(lens), f, *args, q_out=qo, seq_status=st)
    assert st.tolist() == [0, 64, 64, 0]
    assert (qo[3:25] == 7).all() and not (qo[:3] == 7).all() and not (qo[25:] == 7).all()
    changed = (c["k_cache"].view(torch.int16) != kc.view(torch.int16)).any(-1).any(1).sum()
    assert int(changed) == 3 + 4
    kc = c["k_cache"].clone()
    for bad in ([0, 3, 2, 5, 6], [0, 1, 2, 3, 99]):
        qo.fill_(7)
        bnd.attn_append_rope(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), f, *args, q_out=qo, seq_status=st)
        assert st.tolist() == [32] * 4 and (qo == 7).all() and torch.equal(c["k_cache"].view(torch.int16), kc.view(torch.int16))


def test_values_that_are_not_finite_in_8_bits(bnd):
    """A row with a NaN or an infinity reads back as NaN, others are as they were."""
    c = U.cache(19, 1, [0], 1, 64, 16, BF, E4, room=20)
    q, k, v = rows_of(20, 6, 1, 1, 64, BF)
    k, v = k.contiguous(), v.contiguous()
    k[2, 0, 3], v[4, 0, 63] = float("inf"), float("nan")
    args, scales = U.cache_args(c)
    bnd.attn_append_rope(None, k, v, V.starts([6]), freqs(64), *args, **scales)
    got = [x[:6, 0] for x in V.cached(c, 0, 6)]
    for g, t, row in ((got[0], k, 2), (got[1], v, 4)):
        assert np.isnan(g[row]).all() and np.isfinite(np.delete(g, row, 0)).all()


@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (F32, E4)])
@pytest.mark.parametrize("with_q", [False, True])
def test_append_of_no_rows(bnd, dtype, cdtype, with_q):
    """A call without rows writes the status of its empty sequences and nothing else."""
    c = U.cache(43, 3, [5, 0, 40], 2, 64, 16, dtype, cdtype)
    c["cache_len"][1] = 10 ** 6  # past its pages
    args, scales = U.cache_args(c)
    before = {m: c[m].clone() for m in ("k_cache", "v_cache")}
    rows = lambda h: torch.empty(0, h, 64, dtype=dtype, device="cuda")
    st = torch.full((3,), -3, dtype=torch.int32, device="cuda")
    say(f"[append] no rows, {dtype} {cdtype} q: {with_q}")
    q = bnd.attn_append_rope(rows(4) if with_q else None, rows(2), rows(2), V.starts([0, 0, 0]), freqs(64), *args, **scales, seq_status=st)
    bnd.attn_append_rope(None, rows(2), rows(2), V.starts([0, 0, 0]), freqs(64), *args, **scales)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 64, 0] and (q.shape == (0, 4, 64) if with_q else q is None)
    for m, t in before.items():
        assert torch.equal(c[m].view(torch.uint8), t.view(torch.uint8))
