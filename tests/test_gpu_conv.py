"""GPU: the short causal convolution (tree_ssd_conv_prefill, _step, _verify, _commit) against the fp64 definition.
States are inputs as they are, so they have to be equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import layer as Y
from oracle import sequence as S
from tests import layer_util as V
from tests import seq_util as U
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF, F32 = V.BF, V.F32


@pytest.fixture(scope="module")
def bnd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from speculative_tree_verification_amd import binding
    return binding


def taps(seed, C, W, n, dtype):
    g = torch.Generator().manual_seed(seed + 1000)
    rnd = lambda *s: torch.randn(*s, generator=g)
    return (0.6 * rnd(C, W)).cuda(), (0.3 * rnd(C)).cuda(), rnd(n, W - 1, C).to(dtype).cuda()


def outputs(rows, dims, dtype):
    H, P, G, N = dims
    return tuple(torch.full((*rows, *s), 7.0, dtype=dtype, device="cuda") for s in ((H, P), (G, N), (G, N)))


def joined(out):
    return torch.cat([o.flatten(-2) for o in out], -1)


def check(got, ref, W, dtype, act, what):
    y, ya, raw = ref
    return U.within(U.f64(got), y, V.conv_bound(y, ya, raw, W, dtype, act), what)


DIMS = [(4, 64, 1, 128), (3, 8, 3, 8), (2, 40, 1, 16), (5, 3, 1, 7), (1, 1, 1, 1), (80, 64, 1, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [0, 1, 2, 3, 0, 4, 70], [257]])
def test_prompts(bnd, dtype, dims, W, lens):
    H, P, G, N = dims
    C, n, act = H * P + 2 * G * N, len(lens), (W + len(lens)) % 2 == 0
    rows = sum(lens) + 3
    xbc = V.wide(C + W, rows, C, dtype=dtype, lead=16, tail=8)
    w, b, state = taps(C, C, W, n, dtype)
    b = None if W == 3 else b
    before, out = U.f64(state), outputs((rows,), dims, dtype)
    st = torch.full((n,), -3, dtype=torch.int32, device="cuda")
    what = f"conv {dtype} {dims} W={W} {lens}"
    say(f"[conv] {what}")
    bnd.conv_prefill(xbc, w, b, state, V.starts(lens, 1), *out, silu=act, seq_status=st)
    torch.cuda.synchronize()
    got, u, after, at, worst = joined(out), U.f64(xbc), U.f64(state), 1, 0.0
    bias = np.zeros(C) if b is None else U.f64(b)
    for q, L in enumerate(lens):
        *ref, new = Y.conv(u[at:at + L], before[q], U.f64(w), bias, act)
        assert np.array_equal(after[q], new), (what, q)
        if L:
            worst = max(worst, check(got[at:at + L], ref, W, dtype, act, f"{what}, sequence {q}"))
        at += L
    assert (got[0] == 7).all() and (got[at:] == 7).all(), "rows of no sequence"
    assert st.tolist() == [0] * n
    say(f"[conv] {what}: {worst:.3f} of the bound")


def test_many_sequences(bnd):
    """More sequences than lanes, strips of a long one among them; the rows' order is the sequences'."""
    lens = [(5 * q) % 7 for q in range(150)]
    lens[70] = 700
    dims, W, n = (2, 64, 1, 64), 4, 150
    C = 256
    xbc = V.wide(1, sum(lens), C, dtype=BF)
    w, b, state = taps(2, C, W, n, BF)
    before, out = U.f64(state), outputs((sum(lens),), dims, BF)
    bnd.conv_prefill(xbc, w, b, state, V.starts(lens), *out)
    got, u, after, at = joined(out), U.f64(xbc), U.f64(state), 0
    for q, L in enumerate(lens):
        *ref, new = Y.conv(u[at:at + L], before[q], U.f64(w), U.f64(b), True)
        assert np.array_equal(after[q], new), q
        if L:
            check(got[at:at + L], ref, W, BF, True, f"sequence {q}")
        at += L


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_strips(bnd, dtype):
    """Enough rows for the longer strips: every row equals that of the same inputs one token at a time."""
    dims, W, lens = (64, 64, 8, 64), 4, [1, 4099, 33, 2300]
    C = 64 * 64 + 2 * 8 * 64
    xbc = V.wide(3, sum(lens), C, dtype=dtype, tail=64)
    w, b, state = taps(4, C, W, 4, dtype)
    before, out = state.clone(), outputs((sum(lens),), dims, dtype)
    bnd.conv_prefill(xbc, w, b, state, V.starts(lens), *out)
    # steps of a few rows, from states that the definition gives
    at = 0
    for q, L in enumerate(lens):
        both = torch.cat([before[q], xbc[at:at + L]])
        rows = sorted({0, 1, 2, 3, L // 2, L - 1} & set(range(L)))
        past = torch.stack([both[r:r + W - 1] for r in rows])
        one = outputs((len(rows),), dims, dtype)
        bnd.conv_step(torch.stack([xbc[at + r] for r in rows]), w, b, past, *one)
        assert all(torch.equal(a[[at + r for r in rows]], o) for a, o in zip(out, one)), q
        assert torch.equal(state[q], both[L:])
        at += L


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("W", [2, 4])
def test_step(bnd, dtype, dims, W):
    H, P, G, N = dims
    C, n = H * P + 2 * G * N, 5
    xbc = V.wide(C, n, C, dtype=dtype, lead=8, tail=24)
    w, b, state = taps(C, C, W, n, dtype)
    before, out = U.f64(state), outputs((n,), dims, dtype)
    bnd.conv_step(xbc, w, b, state, *out)
    got, u, after = joined(out), U.f64(xbc), U.f64(state)
    for q in range(n):
        *ref, new = Y.conv(u[q:q + 1], before[q], U.f64(w), U.f64(b), True)
        assert np.array_equal(after[q], new)
        check(got[q:q + 1], ref, W, dtype, True, f"step {dims} {q}")


TREES = [(1, "random"), (2, "chain"), (7, "star"), (15, "random"), (64, "chain"), (65, "random"), (255, "random"), (1024, "random")]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,kind", TREES)
@pytest.mark.parametrize("dims,W", [((2, 64, 1, 32), 4), ((3, 5, 1, 3), 3), ((1, 8, 1, 8), 2)])
def test_tree(bnd, dtype, T, kind, dims, W):
    H, P, G, N = dims
    C, n = H * P + 2 * G * N, 3
    xbc = V.wide(T, n, T, C, dtype=dtype, lead=8, tail=8)
    w, b, state = taps(T, C, W, n, dtype)
    par = U.trees(T, n, T, kind)
    before, out = state.clone(), outputs((n, T), dims, dtype)
    st = torch.full((n,), -3, dtype=torch.int32, device="cuda")
    bnd.conv_verify(xbc, w, b, state, par.cuda(), *out, tree_status=st)
    assert torch.equal(state, before) and st.tolist() == [0] * n
    got, u, s0 = U.f64(joined(out)), U.f64(xbc), U.f64(state)
    for q in range(n):
        for i in sorted({0, 1, 2, 3, T // 2, T - 1} & set(range(T))):
            path = S.root_path(par[q].numpy(), i)
            y, ya, raw, _ = Y.conv(u[q, path], s0[q], U.f64(w), U.f64(b), True)
            U.within(got[q, i], y[-1], V.conv_bound(y[-1], ya[-1], raw[-1], W, dtype, True), f"tree {kind} T={T} {q} {i}")


def test_tree_of_many_items(bnd):
    """Enough nodes for the longer strips: each node equals the last token of its root path."""
    n, T, dims, W = 40, 63, (80, 64, 1, 128), 4
    C = 80 * 64 + 256
    xbc = V.wide(5, n, T, C, dtype=BF, tail=80)
    w, b, state = taps(6, C, W, n, BF)
    par = U.trees(7, n, T)
    out = outputs((n, T), dims, BF)
    bnd.conv_verify(xbc, w, b, state, par.cuda(), *out)
    picks = [(q, i) for q in (0, 17, n - 1) for i in (0, 1, 2, 31, 32, T - 1)]
    past, last = [], []
    for q, i in picks:
        path = S.root_path(par[q].numpy(), i)
        past.append(torch.cat([state[q], xbc[q, path]])[-W:-1])
        last.append(xbc[q, i])
    one = outputs((len(picks),), dims, BF)
    bnd.conv_step(torch.stack(last), w, b, torch.stack(past), *one)
    for a, o in zip(out, one):
        assert torch.equal(torch.stack([a[q, i] for q, i in picks]), o)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dims", [(2, 64, 1, 32), (3, 5, 1, 3)])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_commit(bnd, dtype, dims, W):
    H, P, G, N = dims
    C, T = H * P + 2 * G * N, 70
    par = U.trees(8, 6, T, "chain")
    count = [0, 1, 2, 3, 5, 70]
    xbc = V.wide(9, 6, T, C, dtype=dtype, lead=8)
    state = V.wide(10, 6, W - 1, C, dtype=dtype)
    before = state.clone()
    acc = torch.arange(T, dtype=torch.int32).repeat(6, 1).cuda()
    st = torch.full((6,), -3, dtype=torch.int32, device="cuda")
    bnd.conv_commit(xbc, state, par.cuda(), acc, torch.tensor(count, dtype=torch.int32, device="cuda"), H, P, G, N, tree_status=st)
    for q, L in enumerate(count):
        assert torch.equal(state[q], torch.cat([before[q], xbc[q, :L]])[-(W - 1):]), (q, L)
    assert st.tolist() == [0] * 6


def test_commit_of_a_branch(bnd):
    par = torch.tensor([[-1, 0, 0, 1, 2, 4, 4]], dtype=torch.int32)
    xbc, state = V.wide(11, 1, 7, 96, dtype=BF), V.wide(12, 1, 3, 96, dtype=BF)
    acc = torch.tensor([[0, 2, 4, 6]], dtype=torch.int32, device="cuda")
    bnd.conv_commit(xbc, state, par.cuda(), acc, torch.tensor([4], dtype=torch.int32, device="cuda"), 1, 32, 1, 32)
    assert torch.equal(state[0], xbc[0, [2, 4, 6]])


def test_invalid_items_are_left_whole(bnd):
    dims, W, T, n = (1, 32, 1, 32), 4, 9, 5
    xbc = V.wide(13, n, T, 96, dtype=BF)
    w, b, state = taps(14, 96, W, n, BF)
    par = U.trees(15, n, T)
    par[1, 0], par[2, 5] = 0, 5
    good, st = [0, 3, 4], torch.zeros(n, dtype=torch.int32, device="cuda")
    out = outputs((n, T), dims, BF)
    bnd.conv_verify(xbc, w, b, state, par.cuda(), *out, tree_status=st)
    assert st.tolist() == [0, 1, 2, 0, 0]
    assert all((o[[1, 2]] == 7).all() and not (o[good] == 7).all() for o in out)
    before = state.clone()
    acc = torch.zeros(n, 4, dtype=torch.int32)
    acc[3, 1] = 8 if par[3, 8] != 0 else 99
    count = torch.tensor([1, 1, 1, 2, 5], dtype=torch.int32, device="cuda")  # item 4's is above max_path_len
    bnd.conv_commit(xbc, state, par.cuda(), acc.cuda(), count, 1, 32, 1, 32, tree_status=st)
    assert st.tolist() == [0, 1, 2, 4, 4]
    assert torch.equal(state[1:], before[1:]) and torch.equal(state[0, 2], xbc[0, 0])
    # a packing that is none
    rows = xbc.view(-1, 96)
    out = outputs((n * T,), dims, BF)
    for bad in ([0, 3, 2, 5], [-1, 3, 4, 5], [0, 3, 4, 46]):
        state = before[:3].clone()
        st = torch.zeros(3, dtype=torch.int32, device="cuda")
        bnd.conv_prefill(rows, w, b, state, torch.tensor(bad, dtype=torch.int32, device="cuda"), *out, seq_status=st)
        assert st.tolist() == [32] * 3 and torch.equal(state, before[:3]) and all((o == 7).all() for o in out)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite(bnd, value):
    """They reach the W rows whose taps hold them, in their channel."""
    dims, lens = (1, 32, 1, 32), [20, 20]
    xbc = V.wide(16, 40, 96, dtype=BF).contiguous()
    w, b, state = taps(17, 96, 4, 2, BF)
    clean, out = outputs((40,), dims, BF), outputs((40,), dims, BF)
    bnd.conv_prefill(xbc, w, b, state.clone(), V.starts(lens), *clean)
    xbc[18, 40] = value
    s2 = state.clone()
    bnd.conv_prefill(xbc, w, b, s2, V.starts(lens), *out)
    a, o = joined(clean), joined(out)
    hit = torch.zeros_like(a, dtype=torch.bool)
    hit[18:20, 40] = True  # the next sequence does not see it
    assert torch.equal(a[~hit], o[~hit]) and not torch.isfinite(xbc[18, 40])
    assert int((a != o).sum()) == 2 and not torch.isfinite(s2[0, 1, 40]) and torch.isfinite(s2[1].float()).all()


def test_unaligned_and_offset_tensors(bnd):
    """Pointers that are not 16-byte aligned give the aligned call's results."""
    dims, lens, C = (2, 32, 1, 32), [9, 30], 128
    xbc = V.wide(18, 39, C, dtype=BF, lead=1, tail=1)
    assert xbc.data_ptr() % 16 and xbc.stride(0) % 8
    w, b, state = taps(19, C, 4, 2, BF)
    s2 = state.clone()
    odd, even = outputs((39,), dims, BF), outputs((39,), dims, BF)
    bnd.conv_prefill(xbc, w, b, state, V.starts(lens), *odd)
    bnd.conv_prefill(xbc.contiguous(), w, b, s2, V.starts(lens), *even)
    assert all(torch.equal(x, y) for x, y in zip(odd, even)) and torch.equal(state, s2)


def test_empty_calls(bnd):
    w, b, state = taps(20, 96, 4, 2, BF)
    before, none = state.clone(), outputs((0,), (1, 32, 1, 32), BF)
    st = torch.full((2,), -3, dtype=torch.int32, device="cuda")
    bnd.conv_prefill(torch.empty(0, 96, dtype=BF, device="cuda"), w, b, state, V.starts([0, 0]), *none, seq_status=st)
    assert torch.equal(state, before) and st.tolist() == [0, 0]
    bnd.conv_step(torch.empty(0, 96, dtype=BF, device="cuda"), w, b, state[:0], *none)
