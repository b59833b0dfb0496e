"""GPU: the prompt scan (tree_ssd_prefill) and the single-token step
(tree_ssd_step) against the fp64 recurrence, elementwise.

Bounds. With |.| summed along the same paths (ya for y, ha for the state): a
state of L tokens in fp32 sees at most 3 roundings a token plus an exponential
whose argument is a sum of log decays of at most L max|dA|, taken over a tree of
6 levels in a chunk: (8 + 8 max|dA|) L roundings of 2^-24 are a bound, the
read-out adds N + 64. bf16 adds half a step (2^-8) of y and, where the masked
products are rounded before they meet x, half a step of each term: 2^-8 ya.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import sequence as S
from tests import seq_util as U
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bnd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from speculative_tree_verification_amd import binding
    return binding


def bounds(d, L, y, ya, ha, dtype):
    N = d["B"].shape[-1]
    top = float(np.abs(U.f64(d["dt"])).max() * np.abs(U.f64(d["A"])).max()) if d["dt"].numel() else 0.0
    f = ((8 + 8 * min(top, 128.0)) * L + N + 64) * 2.0 ** -24
    by = f * ya + 1e-30
    if dtype == BF:
        by = by + 2.0 ** -8 * (np.abs(y) + 1.02 * ya)
    return by, f * ha + 1e-30


def check_prefill(bnd, d, lens, dtype, start0=0, **kw):
    starts = np.concatenate([[0], np.cumsum(lens)]) + start0
    n, rows = len(lens), d["x"].shape[0]
    seq = torch.tensor(starts, dtype=torch.int32, device="cuda")
    y = torch.full_like(d["x"], 7.0)
    st = torch.full((n,), -3, dtype=torch.int32, device="cuda")
    h = d["h"].clone()
    bnd.prefill(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], h, seq, y=y, seq_status=st, **kw)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * n
    e = {k: U.f64(v) for k, v in d.items()}
    yg, hg = U.f64(y), U.f64(h)
    outside = np.ones(rows, bool)
    outside[starts[0]:starts[-1]] = False
    assert (yg[outside] == 7.0).all()
    for q, L in enumerate(lens):
        r = slice(starts[q], starts[q + 1])
        yr, hr, ya, ha = S.scan(e["x"][r], e["dt"][r], e["A"], e["B"][r], e["C"][r], e["D"], e["h"][q])
        by, bh = bounds(d, L, yr, ya, ha, dtype)
        if L == 0:
            assert torch.equal(h[q], d["h"][q])
            continue
        wy, wh = U.within(yg[r], yr, by, f"y of sequence {q}"), U.within(hg[q], hr, bh, f"state of sequence {q}")
    say(f"[prefill] {lens} {dtype}: y {wy:.3f} h {wh:.3f} of the bound")
    return y, h


SHAPES = [(BF, 4, 64, 128, 1), (BF, 8, 64, 64, 4), (F32, 4, 64, 128, 2), (BF, 3, 24, 40, 1), (F32, 2, 65, 7, 1), (F32, 1, 1, 1, 1),
          (BF, 2, 100, 200, 2), (F32, 2, 256, 256, 1)]


@pytest.mark.parametrize("dtype,H,P,N,G", SHAPES)
@pytest.mark.parametrize("lens", [[1], [63, 64, 65], [0, 5, 0, 0, 130, 1], [129]])
def test_prefill_lengths(bnd, dtype, H, P, N, G, lens):
    say(f"[prefill] {dtype} H={H} P={P} N={N} G={G} {lens}")
    d = U.ssd(len(lens) + P, sum(lens) + 4, len(lens), H, P, N, G, dtype)
    check_prefill(bnd, d, lens, dtype, start0=2)


@pytest.mark.parametrize("dtype,H,P,N,G", SHAPES[:4])
@pytest.mark.parametrize("lens", [[700], [257, 0, 513, 256, 3]])
def test_prefill_segments(bnd, dtype, H, P, N, G, lens):
    """Sequences of several segments, which start from the states that the ones before leave."""
    say(f"[prefill] segments {dtype} {lens}")
    d = U.ssd(1 + P, sum(lens), len(lens), H, P, N, G, dtype, dt_bias=-4.0)
    assert bnd.prefill_workspace_bytes(len(lens), sum(lens), H, P, N, G, dtype) > 0
    check_prefill(bnd, d, lens, dtype)


@pytest.mark.parametrize("H,N,G,lens", [(64, 64, 8, [70, 1, 64, 0, 129, 33, 65, 5, 90]), (80, 128, 1, [65, 130, 0, 63, 1, 100, 64]),
                                        (64, 128, 2, [600, 130])])
def test_prefill_two_heads_a_work_group(bnd, H, N, G, lens):
    """Enough heads and sequences that a work-group takes two heads, with and without segments."""
    d = U.ssd(51 + N, sum(lens) + 3, len(lens), H, 64, N, G, BF)
    check_prefill(bnd, d, lens, BF, start0=1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,longest", [(16, 40), (37, 70), (200, 9), (256, 5), (257, 5), (20, 600)])
def test_prefill_longest_first(bnd, dtype, n, longest):
    """16 to 256 sequences are dealt out by falling length, with equal and empty ones among them."""
    lens = [(13 * i + 5) % (longest + 1) for i in range(n)]
    lens[n // 2] = longest
    d = U.ssd(61 + n, sum(lens) + 1, n, 4, 64, 64, 2, dtype, dt_bias=-4.0)
    check_prefill(bnd, d, lens, dtype)


@pytest.mark.parametrize("H,N,G", [(64, 64, 8), (80, 128, 1), (75, 128, 5)])
def test_prefill_longest_first_in_segments(bnd, H, N, G):
    """Dealt by falling length, cut, two heads a work-group (one where a group has an odd number)."""
    lens = [(29 * i + 3) % 40 for i in range(18)]
    lens[4], lens[11] = 2900, 900
    d = U.ssd(67 + N, sum(lens) + 2, len(lens), H, 64, N, G, BF, dt_bias=-4.0)
    assert bnd.prefill_workspace_bytes(len(lens), sum(lens) + 2, H, 64, N, G, BF) > 0
    check_prefill(bnd, d, lens, BF, start0=1)


@pytest.mark.parametrize("dtype,H,P,N,G", SHAPES[4:])
def test_prefill_segments_of_other_shapes(bnd, dtype, H, P, N, G):
    d = U.ssd(69 + P, 707, 2, H, P, N, G, dtype, dt_bias=-4.0)
    assert bnd.prefill_workspace_bytes(2, 707, H, P, N, G, dtype) > 0
    check_prefill(bnd, d, [690, 17], dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("which", [["dt"], ["h"], ["x"], ["B", "C"], ["x", "dt", "B", "C", "h"]])
def test_prefill_unaligned_in_segments(bnd, dtype, which):
    """Each tensor alone at an odd element: steps by words, the combining pass and the choice of the kernel."""
    d = U.ssd(70, 900, 2, 16, 64, 128, 2, dtype, dt_bias=-4.0)
    for k in which:
        buf = torch.empty(d[k].numel() + 1, dtype=d[k].dtype, device="cuda")
        buf[1:] = d[k].reshape(-1)
        d[k] = buf[1:].view(d[k].shape)
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    lens, seq = [630, 270], torch.tensor([0, 630, 900], dtype=torch.int32, device="cuda")
    e, h0 = {k: U.f64(v) for k, v in d.items()}, U.f64(d["h"])
    y = bnd.prefill(*(d[k] for k in ("x", "dt", "A", "B", "C", "D")), d["h"], seq, seq_status=st)  # h in place, where it is
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0]
    for q, r in enumerate((slice(0, 630), slice(630, 900))):
        yr, hr, ya, ha = S.scan(e["x"][r], e["dt"][r], e["A"], e["B"][r], e["C"][r], e["D"], h0[q])
        by, bh = bounds(d, lens[q], yr, ya, ha, dtype)
        U.within(U.f64(y)[r], yr, by, f"y of sequence {q}, {which}"), U.within(U.f64(d["h"])[q], hr, bh, f"state {q}, {which}")


def test_prefill_many_sequences(bnd):
    """More sequences than threads of the search for a segment."""
    lens = [(7 * i) % 4 for i in range(700)]
    d = U.ssd(5, sum(lens), 700, 2, 64, 64, 1, BF)
    check_prefill(bnd, d, lens, BF)


def test_prefill_plain_and_matrix_kernels_agree(bnd):
    d = U.ssd(9, 300, 2, 4, 64, 128, 2, BF)
    a = check_prefill(bnd, d, [190, 110], BF)
    b = check_prefill(bnd, d, [190, 110], BF, force_generic=True)
    assert (a[1] - b[1]).abs().max() <= 1e-4 * a[1].abs().max()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["strong decay", "no decay", "growing", "zero dt"])
def test_prefill_decays(bnd, dtype, kind):
    d = U.ssd(21, 150, 1, 2, 64, 64, 1, dtype)
    if kind == "strong decay":  # exp underflows for some tokens and not for others
        d["dt"][::3] = 40.0
    elif kind == "no decay":
        d["A"].zero_()
    elif kind == "growing":
        d["A"].abs_().mul_(0.02)
    else:
        d["dt"][10:90] = 0.0
    check_prefill(bnd, d, [150], dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_later_tokens_do_not_reach_back(bnd, dtype):
    """A token that is not finite changes its own and later outputs of its sequence, and no others."""
    lens, bad = [100, 90], 100 + 37
    d = U.ssd(23, 190, 2, 2, 64, 128, 1, dtype)
    seq = torch.tensor([0, 100, 190], dtype=torch.int32, device="cuda")
    clean = bnd.prefill(*(d[k] for k in ("x", "dt", "A", "B", "C", "D")), d["h"].clone(), seq)
    for name in ("x", "B", "C", "dt"):
        for value in (float("nan"), float("inf")):
            e = {k: v.clone() for k, v in d.items()}
            e[name][bad] = value
            h = d["h"].clone()
            y = bnd.prefill(*(e[k] for k in ("x", "dt", "A", "B", "C", "D")), h, seq)
            assert torch.equal(y[:bad], clean[:bad]), (name, value)
            assert not torch.isfinite(y[bad].float()).any() or name == "dt" or value == float("inf"), (name, value)
            if name == "C":
                assert torch.equal(y[bad + 1:], clean[bad + 1:]), value
            elif value != value:
                assert torch.isnan(y[bad:].float()).all() and torch.isnan(h[1]).all(), (name, value)
            assert torch.isfinite(h[0]).all()


@pytest.mark.parametrize("seq", [[0, 5, 4], [-1, 5, 9], [0, 5, 41], [3, 2, 9]])
def test_prefill_bad_packing_writes_nothing(bnd, seq):
    d = U.ssd(31, 40, 2, 2, 64, 64, 1, BF)
    y, h, st = torch.full_like(d["x"], 7.0), d["h"].clone(), torch.zeros(2, dtype=torch.int32, device="cuda")
    bnd.prefill(*(d[k] for k in ("x", "dt", "A", "B", "C", "D")), h, torch.tensor(seq, dtype=torch.int32, device="cuda"),
                y=y, seq_status=st)
    assert st.tolist() == [32, 32] and (y == 7.0).all() and torch.equal(h, d["h"])


def test_prefill_no_tokens(bnd):
    d = U.ssd(33, 0, 3, 2, 64, 64, 1, BF)
    st, h = torch.full((3,), 9, dtype=torch.int32, device="cuda"), d["h"].clone()
    bnd.prefill(*(d[k] for k in ("x", "dt", "A", "B", "C", "D")), h, torch.zeros(4, dtype=torch.int32, device="cuda"),
                seq_status=st)
    assert st.tolist() == [0, 0, 0] and torch.equal(h, d["h"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_in_two_calls_is_one(bnd, dtype):
    """A prompt that arrives in two pieces leaves the state of the whole."""
    d = U.ssd(35, 500, 1, 4, 64, 128, 1, dtype, dt_bias=-4.0)
    one = d["h"].clone()
    names = ("x", "dt", "A", "B", "C", "D")
    bnd.prefill(*(d[k] for k in names), one, torch.tensor([0, 500], dtype=torch.int32, device="cuda"))
    two = d["h"].clone()
    for a, b in ((0, 333), (333, 500)):
        part = {k: d[k][a:b].contiguous() if k in ("x", "dt", "B", "C") else d[k] for k in names}
        bnd.prefill(*(part[k] for k in names), two, torch.tensor([0, b - a], dtype=torch.int32, device="cuda"))
    assert (one - two).abs().max() <= 2e-5 * one.abs().max()


def test_prefill_unaligned_views(bnd):
    """Contiguous tensors that begin at an odd element."""
    d = U.ssd(37, 70, 1, 2, 64, 64, 1, BF)
    for k in ("x", "B", "C", "dt", "h"):
        buf = torch.empty(d[k].numel() + 1, dtype=d[k].dtype, device="cuda")
        buf[1:] = d[k].reshape(-1)
        d[k] = buf[1:].view(d[k].shape)
    check_prefill(bnd, d, [70], BF)


def test_prefill_on_a_side_stream_and_in_a_graph(bnd):
    d = U.ssd(39, 600, 2, 4, 64, 128, 1, BF, dt_bias=-4.0)
    names = ("x", "dt", "A", "B", "C", "D")
    seq = torch.tensor([0, 450, 600], dtype=torch.int32, device="cuda")
    want_h = d["h"].clone()
    want = bnd.prefill(*(d[k] for k in names), want_h, seq)
    side, h = torch.cuda.Stream(), d["h"].clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # the current stream is busy
    y = bnd.prefill(*(d[k] for k in names), h, seq, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(h, want_h)
    h, y = d["h"].clone(), torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        bnd.prefill(*(d[k] for k in names), h, seq, y=y)
    for _ in range(3):
        h.copy_(d["h"])
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(h, want_h)


STEP = [(BF, 4, 64, 128, 1), (BF, 8, 64, 64, 4), (F32, 4, 64, 128, 2), (BF, 3, 24, 40, 1), (F32, 2, 65, 7, 1), (F32, 1, 1, 1, 1),
        (BF, 2, 100, 200, 2), (F32, 2, 256, 256, 1)]


@pytest.mark.parametrize("dtype,H,P,N,G", STEP)
@pytest.mark.parametrize("n", [1, 5, 70])
def test_step(bnd, dtype, H, P, N, G, n):
    d = U.ssd(41 + n, n, n, H, P, N, G, dtype)
    h = d["h"].clone()
    y = bnd.step(*(d[k] for k in ("x", "dt", "A", "B", "C", "D")), h)
    torch.cuda.synchronize()
    e = {k: U.f64(v) for k, v in d.items()}
    for b in range(n):
        yr, hr, ya, ha = S.scan(e["x"][b:b + 1], e["dt"][b:b + 1], e["A"], e["B"][b:b + 1], e["C"][b:b + 1], e["D"], e["h"][b])
        by, bh = bounds(d, 1, yr, ya, ha, dtype)
        U.within(U.f64(y)[b:b + 1], yr, by, "y")
        U.within(U.f64(h)[b], hr, bh, "state")


def test_step_unaligned_views(bnd):
    d = U.ssd(43, 3, 3, 2, 64, 64, 1, BF)
    want_h = d["h"].clone()
    want = bnd.step(*(d[k] for k in ("x", "dt", "A", "B", "C", "D")), want_h)
    o = {}
    for k in ("x", "B", "C", "dt", "h"):
        buf = torch.empty(d[k].numel() + 1, dtype=d[k].dtype, device="cuda")
        buf[1:] = d[k].reshape(-1)
        o[k] = buf[1:].view(d[k].shape)
    y = bnd.step(o["x"], o["dt"], d["A"], o["B"], o["C"], d["D"], o["h"])
    assert torch.equal(y, want) and torch.equal(o["h"], want_h)


def test_prompt_then_steps_is_one_sequence(bnd):
    """A prompt, then token after token: the outputs and the state of one scan."""
    d = U.ssd(45, 140, 1, 4, 64, 128, 1, F32, dt_bias=-4.0)
    names = ("x", "dt", "A", "B", "C", "D")
    one = d["h"].clone()
    y1 = bnd.prefill(*(d[k] for k in names), one, torch.tensor([0, 140], dtype=torch.int32, device="cuda"))
    two = d["h"].clone()
    y2 = torch.zeros_like(y1)
    part = {k: d[k][:130].contiguous() if k in ("x", "dt", "B", "C") else d[k] for k in names}
    y2[:130] = bnd.prefill(*(part[k] for k in names), two, torch.tensor([0, 130], dtype=torch.int32, device="cuda"))
    for t in range(130, 140):
        part = {k: d[k][t:t + 1].contiguous() if k in ("x", "dt", "B", "C") else d[k] for k in names}
        y2[t:t + 1] = bnd.step(*(part[k] for k in names), two)
    assert (one - two).abs().max() <= 2e-5 * one.abs().max()
    assert (y1 - y2).abs().max() <= 2e-5 * y1.abs().max()
