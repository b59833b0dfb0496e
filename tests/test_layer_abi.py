"""Refusals and workspace sizes of the convolution's, the rotation's and the packed rows' attention's entry points: all
before anything is enqueued (no GPU needed)."""
import ctypes

import pytest

from speculative_tree_verification_amd import binding as B
from tests.test_seq_abi import attn, seq

L = B.lib
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call here returns before a launch
OK, NULL, SHAPE, DTYPE, UNSUPPORTED = 0, 1, 2, 3, 4
MOST = (2 ** 32 - 1) // 256  # work-groups of 256 threads whose threads are counted in 32 bits


def tree(**kw):
    v = dict(batch=2, n_nodes=15, n_heads=8, head_dim=64, d_state=128, n_groups=1, in_dtype=1, flags=0, heads_per_block=0)
    v.update(kw)
    return B.Shape(*v.values())


def taps(**kw):
    v = dict(width=4, row_stride=768, silu=1)
    v.update(kw)
    return B.Conv(*v.values())


def rot(**kw):
    v = dict(rot_dim=64, interleaved=0, eps=1e-6, q_stride=512, k_stride=128, v_stride=128)
    v.update(kw)
    return B.Rope(*v.values())


def ref(s):
    return None if s is None else ctypes.byref(s)


def conv_prefill(s, c, p=None):
    p = p or [FAKE] * 8
    return L.tree_ssd_conv_prefill(ref(s), ref(c), *p, None, None)


def conv_step(s, c, p=None):
    return L.tree_ssd_conv_step(ref(s), ref(c), *(p or [FAKE] * 7), None)


def conv_verify(s, c, p=None):
    return L.tree_ssd_conv_verify(ref(s), ref(c), *(p or [FAKE] * 8), None, None)


def conv_commit(s, c, p=None, lmax=4):
    return L.tree_ssd_conv_commit(ref(s), ref(c), *(p or [FAKE] * 5), lmax, None, None)


def rope(s, r, p=None):
    return L.tree_attn_rope(ref(s), ref(r), *(p or [FAKE] * 8), None)


def append(s, r, p=None):
    return L.tree_attn_append_rope(ref(s), ref(r), *(p or [FAKE] * 14), None, None)


def chunk(s, window=0, sinks=0, p=None, ws=FAKE, size=1 << 62):
    return L.tree_attn_prefill(ref(s), window, sinks, *(p or [FAKE] * 9), None, ws, size, None)


def without(n, i):
    p = [FAKE] * n
    p[i] = None
    return p


CONV = [("width", 1, SHAPE), ("width", 0, SHAPE), ("width", 5, UNSUPPORTED), ("row_stride", 767, SHAPE), ("silu", 2, SHAPE), ("silu", -1, SHAPE)]


@pytest.mark.parametrize("field,value,code", CONV)
def test_conv_refuses_taps(field, value, code):
    c = taps(**{field: value})
    assert conv_prefill(seq(), c) == conv_step(tree(n_nodes=1), c) == conv_verify(tree(), c) == conv_commit(tree(), c) == code


@pytest.mark.parametrize("field,value,code", [("n_heads", 0, SHAPE), ("head_dim", 0, SHAPE), ("d_state", 0, SHAPE), ("n_groups", 3, SHAPE),
                                              ("n_groups", 0, SHAPE), ("in_dtype", 2, DTYPE), ("head_dim", 257, UNSUPPORTED),
                                              ("d_state", 257, UNSUPPORTED), ("n_heads", 70000, UNSUPPORTED)])
def test_conv_refuses_shapes(field, value, code):
    c = taps(row_stride=1 << 30)
    assert conv_prefill(seq(**{field: value}), c) == conv_verify(tree(**{field: value}), c) == conv_commit(tree(**{field: value}), c) == code
    assert conv_step(tree(**{"n_nodes": 1, field: value}), c) == code


def test_conv_sizes():
    assert conv_prefill(seq(n_seqs=-1), taps()) == conv_prefill(seq(n_tokens=-1), taps()) == SHAPE
    assert conv_verify(tree(batch=-1), taps()) == conv_verify(tree(n_nodes=-1), taps()) == conv_verify(tree(n_nodes=1025), taps()) == SHAPE
    assert conv_step(tree(n_nodes=2), taps()) == conv_commit(tree(n_nodes=1025), taps()) == SHAPE
    assert conv_commit(tree(), taps(), lmax=-1) == conv_commit(tree(), taps(), lmax=1025) == SHAPE
    assert conv_prefill(seq(n_tokens=2 ** 31 - 1), taps()) == UNSUPPORTED


def test_conv_null_and_empty():
    for f, n, s, optional in ((conv_prefill, 8, seq(), {2}), (conv_step, 7, tree(n_nodes=1), {2}), (conv_verify, 8, tree(), {2}), (conv_commit, 5, tree(), set())):
        assert f(None, taps()) == NULL and f(s, None) == NULL
        for i in set(range(n)) - optional:
            assert f(s, taps(), without(n, i)) == NULL, (f.__name__, i)
    assert conv_prefill(seq(n_seqs=0), taps(), [None] * 8) == OK
    for f, n in ((conv_step, 7), (conv_verify, 8), (conv_commit, 5)):
        assert f(tree(batch=0, n_nodes=1), taps(), [None] * n) == OK
        assert f(tree(n_nodes=0), taps(), [None] * n) == OK


def test_grids_past_32_bits_of_threads_are_refused():
    one = dict(n_heads=1, head_dim=1, d_state=1)
    c = taps(row_stride=3)
    assert conv_step(tree(batch=4 * MOST + 1, n_nodes=1, **one), c) == UNSUPPORTED
    assert conv_commit(tree(batch=4 * MOST + 1, **one), c) == UNSUPPORTED
    assert conv_verify(tree(batch=MOST, n_nodes=1024, **one), c) == UNSUPPORTED
    assert conv_prefill(seq(n_seqs=2 ** 30, n_tokens=2 ** 30, **one), c) == UNSUPPORTED
    assert rope(attn(batch=1, n_nodes=2 ** 31 - 1), rot()) == UNSUPPORTED
    assert rope(attn(batch=2 ** 16, n_nodes=2 ** 16), rot()) == UNSUPPORTED
    assert rope(attn(batch=1, n_nodes=4 * MOST + 1), rot()) == UNSUPPORTED
    assert append(attn(n_nodes=4 * MOST + 1), rot()) == UNSUPPORTED
    assert append(attn(batch=MOST, n_nodes=64), rot()) == UNSUPPORTED
    assert chunk(attn(n_nodes=2 ** 31 - 1)) == UNSUPPORTED
    assert chunk(attn(batch=MOST, n_nodes=MOST, n_heads=8, n_kv_heads=8)) == UNSUPPORTED
    n = ctypes.c_uint64(7)
    assert L.tree_attn_prefill_workspace(ctypes.byref(attn(n_nodes=2 ** 30, n_heads=16, n_kv_heads=2)), ctypes.byref(n)) == UNSUPPORTED
    assert n.value == 7


BAD_ATTN = [("batch", -1, SHAPE), ("n_nodes", -1, SHAPE), ("n_heads", 0, SHAPE), ("n_kv_heads", 3, SHAPE), ("n_kv_heads", 0, SHAPE),
            ("head_dim", 0, SHAPE), ("n_pages", -1, SHAPE), ("max_pages", -1, SHAPE), ("page_size", 0, SHAPE), ("page_size", 65537, SHAPE),
            ("max_pages", 2 ** 27, SHAPE), ("scale", float("nan"), SHAPE), ("scale", 3e38, SHAPE), ("in_dtype", 2, DTYPE),
            ("cache_dtype", 3, DTYPE), ("cache_dtype", 0, UNSUPPORTED), ("head_dim", 257, UNSUPPORTED)]


@pytest.mark.parametrize("field,value,code", BAD_ATTN)
def test_attention_calls_refuse_shapes(field, value, code):
    s, r = attn(**{field: value}), rot(rot_dim=0, q_stride=1 << 20, k_stride=1 << 20, v_stride=1 << 20)
    assert rope(s, r) == append(s, r) == chunk(s) == code


@pytest.mark.parametrize("field,value", [("rot_dim", -2), ("rot_dim", 7), ("rot_dim", 66), ("interleaved", 2), ("interleaved", -1), ("eps", -1e-9),
                                         ("eps", float("nan")), ("eps", float("inf")), ("q_stride", 511), ("k_stride", 127), ("q_stride", 2 ** 28)])
def test_rope_refuses(field, value):
    assert rope(attn(), rot(**{field: value})) == append(attn(), rot(**{field: value})) == SHAPE


def test_append_refuses_strides_of_v():
    assert append(attn(), rot(v_stride=127)) == append(attn(), rot(v_stride=2 ** 28)) == SHAPE


def test_rope_null_and_empty():
    assert rope(None, rot()) == rope(attn(), None) == append(None, rot()) == append(attn(), None) == NULL
    assert rope(attn(batch=0), rot(), [None] * 8) == rope(attn(n_nodes=0), rot(), [None] * 8) == OK
    both = [None, None] + [FAKE] * 6
    assert rope(attn(), rot(), both) == NULL
    for i in (2, 3, 6, 7):  # position, inv_freq, q_out, k_out
        assert rope(attn(), rot(), without(8, i)) == NULL, i
    for i in (1, 2, 3, 4, 7, 8, 9, 10, 11):  # k, v, seq_start, inv_freq, page_table, cache_len, q_out, k_cache, v_cache
        assert append(attn(), rot(), without(14, i)) == NULL, i
    for i in (12, 13):
        assert append(attn(cache_dtype=2), rot(), without(14, i)) == NULL, i
    assert append(attn(batch=0), rot(), [None] * 14) == OK


@pytest.mark.parametrize("window,sinks", [(-1, 0), (0, 1), (5, -1), (0, -1)])
def test_chunk_refuses_windows(window, sinks):
    assert chunk(attn(), window, sinks) == SHAPE


def test_chunk_null_workspace_and_empty():
    assert chunk(None) == NULL
    for i in range(9):
        scales = i in (4, 5)
        assert chunk(attn(cache_dtype=2), p=without(9, i)) == NULL, i
        if not scales:
            assert chunk(attn(), p=without(9, i)) == NULL, i
    long = attn(max_pages=4096)
    need = B.attn_prefill_workspace_bytes(2, 15, 8, 2, 64, 16, 4096)
    assert need > 0
    assert chunk(long, ws=None) == NULL
    assert chunk(long, size=need - 1) == NULL
    assert chunk(long, ws=ctypes.c_void_p(0x1004)) == SHAPE
    assert L.tree_attn_prefill_workspace(ctypes.byref(long), None) == NULL
    assert B.attn_prefill_workspace_bytes(2, 15, 8, 2, 64, 16, 4) == 0  # 64 positions are not split
    assert B.attn_prefill_workspace_bytes(0, 15, 8, 2, 64, 16, 4096) == 0
    assert chunk(attn(batch=0), p=[None] * 9, ws=None, size=0) == OK


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="GPU"):
        B.attn_rope(z(3, 2, 8), None, z(3, dtype=torch.int32), z(4))
    with pytest.raises(ValueError, match="needed"):
        B.attn_rope(None, None, z(3, dtype=torch.int32), z(4))
    with pytest.raises(ValueError, match="one distance"):
        B.attn_rope(z(2, 5, 2, 8)[:, :3], None, z(2, 3, dtype=torch.int32), z(4))
    with pytest.raises(ValueError, match="contiguous"):
        B.attn_rope(z(3, 2, 16)[..., ::2], None, z(3, dtype=torch.int32), z(4))
    with pytest.raises(ValueError, match="position"):
        B.attn_rope(z(3, 2, 8), None, z(2, dtype=torch.int32), z(4))
    with pytest.raises(TypeError, match="inv_freq"):
        B.attn_rope(z(3, 2, 8), None, z(3, dtype=torch.int32), z(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="without q"):
        B.attn_rope(None, z(3, 2, 8), z(3, dtype=torch.int32), z(4), q_out=z(3, 2, 8))
    start, c, table, n = z(2, dtype=torch.int32), z(2, 2, 16, 8), z(1, 1, dtype=torch.int32), z(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="head_dim"):
        B.attn_prefill(z(3, 2, 4), start, c, c, table, n)
    with pytest.raises(TypeError, match="float8"):
        B.attn_prefill(z(3, 2, 8, dtype=bf), start, c, c, table, n)
    with pytest.raises(ValueError, match="GPU"):
        B.attn_append_rope(None, z(3, 2, 8), z(3, 2, 8), start, z(4), c, c, table, n)
    x, b = z(3, 1, 8), z(3, 1, 4)
    with pytest.raises(ValueError, match="state"):
        B.conv_prefill(z(3, 16), z(16, 4), None, z(1, 3, 15), start, x, b, b)
    with pytest.raises(ValueError, match="weight"):
        B.conv_step(z(3, 16), z(16, 3), None, z(3, 3, 16), x, b, b)
    with pytest.raises(ValueError, match="GPU"):
        B.conv_step(z(3, 20)[:, 2:18], z(16, 4), None, z(3, 3, 16), x, b, b)


def test_rows_at_one_distance():
    torch = pytest.importorskip("torch")
    rows = lambda t, r, w: B._need_rows(t, "t", r, w, torch.float32, -1)
    t = torch.zeros(4, 6, 10, 8)
    assert rows(t, (4, 6), (10, 8)) == 80
    assert rows(t[:, :, 2:5], (4, 6), (3, 8)) == 80
    assert rows(t[:, 1:2, 2:5], (4, 1), (3, 8)) == 480  # one row in the inner size: the outer one's distance
    assert rows(t[1:2, 1:2], (1, 1), (10, 8)) == 80     # one row: its own length
    assert rows(t[0, :, 2:5], (6,), (3, 8)) == 80
    assert rows(t.view(4, 6, 80)[..., 8:24], (4, 6), (16,)) == 80


def test_append_of_no_rows():
    """Rows that are none have no pointers (as an empty tensor's)."""
    for q in (None, FAKE):
        assert append(attn(n_nodes=0), rot(), [q, None, None] + [FAKE] * 11) == OK
    assert append(attn(n_nodes=0, n_pages=0, max_pages=0), rot(), [None] * 3 + [FAKE, FAKE] + [None] * 3 + [FAKE] + [None] * 5) == OK


def test_numbers_past_32_bits_are_refused():
    """A number that its argument cannot hold is refused, and not cut to one that it can."""
    torch = pytest.importorskip("torch")
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="meta")
    i32 = torch.int32
    start, c, table, n = z(2, dtype=i32), z(2, 2, 16, 8), z(1, 1, dtype=i32), z(1, dtype=i32)
    for big in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, -2 ** 32 + 5):
        with pytest.raises(ValueError, match="window"):
            B.attn_prefill(z(3, 2, 8), start, c, c, table, n, window=big)
        with pytest.raises(ValueError, match="sinks"):
            B.attn_prefill(z(3, 2, 8), start, c, c, table, n, window=5, sinks=big)
    far = torch.empty_strided((3, 16), (2 ** 32 + 16, 1), device="meta")
    x, b, taps = z(3, 1, 8), z(3, 1, 4), z(16, 4)
    with pytest.raises(ValueError, match="row_stride"):
        B.conv_step(far, taps, None, z(3, 3, 16), x, b, b)
    with pytest.raises(ValueError, match="row_stride"):
        B.conv_prefill(far, taps, None, z(1, 3, 16), start, x, b, b)
    one = z(3, 1, dtype=i32)
    with pytest.raises(ValueError, match="row_stride"):
        B.conv_verify(far[:, None], taps, None, z(3, 3, 16), one, x[:, None], b[:, None], b[:, None])
    with pytest.raises(ValueError, match="row_stride"):
        B.conv_commit(far[:, None], z(3, 3, 16), one, one, z(3, dtype=i32), 1, 8, 1, 4)
    with pytest.raises(ValueError, match="accepted"):
        B.conv_commit(z(3, 1, 16), z(3, 3, 16), one, z(3, 2 ** 32 + 1, dtype=i32), z(3, dtype=i32), 1, 8, 1, 4)
    rows = 2 ** 32 + 3
    with pytest.raises(ValueError, match="n_nodes"):
        B.attn_rope(z(rows, 1, 8), None, z(rows, dtype=i32), z(4))
    with pytest.raises(ValueError, match="n_nodes"):
        B.attn_prefill_workspace_bytes(1, rows, 2, 2, 64, 16, 4)
