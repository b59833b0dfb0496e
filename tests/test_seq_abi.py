"""Refusals and workspace sizes of the prompt scan, the step and the paged
cache's entry points: all before anything is enqueued (no GPU needed)."""
import ctypes
import glob
import os
import re

import pytest

from speculative_tree_verification_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = B.lib
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call here returns before a launch
OK, NULL, SHAPE, DTYPE, UNSUPPORTED = 0, 1, 2, 3, 4


def seq(**kw):
    v = dict(n_seqs=2, n_tokens=40, n_heads=8, head_dim=64, d_state=128, n_groups=1, in_dtype=1, flags=0)
    v.update(kw)
    return B.SeqShape(*v.values())


def attn(**kw):
    v = dict(batch=2, n_nodes=15, n_heads=8, n_kv_heads=2, head_dim=64, n_pages=9, page_size=16, max_pages=4, in_dtype=1,
             cache_dtype=1, flags=0, scale=0.125)
    v.update(kw)
    return B.AttnShape(*v.values())


def prefill(s, ptrs=None, ws=FAKE, size=1 << 62):
    p = [FAKE] * 9 if ptrs is None else ptrs
    return L.tree_ssd_prefill(ctypes.byref(s) if s is not None else None, *p, None, ws, size, None)


def verify(s, ptrs=None, ws=FAKE, size=1 << 62):
    p = [FAKE] * 11 if ptrs is None else ptrs
    return L.tree_attn_verify(ctypes.byref(s) if s is not None else None, *p, None, ws, size, None)


def commit(s, lmax=4, ptrs=None):
    p = [FAKE] * 5 if ptrs is None else ptrs[:5]
    r = [FAKE] * 6 if ptrs is None else ptrs[5:]
    return L.tree_attn_commit(ctypes.byref(s), *p, lmax, *r, None, None)


def append(s, ptrs=None):
    p = [FAKE] * 9 if ptrs is None else ptrs
    return L.tree_attn_append(ctypes.byref(s), *p, None, None)


def test_declared_and_exported():
    text = open(os.path.join(ROOT, "include", "tree_ssd.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(tree_(?:ssd|gdn|attn)_\w+)\s*\(", text))
    assert names == set(B.EXPORTS)
    for n in names:
        assert hasattr(L, n), n


@pytest.mark.parametrize("field,value,code", [
    ("n_seqs", -1, SHAPE), ("n_tokens", -1, SHAPE), ("n_heads", 0, SHAPE), ("head_dim", 0, SHAPE), ("d_state", 0, SHAPE),
    ("n_groups", 3, SHAPE), ("n_groups", 0, SHAPE), ("in_dtype", 2, DTYPE), ("head_dim", 257, UNSUPPORTED),
    ("d_state", 257, UNSUPPORTED), ("n_heads", 70000, UNSUPPORTED)])
def test_prefill_refuses_shapes(field, value, code):
    assert prefill(seq(**{field: value})) == code
    n = ctypes.c_uint64(7)
    assert L.tree_ssd_prefill_workspace(ctypes.byref(seq(**{field: value})), ctypes.byref(n)) == code
    assert n.value == 7


def test_prefill_refuses_grids_past_31_bits():
    assert prefill(seq(n_seqs=2 ** 31 - 1, n_tokens=2 ** 31 - 1, n_heads=4096, n_groups=1)) == UNSUPPORTED


def test_prefill_null_and_workspace():
    assert prefill(None) == NULL
    for i in range(9):
        p = [FAKE] * 9
        p[i] = None
        assert prefill(seq(), p) == NULL, i
    assert prefill(seq(n_seqs=0), [None] * 9, None, 0) == OK
    long = seq(n_tokens=100000)
    need = B.prefill_workspace_bytes(2, 100000, 8, 64, 128)
    assert need > 0
    assert prefill(long, ws=None) == NULL
    assert prefill(long, size=need - 1) == NULL
    assert prefill(long, ws=ctypes.c_void_p(0x1008)) == SHAPE
    assert L.tree_ssd_prefill_workspace(ctypes.byref(long), None) == NULL
    # a prompt of at most one segment needs none
    assert B.prefill_workspace_bytes(1, 256, 80, 64, 128) == 0


@pytest.mark.parametrize("field,value,code", [
    ("batch", -1, SHAPE), ("n_nodes", 2, SHAPE), ("n_nodes", -1, SHAPE), ("n_heads", 0, SHAPE), ("n_groups", 3, SHAPE),
    ("in_dtype", 2, DTYPE), ("head_dim", 257, UNSUPPORTED), ("d_state", 300, UNSUPPORTED)])
def test_step_refuses(field, value, code):
    v = dict(batch=2, n_nodes=1, n_heads=8, head_dim=64, d_state=128, n_groups=1, in_dtype=1, flags=0, heads_per_block=0)
    v[field] = value
    assert L.tree_ssd_step(ctypes.byref(B.Shape(*v.values())), *[FAKE] * 8, None) == code


def test_step_null_and_empty():
    s = B.Shape(2, 1, 8, 64, 128, 1, 1, 0, 0)
    assert L.tree_ssd_step(None, *[FAKE] * 8, None) == NULL
    for i in range(8):
        p = [FAKE] * 8
        p[i] = None
        assert L.tree_ssd_step(ctypes.byref(s), *p, None) == NULL, i
    s.batch = 0
    assert L.tree_ssd_step(ctypes.byref(s), *[None] * 8, None) == OK


BAD_ATTN = [("batch", -1, SHAPE), ("n_nodes", -1, SHAPE), ("n_heads", 0, SHAPE), ("n_kv_heads", 3, SHAPE),
            ("n_kv_heads", 0, SHAPE), ("head_dim", 0, SHAPE), ("n_pages", -1, SHAPE), ("max_pages", -1, SHAPE),
            ("page_size", 0, SHAPE), ("page_size", 65537, SHAPE), ("max_pages", 2 ** 27, SHAPE),
            ("scale", float("nan"), SHAPE), ("scale", float("inf"), SHAPE), ("in_dtype", 2, DTYPE), ("cache_dtype", 3, DTYPE),
            ("cache_dtype", 0, UNSUPPORTED), ("head_dim", 257, UNSUPPORTED)]


@pytest.mark.parametrize("field,value,code", BAD_ATTN + [("n_nodes", 1025, SHAPE)])
def test_attn_verify_and_commit_refuse_shapes(field, value, code):
    assert verify(attn(**{field: value})) == code
    assert commit(attn(**{field: value})) == code


@pytest.mark.parametrize("field,value,code", BAD_ATTN)
def test_attn_append_refuses_shapes(field, value, code):
    assert append(attn(**{field: value})) == code


def test_attn_null_and_workspace():
    assert verify(None) == NULL
    for i in range(11):
        p = [FAKE] * 11
        p[i] = None
        scales = i in (6, 7)
        assert verify(attn(cache_dtype=2), p, None, 0) == NULL, i
        if not scales:
            assert verify(attn(), p, None, 0) == NULL, i
    long = attn(max_pages=4096)
    need = B.attn_verify_workspace_bytes(2, 15, 8, 2, 64, 16, 4096)
    assert need > 0
    assert verify(long, ws=None) == NULL
    assert verify(long, size=need - 1) == NULL
    assert verify(long, ws=ctypes.c_void_p(0x1004)) == SHAPE
    assert B.attn_verify_workspace_bytes(2, 15, 8, 2, 64, 16, 4) == 0  # 64 positions are not split
    assert B.attn_verify_workspace_bytes(0, 15, 8, 2, 64, 16, 4096) == 0
    for f, n in ((commit, 11), (append, 9)):
        for i in range(n):
            p = [FAKE] * n
            p[i] = None
            assert (f(attn(cache_dtype=2), ptrs=p)) == NULL, (f.__name__, i)


def test_attn_commit_path_lengths():
    assert commit(attn(), lmax=-1) == SHAPE
    assert commit(attn(), lmax=1025) == SHAPE


def test_attn_empty_calls_are_noops():
    assert verify(attn(batch=0), [None] * 11, None, 0) == OK
    assert verify(attn(n_nodes=0), [None] * 11, None, 0) == OK
    assert commit(attn(batch=0), ptrs=[None] * 11) == OK
    assert append(attn(batch=0), ptrs=[None] * 9) == OK


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):  # a tensor that is not on a GPU
        B.step(x, torch.zeros(4, 2), torch.zeros(2), torch.zeros(4, 1, 16), torch.zeros(4, 1, 16), torch.zeros(2),
               torch.zeros(4, 2, 8, 16))
    with pytest.raises(ValueError):  # a state of another shape
        B.step(x, torch.zeros(4, 2), torch.zeros(2), torch.zeros(4, 1, 16), torch.zeros(4, 1, 16), torch.zeros(2),
               torch.zeros(4, 2, 8, 15))
    k, table, n = torch.zeros(3, 2, 8), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    start = torch.tensor([0, 3], dtype=torch.int32)
    c8 = torch.zeros(2, 2, 16, 8, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="k_scale"):
        B.attn_append(k, k, start, c8, c8, table, n)
    with pytest.raises(TypeError, match="float8"):
        B.attn_append(k, k, start, c8.view(torch.uint8), c8.view(torch.uint8), table, n)
    c = torch.zeros(2, 2, 16, 8)
    with pytest.raises(ValueError, match="contiguous"):
        B.attn_append(k, k, start, c.transpose(0, 1), c, table, n)
    with pytest.raises(ValueError, match="e4m3"):
        B.attn_append(k, k, start, c, c, table, n, k_scale=torch.zeros(2, 2, 16))


MOST = (2 ** 32 - 1) // 256  # work-groups of 256 threads whose threads are counted in 32 bits


@pytest.mark.parametrize("name,call", [
    ("step", lambda n: L.tree_ssd_step(ctypes.byref(B.Shape(n, 1, 1, 1, 1, 1, 1, 0, 0)), *[FAKE] * 8, None)),
    ("step, two work-groups a state", lambda n: L.tree_ssd_step(ctypes.byref(B.Shape(n // 2 + 1, 1, 1, 64, 128, 1, 1, 0, 0)), *[FAKE] * 8, None)),
    ("prefill", lambda n: prefill(seq(n_seqs=n, n_tokens=n, n_heads=1, head_dim=1, d_state=1))),
    ("prefill, states of 8 work-groups", lambda n: prefill(seq(n_seqs=n // 8 + 1, n_tokens=2000, n_heads=1))),
    ("prefill, states that are not aligned", lambda n: prefill(seq(n_seqs=n // 32 + 1, n_tokens=2000, n_heads=1), [FAKE] * 6 + [ctypes.c_void_p(0x1004)] + [FAKE] * 2)),
    ("verify", lambda n: verify(attn(batch=n, n_nodes=1, n_heads=1, n_kv_heads=1))),
    ("verify, join", lambda n: verify(attn(batch=n // 8 + 1, n_nodes=128, n_heads=1, n_kv_heads=1, max_pages=100))),
    ("commit", lambda n: commit(attn(batch=n), lmax=2)),
    ("commit, long paths", lambda n: commit(attn(batch=n // 4 + 1), lmax=8)),
    ("append", lambda n: append(attn(batch=2, n_nodes=16 * n)))])
def test_grids_past_32_bits_of_threads_are_refused(name, call):
    assert call(MOST + 1) == UNSUPPORTED, name


def test_sizes_below_the_largest_grid_are_not_refused():
    n = ctypes.c_uint64()
    # 100,000 prompts of 80 heads without a cut; 20,000 with one
    for s in (seq(n_seqs=100000, n_tokens=200, n_heads=80), seq(n_seqs=20000, n_tokens=100000, n_heads=80)):
        assert L.tree_ssd_prefill_workspace(ctypes.byref(s), ctypes.byref(n)) == OK
    assert commit(attn(batch=MOST // 4), lmax=8, ptrs=[None] * 11) == NULL  # past the size checks
    assert append(attn(batch=2, n_nodes=16 * (MOST - 2)), ptrs=[None] * 9) == NULL


def test_rows_near_the_largest_int_are_refused():
    """Tokens up to 2^31 - 2^16, below which no sum of a row and a step passes an int; and many sequences of one
    token, whose segments are more than an int holds."""
    one = dict(n_seqs=1, n_heads=1, head_dim=1, d_state=1)
    n = ctypes.c_uint64()
    for tokens, code in ((2 ** 31 - 2 ** 16, OK), (2 ** 31 - 2 ** 16 + 1, UNSUPPORTED), (2 ** 31 - 1, UNSUPPORTED)):
        assert L.tree_ssd_prefill_workspace(ctypes.byref(seq(n_tokens=tokens, **one)), ctypes.byref(n)) == code
    assert prefill(seq(n_tokens=2 ** 31 - 1, **one)) == UNSUPPORTED
    many = dict(one, n_seqs=2 ** 31 - 2 ** 16)
    assert prefill(seq(n_tokens=2 ** 31 - 2 ** 16, **many)) == UNSUPPORTED
    # the bound of the segments is not negative: as many states as 16 million sequences and 500 more segments have
    need = B.prefill_workspace_bytes(16_000_000, 2 ** 31 - 2 ** 16, 1, 1, 1)
    assert need >= 16_000_000 * 20
    assert append(attn(n_nodes=2 ** 31 - 1)) == UNSUPPORTED


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Launching there would hand it this device's addresses."""
    torch = pytest.importorskip("torch")

    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0

    def body(s):
        raise AssertionError("launched")

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with pytest.raises(ValueError, match="stream"):
        B._launch(0, Stream(), body)


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_a_factor_that_passes_the_floats_range_is_refused(scale):
    """The scores' factor is taken times log2(e)."""
    assert verify(attn(scale=scale)) == SHAPE
    assert commit(attn(scale=scale)) == SHAPE
