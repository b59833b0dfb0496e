"""The fp64 oracle of the prompt scan and the paged attention against other
formulations (no GPU): a chain-shaped tree of the existing tree oracle, the
chunked form of the scan, a dense masked softmax, and torch's e4m3 type."""
import numpy as np
import pytest
import torch

from oracle import sequence as S
from tests import seq_util as U


@pytest.mark.parametrize("G", [1, 2])
def test_scan_is_a_chain_shaped_tree(oracle_mod, G):
    from speculative_tree_verification_amd import workloads as W
    inp = W.make_custom(11, batch=2, n_nodes=13, n_heads=4, head_dim=8, d_state=16, n_groups=G, dtype=W.F32)
    inp["parent"] = np.tile(np.arange(-1, 12, dtype=np.int32), (2, 1))
    ref, _ = oracle_mod.verify_full(inp, W.F32)
    d = {k: np.asarray(inp[k], np.float64) for k in ("x", "dt", "A", "B", "C", "D", "h0")}
    for b in range(2):
        y = S.scan(d["x"][b], d["dt"][b], d["A"], d["B"][b], d["C"][b], d["D"], d["h0"][b])[0]
        assert np.abs(y - np.asarray(ref)[b]).max() <= 1e-12 * np.abs(ref).max()


def test_scan_in_two_pieces_is_one():
    d = {k: U.f64(v) for k, v in U.ssd(3, 9, 1, 4, 8, 16, 2, torch.float32, device="cpu").items()}
    whole = S.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["h"][0])
    y1, h1, _, _ = S.scan(d["x"][:4], d["dt"][:4], d["A"], d["B"][:4], d["C"][:4], d["D"], d["h"][0])
    y2, h2, _, _ = S.scan(d["x"][4:], d["dt"][4:], d["A"], d["B"][4:], d["C"][4:], d["D"], h1)
    assert np.allclose(np.concatenate([y1, y2]), whole[0], rtol=1e-13, atol=1e-13)
    assert np.allclose(h2, whole[1], rtol=1e-13, atol=1e-13)


def test_attend_is_a_masked_softmax():
    g = torch.Generator().manual_seed(5)
    T, H, Hk, D, L = 7, 4, 2, 8, 5
    q, k, v = (torch.randn(T, n, D, generator=g, dtype=torch.float64) for n in (H, Hk, Hk))
    kc, vc = (torch.randn(L, Hk, D, generator=g, dtype=torch.float64) for _ in range(2))
    par = U.trees(6, 1, T)[0].numpy()
    o, oa, _ = S.attend(*(t.numpy() for t in (q, k, v)), par, kc.numpy(), vc.numpy(), 0.3)
    mask = torch.zeros(T, L + T, dtype=torch.bool)
    mask[:, :L] = True
    for i in range(T):
        mask[i, [L + j for j in S.root_path(par, i)]] = True
    K, V = torch.cat([kc, k]).repeat_interleave(2, 1), torch.cat([vc, v]).repeat_interleave(2, 1)
    s = torch.einsum("ihd,jhd->hij", q, K) * 0.3
    want = torch.einsum("hij,jhd->ihd", torch.softmax(s.masked_fill(~mask, -np.inf), -1), V)
    assert np.abs(o - want.numpy()).max() < 1e-13
    assert (oa >= np.abs(o) - 1e-13).all()


def test_quantised_rows_are_within_half_a_step():
    v = torch.randn(50, 16, generator=torch.Generator().manual_seed(7)) * torch.logspace(-30, 30, 50)[:, None]
    v[3] = 0
    by, sc = U.quantise(v)
    back = by.float().double() * sc.double()[:, None]
    # normal values: half a step is 2^-4; below 2^-6 of the scale: half of 2^-9
    assert ((back - v.double()).abs() <= torch.maximum(v.double().abs() * 2.0 ** -4, sc.double()[:, None] * 2.0 ** -10) * (1 + 1e-6)).all()
    assert (back[3] == 0).all()
