"""gqa_decode_tree and gqa_decode_scored where a CTA's range runs from one lane
group into the next with several tiles of each: more than 32 sequences, one
row tile, both tensor-core widths.

Bounds: element by element as in test_gpu_tree, and the relative L2 error of
every sequence.  A bf16 rounding moves a value from [1, 2) 2^k by up to 2^-8
2^k either way: 2^-8 / sqrt(3) 2^k in root mean square, of values of
sqrt(7 / 3) 2^k: 2^-8 / sqrt(7) = 1.5e-3 relative.  The softmax weights and
the result are each rounded once, independently, and the values' signs are
random: sqrt(2) 1.5e-3 = 2.1e-3 expected (which has no hard limit below the
element's), held to twice that."""
import numpy as np
import pytest
import torch

import serving_oracle as so
from parity import f64
from test_gpu_tree import BF, DEV, assert_mix, make, random_tree

pytestmark = pytest.mark.gpu

REL_L2 = 2 * 2.1e-3


def assert_sequences(got, want, mag, what=""):
    assert_mix(got, want, mag, BF, what)
    g = f64(got)
    for b in range(len(want)):
        size = np.linalg.norm(want[b])
        if size > 0:
            assert np.linalg.norm(g[b] - want[b]) <= REL_L2 * size, f"{what}: sequence {b}"


def lengths(B, C, least=0):
    return [C - (b * 397) % (C - least + 1) for b in range(B)]


BATCHES = [
    # B, Hq, Hkv, C, d, t, window: lane groups of 2 to 12 tiles
    (60, 6, 3, 1500, 128, 16, None),
    (60, 6, 3, 1500, 64, 16, None),
    (48, 8, 4, 1200, 64, 26, None),
    (40, 16, 4, 900, 128, 31, 600),
    (70, 3, 3, 1000, 64, 7, None),
]


@pytest.mark.parametrize("case", BATCHES, ids=lambda c: f"B{c[0]}Hq{c[1]}Hkv{c[2]}C{c[3]}d{c[4]}t{c[5]}w{c[6]}")
def test_tree_batches(cuda_lib, case):
    B, Hq, Hkv, C, d, t, window = case
    lens = lengths(B, C)
    ins = make(B, Hq, Hkv, C, d, t, lens, t + d)
    par = random_tree(B, t, t, min(3, t - 1))
    want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), lens, window=window)
    dev = [x.to(DEV) for x in ins]
    lt, pd = torch.tensor(lens, dtype=torch.int32, device=DEV), par.to(DEV)
    ws = cuda_lib.decode_tree_workspace(dev[0], dev[1])
    st = cuda_lib.new_status(DEV)
    first = cuda_lib.decode_tree(*dev, pd, lt, window=window, workspace=ws, status=st)
    assert int(st.item()) == 0
    assert_sequences(first, want, mag)
    for _ in range(20):
        o = cuda_lib.decode_tree(*dev, pd, lt, window=window, workspace=ws, status=st)
        assert torch.equal(o, first)
    assert int(st.item()) == 0


@pytest.mark.parametrize("d,Hkv,t", [(64, 4, 12), (128, 4, 12), (64, 2, 40), (128, 2, 36)])
def test_unfinite_drafts_stay_in_their_sequence(cuda_lib, d, Hkv, t):
    """inf and NaN in drafted value rows that some nodes read: between the
    segments those rows are added from global memory, while the next lane
    group's products are already under way.  (24 rows, and 160 and 144: two
    row tiles.)"""
    B, Hq, C = 45, 8, 800
    lens = lengths(B, C)
    ins = make(B, Hq, Hkv, C, d, t, lens, 31)
    par = random_tree(B, t, 77)
    clean = [f64(x) for x in ins]
    clean[4] = clean[4].copy()
    for b in range(0, B, 3):
        for node, col, bad in ((1, 5, float("inf")), (4, d - 1, float("nan"))):
            ins[4][b, :, node, col] = bad
            clean[4][b, :, node, col] = 0.0
    want, mag = so.tree(*clean, par.numpy(), lens)
    dev = [x.to(DEV) for x in ins]
    lt, pd = torch.tensor(lens, dtype=torch.int32, device=DEV), par.to(DEV)
    ws = cuda_lib.decode_tree_workspace(dev[0], dev[1])
    for _ in range(10):
        st = cuda_lib.new_status(DEV)
        o = cuda_lib.decode_tree(*dev, pd, lt, workspace=ws, status=st)
        assert int(st.item()) == 0
        got = f64(o)
        for b in range(0, B, 3):
            for i in range(t):
                line = so.line_of(par[b].numpy(), i)
                for node, col, bad in ((1, 5, np.inf), (4, d - 1, np.nan)):
                    if node in line:
                        assert np.array_equal(got[b, :, i, col], np.full(Hq, bad), equal_nan=True)
                        got[b, :, i, col] = want[b, :, i, col]
        assert_sequences(torch.from_numpy(got), want, mag)


@pytest.mark.parametrize("d,Hkv,t", [(64, 4, 12), (128, 2, 36)])
def test_unfinite_cells_behind_a_window(cuda_lib, d, Hkv, t):
    """A cell that the roots' windows still hold and no deeper node's: the roots
    are not finite, everybody else keeps the bounds."""
    B, Hq, C, window = 45, 8, 800, 300
    lens = [max(n, window) for n in lengths(B, C)]
    ins = make(B, Hq, Hkv, C, d, t, lens, 32)
    par = random_tree(B, t, 78)
    for b in range(0, B, 2):
        ins[2][b, :, lens[b] - (window - 1)] = float("nan") if b % 4 else float("inf")
    want, mag = so.tree(*[np.nan_to_num(f64(x), nan=0.0, posinf=0.0) for x in ins], par.numpy(), lens,
                        window=window)
    dev = [x.to(DEV) for x in ins]
    lt, pd = torch.tensor(lens, dtype=torch.int32, device=DEV), par.to(DEV)
    ws = cuda_lib.decode_tree_workspace(dev[0], dev[1])
    for _ in range(5):
        st = cuda_lib.new_status(DEV)
        got = f64(cuda_lib.decode_tree(*dev, pd, lt, window=window, workspace=ws, status=st))
        assert int(st.item()) == 0
        for b in range(0, B, 2):
            for i in range(t):
                if int(par[b, i]) == -1:
                    assert not np.isfinite(got[b, :, i]).any(), (b, i)
                    got[b, :, i] = want[b, :, i]
        assert_sequences(torch.from_numpy(got), want, mag)


@pytest.mark.parametrize("B,Hq,Hkv,C,d,t", [(50, 6, 3, 1100, 64, 12), (40, 16, 4, 900, 128, 32)])
def test_scored_batches(cuda_lib, B, Hq, Hkv, C, d, t):
    """(36 rows of 64: the weights from the keys; 128 rows of 128: likewise.)"""
    lens = lengths(B, C, t)
    q, kc, vc, _, _ = make(B, Hq, Hkv, C, d, t, lens, 5)
    want, mag, w, big = so.scored(f64(q), f64(kc), f64(vc), lens)
    dev = [x.to(DEV) for x in (q, kc, vc)]
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = cuda_lib.decode_scored_workspace(dev[0], dev[1])
    st = cuda_lib.new_status(DEV)
    first = None
    for _ in range(10):
        got = torch.zeros(B, Hkv, C, device=DEV)
        o = cuda_lib.decode_scored(*dev, got, lt, workspace=ws, status=st)
        if first is None:
            first = o, got
            assert_sequences(o, want, mag)
            # (the bound of test_gpu_cache_upkeep, with no weights before)
            bound = w * (2 * d * 2.0 ** -23 * big + 2.0 ** -17) + 2.0 ** -24 * w
            assert np.max(np.abs(f64(got) - w) - bound) <= 0
        assert torch.equal(o, first[0]) and torch.equal(got, first[1])
    assert int(st.item()) == 0
