"""gqa_decode_scored on buffers that are not 16-byte aligned: CUDA cores, with
the scores kept (few rows) and multiplied again (many).  Bounds as in
test_gpu_cache_upkeep."""
import numpy as np
import pytest
import torch

import serving_oracle as so
from parity import f64
from test_gpu_tree import BF, DEV, assert_mix, make

pytestmark = pytest.mark.gpu


def shifted(x, by=1):
    flat = torch.empty(x.numel() + by, dtype=x.dtype, device=DEV)[by:]
    return flat.view(x.shape).copy_(x)


@pytest.mark.parametrize("B,Hq,Hkv,C,d,t,lens", [
    (1, 4, 1, 300, 64, 5, [300]),                 # 20 rows of 64: from the keys
    (1, 4, 1, 300, 64, 4, [299]),                 # 16 rows of 64: scores kept
    (2, 8, 2, 700, 128, 9, [700, 9]),             # 36 rows, a sequence of its rows alone
    (3, 6, 2, 129, 128, 100, [128, 129, 100]),    # 300 rows, tile edges
    (2, 40, 1, 260, 64, 1, [257, 1]),             # one row of 40 heads
    (2, 4, 2, 1500, 128, 60, [1500, 1027]),       # several parts
    (4, 8, 2, 70, 64, 64, [64, 71, 63, 70]),      # two refused
])
def test_unaligned_scored(cuda_lib, B, Hq, Hkv, C, d, t, lens):
    q, kc, vc, _, _ = make(B, Hq, Hkv, C, d, t, lens, C + t)
    ok = [b for b, n in enumerate(lens) if t <= n <= C]
    want, mag, w, big = so.scored(f64(q), f64(kc), f64(vc), lens)
    base = torch.rand(B, Hkv, C, generator=torch.Generator().manual_seed(2)).to(DEV)
    weights = base.clone()
    st = cuda_lib.new_status(DEV)
    qd = q[:, :, 0] if t == 1 else q
    dev = [shifted(x) for x in (qd, kc, vc)]
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = cuda_lib.decode_scored_workspace(dev[0], dev[1])
    o = cuda_lib.decode_scored(*dev, weights, lt, workspace=ws, status=st)
    assert int(st.item()) == (0 if len(ok) == B else 5)
    assert_mix(o.view(B, Hq, t, d), want, mag, BF)
    got = f64(weights) - f64(base)
    bound = w * (2 * d * 2.0 ** -23 * big + 2.0 ** -17) + 2.0 ** -24 * (f64(base) + w)
    assert np.max(np.abs(got - w) - bound) <= 0
    for b, n in enumerate(lens):
        if b not in ok:
            assert torch.equal(weights[b], base[b])
        else:
            assert torch.equal(weights[b, :, n:], base[b, :, n:])
    twice = base.clone()
    for _ in range(2):
        cuda_lib.decode_scored(*dev, twice, lt, workspace=ws, status=st)
    assert np.max(np.abs(f64(twice) - f64(base) - 2 * w) - 2 * bound - 2.0 ** -23 * w) <= 0


def test_a_key_that_only_the_last_row_reads(cuda_lib):
    """It is not finite: the last row and the weights of all that it reads are
    NaN, the other rows are as if it were not there, aligned or not."""
    B, Hq, Hkv, C, d, t = 1, 8, 2, 400, 128, 10
    lens = [390]
    q, kc, vc, _, _ = make(B, Hq, Hkv, C, d, t, lens, 3)
    want, mag, _, _ = so.scored(f64(q), f64(kc), f64(vc), lens)
    kc[:, :, 389] = float("nan")
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for put in (shifted, lambda x: x.to(DEV)):
        weights = torch.zeros(B, Hkv, C, device=DEV)
        o = cuda_lib.decode_scored(put(q), put(kc), put(vc), weights, lt)
        assert torch.isnan(o[:, :, t - 1]).all()
        assert_mix(o[:, :, :t - 1], want[:, :, :t - 1], mag[:, :, :t - 1], BF)
        assert torch.isnan(weights[:, :, :390]).all() and torch.all(weights[:, :, 390:] == 0)
