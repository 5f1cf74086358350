"""One scored row over more sequences, or more KV heads, than the one-row kernel
takes (65535 of either): the other kernels have no such limit.  Bounds as in
test_gpu_cache_upkeep."""
import numpy as np
import pytest
import torch

from parity import f64
from test_gpu_tree import BF, DEV, F32, assert_mix
from grouped_query_attention_03_b200 import synthetic

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,B,Hq,Hkv,C", [(BF, 65535, 2, 1, 3), (BF, 65536, 2, 1, 3), (BF, 70001, 1, 1, 2),
                                              (BF, 1, 65600, 65600, 3), (F32, 65536, 2, 1, 3)])
def test_many_lanes(cuda_lib, dtype, B, Hq, Hkv, C):
    d, r = 64, Hq // Hkv
    q = synthetic.normal((B, Hq, d), 1, 1.0, dtype, offset=81)
    kc = synthetic.normal((B, Hkv, C, d), 1, 1.0, dtype, offset=82)
    vc = synthetic.normal((B, Hkv, C, d), 1, 1.0, dtype, offset=83)
    lens = 1 + np.arange(B) % C
    # softmax over the first lens cells, all lanes at once
    x = f64(q).reshape(B, Hkv, r, d)
    s = np.einsum("bgrd,bgcd->bgrc", x, f64(kc)) * d ** -0.5
    s[np.broadcast_to(np.arange(C) >= lens[:, None, None, None], s.shape)] = -np.inf
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    want = np.einsum("bgrc,bgcd->bgrd", p, f64(vc)).reshape(B, Hq, d)
    mag = np.einsum("bgrc,bgcd->bgrd", p, np.abs(f64(vc))).reshape(B, Hq, d)
    big = float(np.einsum("bgrd,bgcd->bgrc", np.abs(x), np.abs(f64(kc))).max()) * d ** -0.5
    weights = torch.zeros(B, Hkv, C, device=DEV)
    st = cuda_lib.new_status(DEV)
    o = cuda_lib.decode_scored(q.to(DEV), kc.to(DEV), vc.to(DEV), weights,
                               torch.tensor(lens, dtype=torch.int32, device=DEV), status=st)
    assert int(st.item()) == 0
    assert_mix(o, want, mag, dtype)
    w = p.sum(2)
    bound = w * (2 * d * 2.0 ** -23 * big + 2.0 ** -17)
    assert np.max(np.abs(f64(weights) - w) - bound) <= 0
