"""Host-side refusals of the serving operators (no CUDA call is reached), the
workspace sizes, and the float64 forms the GPU tests compare with, pinned to
the C oracle and to closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import serving_oracle as so
from grouped_query_attention_03_b200 import build as gbuild

OK, NULL, SHAPE, GROUPS, WINDOW, CAPACITY, OVERFLOW, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5, 6, 7, 8
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every case fails first


@pytest.fixture(scope="module")
def gqa():
    gbuild.build()
    from grouped_query_attention_03_b200 import gqa
    gqa.lib()
    return gqa


def call(fn, base, **kw):
    a = dict(base)
    for k, v in kw.items():
        assert k in a, k
        a[k] = v
    return fn(*a.values())


NORM_ROPE = dict(dtype=1, qkv=FAKE, bs=4096, rs=512, qw=None, kw=None, eps=1e-6, inv=FAKE, rot=64, inter=0,
                 pos=None, axes=1, pair=None, q=FAKE, k=FAKE, v=FAKE, B=1, Hq=4, Hkv=2, T=8, d=64, st=None)


def test_norm_rope_refusals(gqa):
    f = gqa.lib().gqa_qk_norm_rope
    bad = lambda **kw: call(f, NORM_ROPE, **kw)  # noqa: E731
    assert bad(dtype=2) == UNSUPPORTED
    assert bad(B=-1) == SHAPE and bad(T=-1) == SHAPE and bad(d=0) == SHAPE and bad(Hkv=0) == SHAPE
    assert bad(Hq=3) == GROUPS
    assert bad(rot=63) == SHAPE and bad(rot=66) == SHAPE and bad(rot=-2) == SHAPE
    assert bad(eps=-1e-6) == SHAPE and bad(eps=float("nan")) == SHAPE
    assert bad(rs=511) == SHAPE and bad(bs=-1) == SHAPE
    assert bad(axes=0) == SHAPE and bad(axes=5) == SHAPE
    pair = (ctypes.c_int32 * 32)(*([0] * 31 + [1]))
    assert bad(pair=pair) == SHAPE and bad(pair=pair, axes=2) == NULL  # axes without positions
    pair[31] = -1
    assert bad(pair=pair) == SHAPE
    assert bad(qkv=None) == NULL and bad(q=None) == NULL and bad(k=None) == NULL and bad(v=None) == NULL
    assert bad(inv=None) == NULL
    assert bad(d=258, rs=8 * 258) == UNSUPPORTED
    assert bad(T=2 ** 31 - 1, rs=2 ** 62) == OVERFLOW
    assert bad(B=2 ** 31 - 1, T=2 ** 31 - 1, Hq=2 ** 20, Hkv=2 ** 20, rs=2 ** 40) == OVERFLOW
    assert bad(B=0, qkv=None) == OK and bad(T=0, q=None) == OK


TREE = dict(dtype=1, q=FAKE, kc=FAKE, vc=FAKE, kd=FAKE, vd=FAKE, par=FAKE, o=FAKE, lens=FAKE, B=1, Hq=4,
            Hkv=2, C=64, d=64, t=8, window=-1, scale=0.125, ws=FAKE, wsb=1 << 40, status=FAKE, st=None)


def test_tree_refusals(gqa):
    f = gqa.lib().gqa_decode_tree
    bad = lambda **kw: call(f, TREE, **kw)  # noqa: E731
    assert bad(dtype=5) == UNSUPPORTED
    assert bad(B=-1) == SHAPE and bad(C=-1) == SHAPE and bad(t=-1) == SHAPE and bad(d=-3) == SHAPE
    assert bad(Hq=5) == GROUPS and bad(window=0) == WINDOW and bad(window=-2) == WINDOW
    assert bad(t=129) == UNSUPPORTED and bad(d=257) == UNSUPPORTED
    for name in ("q", "kc", "vc", "kd", "vd", "o", "lens", "status"):
        assert bad(**{name: None}) == NULL, name
    need = gqa.lib().gqa_decode_tree_workspace_bytes(1, 1, 4, 2, 64, 64, 8)
    assert need > 0
    assert bad(ws=None) == WORKSPACE and bad(wsb=need - 1) == WORKSPACE
    assert bad(ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert bad(B=2 ** 31 - 1, C=2 ** 31 - 1, Hq=2 ** 16, Hkv=2 ** 16) == OVERFLOW
    assert bad(C=2 ** 31 - 1) == UNSUPPORTED
    assert bad(B=0, q=None) == OK and bad(t=0, q=None) == OK


SCORED = dict(dtype=1, q=FAKE, kc=FAKE, vc=FAKE, o=FAKE, w=FAKE, lens=FAKE, B=1, Hq=4, Hkv=2, C=64, d=64, t=1,
              scale=0.125, ws=FAKE, wsb=1 << 40, status=FAKE, st=None)


def test_scored_refusals(gqa):
    f = gqa.lib().gqa_decode_scored
    bad = lambda **kw: call(f, SCORED, **kw)  # noqa: E731
    assert bad(t=65) == CAPACITY and bad(t=129, C=500) == UNSUPPORTED and bad(Hq=5) == GROUPS
    for name in ("q", "kc", "vc", "o", "w", "lens", "status"):
        assert bad(**{name: None}) == NULL, name
    need = gqa.lib().gqa_decode_scored_workspace_bytes(1, 1, 4, 2, 64, 64, 1)
    assert need >= 4 * 4 * 128  # 4 rows of scores, whole tiles
    assert bad(wsb=need - 1) == WORKSPACE
    assert bad(B=0, q=None) == OK and bad(t=0, q=None) == OK


def test_workspace_sizes(gqa):
    for f in (gqa.lib().gqa_decode_tree_workspace_bytes, gqa.lib().gqa_decode_scored_workspace_bytes):
        assert f(1, 1, 3, 2, 64, 64, 1) == 0 and f(1, -1, 4, 2, 64, 64, 1) == 0
        assert f(1, 1, 4, 2, 64, 64, 129) == 0 and f(1, 1, 4, 2, 64, 300, 1) == 0 and f(7, 1, 4, 2, 64, 64, 1) == 0
        small, large = f(1, 1, 4, 2, 64, 64, 1), f(1, 8, 4, 2, 64, 64, 16)
        assert 0 < small <= large


COMMIT = dict(dtype=1, kc=FAKE, vc=FAKE, kd=FAKE, vd=FAKE, path=FAKE, pl=FAKE, lens=FAKE, lo=FAKE, B=1, Hkv=2,
              C=8, d=64, t=4, P=4, status=FAKE, st=None)


def test_commit_refusals(gqa):
    f = gqa.lib().gqa_tree_commit
    bad = lambda **kw: call(f, COMMIT, **kw)  # noqa: E731
    assert bad(dtype=9) == UNSUPPORTED and bad(B=-1) == SHAPE and bad(Hkv=0) == SHAPE and bad(P=-1) == SHAPE
    for name in ("kc", "vc", "kd", "vd", "path", "pl", "lens", "lo", "status"):
        assert bad(**{name: None}) == NULL, name
    assert bad(B=2 ** 31 - 1, C=2 ** 31 - 1, Hkv=2 ** 16) == OVERFLOW
    assert bad(C=0, t=0, d=2 ** 29) == OVERFLOW  # empty, but no row is that wide
    assert bad(B=0, kc=None) == OK


EVICT = dict(dtype=1, kc=FAKE, vc=FAKE, w=FAKE, lens=FAKE, ko=FAKE, vo=FAKE, wo=FAKE, lo=FAKE, kept=FAKE, B=1,
             Hkv=2, C=8, Co=8, d=64, budget=4, recent=2, status=FAKE, st=None)


def test_evict_refusals(gqa):
    f = gqa.lib().gqa_cache_evict
    bad = lambda **kw: call(f, EVICT, **kw)  # noqa: E731
    other = ctypes.c_void_p(0x2000)
    assert bad(dtype=9) == UNSUPPORTED and bad(budget=-1) == SHAPE and bad(recent=-1) == SHAPE and bad(d=0) == SHAPE
    assert bad(recent=5) == CAPACITY and bad(budget=9) == CAPACITY
    for name in ("kc", "vc", "w", "lens", "ko", "vo", "wo", "lo", "kept", "status"):
        assert bad(**{name: None}) == NULL, name
    assert bad(ko=other) == SHAPE and bad(wo=other) == SHAPE  # partly in place
    assert bad(Co=9) == SHAPE                                  # in place, other capacity
    assert bad(ko=other, vo=other, wo=other, C=2 ** 31 - 1) == UNSUPPORTED
    assert bad(B=2 ** 31 - 1, C=2 ** 31 - 1, Hkv=2 ** 16) == OVERFLOW
    assert bad(C=0, Co=0, budget=0, recent=0, d=2 ** 29) == OVERFLOW
    assert bad(B=2 ** 20, Hkv=2 ** 12, C=0, Co=0, budget=0, recent=0) == UNSUPPORTED  # grids
    assert bad(B=0, kc=None) == OK


def test_binding_refuses_before_the_library(gqa):
    x = torch.zeros(2, 3, 8 * 64)
    with pytest.raises(ValueError, match="contiguous rows"):
        gqa.qk_norm_rope(x.transpose(1, 2), 4, 2, 64)
    with pytest.raises(ValueError, match="do not hold"):
        gqa.qk_norm_rope(x, 5, 2, 64)
    with pytest.raises(ValueError, match="positions"):
        gqa.qk_norm_rope(x, 4, 2, 64, positions=torch.zeros(3, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="each of the 32 pairs"):
        gqa.qk_norm_rope(x, 4, 2, 64, inv_freq=torch.zeros(32), axes=[0] * 31)
    with pytest.raises(ValueError, match="CUDA device memory"):
        gqa.qk_norm_rope(x, 4, 2, 64)
    q, kc, kd = torch.zeros(2, 4, 3, 64), torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 3, 64)
    lens = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="drafted"):
        gqa.decode_tree(q, kc, kc, kd[:, :, :2], kd, None, lens, workspace=ws)
    with pytest.raises(ValueError, match="parents"):
        gqa.decode_tree(q, kc, kc, kd, kd, torch.zeros(2, 2, dtype=torch.int32), lens, workspace=ws)
    with pytest.raises(ValueError, match="lengths"):
        gqa.decode_tree(q, kc, kc, kd, kd, None, lens[:1], workspace=ws)
    with pytest.raises(ValueError, match="weights"):
        gqa.decode_scored(q, kc, kc, torch.zeros(2, 2, 15), lens, workspace=ws)
    with pytest.raises(ValueError, match="path"):
        gqa.tree_commit(kc, kc, kd, kd, torch.zeros(2, 2, dtype=torch.int32), lens[:1], lens)
    with pytest.raises(ValueError, match="come together"):
        gqa.cache_evict(kc, kc, torch.zeros(2, 2, 16), lens, 4, 1, k_out=kc)
    with pytest.raises(ValueError, match="CUDA device memory"):
        gqa.decode_tree(q, kc, kc, kd, kd, None, lens, workspace=ws, status=lens[:1])


# ---------------------------------------------- the float64 forms' own pins
def test_tree_form_is_the_oracles_decode_on_a_chain():
    rng = np.random.default_rng(0)
    B, Hq, Hkv, C, d, t = 2, 4, 2, 12, 8, 5
    q = rng.standard_normal((B, Hq, t, d))
    kc, vc = rng.standard_normal((2, B, Hkv, C, d))
    kd, vd = rng.standard_normal((2, B, Hkv, t, d))
    lens = [7, 0]
    k2, v2 = kc.copy(), vc.copy()
    for b, n in enumerate(lens):
        k2[b, :, n:n + t], v2[b, :, n:n + t] = kd[b], vd[b]
    for window in (None, 1, 3, 9):
        want = oracle.decode_multi(q, k2, v2, [n + t for n in lens], window=window)
        got, mag = so.tree(q, kc, vc, kd, vd, None, lens, window=window)
        assert np.abs(got - want).max() < 1e-12 and (mag >= np.abs(got) - 1e-12).all()
    # two chains side by side: each as if the other were not there
    par = np.array([[-1, -1, 0, 1, 2]] * B)
    got, _ = so.tree(q, kc, vc, kd, vd, par, lens)
    one = [0, 2, 4]
    alone, _ = so.tree(q[:, :, one], kc, vc, kd[:, :, one], vd[:, :, one], None, lens)
    assert np.abs(got[:, :, one] - alone).max() < 1e-12


def test_scored_form_is_the_oracles_decode_and_sums_to_the_rows():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((2, 4, 3, 8))
    kc, vc = rng.standard_normal((2, 2, 2, 10, 8))
    o, _, w, _ = so.scored(q, kc, vc, [10, 4])
    assert np.abs(o - oracle.decode_multi(q, kc, vc, [10, 4])).max() < 1e-12
    assert np.allclose(w.sum(-1), 2 * 3) and (w[1, :, 4:] == 0).all()


def test_norm_rope_form():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((1, 2, 3 * 4))
    (q, k, v), _ = so.norm_rope(x, 1, 1, 4, np.ones(4), None, 0.0, np.array([np.pi / 2, 0.0]),
                                np.array([[[0, 1]]]), [0, 0], False)
    assert np.allclose((q ** 2).mean(-1), 1) and np.allclose(v[0, 0], x[0, :, 8:])
    assert np.allclose(k[0, 0, 0], x[0, 0, 4:8])  # position 0
    a = x[0, 1, 4:8]
    assert np.allclose(k[0, 0, 1], [-a[2], a[1], a[0], a[3]])  # a quarter turn of pair (0, 2)


def test_survivors_form():
    w = np.array([3, 1, 3, 0, np.nan, 2, 9, 9], dtype=np.float32)
    assert so.survivors(w, 8, 4, 2) == [0, 2, 6, 7]
    assert so.survivors(w, 8, 3, 2) == [0, 6, 7]   # the lower of the equal ones
    assert so.survivors(w, 8, 7, 2) == [0, 1, 2, 3, 5, 6, 7]
    assert so.survivors(w, 4, 4, 0) == [0, 1, 2, 3]
