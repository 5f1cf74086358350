"""gqa_decode_scored, gqa_cache_evict and gqa_tree_commit, and a run of the
serving operators together, against the float64 definitions.

Bounds: outputs as in test_gpu_tree.  A cell's weight is a sum of softmax
weights p; a score's error is at most d roundings of 2^-23 of S = scale * sum
|q| |k| (the tensor core may truncate), a p's twice that relative, plus fp32
exponentials and the sum of at most 4096 terms: weight * (2 d 2^-23 S +
2^-17).  What is only moved is equal."""
import numpy as np
import pytest
import torch

import serving_oracle as so
from parity import f64
from test_gpu_tree import BF, DEV, F32, assert_mix, make, random_tree
from grouped_query_attention_03_b200 import synthetic

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- scored
SCORED = [
    # dtype, B, Hq, Hkv, C, d, t, lens
    (BF, 1, 4, 1, 64, 64, 1, [1]),
    (BF, 2, 8, 2, 700, 128, 1, [700, 129]),
    (BF, 3, 8, 8, 300, 128, 1, [300, 128, 5]),
    (BF, 2, 16, 1, 500, 64, 1, [401, 256]),
    (BF, 2, 8, 2, 700, 128, 9, [700, 9]),
    (BF, 1, 4, 1, 900, 128, 32, [888]),                # 128 rows
    (BF, 1, 14, 2, 600, 64, 40, [600]),                # 280 rows: two groups
    (BF, 1, 32, 8, 9000, 128, 1, [8999]),
    (BF, 2, 4, 2, 200, 96, 3, [200, 50]),
    (F32, 2, 4, 2, 128, 64, 1, [128, 33]),
    (F32, 1, 6, 2, 300, 128, 17, [290]),
    (F32, 1, 2, 1, 100, 256, 100, [100]),
    # one row: groups of 3, 10, 20 and 32 heads, more sequences than the
    # kernels keep lengths of
    (BF, 2, 6, 2, 300, 64, 1, [300, 7]),
    (BF, 2, 20, 2, 1500, 128, 1, [1500, 777]),
    (BF, 1, 40, 2, 2100, 64, 1, [2099]),
    (BF, 2, 64, 2, 700, 128, 1, [650, 700]),
    (BF, 4500, 1, 1, 20, 64, 1, [1 + b % 20 for b in range(4500)]),
    (BF, 140, 2, 1, 300, 64, 3, [3 + (b * 37) % 298 for b in range(140)]),
    (BF, 140, 32, 1, 200, 128, 4, [4 + (b * 37) % 197 for b in range(140)]),
]


@pytest.mark.parametrize("case", SCORED, ids=lambda c: (
    f"{'f32' if c[0] == F32 else 'bf16'}-B{c[1]}Hq{c[2]}Hkv{c[3]}C{c[4]}d{c[5]}t{c[6]}"))
def test_scored_cases(cuda_lib, case):
    dtype, B, Hq, Hkv, C, d, t, lens = case
    q, kc, vc, _, _ = make(B, Hq, Hkv, C, d, t, lens, C + t, dtype)
    want, mag, w, big = so.scored(f64(q), f64(kc), f64(vc), lens)
    w0 = torch.rand(B, Hkv, C, generator=torch.Generator().manual_seed(1)).to(DEV)
    weights = w0.clone()
    st = cuda_lib.new_status(DEV)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qd = (q[:, :, 0].contiguous() if t == 1 else q).to(DEV)
    o = cuda_lib.decode_scored(qd, kc.to(DEV), vc.to(DEV), weights, lt, status=st)
    assert int(st.item()) == 0 and o.shape == qd.shape
    assert_mix(o.view(B, Hq, t, d), want, mag, dtype)
    got, base = f64(weights), f64(w0)
    bound = w * (2 * d * 2.0 ** -23 * big + 2.0 ** -17) + 2.0 ** -24 * (base + w)
    assert np.max(np.abs(got - base - w) - bound) <= 0
    for b, n in enumerate(lens):  # cells behind the sequence are left alone
        assert np.array_equal(got[b, :, n:], base[b, :, n:])
        assert abs(got[b].sum() - base[b].sum() - Hq * t) <= 1e-3 * Hq * t


def test_scored_equals_decode_and_adds_up(cuda_lib):
    """The same row as gqa_decode's within the bounds, twice the weights after
    two steps, the same bits again."""
    B, Hq, Hkv, C, d = 2, 8, 2, 900, 128
    lens = [900, 333]
    q, kc, vc, _, _ = make(B, Hq, Hkv, C, d, 1, lens, 9)
    q = q[:, :, 0].contiguous()
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    dev = [x.to(DEV) for x in (q, kc, vc)]
    w = torch.zeros(B, Hkv, C, device=DEV)
    a = cuda_lib.decode_scored(*dev, w, lt)
    once = w.clone()
    b = cuda_lib.decode_scored(*dev, w, lt)
    assert torch.equal(a, b) and torch.equal(w, once + once)
    want, mag, _, _ = so.scored(f64(q)[:, :, None], f64(kc), f64(vc), lens)
    assert_mix(a[:, :, None], want, mag, BF)
    assert_mix(cuda_lib.decode(*dev, lt)[:, :, None], want, mag, BF)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_scored_refusals_on_the_device(cuda_lib, dtype, d):
    B, Hq, Hkv, C, t = 4, 4, 2, 50, 3
    q, kc, vc, _, _ = make(B, Hq, Hkv, C, d, t, [C] * B, 9, dtype)
    lens = [2, 51, 50, -7]
    want, mag, w, _ = so.scored(f64(q), f64(kc), f64(vc), lens)
    weights = torch.full((B, Hkv, C), 2.0, device=DEV)
    st = cuda_lib.new_status(DEV)
    o = cuda_lib.decode_scored(q.to(DEV), kc.to(DEV), vc.to(DEV), weights,
                               torch.tensor(lens, dtype=torch.int32, device=DEV), status=st)
    assert int(st.item()) == 5
    assert_mix(o, want, mag, dtype)
    for b in (0, 1, 3):
        assert torch.all(o[b] == 0) and torch.all(weights[b] == 2)
    assert np.abs(f64(weights[2]) - 2 - w[2]).max() < 1e-3


def test_later_rows_do_not_reach_earlier_ones(cuda_lib):
    """The newest cell is not finite: only the last row reads it."""
    for dtype, d in ((BF, 128), (BF, 64), (F32, 64)):
        B, Hq, Hkv, C, t = 1, 4, 2, 300, 4
        lens = [257]
        q, kc, vc, _, _ = make(B, Hq, Hkv, C, d, t, lens, 10, dtype)
        want, mag, _, _ = so.scored(f64(q), np.nan_to_num(f64(kc)), np.nan_to_num(f64(vc), posinf=0.0), lens)
        kc[:, :, 256] = float("nan")
        vc[:, :, 256] = float("nan")
        w = torch.zeros(B, Hkv, C, device=DEV)
        o = cuda_lib.decode_scored(q.to(DEV), kc.to(DEV), vc.to(DEV), w,
                                   torch.tensor(lens, dtype=torch.int32, device=DEV))
        assert_mix(o[:, :, :t - 1], want[:, :, :t - 1], mag[:, :, :t - 1], dtype)
        assert torch.isnan(o[:, :, t - 1].float()).all()


# -------------------------------------------------------------------- evict
def lane_weights(B, Hkv, C, seed, kind):
    g = torch.Generator()
    g.manual_seed(seed)
    u = torch.rand(B, Hkv, C, generator=g)
    if kind == "ties":
        return torch.floor(u * 4) / 4
    if kind == "equal":
        return torch.full_like(u, 0.5)
    if kind == "wild":
        w = torch.exp((u - 0.5) * 80)
        w[u < 0.1] = 0.0
        w[(u > 0.1) & (u < 0.15)] = -0.0
        w[(u > 0.15) & (u < 0.2)] *= -1
        w[(u > 0.2) & (u < 0.22)] = float("inf")
        w[(u > 0.22) & (u < 0.24)] = float("nan")
        w[(u > 0.24) & (u < 0.26)] = float("-inf")
        return w
    return u ** 6


EVICT = [
    # dtype, B, Hkv, C, d, lens, budget, recent, kind
    (BF, 2, 2, 300, 64, [300, 120], 100, 20, "tail"),
    (BF, 2, 2, 300, 64, [300, 101], 100, 100, "tail"),     # recent cells alone
    (BF, 2, 1, 300, 128, [0, 100], 100, 10, "tail"),       # nothing leaves
    (BF, 1, 1, 64, 128, [64], 0, 0, "tail"),               # everything leaves
    (BF, 1, 2, 65, 128, [65], 1, 0, "ties"),
    (BF, 2, 2, 1500, 64, [1500, 1025], 512, 0, "ties"),
    (BF, 1, 3, 1024, 128, [1023], 1000, 3, "equal"),
    (BF, 2, 3, 2100, 64, [2100, 2000], 777, 50, "wild"),
    (BF, 1, 2, 9000, 64, [8900], 4096, 512, "tail"),
    (BF, 1, 1, 40000, 64, [39999], 5000, 100, "wild"),     # 32 keys a thread, 4 CTAs
    (BF, 1, 1, 70000, 8, [69999], 30000, 0, "wild"),       # 8 CTAs
    (BF, 1, 1, 140000, 8, [139999], 5000, 100, "wild"),    # longer than the registers
    (BF, 1, 1, 140000, 8, [139999], 139998, 0, "ties"),
    (BF, 40, 4, 9000, 8, [(b * 997) % 9001 for b in range(40)], 4096, 512, "ties"),  # a CTA per lane
    (BF, 1, 1, 40000, 64, [33000], 32999, 0, "ties"),
    (BF, 1, 2, 100, 33, [100], 37, 5, "ties"),             # odd rows
    (F32, 2, 2, 200, 64, [200, 150], 64, 16, "wild"),
    (F32, 1, 1, 200, 3, [199], 64, 16, "tail"),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: (
    f"{'f32' if c[0] == F32 else 'bf16'}-B{c[1]}Hkv{c[2]}C{c[3]}d{c[4]}m{c[6]}r{c[7]}-{c[8]}"))
def test_evict_cases(cuda_lib, case, in_place):
    dtype, B, Hkv, C, d, lens, budget, recent, kind = case
    kc = synthetic.normal((B, Hkv, C, d), 3, 1.0, dtype, offset=71)
    vc = synthetic.normal((B, Hkv, C, d), 3, 1.0, dtype, offset=72)
    w = lane_weights(B, Hkv, C, C + budget, kind)
    dev = [x.to(DEV) for x in (kc, vc, w)]
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st = cuda_lib.new_status(DEV)
    if in_place:
        kept = cuda_lib.cache_evict(*dev, lt, budget, recent, status=st)
        ko, vo, wo, lo, Co = *dev, lt, C
    else:
        Co = budget + 7
        ko, vo = (torch.full((B, Hkv, Co, d), 5.0, dtype=dtype, device=DEV) for _ in range(2))
        wo = torch.full((B, Hkv, Co), 5.0, device=DEV)
        lo = torch.full((B,), -3, dtype=torch.int32, device=DEV)
        kept = cuda_lib.cache_evict(*dev, lt, budget, recent, k_out=ko, v_out=vo, weights_out=wo,
                                    lens_out=lo, status=st)
        assert lt.tolist() == lens and torch.equal(dev[0].cpu(), kc)
    assert int(st.item()) == 0
    assert lo.tolist() == [min(n, budget) for n in lens]
    for b in range(B):
        for g in range(Hkv):
            stay = so.survivors(w[b, g].numpy(), lens[b], budget, recent)
            m = len(stay)
            assert kept[b, g].tolist() == stay + [-1] * (budget - m), (b, g)
            assert torch.equal(ko[b, g, :m].cpu(), kc[b, g, stay])
            assert torch.equal(vo[b, g, :m].cpu(), vc[b, g, stay])
            got = wo[b, g].cpu()
            assert torch.equal(torch.nan_to_num(got[:m], nan=-7.5), torch.nan_to_num(w[b, g, stay], nan=-7.5))
            assert torch.all(got[m:] == 0)
            if not in_place:  # rows behind the new length are left alone
                assert torch.all(ko[b, g, m:] == 5) and torch.all(vo[b, g, m:] == 5)


def test_evict_refuses_a_bad_length_and_leaves_that_sequence(cuda_lib):
    B, Hkv, C, d = 3, 2, 80, 64
    kc = synthetic.normal((B, Hkv, C, d), 3, 1.0, BF, offset=71)
    vc = synthetic.normal((B, Hkv, C, d), 3, 1.0, BF, offset=72)
    w = lane_weights(B, Hkv, C, 1, "tail")
    lens = [81, 80, -1]
    for in_place in (True, False):
        dev = [x.to(DEV) for x in (kc, vc, w)]
        lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st = cuda_lib.new_status(DEV)
        outs = dev if in_place else [torch.full_like(x[:, :, :32], 9.0) for x in dev]
        outs = [x.contiguous() for x in outs]
        kept = cuda_lib.cache_evict(*dev, lt, 32, 8, k_out=outs[0], v_out=outs[1], weights_out=outs[2],
                                    status=st)
        assert int(st.item()) == 5
        assert lt.tolist() == [81, 32, -1]
        for b in (0, 2):
            assert torch.all(kept[b] == -1)
            for x, x0, y in zip(outs, (kc, vc, w), (9, 9, 9)):
                assert torch.equal(x[b].cpu(), x0[b]) if in_place else torch.all(x[b] == y)
        stay = so.survivors(w[1, 0].numpy(), 80, 32, 8)
        assert torch.equal(outs[0][1, 0, :32].cpu(), kc[1, 0, stay])


def test_evict_and_scored_replay_from_a_graph(cuda_lib):
    """A captured step (scored rows, then eviction in place) replays on what is
    in its buffers then, and leaves rows behind the last sequence alone."""
    B, Hq, Hkv, C, d = 2, 8, 2, 1200, 128
    lens = [1200, 700]
    q, kc, vc, _, _ = make(B, Hq, Hkv, C, d, 1, lens, 21)
    kc, vc = torch.nan_to_num(kc), torch.nan_to_num(vc, posinf=1.0)
    dev = [x.to(DEV) for x in (q[:, :, 0].contiguous(), kc, vc)]
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    w, st = torch.zeros(B, Hkv, C, device=DEV), cuda_lib.new_status(DEV)
    ws = cuda_lib.decode_scored_workspace(dev[0], dev[1])
    kept = torch.empty(B, Hkv, 800, dtype=torch.int32, device=DEV)
    o = torch.empty_like(dev[0])

    def step():
        cuda_lib.decode_scored(*dev, w, lt, out=o, workspace=ws, status=st)
        cuda_lib.cache_evict(dev[1], dev[2], w, lt, 800, 64, kept=kept, status=st)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2):
        dev[0].copy_(synthetic.normal(dev[0].shape, seed, 1.0, BF))
        dev[1].copy_(kc), dev[2].copy_(vc), w.zero_(), lt.copy_(torch.tensor(lens))
        g.replay()
        torch.cuda.synchronize()
        want, mag, wv, _ = so.scored(f64(dev[0])[:, :, None], f64(kc), f64(vc), lens)
        assert_mix(o[:, :, None], want, mag, BF)
        assert int(st.item()) == 0 and lt.tolist() == [800, 700]
        for h in range(Hkv):
            rows = kept[0, h].long().cpu()
            assert torch.equal(dev[1][0, h, :800].cpu(), kc[0, h, rows])
            # the survivors are the heaviest up to the weights' rounding
            lost = np.setdiff1d(np.arange(1200 - 64), rows.numpy())
            stay = rows.numpy()[rows.numpy() < 1200 - 64]
            assert wv[0, h, stay].min() >= wv[0, h, lost].max() * (1 - 1e-4)
            assert kept[1, h, :700].tolist() == list(range(700)) and torch.all(kept[1, h, 700:] == -1)
            assert torch.equal(dev[1][1, h].cpu(), kc[1, h]) and torch.equal(dev[2][0, h, 800:].cpu(), vc[0, h, 800:])


# ------------------------------------------------------------------- commit
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("dtype,B,Hkv,C,d,t,P", [
    (BF, 3, 2, 40, 128, 20, 6), (BF, 1, 1, 9, 64, 1, 1), (BF, 2, 2, 40, 33, 12, 12),
    (F32, 3, 2, 40, 64, 20, 9), (BF, 70, 8, 30, 128, 30, 20),
    (BF, 5, 4, 30, 128, 9, 4), (BF, 7, 6, 30, 128, 9, 4)])  # clusters of 3 and of 6 CTAs
def test_commit(cuda_lib, dtype, B, Hkv, C, d, t, P, apart):
    g = torch.Generator()
    g.manual_seed(B + P)
    kc = synthetic.normal((B, Hkv, C, d), 3, 1.0, dtype, offset=71)
    vc = synthetic.normal((B, Hkv, C, d), 3, 1.0, dtype, offset=72)
    kd = synthetic.normal((B, Hkv, t, d), 3, 1.0, dtype, offset=73)
    vd = synthetic.normal((B, Hkv, t, d), 3, 1.0, dtype, offset=74)
    acc = [(5 * b + P) % (P + 1) for b in range(B)]
    lens = [C - a if b % 2 == 0 else min(3, C - a) for b, a in enumerate(acc)]  # full, or room left
    path = torch.full((B, P), 10 ** 6, dtype=torch.int32)  # entries behind the path are not read
    for b in range(B):
        path[b, :acc[b]] = torch.randperm(t, generator=g)[:acc[b]].sort().values.to(torch.int32)
    kw, vw = kc.clone(), vc.clone()
    for b in range(B):
        idx = path[b, :acc[b]].long()
        kw[b, :, lens[b]:lens[b] + acc[b]] = kd[b][:, idx]
        vw[b, :, lens[b]:lens[b] + acc[b]] = vd[b][:, idx]
    k, v = kc.to(DEV), vc.to(DEV)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    lo = torch.full_like(lt, -1) if apart else lt
    st = cuda_lib.tree_commit(k, v, kd.to(DEV), vd.to(DEV), path.to(DEV),
                              torch.tensor(acc, dtype=torch.int32, device=DEV), lt,
                              lens_out=lo if apart else None)
    assert int(st.item()) == 0
    assert torch.equal(k.cpu(), kw) and torch.equal(v.cpu(), vw)
    assert lo.tolist() == [n + a for n, a in zip(lens, acc)]
    if apart:
        assert lt.tolist() == lens


@pytest.mark.parametrize("apart", [False, True])
def test_commit_is_all_or_nothing(cuda_lib, apart):
    B, Hkv, C, d, t, P = 3, 2, 16, 64, 8, 4
    kc = synthetic.normal((B, Hkv, C, d), 3, 1.0, BF, offset=71)
    kd = synthetic.normal((B, Hkv, t, d), 3, 1.0, BF, offset=73).to(DEV)
    good = dict(lens=[0, 5, 12], acc=[4, 0, 4], path=[[0, 1, 2, 3], [0, 0, 0, 0], [1, 4, 6, 7]])
    for want, change in ((0, {}), (5, dict(lens=[0, 5, 13])), (5, dict(lens=[-1, 5, 12])),
                         (5, dict(lens=[17, 5, 12])), (13, dict(acc=[5, 0, 4])), (13, dict(acc=[-1, 0, 4])),
                         (13, dict(path=[[0, 1, 1, 3], [0] * 4, [1, 4, 6, 7]])),
                         (13, dict(path=[[0, 1, 2, 3], [0] * 4, [1, 4, 6, 8]])),
                         (13, dict(path=[[0, 1, 2, 3], [0] * 4, [-1, 4, 6, 7]]))):
        a = dict(good, **change)
        k, v = kc.to(DEV), kc.to(DEV) + 1
        v0 = v.clone()
        lt = torch.tensor(a["lens"], dtype=torch.int32, device=DEV)
        lo = torch.full_like(lt, -9) if apart else lt
        st = cuda_lib.tree_commit(k, v, kd, kd, torch.tensor(a["path"], dtype=torch.int32, device=DEV),
                                  torch.tensor(a["acc"], dtype=torch.int32, device=DEV), lt,
                                  lens_out=lo if apart else None)
        assert int(st.item()) == want, change
        if want:
            assert torch.equal(k.cpu(), kc) and torch.equal(v, v0)
            assert lo.tolist() == a["lens"]
        else:
            assert lo.tolist() == [4, 5, 16]


def test_large_commit_in_place(cuda_lib):
    """More columns than one cluster takes: two launches."""
    B, Hkv, C, d, t, P = 80, 16, 24, 128, 8, 3
    kc = torch.zeros(B, Hkv, C, d, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    kd = synthetic.normal((B, Hkv, t, d), 3, 1.0, BF, offset=73).to(DEV)
    path = torch.tensor([[1, 3, 6]] * B, dtype=torch.int32, device=DEV)
    acc = torch.full((B,), 3, dtype=torch.int32, device=DEV)
    lt = torch.arange(B, dtype=torch.int32, device=DEV) % 20
    want = lt + 3
    lens = lt.tolist()
    cuda_lib.tree_commit(kc, vc, kd, kd, path, acc, lt)
    assert torch.equal(lt, want)
    for b, n in enumerate(lens):
        assert torch.equal(kc[b, :, n:n + 3], kd[b][:, [1, 3, 6]])
        assert torch.all(kc[b, :, :n] == 0) and torch.all(kc[b, :, n + 3:] == 0)


# ----------------------------------------------------------- used together
def test_a_serving_run(cuda_lib):
    """Prompt -> scored rows -> eviction -> drafted tree -> commit -> decode,
    each step's state feeding the next, in one captured graph and eagerly,
    against the same run in float64."""
    B, Hq, Hkv, d, T, t = 2, 8, 2, 64, 90, 5
    C, budget, recent = 128, 48, 8
    H = Hq + 2 * Hkv
    fr = (1e4 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().to(DEV)
    qw = (1 + synthetic.normal((d,), 1, 0.2, F32)).to(BF).to(DEV)
    x = synthetic.normal((B, T, H * d), 1, 1.0, BF).to(DEV)
    xt = synthetic.normal((B, t, H * d), 2, 1.0, BF).to(DEV)
    x1 = synthetic.normal((B, 1, H * d), 3, 1.0, BF).to(DEV)
    par = torch.tensor([[-1, 0, 0, 1, 1], [-1, 0, 1, 2, -2]], dtype=torch.int32, device=DEV)
    depth = torch.tensor([[0, 1, 1, 2, 2], [0, 1, 2, 3, 0]], dtype=torch.int32, device=DEV)
    path = torch.tensor([[0, 1, 4], [0, 1, 2]], dtype=torch.int32, device=DEV)
    acc = torch.tensor([3, 2], dtype=torch.int32, device=DEV)
    kc = torch.zeros(B, Hkv, C, d, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    w = torch.zeros(B, Hkv, C, device=DEV)
    lt = torch.zeros(B, dtype=torch.int32, device=DEV)
    st = cuda_lib.new_status(DEV)
    rot = dict(q_weight=qw, k_weight=qw, inv_freq=fr)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    ws1 = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    tree_pos, step_pos = (T + depth).contiguous(), (T + acc)[:, None].contiguous()
    kept = torch.empty(B, Hkv, budget, dtype=torch.int32, device=DEV)

    def go():
        kc.zero_(), vc.zero_(), w.zero_(), lt.zero_()
        q, k, v = cuda_lib.qk_norm_rope(x, Hq, Hkv, d, **rot)
        cuda_lib.cache_append(kc, vc, k, v, lt, status=st)
        o_s = cuda_lib.decode_scored(q[:, :, T - 16:].contiguous(), kc, vc, w, lt, workspace=ws, status=st)
        w_s = w.clone()
        cuda_lib.cache_evict(kc, vc, w, lt, budget, recent, kept=kept, status=st)
        qt, kt, vt = cuda_lib.qk_norm_rope(xt, Hq, Hkv, d, positions=tree_pos, **rot)
        o_t = cuda_lib.decode_tree(qt, kc, vc, kt, vt, par, lt, workspace=ws, status=st)
        cuda_lib.tree_commit(kc, vc, kt, vt, path, acc, lt, status=st)
        q1, k1, v1 = cuda_lib.qk_norm_rope(x1, Hq, Hkv, d, positions=step_pos, **rot)
        o_1 = cuda_lib.decode_append(q1[:, :, 0], kc, vc, k1, v1, lt, workspace=ws1, status=st)
        return q, k, v, o_s, w_s, qt, kt, vt, o_t, q1, k1, v1, o_1

    eager = [y.clone() for y in go()]
    lens_after = lt.tolist()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = go()
    g.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for a, b in zip(eager, captured):
        assert torch.equal(a, b)
    q, k, v, o_s, w_s, qt, kt, vt, o_t, q1, k1, v1, o_1 = [f64(y) for y in eager]
    # attention of the last 16 prompt rows, and what each cell received
    want, mag, wv, big = so.scored(q[:, :, T - 16:], k, v, [T] * B)
    assert_mix(eager[3], want, mag, BF)
    assert np.abs(w_s[:, :, :T] - wv).max() <= wv.max() * (2 * d * 2.0 ** -23 * big + 2.0 ** -17)
    # the eviction, by the library's own weights
    K, V = [[None] * Hkv for _ in range(B)], [[None] * Hkv for _ in range(B)]
    for b in range(B):
        for h in range(Hkv):
            stay = so.survivors(w_s[b, h].astype(np.float32), T, budget, recent)
            assert kept[b, h].tolist() == stay
            K[b][h], V[b][h] = k[b, h, stay], v[b, h, stay]
    want, mag = so.tree(qt, np.array(K), np.array(V), kt, vt, par.cpu().numpy(), [budget] * B)
    assert_mix(eager[8], want, mag, BF)
    assert lens_after == [budget + 4, budget + 3]
    for b, (p, a) in enumerate(zip(path.tolist(), acc.tolist())):
        for h in range(Hkv):
            K[b][h] = np.concatenate([K[b][h], kt[b, h, p[:a]], k1[b, h]])
            V[b][h] = np.concatenate([V[b][h], vt[b, h, p[:a]], v1[b, h]])
            n = lens_after[b]
            assert np.array_equal(f64(kc)[b, h, :n], K[b][h]) and np.array_equal(f64(vc)[b, h, :n], V[b][h])
        for h in range(Hq):
            o, m, _ = so._mix(q1[b, h, 0], K[b][h // (Hq // Hkv)], V[b][h // (Hq // Hkv)], d ** -0.5)
            assert_mix(eager[12][b, h], o, m, BF)
