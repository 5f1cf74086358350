"""gqa_decode_tree against the float64 definition.

Bounds.  An output is sum_j p_j v_j.  With bf16 tensors the kernel rounds
each p_j once to bf16 for the tensor cores (2^-8 relative) and the result once
(2^-8), so |error| <= 2^-8 (sum p |v| + |o|), and fp32 arithmetic adds less
than 2^-12 of sum p |v| at these sizes (scores of at most 128 products of
about unit values: 128 * 2^-23 * 7 < 2^-13, twice for a quotient).  fp32
tensors are held to the library's 1e-5."""
import numpy as np
import pytest
import torch

import serving_oracle as so
from parity import F32_MAX_ABS, f64
from grouped_query_attention_03_b200 import synthetic

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def assert_mix(got, want, mag, dtype, what=""):
    got = f64(got)
    assert np.isfinite(got).all(), what
    if dtype == F32:
        bound = np.full(want.shape, F32_MAX_ABS)
    else:
        bound = 2.0 ** -8 * (mag + np.abs(want)) + 2.0 ** -12 * mag
    worst = np.max(np.abs(got - want) - bound)
    assert worst <= 0, f"{what}: {worst:.3e} over its bound"


def make(B, Hq, Hkv, C, d, t, lens, seed, dtype=BF, junk=True):
    q = synthetic.normal((B, Hq, t, d), seed, 1.0, dtype, offset=51)
    kc = synthetic.normal((B, Hkv, C, d), seed, 1.0, dtype, offset=52)
    vc = synthetic.normal((B, Hkv, C, d), seed, 1.0, dtype, offset=53)
    kd = synthetic.normal((B, Hkv, t, d), seed, 1.0, dtype, offset=54)
    vd = synthetic.normal((B, Hkv, t, d), seed, 1.0, dtype, offset=55)
    if junk:  # cells behind the sequence belong to nobody
        for b, n in enumerate(lens):
            if 0 <= n < C:
                kc[b, :, n:] = float("nan")
                vc[b, :, n:] = float("inf")
    return q, kc, vc, kd, vd


def random_tree(B, t, seed, pad=0):
    g = torch.Generator()
    g.manual_seed(seed)
    par = torch.empty((B, t), dtype=torch.int32)
    for b in range(B):
        for i in range(t):
            par[b, i] = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        if pad:
            par[b, t - min(pad, t - 1):] = -2
    return par


def run(lib, ins, par, lens, **kw):
    dev = [x.to(DEV) for x in ins]
    st = lib.new_status(DEV)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    o = lib.decode_tree(*dev, None if par is None else par.to(DEV), lt, status=st, **kw)
    torch.cuda.synchronize()
    return o, int(st.item())


CASES = [
    # dtype, B, Hq, Hkv, C, d, t, lens, window, padding nodes
    (BF, 1, 4, 1, 300, 64, 8, [300], None, 0),            # one lane, full cache
    (BF, 1, 8, 2, 1088, 64, 8, [1000], None, 0),
    (BF, 2, 8, 2, 700, 128, 7, [0, 1], None, 2),          # empty and one-cell caches
    (BF, 3, 4, 4, 260, 128, 1, [128, 129, 127], None, 0),  # one node, tile edges
    (BF, 2, 4, 1, 500, 128, 32, [499, 256], None, 5),     # 128 rows: a full row tile
    (BF, 2, 3, 1, 500, 128, 43, [130, 400], None, 0),     # 129 rows: a second tile of 1
    (BF, 1, 8, 1, 900, 128, 32, [777], None, 0),          # 256 rows: two full tiles
    (BF, 2, 14, 2, 513, 64, 43, [512, 77], None, 9),      # group of 7, 301 rows
    (BF, 2, 8, 1, 600, 128, 128, [555, 3], None, 100),    # 1024 rows, mostly padding
    (BF, 5, 4, 2, 2000, 128, 20, [1999, 3, 700, 0, 1234], None, 3),
    (BF, 2, 8, 2, 700, 128, 20, [650, 300], 128, 4),      # window
    (BF, 2, 8, 2, 700, 64, 40, [650, 100], 5, 0),         # window inside the tree
    (BF, 2, 8, 2, 700, 128, 16, [650, 300], 1, 0),        # self only
    (BF, 1, 8, 2, 3000, 128, 60, [2900], 1025, 0),
    (BF, 1, 4, 2, 200, 96, 9, [150], None, 2),            # CUDA cores
    (BF, 2, 4, 2, 200, 80, 30, [150, 0], 40, 2),
    (BF, 1, 2, 1, 100, 33, 5, [99], None, 0),             # odd width
    (F32, 2, 4, 2, 128, 64, 7, [127, 60], 32, 0),
    (F32, 1, 8, 1, 700, 128, 33, [650], None, 3),
    (F32, 2, 2, 2, 300, 256, 12, [299, 0], None, 0),
    (F32, 1, 3, 1, 64, 32, 128, [50], 20, 30),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: (
    f"{'f32' if c[0] == F32 else 'bf16'}-B{c[1]}Hq{c[2]}Hkv{c[3]}C{c[4]}d{c[5]}t{c[6]}w{c[8]}"))
def test_tree_cases(cuda_lib, case):
    dtype, B, Hq, Hkv, C, d, t, lens, window, pad = case
    ins = make(B, Hq, Hkv, C, d, t, lens, C + t, dtype)
    par = random_tree(B, t, C * 7 + t, pad)
    for b in range(B):  # padding rows hold anything
        for i in range(t):
            if par[b, i] == -2:
                for x in (ins[3], ins[4]):
                    x[b, :, i] = float("nan")
    want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), lens, window=window)
    o, st = run(cuda_lib, ins, par, lens, window=window)
    assert st == 0
    assert_mix(o, want, mag, dtype)


def test_chain_is_the_default_tree_and_the_multi_row_decode(cuda_lib):
    B, Hq, Hkv, C, d, t = 2, 8, 2, 600, 128, 9
    lens = [500, 37]
    ins = make(B, Hq, Hkv, C, d, t, lens, 3)
    chain = torch.arange(-1, t - 1, dtype=torch.int32).repeat(B, 1)
    o, st = run(cuda_lib, ins, None, lens)
    o2, st2 = run(cuda_lib, ins, chain, lens)
    assert st == st2 == 0 and torch.equal(o, o2)
    q, kc, vc, kd, vd = [x.to(DEV) for x in ins]
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cuda_lib.cache_append(kc, vc, kd, vd, lt)
    want, mag = so.tree(*[f64(x) for x in ins], None, lens)
    assert_mix(cuda_lib.decode_multi(q, kc, vc, lt), want, mag, BF)
    assert_mix(o, want, mag, BF)


@pytest.mark.parametrize("d,t,dtype", [(128, 12, BF), (64, 40, BF), (96, 12, BF), (64, 12, F32)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_node_may_not_read_never_reaches_it(cuda_lib, d, t, dtype, bad):
    """One drafted row is not finite: its descendants see it, nobody else;
    and a cell that only shallow nodes' windows still hold."""
    B, Hq, Hkv, C = 2, 4, 1, 300
    lens, window = [290, 140], 120
    ins = make(B, Hq, Hkv, C, d, t, lens, 17, dtype)
    par = random_tree(B, t, 99)
    par[:, 1] = -1
    sick = 1
    ins[3][:, :, sick] = bad
    ins[4][:, :, sick] = bad
    for b in range(B):  # the roots' first cell; every deeper node starts later
        ins[2][b, :, lens[b] - (window - 1)] = bad
    want, mag = so.tree(*[np.nan_to_num(f64(x), nan=0.0, posinf=0.0, neginf=0.0) for x in ins],
                        par.numpy(), lens, window=window)
    o, st = run(cuda_lib, ins, par, lens, window=window)
    assert st == 0
    got = f64(o)
    clean = 0
    for b in range(B):
        for i in range(t):
            line = so.line_of(par[b].numpy(), i)
            if sick in line or len(line) == 1:
                assert not np.isfinite(got[b, :, i]).any(), (b, i)
            else:
                clean += 1
                assert_mix(o[b, :, i], want[b, :, i], mag[b, :, i], dtype, f"node {i}")
    assert clean > 0


def test_an_unfinite_value_adds_only_to_its_own_column(cuda_lib):
    """inf in one column of a value row: that column is inf for the rows that
    read it, the others keep their bounds (the row still counts in full)."""
    B, Hq, Hkv, C, d, t = 1, 4, 2, 200, 128, 6
    lens = [150]
    ins = make(B, Hq, Hkv, C, d, t, lens, 23)
    par = torch.tensor([[-1, 0, 0, 1, 1, 2]], dtype=torch.int32)
    ins[4][:, :, 1, 77] = float("inf")
    clean = [f64(x) for x in ins]
    clean[4][:, :, 1, 77] = 0.0
    want, mag = so.tree(*clean, par.numpy(), lens)
    o, st = run(cuda_lib, ins, par, lens)
    assert st == 0
    got = f64(o)
    for i in range(t):
        if 1 in so.line_of(par[0].numpy(), i):
            assert np.isposinf(got[0, :, i, 77]).all()
            got[0, :, i, 77] = want[0, :, i, 77]
    assert_mix(torch.from_numpy(got), want, mag, BF)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_tree_refusals_on_the_device(cuda_lib, dtype, d):
    B, Hq, Hkv, C, t = 3, 4, 2, 64, 6
    ins = make(B, Hq, Hkv, C, d, t, [64, 64, 64], 5, dtype)
    good = random_tree(B, t, 1)
    want, mag = so.tree(*[f64(x) for x in ins], good.numpy(), [64, 65, -1])
    o, st = run(cuda_lib, ins, good, [64, 65, -1])
    assert st == 5
    assert_mix(o, want, mag, dtype)
    assert torch.all(o[1:] == 0)
    for node, parent in ((2, 2), (2, 5), (3, -3), (0, 0)):
        par = good.clone()
        par[1, node] = parent
        want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), [64, 64, 0])
        o, st = run(cuda_lib, ins, par, [64, 64, 0])
        assert st == 13, (node, parent)
        assert_mix(o, want, mag, dtype, f"{node} -> {parent}")
        assert torch.all(o[1, :, node] == 0)
    par = torch.tensor([[-1, 0, -2, 2, 1, -1]] * 3, dtype=torch.int32)  # 3 hangs on padding
    want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), [64, 64, 0])
    o, st = run(cuda_lib, ins, par, [64, 64, 0])
    assert st == 13 and torch.all(o[:, :, 2:4] == 0)
    assert_mix(o, want, mag, dtype)


def test_unaligned_buffers_run_the_other_kernel(cuda_lib):
    B, Hq, Hkv, C, d, t = 1, 4, 2, 150, 64, 6
    ins = make(B, Hq, Hkv, C, d, t, [140], 8)
    par = random_tree(B, t, 3)
    want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), [140])
    moved = []
    for x in ins:
        flat = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)
        flat[1:] = x.flatten().to(DEV)
        moved.append(flat[1:].view(x.shape))
    st = cuda_lib.new_status(DEV)
    o = cuda_lib.decode_tree(*moved, par.to(DEV), torch.tensor([140], dtype=torch.int32, device=DEV),
                             status=st)
    assert int(st.item()) == 0
    assert_mix(o, want, mag, BF)


def test_scale_of_either_sign(cuda_lib):
    B, Hq, Hkv, C, d, t = 1, 4, 2, 300, 128, 5
    ins = make(B, Hq, Hkv, C, d, t, [250], 8)
    par = random_tree(B, t, 3)
    for scale in (0.0, -0.05, 0.3):
        want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), [250], scale=scale)
        o, st = run(cuda_lib, ins, par, [250], scale=scale)
        assert st == 0
        assert_mix(o, want, mag, BF, f"scale {scale}")


def test_one_workspace_many_shapes_streams_and_graphs(cuda_lib):
    """One workspace, zeroed once; a captured call replays with new inputs in
    the same buffers; a second stream ordered by events."""
    shapes = [(2, 8, 2, 900, 128, 20, [888, 400]), (1, 8, 1, 600, 64, 64, [600]), (1, 4, 4, 300, 128, 3, [5])]
    ws = torch.zeros(cuda_lib.lib().gqa_decode_tree_workspace_bytes(1, 2, 8, 2, 900, 128, 128) +
                     (8 << 20), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    for rep in range(2):
        for B, Hq, Hkv, C, d, t, lens in shapes:
            ins = make(B, Hq, Hkv, C, d, t, lens, t + rep)
            par = random_tree(B, t, t)
            want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), lens)
            dev = [x.to(DEV) for x in ins]
            lt, pd = torch.tensor(lens, dtype=torch.int32, device=DEV), par.to(DEV)
            st = cuda_lib.new_status(DEV)
            o = torch.empty_like(dev[0])
            side.wait_stream(torch.cuda.current_stream())
            cuda_lib.decode_tree(*dev, pd, lt, out=o, workspace=ws, status=st, stream=side)
            torch.cuda.current_stream().wait_stream(side)
            first = o.clone()
            assert_mix(o, want, mag, BF)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                cuda_lib.decode_tree(*dev, pd, lt, out=o, workspace=ws, status=st)
            for _ in range(3):
                o.fill_(7)
                g.replay()
                assert torch.equal(o, first)  # the same bits every time
            dev[0].copy_(dev[0].flip(2))
            ins2 = [f64(dev[0])] + [f64(x) for x in ins[1:]]
            want, mag = so.tree(*ins2, par.numpy(), lens)
            g.replay()
            assert_mix(o, want, mag, BF)
            assert int(st.item()) == 0


def test_a_long_cache_splits_over_all_sms(cuda_lib):
    """One lane of 20000 cells (about 150 parts) and many short lanes."""
    B, Hq, Hkv, C, d, t = 1, 2, 1, 20000, 128, 3
    ins = make(B, Hq, Hkv, C, d, t, [20000], 11)
    par = random_tree(B, t, 3)
    want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), [20000])
    o, st = run(cuda_lib, ins, par, [20000])
    assert st == 0
    assert_mix(o, want, mag, BF)
    lens = [(37 * b) % 60 for b in range(300)]
    ins = make(300, 4, 2, 64, 64, 4, lens, 12)
    par = random_tree(300, 4, 5, 1)
    want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), lens)
    o, st = run(cuda_lib, ins, par, lens)
    assert st == 0
    assert_mix(o, want, mag, BF)


RUNNING = [
    # B, Hq, Hkv, C, d, t, window, padding: more than 32 sequences, so that a
    # CTA's range runs from one lane group into the next
    (40, 8, 2, 3000, 128, 20, None, 3),
    (40, 8, 1, 1500, 128, 40, None, 9),    # 320 rows: pairs of row tiles, two groups
    (33, 4, 2, 2000, 64, 70, 700, 5),      # 140 rows: a second tile of 12, window
    (150, 2, 1, 900, 128, 5, None, 0),     # more lengths than the kernel keeps at hand
]


@pytest.mark.parametrize("case", RUNNING, ids=lambda c: f"B{c[0]}Hq{c[1]}Hkv{c[2]}d{c[4]}t{c[5]}w{c[6]}")
def test_ranges_that_cross_lane_groups(cuda_lib, case):
    """Early, whole, middle and last parts; refused sequences in between."""
    B, Hq, Hkv, C, d, t, window, pad = case
    lens = [(b * 733) % (C + 1) for b in range(B)]
    lens[1], lens[B // 2], lens[3] = -5, C + 1, C
    ins = make(B, Hq, Hkv, C, d, t, lens, t)
    par = random_tree(B, t, t, pad)
    want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), lens, window=window)
    o, st = run(cuda_lib, ins, par, lens, window=window)
    assert st == 5
    assert_mix(o, want, mag, BF)
    again, _ = run(cuda_lib, ins, par, lens, window=window)
    assert torch.equal(o, again)


def test_an_empty_cache(cuda_lib):
    """Capacity 0: the drafts alone."""
    for d, dtype in ((128, BF), (64, F32)):
        ins = make(2, 4, 2, 0, d, 6, [0, 0], 3, dtype)
        par = random_tree(2, 6, 4)
        want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), [0, 0])
        o, st = run(cuda_lib, ins, par, [0, 0])
        assert st == 0
        assert_mix(o, want, mag, dtype)


def test_one_workspace_with_the_other_decodes(cuda_lib):
    """decode, decode_tree and decode_scored take turns on one workspace, and
    two calls run at once on two streams with a workspace each."""
    B, Hq, Hkv, C, d, t = 2, 8, 2, 2500, 128, 12
    lens = [2500, 1300]
    ins = make(B, Hq, Hkv, C, d, t, lens, 3)
    par = random_tree(B, t, 4)
    q, kc, vc, kd, vd = [x.to(DEV) for x in ins]
    lt, pd = torch.tensor(lens, dtype=torch.int32, device=DEV), par.to(DEV)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    q1 = q[:, :, 0].contiguous()
    alone = (cuda_lib.decode_tree(q, kc, vc, kd, vd, pd, lt), cuda_lib.decode(q1, kc, vc, lt),
             cuda_lib.decode_scored(q1, kc, vc, torch.zeros(B, Hkv, C, device=DEV), lt),
             cuda_lib.decode_scored(q, kc, vc, torch.zeros(B, Hkv, C, device=DEV), lt))
    for _ in range(3):
        w1, w2 = torch.zeros(B, Hkv, C, device=DEV), torch.zeros(B, Hkv, C, device=DEV)
        got = (cuda_lib.decode_tree(q, kc, vc, kd, vd, pd, lt, workspace=ws),
               cuda_lib.decode(q1, kc, vc, lt, workspace=ws),
               cuda_lib.decode_scored(q1, kc, vc, w1, lt, workspace=ws),
               cuda_lib.decode_scored(q, kc, vc, w2, lt, workspace=ws))
        for a, b in zip(alone, got):
            assert torch.equal(a, b)
    side = [torch.cuda.Stream() for _ in range(2)]
    wss = [cuda_lib.decode_tree_workspace(q, kc) for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(10):
        for s, w, o in zip(side, wss, outs):
            cuda_lib.decode_tree(q, kc, vc, kd, vd, pd, lt, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[0])


@pytest.mark.parametrize("d", [4, 20, 32, 33, 64, 80, 128, 200, 256])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_cuda_core_rows_of_every_kind(cuda_lib, dtype, d):
    """1 to 17 rows of a group (shared features, shared keys, two groups),
    vectors and single elements, one part and several, windows."""
    if dtype == BF and d in (64, 128):
        shift = 1  # not 16-byte aligned: CUDA cores
    else:
        shift = 0
    for r, t, lens, window in ((1, 1, [40], None), (3, 1, [0], None), (1, 5, [33], 7), (2, 4, [200], None),
                               (3, 3, [95], 40), (4, 4, [31], None), (1, 17, [300], 21), (2, 40, [65], None)):
        for off in {shift, 1}:
            C = lens[0] + 3
            ins = make(1, r, 1, C, d, t, lens, t + d, dtype)
            par = random_tree(1, t, t + r, min(2, t - 1))
            want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), lens, window=window)
            dev = []
            for x in ins:
                flat = torch.empty(x.numel() + off, dtype=dtype, device=DEV)[off:]
                dev.append(flat.view(x.shape).copy_(x))
            st = cuda_lib.new_status(DEV)
            o = cuda_lib.decode_tree(*dev, par.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                     window=window, status=st)
            assert int(st.item()) == 0
            assert_mix(o, want, mag, dtype, f"r{r} t{t} {lens} w{window} off{off}")
