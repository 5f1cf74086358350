"""gqa_qk_norm_rope against the float64 definition.

Bound per output y = u cos a -+ v sin a (u, v normalised): the storage
rounding, eps / 2 of the type times |y|; in fp32 the sum of squares (at most
256 terms in a tree and chains of 8: under 16 roundings), the reciprocal
root, weight, cosine and sine (2 ulp each) and the rotation, together under
2^-19 (|u| + |v|), the angle's 2^-24 half turns among them."""
import numpy as np
import pytest
import torch

import serving_oracle as so
from parity import f64
from grouped_query_attention_03_b200 import synthetic

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def check(got, want, mag, dtype):
    half_step = torch.finfo(dtype).eps / 2
    for g, w, m in zip(got, want, mag):
        assert g.shape == w.shape and g.dtype == dtype
        err = np.abs(f64(g) - w) - (half_step * np.abs(w) + 2.0 ** -19 * m)
        assert err.max() <= 0, f"{err.max():.3e} over its bound"


def freqs(half, theta=1e4):
    return (theta ** (-torch.arange(half, dtype=torch.float64) / max(1, half))).float()


CASES = [
    # dtype, B, T, Hq, Hkv, d, rot, axes, interleaved, norms
    (BF, 1, 1, 4, 1, 64, 64, 1, False, "qk"),
    (BF, 8, 1, 32, 8, 128, 128, 1, False, "qk"),
    (BF, 2, 37, 8, 2, 128, 128, 1, True, "qk"),
    (BF, 2, 37, 8, 2, 128, 64, 1, False, "qk"),      # partial rotation
    (BF, 3, 130, 6, 2, 64, 32, 3, False, "qk"),
    (BF, 2, 65, 7, 1, 128, 128, 3, True, "q"),
    (BF, 1, 50, 3, 3, 96, 96, 2, False, "k"),        # 12 of 16 lanes
    (BF, 1, 50, 4, 2, 80, 80, 1, False, "qk"),       # halves of 40 elements
    (BF, 2, 19, 4, 2, 80, 40, 1, False, "qk"),       # halves of 20: row kernel
    (BF, 2, 19, 4, 2, 80, 36, 4, True, "qk"),        # pairs end inside a vector
    (BF, 1, 21, 2, 1, 256, 256, 1, False, "qk"),
    (BF, 1, 21, 2, 1, 33, 32, 1, False, "qk"),       # odd width
    (BF, 1, 5, 2, 1, 1, 0, 1, False, "qk"),
    (BF, 2, 300, 16, 4, 128, 0, 1, False, "qk"),     # norms alone
    (BF, 2, 300, 16, 4, 128, 128, 1, False, ""),     # rotation alone
    (F32, 2, 128, 4, 2, 64, 64, 1, False, "qk"),
    (F32, 2, 33, 4, 2, 128, 128, 3, True, "qk"),
    (F32, 1, 17, 3, 1, 256, 256, 1, False, "qk"),    # 64 vectors: row kernel
    (F32, 1, 17, 3, 1, 20, 12, 1, False, "qk"),
    (F32, 3, 1, 4, 2, 64, 64, 1, False, ""),
]


def make(dtype, B, T, Hq, Hkv, d, rot, axes, norms, seed):
    x = synthetic.normal((B, T, (Hq + 2 * Hkv) * d), seed, 1.5, dtype, offset=61)
    w = [1 + synthetic.normal((d,), seed, 0.3, F32, offset=62 + i) for i in range(2)]
    qw = w[0].to(dtype) if "q" in norms else None
    kw = w[1].to(dtype) if "k" in norms else None
    g = torch.Generator()
    g.manual_seed(seed)
    pos = torch.randint(-1000, 200000, (axes, B, T), generator=g, dtype=torch.int32)
    ax = [int(a) for a in torch.randint(0, axes, (rot // 2,), generator=g)]
    return x, qw, kw, freqs(rot // 2) if rot else None, pos, ax


@pytest.mark.parametrize("case", CASES, ids=lambda c: (
    f"{'f32' if c[0] == F32 else 'bf16'}-B{c[1]}T{c[2]}Hq{c[3]}Hkv{c[4]}d{c[5]}r{c[6]}a{c[7]}"
    f"{'i' if c[8] else 'h'}-{c[9]}"))
def test_norm_rope_cases(cuda_lib, case):
    dtype, B, T, Hq, Hkv, d, rot, axes, inter, norms = case
    x, qw, kw, fr, pos, ax = make(dtype, B, T, Hq, Hkv, d, rot, axes, norms, d + T)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    got = cuda_lib.qk_norm_rope(dev(x), Hq, Hkv, d, q_weight=dev(qw), k_weight=dev(kw), eps=EPS,
                                inv_freq=dev(fr), interleaved=inter, positions=dev(pos), axes=ax)
    num = lambda t: None if t is None else f64(t)  # noqa: E731
    want, mag = so.norm_rope(f64(x), Hq, Hkv, d, num(qw), num(kw), EPS, num(fr), pos.numpy(), ax, inter)
    check(got, want, mag, dtype)
    assert torch.equal(got[2].cpu(), x.view(B, T, -1, d)[:, :, Hq + Hkv:Hq + 2 * Hkv].transpose(1, 2))


def test_angles_of_far_positions(cuda_lib):
    """|position| up to 2^31 - 1: the rotation of (1, 0) is (cos a, sin a) of
    the exact angle, to fp32."""
    fr = freqs(64, 1e6)
    pos = torch.tensor([[0, 1, -1, 4095, 10 ** 6 + 3, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31]],
                       dtype=torch.int32)
    T = pos.shape[1]
    x = torch.zeros(1, T, 3, 128)
    x[..., :64] = 1.0
    q, k, _ = cuda_lib.qk_norm_rope(x.view(1, T, -1).to(DEV), 1, 1, 128, inv_freq=fr.to(DEV),
                                    positions=pos.to(DEV))
    # exact fractions of a turn: the angle in long double, modulo 2 pi
    from fractions import Fraction
    import math
    two_pi = Fraction(2) * Fraction("3.14159265358979323846264338327950288419716939937510")
    want = np.zeros((T, 128))
    for j, pj in enumerate(pos[0].tolist()):
        for i, f in enumerate(fr.tolist()):
            a = Fraction(pj) * Fraction(f)
            a = float(a - two_pi * (a // two_pi))
            want[j, i], want[j, 64 + i] = math.cos(a), math.sin(a)
    for y in (q, k):
        # 2^-31 * 2^53 rounding of a frequency: 2^-23 turns at the farthest
        assert np.abs(f64(y)[0, 0] - want).max() <= 2.0 ** -21


def test_default_positions_strides_and_step_form(cuda_lib):
    """Rows inside a wider projection, a batch apart; positions None = 0..T-1;
    T = 1 outputs feed the fused decode step."""
    B, T, Hq, Hkv, d = 2, 9, 4, 2, 64
    width = (Hq + 2 * Hkv) * d
    wide = synthetic.normal((B, T, width + 24), 4, 1.0, BF, offset=61).to(DEV)
    x = wide[:, :, 8:8 + width]
    fr = freqs(32).to(DEV)
    got = cuda_lib.qk_norm_rope(x, Hq, Hkv, d, inv_freq=fr)
    pos = torch.arange(T, dtype=torch.int32).expand(1, B, T).numpy()
    want, mag = so.norm_rope(f64(x), Hq, Hkv, d, None, None, EPS, f64(fr), pos, [0] * 32, False)
    check(got, want, mag, BF)
    odd = wide[:, :, 3:3 + width]  # not 16-byte aligned: row kernel
    got = cuda_lib.qk_norm_rope(odd, Hq, Hkv, d, inv_freq=fr)
    want, mag = so.norm_rope(f64(odd), Hq, Hkv, d, None, None, EPS, f64(fr), pos, [0] * 32, False)
    check(got, want, mag, BF)
    one = cuda_lib.qk_norm_rope(x[:, 4:5], Hq, Hkv, d, inv_freq=fr,
                                positions=torch.full((B, 1), 4, dtype=torch.int32, device=DEV))
    want, mag = so.norm_rope(f64(x[:, 4:5]), Hq, Hkv, d, None, None, EPS, f64(fr), pos[:, :, 4:5],
                             [0] * 32, False)
    check(one, want, mag, BF)
    flipped = wide[:1].expand(3, T, width + 24)[:, :, :width]  # batch stride 0
    got = cuda_lib.qk_norm_rope(flipped, Hq, Hkv, d, inv_freq=fr)
    for y in got:
        assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


def test_values_pass_and_unrotated_elements_stay_apart(cuda_lib):
    """inf and NaN in a value head, and in unrotated elements of a head
    without norm, stay where they are."""
    B, T, Hq, Hkv, d = 1, 4, 2, 1, 64
    x = synthetic.normal((B, T, (Hq + 2 * Hkv) * d), 4, 1.0, BF, offset=61)
    y = x.view(B, T, 4, d)
    y[0, 1, 3, 5] = float("inf")
    y[0, 2, 3, 6] = float("nan")
    y[0, 1, 0, 40] = float("-inf")
    for inter in (False, True):
        q, k, v = cuda_lib.qk_norm_rope(x.to(DEV), Hq, Hkv, d, inv_freq=freqs(16).to(DEV), interleaved=inter)
        assert torch.equal(torch.nan_to_num(v.cpu()[0, 0]), torch.nan_to_num(y[0, :, 3]))
        assert torch.equal(q.cpu()[0, 0, :, 32:], y[0, :, 0, 32:])
        assert torch.isfinite(q.cpu()[0, 0, :, :32].float()).all() and torch.isfinite(k.cpu().float()).all()


def test_zero_rows_and_capture(cuda_lib):
    B, T, Hq, Hkv, d = 2, 40, 4, 2, 128
    x = torch.zeros(B, T, (Hq + 2 * Hkv) * d, dtype=BF, device=DEV)
    w = torch.ones(d, dtype=BF, device=DEV)
    fr = freqs(64).to(DEV)
    out = tuple(torch.empty(B, h, T, d, dtype=BF, device=DEV) for h in (Hq, Hkv, Hkv))
    cuda_lib.qk_norm_rope(x, Hq, Hkv, d, q_weight=w, k_weight=w, inv_freq=fr, out=out)
    assert all(torch.all(o == 0) for o in out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.qk_norm_rope(x, Hq, Hkv, d, q_weight=w, k_weight=w, inv_freq=fr, out=out)
    x.copy_(synthetic.normal(x.shape, 3, 1.0, BF))
    g.replay()
    pos = np.broadcast_to(np.arange(T, dtype=np.int32), (1, B, T))
    want, mag = so.norm_rope(f64(x), Hq, Hkv, d, f64(w), f64(w), EPS, f64(fr), pos, [0] * 64, False)
    check(out, want, mag, BF)
