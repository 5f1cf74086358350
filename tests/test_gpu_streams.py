"""Calls on another stream than the current one that bring no output, workspace
or status word: what they allocate is cleared on their own stream, while the
current one is busy."""
import pytest
import torch

import serving_oracle as so
from parity import f64
from test_gpu_tree import BF, DEV, assert_mix, make, random_tree

pytestmark = pytest.mark.gpu


def test_a_call_on_another_stream(cuda_lib):
    B, Hq, Hkv, C, d, t = 2, 8, 2, 2500, 128, 6
    lens = [2500, 1201]
    ins = make(B, Hq, Hkv, C, d, t, lens, 3)
    par = random_tree(B, t, 4)
    want, mag = so.tree(*[f64(x) for x in ins], par.numpy(), lens)
    want_s, mag_s, w, _ = so.scored(f64(ins[0]), f64(ins[1]), f64(ins[2]), lens)
    dev = [x.to(DEV) for x in ins]
    lt, pd = torch.tensor(lens, dtype=torch.int32, device=DEV), par.to(DEV)
    weights = torch.zeros(B, Hkv, C, device=DEV)
    q1 = dev[0][:, :, t - 1].contiguous()
    side = torch.cuda.Stream()
    for _ in range(3):
        weights.zero_()
        # memory that was written to and freed is what the next call may get
        junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in (1 << 20, 4 << 20, 16 << 20)]
        torch.cuda.synchronize()
        del junk
        torch.cuda._sleep(20_000_000)  # the current stream is busy for about 10 ms
        o = cuda_lib.decode_tree(*dev, pd, lt, stream=side)
        o_s = cuda_lib.decode_scored(dev[0], dev[1], dev[2], weights, lt, stream=side)
        o_1 = cuda_lib.decode(q1, dev[1], dev[2], lt, stream=side)
        side.synchronize()
        first = [x.clone() for x in (o, o_s, o_1)]
        torch.cuda.synchronize()
        assert_mix(first[0], want, mag, BF)
        assert_mix(first[1], want_s, mag_s, BF)
        assert_mix(first[2], want_s[:, :, t - 1], mag_s[:, :, t - 1], BF)
