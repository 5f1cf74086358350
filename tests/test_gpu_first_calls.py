"""The first calls of a process, from many threads at once: what the library
looks up once (the driver's tensor-map encoder, each device's facts, kernel
attributes) is there for all of them."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
from grouped_query_attention_03_b200 import gqa
gqa.lib()
N = 16
x = [torch.randn(1, 4, 3, 64, device="cuda").bfloat16() for _ in range(N)]
kc = torch.randn(1, 2, 40, 64, device="cuda").bfloat16()
kd = torch.randn(1, 2, 3, 64, device="cuda").bfloat16()
lens = torch.tensor([40], dtype=torch.int32, device="cuda")
ws = [torch.zeros(1 << 21, dtype=torch.uint8, device="cuda") for _ in range(N)]
st = [gqa.new_status("cuda") for _ in range(N)]
out = [torch.empty_like(q) for q in x]
torch.cuda.synchronize()
go, bad = threading.Barrier(N), []


def call(k):
    if BOUND:  # the thread has used this device before
        torch.zeros(1, device="cuda")
    go.wait()
    try:
        gqa.decode_tree(x[k], kc, kc, kd, kd, None, lens, out=out[k], workspace=ws[k], status=st[k])
    except Exception as e:
        bad.append(str(e))


if not BOUND:  # the library has been used before, by another thread
    gqa.decode_tree(x[0], kc, kc, kd, kd, None, lens, out=out[0], workspace=ws[0], status=st[0])
threads = [threading.Thread(target=call, args=(k,)) for k in range(N)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not bad, bad
for k in range(N):
    assert int(st[k].item()) == 0
    again = gqa.decode_tree(x[k], kc, kc, kd, kd, None, lens, workspace=ws[k])
    assert torch.equal(again, out[k])
print("all there")
"""


EVERY_CALL = """
import threading
import torch
from grouped_query_attention_03_b200 import gqa
gqa.lib()
B, Hq, Hkv, C, d, t = 1, 4, 2, 160, 64, 5


def z(*shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device="cuda").to(dtype)


def i(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


bad, done = [], []
p, q, q1 = z(B, Hq, C, d), z(B, Hq, t, d), z(B, Hq, d)
k, v, new, kd = z(B, Hkv, C, d), z(B, Hkv, C, d), z(B, Hkv, 1, d), z(B, Hkv, t, d)
x, w = z(B, t, (Hq + 2 * Hkv) * d), torch.zeros(B, Hkv, C, device="cuda")
ws = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
st = gqa.new_status("cuda")
outs = [torch.empty_like(y) for y in (p, q, q1)]
nr = tuple(torch.empty(B, h, t, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
kept = torch.empty(B, Hkv, 100, dtype=torch.int32, device="cuda")
seg, lens, full, path, one = torch.zeros(B, C, dtype=torch.int32, device="cuda"), i(100), i(160), i(0).view(1, 1), i(1)
pair, slot = i(150), [i(20) for _ in range(4)]
o_p, o_t, o_1 = outs
calls = {
    "prefill": lambda: gqa.prefill(p, k, v, out=o_p, status=st),
    "prefill_packed": lambda: gqa.prefill_packed(p, k, v, seg, out=o_p, status=st),
    "decode": lambda: gqa.decode(q1, k, v, full, out=o_1, workspace=ws, status=st),
    "decode_append": lambda: gqa.decode_append(q1, k, v, new, new, slot[0], out=o_1, workspace=ws, status=st),
    "decode_multi": lambda: gqa.decode_multi(q, k, v, full, out=o_t, status=st),
    "decode_noalloc": lambda: gqa.decode_noalloc(q1, k, v, full, out=o_1, status=st),
    "cache_append": lambda: gqa.cache_append(k, v, kd, kd, slot[1], status=st),
    "ring_append": lambda: gqa.ring_append(k, v, kd, kd, slot[2], status=st),
    "ring_decode_append": lambda: gqa.ring_decode_append(q1, k, v, new, new, slot[3], out=o_1, workspace=ws, status=st),
    "qk_norm_rope": lambda: gqa.qk_norm_rope(x, Hq, Hkv, d, out=nr),
    "decode_tree": lambda: gqa.decode_tree(q, k, v, kd, kd, None, lens, out=o_t, workspace=ws, status=st),
    "scored, one row": lambda: gqa.decode_scored(q1, k, v, w, full, out=o_1, workspace=ws, status=st),
    "scored": lambda: gqa.decode_scored(q, k, v, w, full, out=o_t, workspace=ws, status=st),
    "tree_commit": lambda: gqa.tree_commit(k, v, kd, kd, path, one, pair, status=st),
    "cache_evict": lambda: gqa.cache_evict(k, v, w, full, 100, 10, kept=kept, status=st),
}
torch.cuda.synchronize()


def call(name):
    try:
        calls[name]()
        done.append(name)
    except Exception as e:
        bad.append((name, str(e)))


for name in calls:  # one new thread each, in turn
    t = threading.Thread(target=call, args=(name,))
    t.start()
    t.join()
torch.cuda.synchronize()
assert not bad, bad
assert int(st.item()) == 0 and len(done) == len(calls)
print("all there")
"""


def run(bound):
    return subprocess.run([sys.executable, "-c", f"BOUND = {bound}\n" + PROGRAM], cwd=ROOT, capture_output=True,
                          text=True, timeout=120)


def test_first_calls_from_many_threads(cuda_lib):
    for _ in range(3):
        r = run(True)
        assert r.returncode == 0 and "all there" in r.stdout, r.stderr[-2000:]


def test_threads_that_have_not_used_the_device(cuda_lib):
    """Buffers from another thread, and no CUDA call before the library's."""
    r = run(False)
    assert r.returncode == 0 and "all there" in r.stdout, r.stderr[-2000:]


def test_every_kind_of_call_from_a_new_thread(cuda_lib):
    r = subprocess.run([sys.executable, "-c", EVERY_CALL], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "all there" in r.stdout, r.stderr[-2000:]
