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


def run(bound):
    return subprocess.run([sys.executable, "-c", f"BOUND = {bound}\n" + PROGRAM], cwd=ROOT, capture_output=True,
                          text=True, timeout=120)


def test_first_calls_from_many_threads(cuda_lib):
    for _ in range(3):
        r = run(True)
        assert r.returncode == 0 and "all there" in r.stdout, r.stderr[-2000:]
