"""What a call with `stream=` allocates itself (output, workspace, status word)
is allocated, and cleared, on that stream: no CUDA call is reached here, the
stream is a stand-in that the binding has to enter."""
import contextlib

import pytest
import torch

from grouped_query_attention_03_b200 import build as gbuild

B, HQ, HKV, C, D, T = 2, 4, 2, 8, 64, 3


@pytest.fixture(scope="module")
def gqa():
    gbuild.build()
    from grouped_query_attention_03_b200 import gqa
    gqa.lib()
    return gqa


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def calls():
    q1, qt = z(B, HQ, D), z(B, HQ, T, D)
    kc, new, kt = z(B, HKV, C, D), z(B, HKV, 1, D), z(B, HKV, T, D)
    lens, w = z(B, dtype=torch.int32), z(B, HKV, C)
    path = z(B, 2, dtype=torch.int32)
    return {
        "prefill": (z(B, HQ, C, D), kc, kc),
        "prefill_packed": (z(B, HQ, C, D), kc, kc, z(B, C, dtype=torch.int32)),
        "decode": (q1, kc, kc, lens),
        "decode_append": (q1, kc, kc, new, new, lens),
        "decode_multi": (qt, kc, kc, lens),
        "decode_noalloc": (q1, kc, kc, lens),
        "cache_append": (kc, kc, kt, kt, lens),
        "ring_append": (kc, kc, kt, kt, lens),
        "ring_decode_append": (q1, kc, kc, new, new, lens),
        "qk_norm_rope": (z(B, T, (HQ + 2 * HKV) * D), HQ, HKV, D),
        "decode_tree": (qt, kc, kc, kt, kt, None, lens),
        "tree_commit": (kc, kc, kt, kt, path, lens, lens),
        "decode_scored": (qt, kc, kc, w, lens),
        "cache_evict": (kc, kc, w, lens, 4, 1),
    }


@pytest.mark.parametrize("name", sorted(calls()))
@pytest.mark.parametrize("given", [False, True], ids=["own stream", "stream="])
def test_allocations_belong_to_the_calls_stream(gqa, monkeypatch, name, given):
    inside, made, current = [], [], object()

    @contextlib.contextmanager
    def enter(stream):
        inside.append(stream)
        yield
        inside.pop()

    def watched(fn):
        def make(*a, **kw):
            made.append(inside[-1] if inside else None)
            return fn(*a, **kw)
        return make

    args = calls()[name]
    if name == "qk_norm_rope":  # asks for a CUDA tensor before it allocates nothing more
        monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(gqa, "_run", lambda *a: None)
    monkeypatch.setattr(gqa, "_ptr", lambda *a, **kw: 0)
    monkeypatch.setattr(gqa, "_stream", lambda s, dev: 0)
    for f in ("zeros", "empty", "empty_like"):
        monkeypatch.setattr(torch, f, watched(getattr(torch, f)))
    getattr(gqa, name)(*args, stream=current if given else None)
    assert made and all(m is (current if given else None) for m in made), made
