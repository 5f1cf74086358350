"""Queries of a wrong rank are refused before the library is called."""
import pytest
import torch

from grouped_query_attention_03_b200 import build as gbuild


@pytest.fixture(scope="module")
def gqa():
    gbuild.build()
    from grouped_query_attention_03_b200 import gqa
    gqa.lib()
    return gqa


@pytest.mark.parametrize("shape", [(2, 64), (2, 4, 2, 3, 64), (2, 4, 1, 1, 1, 64)])
def test_scored_queries_have_three_or_four_dimensions(gqa, monkeypatch, shape):
    monkeypatch.setattr(gqa, "_run", lambda *a: pytest.fail("the library was called"))
    monkeypatch.setattr(gqa, "_ptr", lambda *a, **kw: 0)
    monkeypatch.setattr(gqa, "_stream", lambda s, dev: 0)
    q, kc, w = torch.zeros(shape), torch.zeros(2, 2, 8, 64), torch.zeros(2, 2, 8)
    lens = torch.ones(2, dtype=torch.int32)
    for ws in (None, torch.zeros(256, dtype=torch.uint8)):
        with pytest.raises(ValueError, match=r"q must be \[B,Hq,d\] or \[B,Hq,t,d\]"):
            gqa.decode_scored(q, kc, kc, w, lens, workspace=ws)
    with pytest.raises(ValueError, match="q must be"):
        gqa.decode_scored_workspace(q, kc)
