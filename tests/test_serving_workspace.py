"""Workspace sizes of the tree and scored decode (host only), and the binding's
workspaces."""
import pytest
import torch

from grouped_query_attention_03_b200 import build as gbuild


@pytest.fixture(scope="module")
def gqa():
    gbuild.build()
    from grouped_query_attention_03_b200 import gqa
    gqa.lib()
    return gqa


def partials(B, Hq, Hkv, d, t):
    """An upper bound on partial sums and statistics: one slot of at most 256
    rows per lane group of that many rows, and 1024 more, d + 2 floats a row."""
    R = Hq // Hkv * t
    slots = B * Hkv * ((R + 15) // 16) * 16 + 1024 * min(R + 15, 256)
    return slots * (d + 3) * 4 + B * Hq * t * 8 + (1 << 16)


@pytest.mark.parametrize("B,Hq,Hkv,d,t", [(8, 32, 8, 128, 32), (1, 32, 8, 128, 32), (8, 64, 8, 128, 128),
                                          (4, 8, 1, 64, 3), (1, 4, 4, 64, 17)])
def test_many_scored_rows_need_no_room_for_scores(gqa, B, Hq, Hkv, d, t):
    """bf16, d = 64 or 128, more than d / 4 rows in a KV group: the scores are
    not kept, whatever the buffers' alignment, so the capacity does not count."""
    f = gqa.lib().gqa_decode_scored_workspace_bytes
    sizes = {f(1, B, Hq, Hkv, C, d, t) for C in (8192, 32768, 131072)}
    assert len(sizes) == 1
    # (CUDA-core parts: at most 592 CTAs of 16 rows beside the lane groups' own)
    assert 0 < max(sizes) <= 2 * partials(B, Hq, Hkv, d, t)


def test_where_scores_are_kept(gqa):
    f = gqa.lib().gqa_decode_scored_workspace_bytes
    for dtype, Hq, d, t in ((1, 8, 128, 1), (1, 8, 128, 4), (1, 8, 96, 32), (0, 8, 128, 32), (0, 8, 64, 1)):
        assert f(dtype, 2, Hq, 2, 4096, d, t) >= 2 * Hq * t * 4096 * 4


def test_tree_sizes_do_not_depend_on_a_long_capacity(gqa):
    f = gqa.lib().gqa_decode_tree_workspace_bytes
    assert f(1, 8, 32, 8, 32768, 128, 32) == f(1, 8, 32, 8, 131072, 128, 32)


def test_the_bindings_workspaces_start_with_zeros(gqa):
    for n in (0, 5, 300, 5000, (1 << 22) + 77):
        ws = gqa._workspace(n, torch.device("cpu"))
        assert ws.dtype == torch.uint8 and ws.numel() >= max(n, 256)
        assert not ws[:gqa.WORKSPACE_ZERO_BYTES].any()
