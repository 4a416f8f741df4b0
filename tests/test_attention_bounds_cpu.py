"""The bounds that a caller gives the cache attention (host only)."""
import pytest

import w4a16_bit_matmul_amd as wq


@pytest.mark.parametrize("T,B,most", [(8, 2, 9), (8, 2, 10 ** 6), (2, 2, 3), (1, 1, 64)])
def test_max_queries_past_all_queries_counts_as_all(T, B, most):
    """As in the call itself, so that a workspace of these bytes fits it."""
    sizes = (64, 8, 128, B, 16, 65536)
    assert wq.wq_kv_attention_workspace_bytes(T, *sizes, most) == wq.wq_kv_attention_workspace_bytes(T, *sizes, T) > 0
    assert wq.wq_kv_attention_plan(T, *sizes, most) == wq.wq_kv_attention_plan(T, *sizes, T)


def test_no_queries():
    assert wq.wq_kv_attention_workspace_bytes(0, 64, 8, 128, 2, 16, 65536, 5) == 0
    assert wq.wq_kv_attention_plan(0, 64, 8, 128, 2, 16, 65536, 5) == ""


def test_all_queries_for_each_of_many_sequences_is_refused():
    with pytest.raises(wq.WQError):
        wq.wq_kv_attention_plan(4096, 64, 8, 128, 1024, 16, 4096, 4096)
    assert "grid=8192" in wq.wq_kv_attention_plan(4096, 64, 8, 128, 1024, 16, 4096, 4)
