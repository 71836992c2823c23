"""The host side of the attention binding, without a GPU."""
import pytest
import torch

from int4_routed_expert_quantize_gb300 import attn


def test_page_table_rows_are_where_the_tensor_has_them():
    """an expanded row has stride 0 and holds no second row behind it; rows that overlap are refused"""
    flat = torch.arange(40, dtype=torch.int32)
    assert attn._row_stride(flat.view(4, 10)) == 10
    assert attn._row_stride(flat.view(4, 10)[:, :7]) == 10
    assert attn._row_stride(flat.view(4, 10)[:1]) == 10
    assert attn._row_stride(flat[None, :5].expand(3, -1)) == 0
    assert attn._row_stride(torch.as_strided(flat, (1, 10), (3, 1))) == 10
    for rows, width, stride in ((3, 10, 4), (2, 2, 1)):
        with pytest.raises(ValueError):
            attn._row_stride(torch.as_strided(flat, (rows, width), (stride, 1)))
