"""The binding's block tables: what paged_rows takes and what it refuses."""
import ctypes

import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs


def rows(n=64, width=576, dtype=torch.bfloat16):
    return torch.zeros(n, width, dtype=dtype)


def test_lists_are_counted():
    one, three = torch.zeros(5, dtype=torch.int32), torch.zeros(3, 5, dtype=torch.int32)
    p = hs.paged_rows(rows(), one, 16)
    assert (p.lists, p.page_stride, p.page_rows, p.count) == (1, 5, 16, 64)
    p = hs.paged_rows(rows(), three, 16)
    assert (p.lists, p.page_stride) == (3, 5)
    assert hs.hs_paged_rows.lists.offset == 36 and ctypes.sizeof(hs.hs_paged_rows) == 40
    for bad in (torch.zeros(2, 3, 5, dtype=torch.int32), torch.zeros((), dtype=torch.int32), torch.zeros(0, 5, dtype=torch.int32),
                torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError):
            hs.paged_rows(rows(), bad, 16)
