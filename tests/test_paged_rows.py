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


def test_pages_are_int32():
    """torch's default integer type, taken for int32, would make every other page 0."""
    for dtype in (torch.int64, torch.int16, torch.float32):
        with pytest.raises(ValueError, match="int32"):
            hs.paged_rows(rows(), torch.zeros(4, dtype=dtype), 16)


def test_rows_are_counted_by_their_bytes():
    pages = torch.zeros(4, dtype=torch.int32)
    for good in (rows(), rows(64, 1152, torch.uint8), rows(64, 656, torch.uint8), rows(64, 288, torch.float32),
                 torch.zeros(64, 9, 64, dtype=torch.bfloat16), rows(0)):
        assert hs.paged_rows(good, pages, 16).count == good.shape[0]
    for bad in (torch.zeros(4, 16, 576, dtype=torch.bfloat16), rows(64, 576, torch.float32), rows(64, 512), rows(64, 576, torch.uint8),
                torch.zeros(64 * 576, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="1152 or 656"):
            hs.paged_rows(bad, pages, 16)


def test_rows_have_the_pools_bytes(monkeypatch):
    """Rows of one format beside a pool of the other are refused before the library is called."""
    pages = torch.zeros(4, dtype=torch.int32)
    bf16, fp8 = hs.paged_rows(rows(), pages, 16), hs.paged_rows(rows(64, 656, torch.uint8), pages, 16)
    monkeypatch.setitem(hs._pool_row_bytes, 7, 1152)
    monkeypatch.setitem(hs._pool_row_bytes, 8, 656)
    monkeypatch.setattr(hs, "load", lambda: (_ for _ in ()).throw(KeyError("called")))
    for pool, good, bad in ((7, bf16, fp8), (8, fp8, bf16)):
        with pytest.raises(ValueError, match="bytes"):
            hs.hs_append(pool, 0, 1, hs.hs_append_desc(), bad, False, 0)
        with pytest.raises(ValueError, match="bytes"):
            hs.hs_mla_prefix(pool, 1, 0, bad, 16, None, 1.0, None, None, 0, 0, 0, None, 0)
        with pytest.raises(KeyError, match="called"):
            hs.hs_append(pool, 0, 1, hs.hs_append_desc(), good, False, 0)
    with pytest.raises(KeyError, match="called"):  # a struct that somebody else filled, a pool from elsewhere
        hs.hs_append(7, 0, 1, hs.hs_append_desc(), hs.hs_paged_rows(), False, 0)
    with pytest.raises(KeyError, match="called"):
        hs.hs_append(9, 0, 1, hs.hs_append_desc(), fp8, False, 0)
