"""The binding's append descriptors beyond their shapes: what hs_append refuses of them."""
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs


def desc(n=3, **kw):
    kv = torch.zeros(n, 576, dtype=torch.bfloat16)
    return hs.append_desc(kv, torch.zeros(32), torch.zeros(n, dtype=torch.int32), **kw)


@pytest.fixture
def library(monkeypatch):
    """A library that is never called: reaching it raises KeyError."""
    monkeypatch.setattr(hs, "load", lambda: (_ for _ in ()).throw(KeyError("called")))


def test_no_more_tokens_than_the_tensors_hold(library):
    for ntok in (4, 1 << 30):
        with pytest.raises(ValueError, match="3"):
            hs.hs_append(1, 0, ntok, desc(), None, True, 0)
    for ntok in (3, 1, 0, -1):
        with pytest.raises(KeyError, match="called"):
            hs.hs_append(1, 0, ntok, desc(), None, True, 0)
    with pytest.raises(KeyError, match="called"):  # a struct that somebody else filled
        hs.hs_append(1, 0, 1 << 30, hs.hs_append_desc(), None, True, 0)
