"""What the binding of hs_mla_prefix refuses of its tensors."""
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs

H, BF, F32 = hs.MLA_HEADS, torch.bfloat16, torch.float32


@pytest.fixture
def library(monkeypatch):
    """A library that is never called: reaching it raises KeyError."""
    monkeypatch.setattr(hs, "load", lambda: (_ for _ in ()).throw(KeyError("called")))


def call(**kw):
    a = dict(batch=2, q=torch.zeros(2, H, 576, dtype=BF), prefix=hs.hs_paged_rows(), max_length=64, prefix_length=None,
             sm_scale=1.0, own_out=None, own_lse=None, out=torch.zeros(2, H, 512, dtype=BF), out_type=hs.HS_TYPE_BF16,
             lse=torch.zeros(2, H), workspace=None, stream=0)
    a.update(kw)
    hs.hs_mla_prefix(1, **a)


def test_good_calls_pass(library):
    own = dict(own_out=torch.zeros(2, H, 512), own_lse=torch.zeros(2, H))
    for kw in ({}, own, dict(out=torch.zeros(2, H, 512), out_type=hs.HS_TYPE_F32), dict(batch=1), dict(batch=0),
               dict(q=1 << 20, out=1 << 20, lse=1 << 20), dict(prefix_length=torch.zeros(1, dtype=torch.int32)),
               dict(q=torch.zeros(2 * H * 576, dtype=BF)), dict(batch=-1), dict(out_type=7)):
        with pytest.raises(KeyError, match="called"):
            call(**kw)


@pytest.mark.parametrize("kw", [
    dict(out_type=hs.HS_TYPE_F32),  # would be written past its end
    dict(out=torch.zeros(2, H, 512)),
    dict(out=torch.zeros(2, H, 512, dtype=torch.float16)),
    dict(out=torch.zeros(1, H, 512, dtype=BF)),
    dict(out=torch.zeros(2, H, 576, dtype=BF)[..., :512]),
    dict(q=torch.zeros(2, H, 576)),
    dict(q=torch.zeros(2, H, 512, dtype=BF)),
    dict(q=torch.zeros(2, 576, H, dtype=BF).transpose(1, 2)),
    dict(lse=torch.zeros(2, H, dtype=BF)),
    dict(lse=torch.zeros(H)),
    dict(own_out=torch.zeros(2, H, 512, dtype=BF), own_lse=torch.zeros(2, H)),
    dict(own_out=torch.zeros(1, H, 512), own_lse=torch.zeros(2, H)),
    dict(own_out=torch.zeros(2, H, 512), own_lse=torch.zeros(2, H, dtype=torch.float64)),
    dict(prefix_length=torch.zeros(1, dtype=torch.int64)),
    dict(prefix_length=torch.zeros(0, dtype=torch.int32))])
def test_bad_tensors_are_refused(library, kw):
    with pytest.raises(ValueError, match="contiguous tensors"):
        call(**kw)
