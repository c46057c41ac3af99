"""Lists of the 4-bit operators as torch keeps them in page-locked host memory, and tensors that only look like such."""
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from test_gpu_int4_decode import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g

    g.build()


def test_a_page_locked_list():
    c = Case(3, 300, slots=400, seed=90)
    want, locked = c.run(), c.e.cpu().pin_memory()
    got = c.run(entries=locked)
    c.check(*got)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    values = [torch.empty(3, 300, 576, device="cuda") for _ in range(2)]
    for e, v in zip((c.e, locked), values):
        hs.hs_gather_values(c.pool, 1, 3, e, 300, None, 0, v, hs.HS_TYPE_F32)
    assert torch.equal(*values)
    c.close()


def test_an_ordinary_host_list_is_refused():
    c = Case(2, 64, slots=64, seed=91)
    for call in (lambda: c.run(entries=c.e.cpu()), lambda: c.run(out=torch.empty(2, 128, 512, dtype=torch.bfloat16), lse=torch.empty(2, 128))):
        with pytest.raises(ValueError, match="memory"):
            call()
    c.check(*c.run())
    c.close()
