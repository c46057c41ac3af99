"""hs_mla_prefix over the ways a batch is cut (whole requests, splits, both in one launch, more splits than a warp has lanes)
with either output type, in place and with one workspace for all; outputs and tolerances as in test_gpu_prefix.py."""
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from test_gpu_prefix import Case

pytestmark = pytest.mark.gpu

SPLIT_BYTES = hs.MLA_HEADS * (hs.MLA_D_V * 4 + 8)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g

    g.build()


@pytest.fixture(scope="module")
def pool():
    buf = hs.PoolBuffers(1, 2, 64, 16, 16, 1152)
    yield buf.create()
    torch.cuda.synchronize()
    assert hs.hs_get_error(buf.handle) == 0
    buf.close()


def test_one_workspace_for_every_call(pool):
    """A workspace of the bound's size serves a decode batch that shrinks and a prefix that grows."""
    n = hs.hs_mla_prefix_workspace_bound(pool, 100, 9001)
    work = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    assert hs.hs_mla_prefix_workspace(pool, 76, 9001) < hs.hs_mla_prefix_workspace(pool, 7, 9001) <= n
    for batch, length in ((100, 700), (76, 300), (40, 2000), (7, 9001), (1, 9001), (1, 500)):
        c = Case(batch, length, 64, seed=batch)
        c.check(*c.run(pool, work=work))
