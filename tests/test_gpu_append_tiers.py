"""hs_append into tiers that hold only some of the tokens: what is held is written and right, everything else stays."""
import numpy as np
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from test_gpu_append import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g

    g.build()


@pytest.mark.parametrize("lists", [1, 2])
def test_requests_without_a_list(lists):
    """Block tables with fewer lists than the pool has requests. What lies behind them in memory are page numbers too, of
    pages that nobody may write."""
    s = Setup(40)
    s.desc()
    every = s.pages.cuda()  # the table lies within it: words behind its end are page numbers
    d = s.desc()
    s.pages_d = every[:lists] if lists > 1 else every[0]
    hs.hs_append(s.pool, 1, s.n, d, s.paged(), True)
    torch.cuda.synchronize()
    s.pages[lists:] = -1
    at, rows = s.at(), s.rows.cpu().numpy()
    assert (at >= 0).any() and (at < 0).any()
    rest = np.setdiff1d(np.arange(rows.shape[0]), at[at >= 0])
    assert (rows[rest] == 9).all() and (rows[at[at >= 0]] != 9).any(axis=1).all()
    s.check_all(paged=False)
    assert hs.hs_get_error(s.pool) == 0
