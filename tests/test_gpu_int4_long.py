"""hs_mla_decode_int4 over long lists, and over rows whose rotary keys are infinite, in every cut of a request. Tolerances as in
test_gpu_int4_decode.py: they hold for any length, and for the rows that are left where an infinite score has no weight."""
import math

import numpy as np
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from oracle import int4_rows as ora
from test_gpu_int4_decode import Case, check_request

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g

    g.build()


@pytest.mark.parametrize("batch,k", [(1, 131073), (3, 70001), (9, 20011)])
def test_long_lists(batch, k):
    """More tiles than a split's stages and phases ever were in the other tests; a list's rows come again and again."""
    c = Case(batch, k, slots=3000, away=500, seed=batch, padded=0.02)
    for t in (hs.HS_TYPE_BF16, hs.HS_TYPE_F32):
        c.check(*c.run(t), requests=sorted({0, batch - 1}))
    c.close()


@pytest.mark.parametrize("batch,k", [(1, 40), (1, 200), (2, 700), (2, 2048), (40, 600)])
def test_infinite_keys(batch, k):
    """An infinite value in the rotary key of a row gives the heads whose query has the other sign there a weight of 0, and the heads
    of the same sign no number."""
    c = Case(batch, k, slots=k, seed=k, garbage=False, scale=0.05)
    at, col = int(c.entries[0][k // 2]), 512 + 17
    raw = c.hot[0, at].copy()
    raw[288:].view(np.uint16)[col - 512] = 0x7F80
    c.buf.hot_view()[c.layer, 0, at].copy_(torch.from_numpy(raw))
    out, lse = c.run(hs.HS_TYPE_F32)
    torch.cuda.synchronize()
    sign = c.q[0, :, col].sign()
    assert (sign != 0).all() and (sign > 0).any() and (sign < 0).any()
    assert torch.isnan(out[0][sign > 0]).all() and not torch.isfinite(lse[0][sign > 0]).any()
    rest = ora.values(np.delete(c.rows(0), k // 2, axis=0))
    q, o, s = c.q[0].clone(), out[0].clone(), lse[0].clone()
    first = int((sign < 0).nonzero()[0])  # the heads that have no number are checked as another head
    for x in (q, o, s):
        x[sign > 0] = x[first].clone()
    check_request(q, rest, c.scale, o, s)
    c.check(out, lse, requests=range(1, batch))
    c.close()
