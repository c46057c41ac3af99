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


@pytest.mark.parametrize("out_type", [hs.HS_TYPE_BF16, hs.HS_TYPE_F32])
@pytest.mark.parametrize("batch,length", [(1, 9001), (2, 9001), (1, 40000)])
def test_more_splits_than_a_warp_has_lanes(pool, batch, length, out_type):
    """A lane of the joining kernel then holds the weights of several splits; of a list with missing pages too, and with a
    prefix that leaves most of the splits without a tile."""
    for holes in (0.0, 0.5):
        c = Case(batch, length, 64, seed=length, holes=holes)
        assert hs.hs_mla_prefix_workspace(pool, batch, length) // SPLIT_BYTES // batch > 32
        c.check(*c.run(pool, out_type))
        c.own(shift=4.0)
        c.check(*c.run(pool, out_type))
    c = Case(batch, 700, 64, seed=1, room=length)
    c.check(*c.run(pool, out_type, length_d=torch.tensor([700], dtype=torch.int32, device="cuda")))


SHAPES = {"whole": [(17, 500), (76, 300), (150, 200)], "split": [(3, 600), (9, 3000)], "mixed": [(90, 1500), (100, 2047)]}


def cut(pool, batch, length):
    n = hs.hs_mla_prefix_workspace(pool, batch, length) // SPLIT_BYTES
    return "whole" if n == 0 else "split" if n % batch == 0 else "mixed"


@pytest.mark.parametrize("kind,batch,length", [(k, *s) for k, v in SHAPES.items() for s in v])
def test_fp32_outputs_and_in_place(pool, kind, batch, length):
    """Both output types with and without own rows, then the own outputs themselves as the outputs: the same bits."""
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert cut(pool, batch, length) == kind
    c = Case(batch, length, 32, seed=batch)
    c.check(*c.run(pool, hs.HS_TYPE_F32))
    c.check(*c.run(pool))
    c.own(shift=4.0)
    c.own_lse[0, 3] = c.own_lse[batch - 1, 127] = -float("inf")  # heads without own rows: what their output holds is not read
    c.own_out[0, 3] = c.own_out[batch - 1, 127] = float("nan")
    c.own_lse[batch // 2, 64:96] = -float("inf")  # a whole warp's heads
    c.check(*c.run(pool))
    want = c.run(pool, hs.HS_TYPE_F32)
    c.check(*want)
    got = c.run(pool, hs.HS_TYPE_F32, out=c.own_out, lse=c.own_lse)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
