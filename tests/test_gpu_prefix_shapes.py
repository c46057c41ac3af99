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


def test_a_pool_without_rows(pool):
    """count = 0, and a count below one page: no page is held."""
    c = Case(3, 300, 16, seed=2).own()
    c.at = c.at[:0]
    for count in (0, 15):
        p = hs.paged_rows(c.rows, c.pages, 16)
        p.count = count
        out = torch.empty(3, hs.MLA_HEADS, hs.MLA_D_V, device="cuda")
        lse = torch.empty(3, hs.MLA_HEADS, device="cuda")
        work = torch.empty(hs.hs_mla_prefix_workspace_bound(pool, 3, 300) or 16, dtype=torch.uint8, device="cuda")
        hs.hs_mla_prefix(pool, 3, c.q, p, 300, None, c.scale, c.own_out, c.own_lse, out, hs.HS_TYPE_F32, lse, work)
        c.check(out, lse)


def test_outputs_past_four_gigabytes(pool):
    """20,000 requests: the offsets of their queries pass 2 GB, those of their outputs 5 GB."""
    batch, n, sample = 20000, 5, [0, 1, 9999, 16383, 16384, 19998, 19999]
    c = Case(len(sample), n, 16, seed=4)
    q = torch.zeros(batch, hs.MLA_HEADS, 576, dtype=torch.bfloat16, device="cuda")
    q[sample] = c.q
    out = torch.full((batch, hs.MLA_HEADS, hs.MLA_D_V), float("nan"), device="cuda")
    lse = torch.full((batch, hs.MLA_HEADS), float("nan"), device="cuda")
    assert hs.hs_mla_prefix_workspace(pool, batch, n) == 0
    hs.hs_mla_prefix(pool, batch, q, hs.paged_rows(c.rows, c.pages, 16), n, None, c.scale, None, None, out, hs.HS_TYPE_F32,
                     lse, None)
    c.check(out[sample], lse[sample])
    rest = torch.ones(batch, dtype=torch.bool, device="cuda")
    rest[sample] = False
    mean = c.rows[c.at.cuda(), :512].float().mean(0)  # scores of 0: every row weighs the same
    assert ((out[rest] - mean).abs().amax(dim=(0, 1)) <= 2.0 ** -18 * c.rows[c.at.cuda(), :512].float().abs().mean(0) + 1e-6).all()
    assert ((lse[rest] - torch.tensor(5.0).log().item()).abs() <= 2.0 ** -18).all()


def test_a_captured_decode_step():
    """Append, resolve, sparse attention and prefix attention as one graph, replayed for three steps whose positions,
    selections and prefix length are refilled in place; each step against attention over the union."""
    B, plen, ctx, k, page = 3, 200, 512, 16, 16
    H, DV = hs.MLA_HEADS, hs.MLA_D_V
    g = torch.Generator().manual_seed(7)
    buf = hs.PoolBuffers(1, B, ctx, 64, k, 1152)
    buf.host.numpy()[:] = 0
    pool = buf.create()
    freq = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float().cuda()
    rows = torch.randn(20 * page, 576, generator=g).to(torch.bfloat16).cuda()
    table = torch.randperm(20, generator=g)[: -(-plen // page)].int().cuda()
    shared = hs.paged_rows(rows, table, page)
    n = 40
    own = torch.randn(B * n, 576, generator=g).to(torch.bfloat16).cuda()
    d = hs.append_desc(own, freq, (plen + torch.arange(n)).repeat(B).int().cuda(), req_ids=torch.arange(B).repeat_interleave(n).int().cuda())
    hs.hs_append(pool, 0, B * n, d, None, True)
    new, q_in = torch.zeros(B, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, H, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros_like(q_in)
    pos, topk = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, k, dtype=torch.int32, device="cuda")
    length, slots = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(B, k, dtype=torch.int32, device="cuda")
    step = hs.append_desc(new, freq, pos, q_rope=q_in[..., DV:], q=q)
    out, lse = torch.empty(B, H, DV, device="cuda"), torch.empty(B, H, device="cuda")
    work = torch.empty(hs.hs_mla_prefix_workspace_bound(pool, B, plen) or 16, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.copy_(q_in)
        hs.hs_append(pool, 0, B, step, None, True)
        hs.hs_step_begin(pool)
        hs.hs_resolve(pool, 0, B, topk, k, slots)
        hs.hs_mla_decode(pool, 0, B, q, slots, k, None, 0, 192 ** -0.5, out, lse)
        hs.hs_mla_prefix(pool, B, q, shared, plen, length, 192 ** -0.5, out, lse, out, hs.HS_TYPE_F32, lse, work)
    for i, used in enumerate((200, 77, 0)):
        new.copy_(torch.randn(B, 576, generator=g))
        q_in.copy_(torch.randn(B, H, 576, generator=g))
        pos.fill_(plen + n + i)
        sel = torch.stack([plen + torch.randperm(n + 1 + i, generator=g)[:k] for _ in range(B)])
        sel[:, 0] = torch.where((sel == plen + n + i).any(1), sel[:, 0], plen + n + i)  # the step's own token is among them
        topk.copy_(sel)
        length.fill_(used)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        hist = torch.from_numpy(buf.host.numpy().reshape(B, ctx, 1152)).view(torch.bfloat16).double()
        t = torch.arange(used)
        pre = rows.cpu().double()[table.cpu().long()[t // page] * page + t % page]
        for b in range(B):
            keys = torch.cat((pre, hist[b][sel[b]]))
            assert hist[b][plen + n + i].any()
            s = 192 ** -0.5 * q[b].cpu().double() @ keys.t()
            p = torch.softmax(s, -1)
            # hs_mla_decode rounds its weights and sums the rounded ones: 2 * 2^-8 of the mean at most
            assert ((out[b].cpu().double() - p @ keys[:, :DV]).abs() <= 2.1 * 2.0 ** -8 * (p @ keys[:, :DV].abs())).all()
            assert (lse[b].cpu().double() - torch.logsumexp(s, -1)).abs().max() <= 2.0 ** -7
    assert hs.hs_get_error(pool) == 0
    buf.close()
