"""hs_append and hs_mla_prefix read their positions and lengths when they run: arrays that the operation just before them in
the stream writes, with nothing in between. A kernel of this library starts while the one before it still runs and waits for
its end, so an index that was read ahead of that wait would be an old one."""
import math

import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g

    g.build()


def test_positions_and_lengths_from_the_call_before():
    """A resolve's slots serve as the positions of an append and as the length of a prefix, right behind it."""
    ctx, k, rounds, page = 512, 64, 24, 16
    g = torch.Generator().manual_seed(1)
    buf = hs.PoolBuffers(1, 1, ctx, k, k, 1152)
    buf.host.numpy()[:] = 0
    pool = buf.create()
    kv = torch.randn(k, 576, generator=g).to(torch.bfloat16).cuda()
    prefix_rows = torch.randn(k, 576, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(1, hs.MLA_HEADS, 576, generator=g).to(torch.bfloat16).cuda()
    freq, ids = torch.zeros(32, device="cuda"), torch.zeros(k, dtype=torch.int32, device="cuda")
    table = torch.arange(ctx // page, dtype=torch.int32, device="cuda")
    slots = torch.full((k,), -1, dtype=torch.int32, device="cuda")  # one buffer, rewritten by every resolve
    desc = hs.append_desc(kv, freq, slots, req_ids=ids)
    shared = hs.paged_rows(prefix_rows, torch.arange(k // page, dtype=torch.int32, device="cuda"), page)
    sel = [torch.randperm(ctx, generator=g)[:k].int().cuda() for _ in range(rounds)]
    rows = [torch.zeros(ctx, 576, dtype=torch.bfloat16, device="cuda") for _ in range(rounds)]
    outs = [(torch.zeros(1, hs.MLA_HEADS, 512, device="cuda"), torch.zeros(1, hs.MLA_HEADS, device="cuda"))
            for _ in range(rounds)]
    seen = torch.zeros(rounds, k, dtype=torch.int32, device="cuda")
    paged = [hs.paged_rows(r, table, page) for r in rows]
    n = hs.hs_mla_prefix_workspace(pool, 1, k)
    work = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    for with_copy in (True, False):  # the expected slots first, each taken right away; then the calls alone, once more
        hs.hs_pool_reset(pool)
        for r in rows:
            r.zero_()
        for i in range(rounds):
            hs.hs_step_begin(pool)
            hs.hs_resolve(pool, 0, 1, sel[i], k, slots)
            hs.hs_append(pool, 0, k, desc, paged[i], False)
            hs.hs_resolve(pool, 0, 1, sel[i], k, slots)
            hs.hs_mla_prefix(pool, 1, q, shared, k, slots[:1], 0.05, None, None, outs[i][0], hs.HS_TYPE_F32, outs[i][1], work)
            if with_copy:
                seen[i] = slots
        torch.cuda.synchronize()
        assert len({tuple(s) for s in seen.tolist()}) > rounds // 2
        for i, s in enumerate(seen.long()):
            want = torch.zeros_like(rows[i])
            want[s] = kv
            assert torch.equal(rows[i], want), i
            score = 0.05 * q[0].double() @ prefix_rows[: int(s[0])].double().t()
            if int(s[0]):
                assert (outs[i][1][0].double() - torch.logsumexp(score, -1)).abs().max() < 1e-3, i
            else:
                assert (outs[i][1] == -math.inf).all(), i
    assert hs.hs_get_error(pool) == 0
    buf.close()
