"""hs_append into tiers that hold only some of the tokens (what is held is written and right, everything else stays), hot
slots of every kind of pool, and the codes of 656-byte rows down to the smallest."""
import numpy as np
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from test_append_tolerance import latents_within, spread_latents
from test_gpu_append import TYPES, Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g

    g.build()


def check_held(s):
    """The paged rows, where the pool holds some of the live tokens: theirs are right, the others are untouched."""
    at, rows = s.at(), s.rows.cpu().numpy()
    on = at >= 0
    assert on.any() and not on.all()
    kv, want = s.expected()
    s.expected = lambda: (kv[on], want[on])
    s.check_rows(rows[at[on]])
    del s.expected
    rest = np.setdiff1d(np.arange(rows.shape[0]), at[on])
    assert (rows[rest] == 9).all()


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
    check_held(s)
    s.check_all(paged=False)
    assert hs.hs_get_error(s.pool) == 0


@pytest.mark.parametrize("row_bytes", [1152, 656])
def test_rows_of_the_pages_that_are_held(row_bytes):
    s = Setup(50, row_bytes)
    s.pages[0, ::2] = -1
    s.pages[1, 3:6] = s.rows.shape[0] // s.page
    s.pages[2, 1], s.pages[2, 2] = (1 << 31) - 1, -(1 << 31)
    s.run()
    s.pages[s.pages >= s.rows.shape[0] // s.page] = -1
    check_held(s)
    s.check_all(paged=False)
    s = Setup(50, row_bytes)  # lists shorter than the context
    full = s.pages
    s.pages = full[:, :7].contiguous()
    s.run()
    s.pages = full.clone()
    s.pages[:, 7:] = -1
    check_held(s)
    s.check_all(paged=False)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_fp8_latents_down_to_the_smallest(dtype, norm):
    """Most codes are small against their group's largest, a third below the normal range: none is lost."""
    s = Setup(40, 656, TYPES[dtype], norm=norm)
    s.kv[:, :512] = torch.from_numpy(spread_latents(40, seed=3)).to(s.kv.dtype).cuda()
    s.run()
    z = s.expected()[1][:, :512]
    for got in (s.rows.cpu().numpy()[s.at()],
                s.buf.host.numpy().reshape(2, s.requests, s.ctx, 656)[1][s.req.numpy(), s.pos.numpy()]):
        assert latents_within(got, z, 1.01 * 2.0 ** -14 if norm else 0.0)
    s.check_all()


@pytest.mark.parametrize("noio", [False, True])
@pytest.mark.parametrize("row_bytes", [1152, 656])
def test_hot_slots_of_every_pool(row_bytes, noio):
    """Tokens in hot slots are rewritten there, in the history that the pool fetches from and in the paged rows by one call:
    the three hold the same bytes, of the new rows, and slots of other tokens keep the old ones."""
    s = Setup(24, row_bytes, requests=2, ctx=64, noio=noio)
    s.req[:] = torch.arange(24) // 12
    s.pos[:] = torch.arange(24) % 12
    s.run()
    topk = torch.full((2, 16), -1, dtype=torch.int32)
    topk[:, :8] = torch.randperm(12, generator=torch.Generator().manual_seed(2))[:8]
    topk[:, 8] = 40  # a token of the history that is not appended
    topk_d = topk.cuda()
    out = torch.empty_like(topk_d)
    hs.hs_step_begin(s.pool)
    hs.hs_resolve(s.pool, 1, 2, topk_d, 16, out)
    before = s.buf.hot_view().clone()
    s.kv.copy_(torch.randn(24, 576, generator=torch.Generator().manual_seed(5)))
    s.run()
    s.check_all(noio=noio)
    hot = s.buf.hot_view()
    src = (s.buf.noio_src.cpu().numpy() if noio else s.buf.host.numpy()).reshape(2, 2, 64, row_bytes)[1]
    rows, slots = s.rows.cpu().numpy(), out.cpu().long()
    changed = torch.zeros(hot.shape[:3], dtype=torch.bool)
    for r in range(2):
        for i in range(8):
            t, slot = int(topk[r, i]), int(slots[r, i])
            got = hot[1, r, slot].cpu().numpy()
            page = int(s.pages[r, t // s.page])
            assert (got == src[r, t]).all() and (got == rows[page * s.page + t % s.page]).all()
            changed[1, r, slot] = True
    keep = ~changed
    assert torch.equal(hot.cpu()[keep], before.cpu()[keep]) and (hot[1, 0, int(slots[0, 8])] == 7).all()
    assert hs.hs_get_error(s.pool) == 0


@pytest.mark.parametrize("page", [256, 65536])
def test_large_pages(page):
    s = Setup(60, ctx=700, page=page)
    s.run()
    s.check_all()


def test_positions_in_mapped_host_memory():
    """positions and req_ids are read over the host link and afresh by every call."""
    s = Setup(40, heads=3)
    s.desc()
    pos, req = s.pos.pin_memory(), s.req.pin_memory()
    d = hs.append_desc(s.kv, torch.from_numpy((10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32)).cuda(), pos,
                       req_ids=req, norm_weight=s.weight, norm_eps=1e-5, q_rope=s.q_rope, q=s.q)
    for i in range(3):
        if i:
            s.pos = torch.cat([torch.randperm(s.ctx, generator=torch.Generator().manual_seed(i))[:40].int()])
            s.pos[i] = -1
            pos.copy_(s.pos)
            s.rows.fill_(9)
            s.buf.host.numpy()[:] = 7
            s.q_before = s.q.clone()
            torch.cuda.synchronize()
        hs.hs_append(s.pool, 1, s.n, d, s.paged(), True)
        torch.cuda.synchronize()
        s.check_all()


def test_two_appends_at_once():
    """Two streams write different tokens of one pool at the same time."""
    s = Setup(240, heads=4)
    s.desc()
    half, streams, descs = s.n // 2, [torch.cuda.Stream() for _ in range(2)], []
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32)).cuda()
    for i in range(2):
        at = slice(i * half, (i + 1) * half)
        descs.append(hs.append_desc(s.kv[at], freq, s.pos_d[at], req_ids=s.req_d[at], norm_weight=s.weight, norm_eps=1e-5,
                                    q_rope=s.q_rope[at], q=s.q[at]))
    paged = s.paged()
    torch.cuda.synchronize()
    for _ in range(20):
        for d, stream in zip(descs, streams):
            hs.hs_append(s.pool, 1, half, d, paged, True, stream=stream)
    torch.cuda.synchronize()
    s.check_all()
