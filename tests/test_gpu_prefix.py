"""hs_mla_prefix against attention in 64 bits: lengths, pages, holes, joins, types, workspaces, graphs.

Tolerance, from the arithmetic, for each output by itself. Scores: 576 exact products accumulate in 32 bits, so a score is
off by at most d = scale * 576 * 2^-23 * sum |q_i r_i| (a truncating accumulator loses at most a unit of 2^-23 an addition)
plus the argument's rounding, 2^-22 * |s|. A weight is then off by d + 2^-20 of itself (the exponential's own error is
below 2^-21) and, in the value product, by its rounding to bf16, at most 2^-8. The output, a weighted mean, is off by at
most A * (2^-8 + 2 d + n 2^-23 + 2^-18), with A the same mean of |values| and n its length, and its own rounding: 2^-8 of
itself for bf16. lse is off by at most d + n 2^-24 + 2^-18 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs

pytestmark = pytest.mark.gpu

H, DQK, DV = hs.MLA_HEADS, hs.MLA_D_QK, hs.MLA_D_V
SCALE = 1.0 / math.sqrt(192.0)


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


class Case:
    def __init__(self, batch, length, page=64, seed=0, holes=0.0, garbage=True, room=None, scale=SCALE, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.batch, self.length, self.page, self.scale = batch, length, page, scale
        self.room = length if room is None else room
        n = -(-self.room // page) if self.room else 1
        self.table = torch.randperm(n + 3, generator=g)[:n].int()
        self.table[torch.rand(n, generator=g) < holes] = -1
        self.rows = (spread * torch.randn((n + 3) * page, DQK, generator=g)).to(torch.bfloat16)
        self.q = torch.randn(batch, H, DQK, generator=g).to(torch.bfloat16).cuda()
        t = torch.arange(length)
        p = self.table[t // page].long() if length else t
        self.at = (p * page + t % page)[p >= 0]
        if garbage:  # what no token names holds NaN and infinities
            off = torch.ones(self.rows.shape[0], dtype=torch.bool)
            off[self.at] = False
            self.rows[off] = torch.tensor([math.nan, math.inf, -math.inf, 3e38]).repeat(DQK // 4).to(torch.bfloat16)
        self.rows, self.pages = self.rows.cuda(), self.table.cuda()
        self.own_out = self.own_lse = None

    def own(self, seed=5, shift=0.0):
        g = torch.Generator().manual_seed(seed)
        self.own_out = torch.randn(self.batch, H, DV, generator=g).cuda()
        self.own_lse = (torch.randn(self.batch, H, generator=g) + shift).cuda()
        return self

    def run(self, pool, out_type=hs.HS_TYPE_BF16, length_d=None, out=None, lse=None, work=None, stream=None):
        if out is None:
            out = torch.full((self.batch, H, DV), math.nan, device="cuda",
                             dtype=torch.float32 if out_type == hs.HS_TYPE_F32 else torch.bfloat16)
            lse = torch.full((self.batch, H), math.nan, device="cuda")
        n = hs.hs_mla_prefix_workspace(pool, self.batch, self.room)
        if work is None:
            work = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
        hs.hs_mla_prefix(pool, self.batch, self.q, hs.paged_rows(self.rows, self.pages, self.page), self.room, length_d,
                         self.scale, self.own_out, self.own_lse, out, out_type, lse, work, stream=stream)
        return out, lse

    def check(self, out, lse):
        torch.cuda.synchronize()
        k = self.rows[self.at.cuda()].double()
        n = len(self.at)
        for b0 in range(0, self.batch, 8):
            sl = slice(b0, b0 + 8)
            q = self.q[sl].double().reshape(-1, DQK)
            if n:
                s = self.scale * q @ k.t()
                d = self.scale * 576 * 2.0 ** -23 * (q.abs() @ k.abs().t()).amax(-1, keepdim=True) + 2.0 ** -22 * s.abs().amax(-1, keepdim=True)
                want_lse = torch.logsumexp(s, -1, keepdim=True)
                w = (s - want_lse).exp()
                want, mean = w @ k[:, :DV], w @ k[:, :DV].abs()
            else:
                want_lse = torch.full((q.shape[0], 1), -math.inf, dtype=torch.float64, device="cuda")
                want = mean = torch.zeros(q.shape[0], DV, dtype=torch.float64, device="cuda")
                d = torch.zeros_like(want_lse)
            if self.own_out is not None:
                ol, oo = self.own_lse[sl].double().reshape(-1, 1), self.own_out[sl].double().reshape(-1, DV)
                both = torch.logaddexp(want_lse, ol)
                wa = torch.where(want_lse == -math.inf, 0.0, (want_lse - both).exp())
                wb = torch.where(ol == -math.inf, 0.0, (ol - both).exp())
                oo = torch.where(wb > 0, oo, 0.0)
                want, mean, want_lse = wa * want + wb * oo, wa * mean + wb * oo.abs(), both
            tol = mean * (2.0 ** -8 + 2 * d + n * 2.0 ** -23 + 2.0 ** -18)
            if out.dtype == torch.bfloat16:
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
            got, glse = out[sl].double().reshape(-1, DV), lse[sl].double().reshape(-1, 1)
            assert torch.isfinite(got).all()
            assert ((got - want).abs() <= tol + 1e-37).all(), (b0, float(((got - want).abs() / (tol + 1e-37)).max()))
            none = want_lse == -math.inf
            assert torch.equal(glse == -math.inf, none)
            ltol = d + n * 2.0 ** -24 + 2.0 ** -18 + 2.0 ** -22 * want_lse.abs()
            assert ((glse - want_lse).abs() <= ltol)[~none].all()
            assert not got[none.flatten()].any()


@pytest.mark.parametrize("length", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000])
@pytest.mark.parametrize("batch,page", [(1, 64), (3, 16)])
def test_lengths(pool, batch, page, length):
    c = Case(batch, length, page, seed=length)
    c.check(*c.run(pool))


@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 256, 65536])
@pytest.mark.parametrize("length", [77, 700])
def test_pages(pool, page, length):
    c = Case(2, length, page, seed=page)
    c.check(*c.run(pool))


@pytest.mark.parametrize("batch,length", [(17, 500), (76, 300), (77, 129), (150, 200), (5, 9001)])
def test_batches(pool, batch, length):
    c = Case(batch, length, 32, seed=batch).own(shift=5.0)
    c.check(*c.run(pool))


@pytest.mark.parametrize("page", [1, 16, 128])
@pytest.mark.parametrize("holes", [0.3, 0.9, 1.0])
def test_missing_pages(pool, page, holes):
    for join in (False, True):
        c = Case(3, 1500, page, seed=9, holes=holes)
        c.check(*(c.own() if join else c).run(pool))


def test_pages_out_of_range_are_missing(pool):
    c = Case(2, 400, 16, seed=3, holes=0.2)
    gone = torch.nonzero(c.table < 0).flatten()
    for i, v in zip(gone, (c.rows.shape[0] // 16, (1 << 31) - 1, -(1 << 31), 1 << 27)):
        c.pages[i] = v
    c.check(*c.run(pool))
    c = Case(2, 400, 16, seed=3)  # rows that do not fill their last page: that page is missing
    last = c.rows.shape[0] // 16 - 1
    c.rows = c.rows[:-3]
    t = torch.arange(400)
    p = c.table[t // 16].long()
    c.at = (p * 16 + t % 16)[p != last]
    c.check(*c.run(pool))


@pytest.mark.parametrize("length", [0, 1, 63, 64, 200, 511, 512, 700, -5])
def test_length_on_the_device(pool, length):
    """The length is read when the kernel runs and clamped; the splits are laid out for the longest."""
    used = max(0, min(length, 512))
    c = Case(4, used, 16, seed=1, room=512).own()
    c.check(*c.run(pool, length_d=torch.tensor([length], dtype=torch.int32, device="cuda")))


def test_nothing_to_read(pool):
    c = Case(2, 0)
    out, lse = c.run(pool)
    c.check(out, lse)
    c.own()
    c.own_lse[1, 5] = -math.inf  # no rows of its own either, and what its output holds is not looked at
    c.own_out[1, 5] = math.nan
    out, lse = c.run(pool, hs.HS_TYPE_F32)
    c.check(out, lse)


@pytest.mark.parametrize("shift", [-200.0, 0.0, 6.0, 300.0])
def test_join(pool, shift):
    c = Case(3, 600, 32, seed=4).own(shift=shift)
    c.own_lse[0, 3] = -math.inf
    c.own_out[0, 3] = math.nan
    c.check(*c.run(pool, hs.HS_TYPE_F32))
    c.check(*c.run(pool))
    out, lse = c.own_out.clone(), c.own_lse.clone()  # in place
    want = c.run(pool, hs.HS_TYPE_F32)
    c.own_out, c.own_lse = out, lse
    got = c.run(pool, hs.HS_TYPE_F32, out=out, lse=lse)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_peaked_scores(pool):
    """A scale of 1 spreads the scores over hundreds of powers of two; rising ones move the maximum in every block."""
    c = Case(2, 2000, 64, seed=6, scale=1.0)
    c.check(*c.run(pool))
    c = Case(2, 1500, 64, seed=7, scale=1.0)
    lift = torch.linspace(0, 30, 1500)
    c.q[..., :DV] = 0
    c.rows[c.at.cuda(), DV:] = (torch.randn(1500, 64, generator=torch.Generator().manual_seed(1)) * 0.1 +
                                lift[:, None] * 0.02).to(torch.bfloat16).cuda()
    c.q[..., DV:] = c.q[..., DV:].abs()
    c.check(*c.run(pool))


@pytest.mark.parametrize("scale", [-0.05, 0.0, 1e-6])
def test_scales(pool, scale):
    """A negative scale turns the order of the scores round; with none every row weighs the same."""
    for holes in (0.0, 0.4):
        c = Case(2, 700, 16, seed=3, holes=holes)
        c.scale = abs(scale)
        if scale < 0:
            c.q = -c.q
        want = c.run(pool)
        c.check(*want)
        if scale < 0:
            c.q, c.scale = -c.q, scale
            got = c.run(pool)
            torch.cuda.synchronize()
            assert torch.allclose(got[0].float(), want[0].float(), rtol=2 ** -6, atol=2 ** -8)
            assert torch.allclose(got[1], want[1], rtol=1e-5, atol=1e-5)


def test_queries_and_units_of_many_shapes(pool):
    """Whole requests and splits in one launch (a batch past a multiple of the pairs), single tiles, and a prefix shorter
    than the splits that the longest one was cut into."""
    for batch, room, used in ((90, 1500, 1500), (230, 600, 600), (100, 3000, 200), (100, 3000, 0), (3, 30000, 700), (1, 300, 256)):
        c = Case(batch, used, 64, seed=batch, room=room).own(shift=3.0)
        c.check(*c.run(pool, length_d=torch.tensor([used], dtype=torch.int32, device="cuda")))


def test_first_call_under_capture():
    """Nothing has been called before in the process: the first call of each operator is captured, and replayed."""
    import subprocess
    import sys

    code = """
import sys, torch
sys.path[:0] = [%r, %r]
import hierarchical_sparse_attention_hs_gb300 as hs
from test_gpu_prefix import Case
buf = hs.PoolBuffers(1, 4, 64, 16, 16, 1152)
pool = buf.create()
c = Case(3, 500, 16, seed=1)
out, lse = torch.zeros(3, 128, 512, dtype=torch.bfloat16, device='cuda'), torch.zeros(3, 128, device='cuda')
work = torch.zeros(64 << 20, dtype=torch.uint8, device='cuda')
kv = torch.randn(4, 576).to(torch.bfloat16).cuda()
d = hs.append_desc(kv, torch.zeros(32).cuda(), torch.arange(4, dtype=torch.int32).cuda())
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    hs.hs_append(pool, 0, 4, d)
    hs.hs_mla_prefix(pool, 3, c.q, hs.paged_rows(c.rows, c.pages, 16), 500, None, c.scale, None, None, out, 0, lse, work)
g.replay()
c.check(out, lse)
got = torch.from_numpy(buf.host.numpy().reshape(4, 64, 1152)).view(torch.bfloat16)
assert all(torch.equal(got[i, i], kv[i].cpu()) for i in range(4))
print('captured')
""" % (str(__import__("pathlib").Path(__file__).resolve().parents[1]), str(__import__("pathlib").Path(__file__).resolve().parent))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_not_a_number_shows(pool):
    c = Case(2, 200, 16, seed=2)
    c.q[1, 7, 3] = math.nan
    out, lse = c.run(pool)
    torch.cuda.synchronize()
    assert torch.isnan(out[1, 7]).all() and torch.isnan(lse[1, 7])
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, :7]).all() and torch.isfinite(out[1, 8:]).all()


@pytest.mark.parametrize("page", [1, 2, 16])
def test_infinite_values_stay_where_they_are(pool, page):
    """An infinite latent of a row that is attended to: its score is infinite, so a head's outputs are all not a number
    (+inf) or only the column of the value is (-inf: weight 0 times infinity), as the formula has it. Rows next to pages that
    the pool does not hold change nothing."""
    c = Case(2, 300, page, seed=12, holes=0.4, garbage=False)
    c.q[1, :, 5] = 0.25  # the second request's scores of that row: the value's sign
    c.q[0, :, 5] = -0.25
    c.rows[c.at[17], 5] = math.inf
    out, lse = c.run(pool)
    torch.cuda.synchronize()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.isnan(out[0, :, 5]).all() and torch.isfinite(lse[0]).all()
    got, c.rows[c.at[17]] = out[0].double(), 0
    rest = torch.cat([c.at[:17], c.at[18:]]).cuda()
    k = c.rows[rest].double()
    s = c.scale * c.q[0].double() @ k.t()
    want = torch.softmax(s, -1) @ k[:, :DV]
    keep = torch.arange(DV, device="cuda") != 5
    assert ((got - want).abs()[:, keep] <= 2.1 * 2.0 ** -8 * (torch.softmax(s, -1) @ k[:, :DV].abs())[:, keep]).all()


def test_repeated_pages_and_results(pool):
    """A page may appear twice (its rows then count twice), and the same call gives the same bits."""
    c = Case(9, 900, 16, seed=8)
    c.pages[5] = c.pages[2]
    p = c.pages.cpu().long()[torch.arange(900) // 16]
    c.at = p * 16 + torch.arange(900) % 16
    a = c.run(pool)
    c.check(*a)
    b = c.run(pool)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rows_past_four_gigabytes(pool):
    """Row offsets pass 32 bits."""
    count, page = (5 << 30) // 1152 // 64 * 64, 64
    c = Case(2, 500, page, seed=11, garbage=False)
    rows = torch.empty(count, DQK, dtype=torch.bfloat16, device="cuda")
    table = count // page - 1 - torch.arange(len(c.table)).int() * 3
    at = table.long()[torch.arange(500) // page] * page + torch.arange(500) % page
    rows[at.cuda()] = c.rows[c.at.cuda()]
    c.rows, c.at = rows, at
    c.pages.copy_(table)
    c.check(*c.run(pool))


def test_streams_workspaces_and_graphs(pool):
    a, b = Case(3, 900, 16, seed=1), Case(3, 800, 16, seed=2, room=1024).own()
    want_a = a.run(pool)
    length = torch.tensor([800], dtype=torch.int32, device="cuda")
    b.check(*b.run(pool, length_d=length))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    works = [torch.empty(hs.hs_mla_prefix_workspace(pool, 3, c.room) or 16, dtype=torch.uint8, device="cuda") for c in (a, b)]
    o1 = (torch.zeros(3, H, DV, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, H, device="cuda"))
    o2 = (torch.zeros(3, H, DV, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, H, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(pool, out=o1[0], lse=o1[1], work=works[0], stream=s1)
        b.run(pool, out=o2[0], lse=o2[1], work=works[1], stream=s2, length_d=length)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(o1, want_a))
    b.check(*o2)
    # two graphs, captured with one workspace and replayed one after the other
    work = max(works, key=lambda w: w.numel())
    graphs = []
    for c, o, ln in ((a, o1, None), (b, o2, length)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(pool, out=o[0], lse=o[1], work=work, length_d=ln)
        graphs.append(g)
    for o in (*o1, *o2):
        o.zero_()
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(o1, want_a))
    b.check(*o2)
    # the same graph over a prefix that is shorter, then longer
    for n in (130, 1024, 0):
        length.fill_(n)
        graphs[1].replay()
        t = torch.arange(n)
        b.at = b.table[t // 16].long() * 16 + t % 16 if n else t
        rows = b.rows.clone()
        if n == 1024:  # these tokens have rows now
            bad = ~torch.isfinite(b.rows).all(-1)
            b.rows[bad] = 0.5
            torch.cuda.synchronize()
            graphs[1].replay()
        b.check(*o2)
        b.rows.copy_(rows)


def test_workspace_is_checked(pool):
    c = Case(1, 5000, 64)
    n = hs.hs_mla_prefix_workspace(pool, 1, 5000)
    if n == 0:
        pytest.skip("this size is not split on this device")
    for w in (None, torch.empty(n - 1, dtype=torch.uint8, device="cuda"),
              torch.empty(n + 256, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(hs.HsError) as e:
            if w is None:
                hs.hs_mla_prefix(pool, 1, c.q, hs.paged_rows(c.rows, c.pages, 64), 5000, None, SCALE, None, None,
                                 torch.empty(1, H, DV, dtype=torch.bfloat16, device="cuda"), hs.HS_TYPE_BF16,
                                 torch.empty(1, H, device="cuda"), None)
            else:
                c.run(pool, work=w)
        assert e.value.code == hs.HS_ERR_INVALID_ARG


def test_append_resolve_decode_and_prefix_together():
    """A decode step as a user makes it: a prompt's rows are appended to the ordinary pages that three requests share,
    each request's own rows to its history, the step's queries turn on the way; then a resolve, the sparse attention over
    each request's own selection, and the prefix attention that joins the two. Compared with attention over the union."""
    B, plen, ctx, k, page = 3, 200, 512, 16, 16
    g = torch.Generator().manual_seed(3)
    buf = hs.PoolBuffers(1, B, ctx, 64, k, 1152)
    buf.host.numpy()[:] = 0
    pool = buf.create()
    freq = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float().cuda()
    rows = torch.zeros(20 * page, DQK, dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(20, generator=g)[: -(-plen // page)].int().cuda()
    prompt = torch.randn(plen, DQK, generator=g).to(torch.bfloat16).cuda()
    shared = hs.paged_rows(rows, table, page)
    d = hs.append_desc(prompt, freq, torch.arange(plen, dtype=torch.int32).cuda(),
                       req_ids=torch.zeros(plen, dtype=torch.int32).cuda())
    hs.hs_append(pool, 0, plen, d, shared, False)
    n = 40  # each request's own tokens follow the prompt
    own = torch.randn(B * n, DQK, generator=g).to(torch.bfloat16).cuda()
    req = torch.arange(B).repeat_interleave(n).int().cuda()
    pos = (plen + torch.arange(n)).repeat(B).int().cuda()
    d2 = hs.append_desc(own, freq, pos, req_ids=req)
    hs.hs_append(pool, 0, B * n, d2, None, True)
    new = torch.randn(B, DQK, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(B, H, DQK, generator=g).to(torch.bfloat16).cuda()
    step_pos = torch.full((B,), plen + n, dtype=torch.int32, device="cuda")
    d3 = hs.append_desc(new, freq, step_pos, q_rope=q[..., DV:], q=q)
    hs.hs_append(pool, 0, B, d3, None, True)
    sel = torch.stack([plen + torch.randperm(n + 1, generator=g)[:k] for _ in range(B)]).int()
    topk, slots = sel.cuda(), torch.empty(B, k, dtype=torch.int32, device="cuda")
    hs.hs_step_begin(pool)
    hs.hs_resolve(pool, 0, B, topk, k, slots)
    part, plse = torch.empty(B, H, DV, device="cuda"), torch.empty(B, H, device="cuda")
    hs.hs_mla_decode(pool, 0, B, q, slots, k, None, 0, SCALE, part, plse)
    out, lse = torch.empty(B, H, DV, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H, device="cuda")
    w = torch.empty(hs.hs_mla_prefix_workspace(pool, B, plen) or 16, dtype=torch.uint8, device="cuda")
    hs.hs_mla_prefix(pool, B, q, shared, plen, None, SCALE, part, plse, out, hs.HS_TYPE_BF16, lse, w)
    torch.cuda.synchronize()
    assert hs.hs_get_error(pool) == 0
    hist = torch.from_numpy(buf.host.numpy().reshape(B, ctx, 1152)).view(torch.bfloat16).double()
    t = torch.arange(plen)
    pre = rows.cpu().double()[table.cpu().long()[t // page] * page + t % page]
    for b in range(B):
        keys = torch.cat((pre, hist[b][sel[b].long()]))
        s = SCALE * q[b].cpu().double() @ keys.t()
        want = torch.softmax(s, -1) @ keys[:, :DV]
        mean = torch.softmax(s, -1) @ keys[:, :DV].abs()
        # hs_mla_decode rounds its weights and sums the rounded ones: 2 * 2^-8 of the mean at most, and 2^-8 of the output
        assert ((out[b].cpu().double() - want).abs() <= 2.1 * 2.0 ** -8 * mean + 2.0 ** -8 * want.abs()).all()
        assert (lse[b].cpu().double() - torch.logsumexp(s, -1)).abs().max() <= 2.0 ** -7
    buf.close()


@pytest.mark.parametrize("batch,length", [(2, 3000), (160, 130)])
def test_a_wait_that_runs_out_is_reported(batch, length):
    """With the stall hook nothing is copied or multiplied; every role's wait runs out, the kernel returns, the error word
    says so, and the next call on the same pool is right (split and unsplit)."""
    buf = hs.PoolBuffers(1, 2, 64, 16, 16, 1152)
    p = buf.create()
    c = Case(batch, length, 64, seed=1)
    try:
        hs.hs_debug_attention(64, True)
        c.run(p)
        torch.cuda.synchronize()
    finally:
        hs.hs_debug_attention()
    assert hs.hs_get_error(p, clear=True) == hs.HS_DEVERR_TIMEOUT
    c.check(*c.run(p))
    assert hs.hs_get_error(p) == 0
    buf.close()
