"""hs_append against the float64 oracle: row formats, types, rotations, tiers, padding, strides, graphs.

Tolerance, from the arithmetic. The norm's sum of 512 squares and the rotation are computed in 32 bits: a normed latent is
off by less than 2^-14 of itself (512 additions of relative error 2^-24, halved by the root, and a few more roundings); a
turned value by less than (|x| + |y|) 2^-20 (sine and cosine to a few units in the last place of 2^-24, the angle to 2^-24
of itself below a half turn). One rounding to bf16 adds at most 2^-8 of the value; one to e4m3 at most 2^-4 of it, or
2^-10 (half a step of 2^-9) below the normal range, in units of the scale.
"""
import numpy as np
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from oracle import append_rows as ora

pytestmark = pytest.mark.gpu

FREQ = (10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g

    g.build()


class Setup:
    """A pool of two layers, an ordinary paged pool beside it, and one append's inputs."""

    def __init__(self, n, row_bytes=1152, dtype=torch.bfloat16, heads=0, norm=True, interleaved=True, requests=3, ctx=300,
                 page=16, seed=0, noio=False, first=5, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.rb, self.heads, self.interleaved, self.page = n, row_bytes, heads, interleaved, page
        self.buf = hs.PoolBuffers(2, requests, ctx, 32, 16, row_bytes, noio=noio)
        self.buf.host.numpy()[:] = 7
        if noio:
            self.buf.upload_noio()
        self.pool = self.buf.create()
        self.req = torch.sort(torch.randint(0, requests, (n,), generator=g)).values.int()
        self.pos = torch.zeros(n, dtype=torch.int32)
        for r in range(requests):
            m = self.req == r
            self.pos[m] = torch.randperm(ctx - first, generator=g)[: int(m.sum())].int() + first
        self.kv = (scale * torch.randn(n, 576, generator=g)).to(dtype).cuda()
        self.weight = (1 + 0.3 * torch.randn(512, generator=g)).cuda() if norm else None
        self.q_rope = torch.randn(n, heads, 64, generator=g).to(dtype).cuda() if heads else None
        self.q = torch.randn(n, heads, 576, generator=g).to(torch.bfloat16).cuda() if heads else None
        self.q_before = self.q.clone() if heads else None
        per = -(-ctx // page)
        order = torch.randperm(requests * per + 4, generator=g).int()
        self.pages = order[: requests * per].view(requests, per).contiguous()
        self.rows = torch.full(((requests * per + 4) * page, row_bytes), 9, dtype=torch.uint8, device="cuda")
        self.ctx, self.requests = ctx, requests

    def desc(self, **kw):
        self.req_d, self.pos_d, self.pages_d = self.req.cuda(), self.pos.cuda(), self.pages.cuda()
        a = dict(req_ids=self.req_d, norm_weight=self.weight, norm_eps=1e-5, interleaved=self.interleaved,
                 q_rope=self.q_rope, q=self.q)
        a.update(kw)
        return hs.append_desc(self.kv, torch.from_numpy(FREQ).cuda(), self.pos_d, **a)

    def paged(self):
        return hs.paged_rows(self.rows, self.pages_d, self.page)

    def run(self, layer=1, paged=True, to_history=True, **kw):
        d = self.desc(**kw)
        hs.hs_append(self.pool, layer, self.n, d, self.paged() if paged else None, to_history)
        torch.cuda.synchronize()

    def live(self):
        ok = (self.pos >= 0) & (self.pos < self.ctx) & (self.req >= 0) & (self.req < self.requests)
        return torch.nonzero(ok).flatten().numpy()

    def at(self):
        """Row of the paged pool of each live token (-1: none)."""
        i = self.live()
        page = self.pages[self.req[i].long(), (self.pos[i] // self.page).long()]
        return torch.where(page >= 0, page * self.page + self.pos[i] % self.page, -1).numpy()

    def expected(self):
        i, w = self.live(), None if self.weight is None else self.weight.double().cpu().numpy()
        kv = self.kv.double().cpu().numpy()[i]
        return kv, ora.rows(kv, self.pos.numpy()[i], FREQ, self.interleaved, w, 1e-5)

    def check_rows(self, got):
        """got: the bytes [len(live)][row_bytes] that some tier holds for the live tokens."""
        kv, want = self.expected()
        z, key = want[:, :512], want[:, 512:]
        pair = np.abs(kv[:, 512:])
        other = pair.reshape(-1, 32, 2)[..., ::-1].reshape(-1, 64) if self.interleaved else np.roll(pair, 32, axis=1)
        ktol = 2.0 ** -8 * np.abs(key) + 1.01 * 2.0 ** -20 * (pair + other) + 2.0 ** -133
        got = np.ascontiguousarray(got)
        if self.rb == 1152:
            v = ora.bf16_value(got.view(np.uint16))
            assert (np.abs(v[:, :512] - z) <= (2.0 ** -8 + 2.0 ** -14 * 1.01) * np.abs(z) + 2.0 ** -133).all()
            assert (np.abs(v[:, 512:] - key) <= ktol).all()
            return
        sc = np.ascontiguousarray(got[:, 512:528]).view(np.float32).astype(np.float64)
        ref = ora.scales(z)
        assert (np.abs(sc - ref) <= 2.0 ** -13 * ref).all()
        y = z.reshape(-1, 4, 128) / ref[..., None]
        v = ora.e4m3_value(got[:, :512]).reshape(-1, 4, 128) * (sc / ref)[..., None]
        assert (np.abs(v - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + 448 * 2.0 ** -12).all()
        assert (np.abs(ora.bf16_value(np.ascontiguousarray(got[:, 528:]).view(np.uint16)) - key) <= ktol).all()

    def check_q(self):
        i = self.live()
        x = self.q_rope_in if hasattr(self, "q_rope_in") else self.q_rope
        x = x.double().cpu().numpy()[i]
        want = ora.turn(x, self.pos.numpy()[i], FREQ, self.interleaved)
        m = np.abs(x)
        o = m.reshape(*m.shape[:-1], 32, 2)[..., ::-1].reshape(m.shape) if self.interleaved else np.roll(m, 32, axis=-1)
        got = self.q.double().cpu().numpy()
        assert (np.abs(got[i][..., 512:] - want) <= 2.0 ** -8 * np.abs(want) + 1.01 * 2.0 ** -20 * (m + o)).all()
        before = self.q_before.double().cpu().numpy()
        assert np.array_equal(got[..., :512], before[..., :512])
        dead = np.setdiff1d(np.arange(self.n), i)
        assert np.array_equal(got[dead], before[dead])

    def check_all(self, layer=1, history=True, paged=True, noio=False):
        i, at = self.live(), self.at()
        if paged:
            rows = self.rows.cpu().numpy()
            on = at >= 0
            if on.all():
                self.check_rows(rows[at])
            rest = np.setdiff1d(np.arange(rows.shape[0]), at[on])
            assert (rows[rest] == 9).all()
        if history:
            src = self.buf.noio_src.cpu().numpy() if noio else self.buf.host.numpy()
            src = src.reshape(2, self.requests, self.ctx, self.rb)
            assert (src[1 - layer] == 7).all()
            req, pos = self.req.numpy()[i], self.pos.numpy()[i]
            self.check_rows(src[layer][req, pos])
            touched = np.zeros((self.requests, self.ctx), bool)
            touched[req, pos] = True
            assert (src[layer][~touched] == 7).all()
        if self.q is not None:
            self.check_q()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("row_bytes", [1152, 656])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_and_queries(dtype, row_bytes, interleaved, norm):
    s = Setup(37, row_bytes, TYPES[dtype], heads=5, norm=norm, interleaved=interleaved)
    s.run()
    s.check_all()
    assert hs.hs_get_error(s.pool) == 0


@pytest.mark.parametrize("n,heads,page", [(1, 128, 64), (1, 1, 1), (2, 16, 16), (3, 17, 32), (33, 128, 128), (600, 31, 8),
                                          (900, 0, 1)])
def test_sizes(n, heads, page):
    s = Setup(n, heads=heads, page=page, requests=4)
    s.run()
    s.check_all()


def test_many_tokens_loop_over_the_grid():
    """More rows and more query items than the grid has warps."""
    for rb in (1152, 656):
        s = Setup(20000, rb, heads=16 if rb == 656 else 0, requests=3, ctx=16384, page=64)
        s.run(to_history=False)
        s.check_all(history=False)


def test_padding_and_out_of_range():
    s = Setup(40, heads=3)
    s.pos[[0, 7, 39]] = -1
    s.pos[11] = -(1 << 31)
    s.run()
    s.check_all()
    assert hs.hs_get_error(s.pool) == 0
    s = Setup(40, heads=3)
    s.pos[3], s.pos[9], s.req[20], s.req[21] = s.ctx, (1 << 31) - 1, s.requests, -1
    s.run()
    s.check_all()
    assert hs.hs_get_error(s.pool, clear=True) == hs.HS_DEVERR_RANGE
    s = Setup(9)
    s.pos[:] = -1
    s.run()
    assert (s.rows == 9).all() and (torch.from_numpy(s.buf.host.numpy()) == 7).all()


def test_pages_that_the_pool_does_not_hold():
    s = Setup(50)
    s.pages[0, ::2] = -1
    s.pages[1, 3:6] = s.rows.shape[0] // s.page  # just behind the rows
    s.pages[2, 1] = (1 << 31) - 1
    s.pages[2, 2] = -(1 << 31)
    keep = s.pages.clone()
    s.run()
    s.pages[s.pages >= s.rows.shape[0] // s.page] = -1
    s.check_all()
    assert torch.equal(s.pages_d.cpu(), keep)
    s = Setup(50)  # a list shorter than the context
    full = s.pages
    s.pages = s.pages[:, :7].contiguous()
    s.run()
    s.pages = full.clone()
    s.pages[:, 7:] = -1
    s.check_all()


def test_tiers_alone_and_no_request_ids():
    s = Setup(3, heads=2)
    s.req = torch.arange(3, dtype=torch.int32)  # token i is request i
    s.run(req_ids=None)
    s.check_all()
    s = Setup(8)
    s.run(paged=False)
    s.check_all(paged=False)
    assert (s.rows == 9).all()
    s = Setup(8, heads=4)
    s.run(paged=False, to_history=False)  # the queries alone
    s.check_q()
    assert (s.rows == 9).all() and (torch.from_numpy(s.buf.host.numpy()) == 7).all()
    s = Setup(8, noio=True)  # a pool with a device copy as its row source
    s.run()
    s.check_all(noio=True)
    assert (torch.from_numpy(s.buf.host.numpy()) == 7).all()


def test_far_positions():
    """Angles of positions beyond a million, where a 32-bit product is off by a tenth of a radian and more."""
    s = Setup(64, heads=2, requests=1, ctx=1 << 20, page=64, first=(1 << 20) - 700, norm=False)
    s.run(to_history=False)
    s.check_all(history=False)


def test_rows_past_four_gigabytes():
    """Row offsets of the paged pool pass 32 bits."""
    s = Setup(40, requests=2, ctx=128, page=64)
    count = (5 << 30) // 1152 // 64 * 64
    s.rows = torch.empty((count, 1152), dtype=torch.uint8, device="cuda")
    s.pages = (count // 64 - 1 - torch.arange(4).int() * 3).view(2, 2).contiguous()
    s.rows[-700:] = 9
    s.run()
    i = s.at()
    assert int(i.min()) * 1152 > 1 << 32
    s.check_rows(s.rows[torch.from_numpy(i).cuda()].cpu().numpy())
    rest = np.setdiff1d(np.arange(count - 700, count), i)
    assert (s.rows[torch.from_numpy(rest).cuda()] == 9).all()


def test_values_at_the_edges():
    s = Setup(6, 656, torch.float32, norm=False)
    s.kv[0] = 0
    s.kv[1, :512] = 0
    s.kv[1, 5] = 1e-42
    s.kv[2] *= 1e30
    s.kv[3, :512] = 2.0 ** -120
    s.kv[4, :512] = 448.0
    s.run()
    i = s.live()
    got = s.rows.cpu().numpy()[s.at()]
    assert np.isfinite(ora.e4m3_value(got[:, :512])).all()
    s.check_rows(got)
    assert len(i) == 6
    s = Setup(5, norm=True)  # a latent of zeros under the norm
    s.kv[2, :512] = 0
    s.run()
    s.check_all()


def test_strides_and_in_place_queries():
    s = Setup(21, heads=6)
    wide = torch.randn(21, 2112, dtype=torch.float32).to(torch.bfloat16).cuda()  # a fused projection's output
    wide[:, 1536:] = s.kv
    s.kv = wide[:, 1536:]
    qwide = torch.randn(21, 8, 192, dtype=torch.float32).to(torch.bfloat16).cuda()
    qwide[:, :6, 128:] = s.q_rope
    s.q_rope = qwide[:, :6, 128:]
    big = torch.randn(21, 7, 640).to(torch.bfloat16).cuda()
    big[:, :6, :576] = s.q
    s.q = big[:, :6, :576]
    rest = big.clone()
    s.run()
    s.check_all()
    assert torch.equal(big[:, 6], rest[:, 6]) and torch.equal(big[..., 576:], rest[..., 576:])
    for interleaved in (False, True):
        s = Setup(9, heads=20, interleaved=interleaved)
        s.q_rope_in = s.q[..., 512:].clone()
        s.q_rope = s.q[..., 512:]
        s.run()
        s.check_all()


def test_hot_slots_follow_a_rewrite():
    """A token that occupies a hot slot is rewritten there too: a later gather through out_slots serves the new row."""
    s = Setup(12, requests=2, ctx=64)
    s.req[:], s.pos[:] = 0, torch.arange(12, dtype=torch.int32)
    s.run()
    topk = torch.full((2, 16), -1, dtype=torch.int32)
    topk[0, :8] = torch.arange(8)
    topk = topk.cuda()
    out = torch.empty_like(topk)
    hs.hs_step_begin(s.pool)
    hs.hs_resolve(s.pool, 1, 2, topk, 16, out)
    a, b = (torch.zeros(2, 16, 1152, dtype=torch.uint8, device="cuda") for _ in range(2))
    for seed in (1, 2):
        s.kv.copy_(torch.randn(12, 576, generator=torch.Generator().manual_seed(seed)))
        s.run(paged=False)
        hs.hs_gather(s.pool, 1, 2, out, 16, a)
        hs.hs_gather_history(s.pool, 1, 2, topk, 16, b)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
        s.check_rows(a[0, :8].cpu().numpy()) if len(s.live()) == 8 else s.check_rows(
            np.concatenate([a[0, :8].cpu().numpy(), s.buf.host.numpy().reshape(2, 2, 64, 1152)[1, 0, 8:12]]))
    # the other layer's slots of the same tokens are its own
    assert (s.buf.hot_view()[0] == 0).all()


def test_other_stream_and_captured_graph():
    s = Setup(16, heads=4)
    side = torch.cuda.Stream()
    d, p = s.desc(), None
    p = s.paged()
    torch.cuda.synchronize()
    hs.hs_append(s.pool, 1, 16, d, p, True, stream=side)
    side.synchronize()
    s.check_all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_append(s.pool, 1, 16, d, p, True)
    for seed in (3, 4):
        g = torch.Generator().manual_seed(seed)
        s.kv.copy_(torch.randn(16, 576, generator=g))
        s.q_rope.copy_(torch.randn(16, 4, 64, generator=g))
        s.pos = torch.randperm(s.ctx, generator=g)[:16].int()
        s.pos[5] = -1
        s.pos_d.copy_(s.pos)
        s.rows.fill_(9)
        s.buf.host.numpy()[:] = 7
        s.q_before = s.q.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.check_all()
