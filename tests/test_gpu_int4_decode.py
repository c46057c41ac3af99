"""hs_mla_decode_int4 against attention in 64 bits over the values that the 4-bit rows stand for.

Tolerance, from the arithmetic, for each output by itself. The rows' values are exact operands (a number times a scale has
seven bits). A query is exact too, but for values 2^-28 below the head's largest, off by at most 2^-40 of that one. 576
products accumulate in 32 bits, so a score is off by at most d = scale * 576 * 2^-23 * sum |q_i r_i| (a truncating
accumulator loses at most a unit of 2^-23 an addition) plus the argument's rounding, 2^-22 * |s|. A weight is then off by d +
2^-20 of itself (the exponential's own error is below 2^-21) and, in the value product, by its rounding to 16 bits: at most
2^-11 of it, or 2^-31 of a weight of the head's running maximum below the normal range. The output, a weighted mean, is off
by at most A * (2^-11 + 2 d + n 2^-23 + 2^-18), with A the same mean of |values| and n the length, plus n 2^-31 of the largest
value over the weights' sum (at least 2^-8 of the maximum's weight where the running maximum lags by 8 bits, which the sum
then exceeds by as much: the sum is at least the running maximum's weight), and its own rounding: 2^-8 of itself for bf16.
lse is off by at most d + n 2^-24 + 2^-18 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from oracle import int4_rows as ora

pytestmark = pytest.mark.gpu

H, DQK, DV = hs.MLA_HEADS, hs.MLA_D_QK, hs.MLA_D_V
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g

    g.build()


def model_rows(n, seed, size=1.0):
    """Rows as hs_append writes them, from N(0, 1) latents with some large channels."""
    g = np.random.default_rng(seed)
    z = (size * g.standard_normal((n, 512)) * np.exp(0.4 * g.standard_normal((1, 512)))).astype(np.float32)
    key = torch.from_numpy(g.standard_normal((n, 64)).astype(np.float32) * size).to(torch.bfloat16).view(torch.uint8).numpy()
    return np.concatenate([ora.pack(z), key], 1)


class Case:
    """A pool of two layers whose hot buffer and rows beside it hold rows, and lists that name them."""

    def __init__(self, batch, k, slots=64, away=0, seed=0, scale=SCALE, padded=0.0, garbage=True, size=1.0, qsize=1.0, max_batch=None):
        g = np.random.default_rng(seed)
        self.batch, self.k, self.scale, self.layer = batch, k, scale, 1
        mb = max_batch or batch
        self.buf = hs.PoolBuffers(2, mb, 32, slots, 8, 416)
        self.pool = self.buf.create()
        self.hot = model_rows(mb * slots, seed, size).reshape(mb, slots, 416)
        self.away = model_rows(max(away, 1), seed + 1, size)
        self.entries = np.empty((batch, k), np.int32)
        for b in range(batch):
            self.entries[b] = g.permutation(slots)[:k] if k <= slots else g.integers(0, slots, k)
        if away:
            far = g.random((batch, k)) < 0.4
            self.entries[far] = -2 - g.integers(0, away, (batch, k))[far]
        self.entries[g.random((batch, k)) < padded] = -1
        raw = self.hot.copy()
        if garbage:  # what no entry names holds scales and keys that are NaN and infinite
            for b in range(mb):
                off = np.ones(slots, bool)
                if b < batch:
                    off[self.entries[b][self.entries[b] >= 0]] = False
                raw[b][off] = 0xFF
        self.buf.hot.fill_(0xFF)
        self.buf.hot_view()[self.layer].copy_(torch.from_numpy(raw))
        self.away_d = torch.from_numpy(self.away).cuda() if away else None
        self.q = (qsize * torch.randn(batch, H, DQK, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).cuda()
        self.e = torch.from_numpy(self.entries).cuda()

    def run(self, out_type=hs.HS_TYPE_BF16, entries=None, stream=None, out=None, lse=None):
        if out is None:
            out = torch.full((self.batch, H, DV), math.nan, device="cuda",
                             dtype=torch.float32 if out_type == hs.HS_TYPE_F32 else torch.bfloat16)
            lse = torch.full((self.batch, H), math.nan, device="cuda")
        hs.hs_mla_decode_int4(self.pool, self.layer, self.batch, self.q, self.e if entries is None else entries, self.k,
                              self.away_d, 0 if self.away_d is None else self.away_d.shape[0], self.scale, out, out_type, lse,
                              stream=stream)
        return out, lse

    def rows(self, b):
        e = self.entries[b].astype(np.int64)
        raw = np.concatenate([self.hot[b], self.away])
        at = np.where(e >= 0, e, len(self.hot[b]) - 2 - e)
        ok = ((e >= 0) & (e < len(self.hot[b]))) | ((e <= -2) & (at < len(raw)) if self.away_d is not None else False)
        return raw[at[ok]]

    def check(self, out, lse, requests=None):
        torch.cuda.synchronize()
        assert hs.hs_get_error(self.pool) == 0
        for b in range(self.batch) if requests is None else requests:
            check_request(self.q[b], ora.values(self.rows(b)), self.scale, out[b], lse[b], b)

    def close(self):
        torch.cuda.synchronize()
        self.buf.close()


def check_request(q, rows, scale, out, lse, what=None):
    k = torch.from_numpy(rows).cuda()
    n, q = len(rows), q.double()
    if n:
        s = scale * q @ k.t()
        d = abs(scale) * 576 * 2.0 ** -23 * (q.abs() @ k.abs().t()).amax(-1, keepdim=True) + 2.0 ** -22 * s.abs().amax(-1, keepdim=True)
        want_lse = torch.logsumexp(s, -1, keepdim=True)
        w = (s - want_lse).exp()
        want, mean, most = w @ k[:, :DV], w @ k[:, :DV].abs(), k[:, :DV].abs().max()
    else:
        want_lse = torch.full((H, 1), -math.inf, dtype=torch.float64, device="cuda")
        want = mean = torch.zeros(H, DV, dtype=torch.float64, device="cuda")
        d, most = torch.zeros_like(want_lse), 0.0
    tol = mean * (2.0 ** -11 + 2 * d + n * 2.0 ** -23 + 2.0 ** -18) + n * 2.0 ** -31 * most
    if out.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    got, glse = out.double(), lse.double()[:, None]
    assert torch.isfinite(got).all(), what
    assert ((got - want).abs() <= tol + 1e-37).all(), (what, float(((got - want).abs() / (tol + 1e-37)).max()))
    if n == 0:
        assert (glse == -math.inf).all() and not got.any()
    else:
        assert ((glse - want_lse).abs() <= d + n * 2.0 ** -24 + 2.0 ** -18 + 2.0 ** -22 * want_lse.abs()).all(), what


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 193, 255, 256, 257, 511, 513, 1000])
@pytest.mark.parametrize("batch", [1, 3])
def test_lengths(batch, k):
    c = Case(batch, k, slots=1024, seed=k)
    c.check(*c.run())
    c.check(*c.run(hs.HS_TYPE_F32))
    c.close()


@pytest.mark.parametrize("batch,k", [(2, 2048), (1, 4097), (9, 1500), (9, 2100), (17, 700), (20, 513), (30, 1100), (39, 600),
                                     (77, 300), (80, 1300), (160, 70), (190, 500)])
def test_batches(batch, k):
    c = Case(batch, k, slots=600, away=50, seed=batch, padded=0.05)
    c.check(*c.run(hs.HS_TYPE_F32 if batch % 2 else hs.HS_TYPE_BF16), requests=sorted({0, 1, batch // 2, batch - 1} & set(range(batch))))
    c.close()


@pytest.mark.parametrize("padded", [0.1, 0.9, 1.0])
@pytest.mark.parametrize("k", [3, 300, 1200])
def test_padding(k, padded):
    """Entries of no row in every place; a request without a row; entries past the slots and past the rows beside them."""
    c = Case(4, k, slots=256, away=30, seed=3, padded=padded)
    c.entries[2] = -1
    c.entries[1][:: 5] = 256
    c.entries[1][1:: 5] = 2 ** 31 - 1
    c.entries[0][:: 7] = -2 - 30
    c.entries[0][1:: 7] = -2 ** 31
    c.e = torch.from_numpy(c.entries).cuda()
    for t in (hs.HS_TYPE_BF16, hs.HS_TYPE_F32):
        c.check(*c.run(t))
    c.close()


def test_leading_and_trailing_padding():
    """Whole tiles and parts of tiles without a row, at the front, in the middle and at the end."""
    c = Case(6, 1100, slots=512, seed=8)
    for b, (lo, hi) in enumerate([(0, 1), (1099, 1100), (300, 301), (256, 512), (0, 600), (64, 65)]):
        keep = c.entries[b, lo:hi].copy()
        c.entries[b] = -1
        c.entries[b, lo:hi] = keep
    c.e = torch.from_numpy(c.entries).cuda()
    for t in (hs.HS_TYPE_BF16, hs.HS_TYPE_F32):
        c.check(*c.run(t))
    c.close()


def test_placement_does_not_matter():
    """The same rows through slots, beside the hot buffer and from the history: bit-identical, and twice the same."""
    c = Case(3, 700, slots=800, seed=4, garbage=False)
    want = c.run(hs.HS_TYPE_F32)
    for t in c.run(hs.HS_TYPE_F32), :
        assert torch.equal(t[0], want[0]) and torch.equal(t[1], want[1])
    rows = torch.from_numpy(c.hot.reshape(-1, 416)).cuda()
    e = -2 - (c.e + 800 * torch.arange(3, device="cuda", dtype=torch.int32)[:, None])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    hs.hs_mla_decode_int4(c.pool, 0, 3, c.q, e.contiguous(), 700, rows, 2400, SCALE, out, hs.HS_TYPE_F32, lse)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    buf = hs.PoolBuffers(2, 3, 800, 16, 8, 416)
    buf.host.numpy()[3 * 800 * 416:] = c.hot.reshape(-1)
    hs.hs_mla_decode_int4_history(buf.create(), 1, 3, c.q, c.e, 700, SCALE, out, hs.HS_TYPE_F32, lse)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    c.check(*want)
    buf.close()
    c.close()


@pytest.mark.parametrize("scale", [1.0, 5.0, 1e-6, 0.0, -0.3])
def test_scales(scale):
    """Peaked and flat softmaxes (the output is rescaled again and again, or never), no scale, a negative one."""
    c = Case(2, 900, slots=900, seed=6, scale=scale)
    c.check(*c.run(hs.HS_TYPE_F32))
    c.close()


def test_rising_scores():
    """Every tile's largest score exceeds all before it by far: the output is rescaled at each."""
    c = Case(1, 1024, slots=1024, seed=7, garbage=False)
    s = torch.from_numpy(ora.values(c.hot[0])).cuda() @ c.q[0, 5].double()
    c.entries[0] = s.argsort().int().cpu().numpy()
    c.e = torch.from_numpy(c.entries).cuda()
    c.scale = 2.0
    c.check(*c.run(hs.HS_TYPE_F32))
    c.entries[0] = c.entries[0][::-1]
    c.e = torch.from_numpy(c.entries).cuda()
    c.check(*c.run(hs.HS_TYPE_F32))
    c.close()


@pytest.mark.parametrize("size,qsize", [(1e-4, 1e3), (2000.0, 1e-3), (1.0, 1e-30), (1.0, 1e30), (1e-4, 1e-4)])
def test_magnitudes(size, qsize):
    """Latents near the ends of the scales' range, queries far outside a half's."""
    c = Case(2, 300, slots=300, seed=9, size=size, qsize=qsize, scale=0.1 / (size * qsize))
    c.check(*c.run(hs.HS_TYPE_F32))
    c.close()


def test_queries_of_mixed_magnitude():
    """One value far above the rest of its head, a head of zeros, one of subnormal numbers."""
    c = Case(1, 300, slots=300, seed=10)
    c.q[0, 0, 3] = 1e4
    c.q[0, 1, 570] = -1e5
    c.q[0, 2] = 0
    c.q[0, 3] = torch.randint(-100, 100, (576,), device="cuda").to(torch.int16).abs().view(torch.bfloat16)
    c.check(*c.run(hs.HS_TYPE_F32))
    c.close()


def test_values_that_are_not_finite_stay_in_their_request():
    c = Case(3, 300, slots=300, seed=11)
    c.buf.hot_view()[1, 1, int(c.entries[1][7]), 256 + 3] = 255  # a block of NaN in a row of request 1
    c.q[2, 9, 100] = math.nan
    out, lse = c.run()
    c.check(out, lse, requests=[0])
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.isnan(out[2, 9]).all() and torch.isfinite(out[2, :9]).all() and torch.isfinite(out[2, 10:]).all()
    c.close()


def test_rows_past_4_gb():
    count = (1 << 32) // 416 + 500
    rows = torch.full((count, 416), 255, dtype=torch.uint8, device="cuda")
    some = model_rows(200, 12)
    at = np.concatenate([np.arange(100), np.arange(count - 100, count)])
    rows[torch.from_numpy(at).cuda()] = torch.from_numpy(some).cuda()
    buf = hs.PoolBuffers(1, 1, 16, 8, 8, 416)
    e = torch.from_numpy((-2 - at).astype(np.int32)).view(1, -1).cuda()
    q = torch.randn(1, H, DQK, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    out, lse = torch.empty(1, H, DV, device="cuda"), torch.empty(1, H, device="cuda")
    hs.hs_mla_decode_int4(buf.create(), 0, 1, q, e, 200, rows, count, SCALE, out, hs.HS_TYPE_F32, lse)
    check_request(q[0], ora.values(some), SCALE, out[0], lse[0])
    torch.cuda.synchronize()
    buf.close()


def test_two_calls_at_once_and_a_replayed_graph():
    c = [Case(5, 800, slots=800, seed=20 + i) for i in range(2)]
    want = [x.run() for x in c]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in c]
    graphs, outs = [], []
    for x, s in zip(c, streams):
        outs.append([torch.empty_like(t) for t in want[0]])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            x.run(out=outs[-1][0], lse=outs[-1][1])
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o[0].zero_(), o[1].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    c[0].entries[:] = np.roll(c[0].entries, 3, axis=1)  # another selection in the captured list's place
    c[0].entries[1, 100:] = -1
    c[0].e.copy_(torch.from_numpy(c[0].entries))
    graphs[0].replay()
    c[0].check(*outs[0])
    for x in c:
        x.check(*x.run())
        x.close()


def test_a_list_in_mapped_host_memory():
    c = Case(2, 500, slots=500, seed=30)
    mem = hs.HostBuffer(2 * 500 * 4)
    e = np.ctypeslib.as_array((np.ctypeslib.ctypes.c_int32 * 1000).from_address(mem.ptr)).reshape(2, 500)
    for shift in (0, 1):
        c.entries[:] = np.roll(c.entries, shift, axis=1)
        e[:] = c.entries
        c.check(*c.run(entries=mem.ptr))
    mem.close()
    c.close()


def test_a_decode_step():
    """Append, resolve, attend, read back: two steps of a captured graph whose second one evicts and rewrites."""
    batch, ctx, k = 4, 512, 48
    buf = hs.PoolBuffers(1, batch, ctx, 96, k, 416)
    host = model_rows(batch * ctx, 40).reshape(batch, ctx, 416)
    buf.host.numpy()[:] = host.reshape(-1)
    pool = buf.create()
    kv = torch.zeros(batch, 576, dtype=torch.bfloat16, device="cuda")
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32)).cuda()
    pos = torch.zeros(batch, dtype=torch.int32, device="cuda")
    topk = torch.zeros(batch, k, dtype=torch.int32, device="cuda")
    q = torch.zeros(batch, H, DQK, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty_like(topk)
    out, lse = torch.empty(batch, H, DV, device="cuda"), torch.empty(batch, H, device="cuda")
    values = torch.empty(batch, k, DQK, device="cuda")
    d = hs.append_desc(kv, freq, pos)

    def step():
        hs.hs_append(pool, 0, batch, d)
        hs.hs_step_begin(pool)
        hs.hs_resolve(pool, 0, batch, topk, k, slots)
        hs.hs_mla_decode_int4(pool, 0, batch, q, slots, k, None, 0, SCALE, out, hs.HS_TYPE_F32, lse)
        hs.hs_gather_values(pool, 0, batch, slots, k, None, 0, values, hs.HS_TYPE_F32)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    hs.hs_pool_reset(pool)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    g = torch.Generator().manual_seed(5)
    for n in range(4):
        kv.copy_(torch.randn(batch, 576, generator=g))
        pos.copy_(torch.randint(0, ctx, (batch,), generator=g))
        pick = torch.stack([torch.randperm(ctx, generator=g)[:k] for _ in range(batch)]).int()
        pick[:, 0] = pos.cpu()
        for b in range(batch):  # distinct tokens
            rest = [t for t in pick[b, 1:].tolist() if t != int(pos[b])]
            pick[b, 1:] = -1
            pick[b, 1:1 + len(rest)] = torch.tensor(rest, dtype=torch.int32)
        topk.copy_(pick)
        q.copy_(torch.randn(batch, H, DQK, generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        now = buf.host.numpy().reshape(batch, ctx, 416)
        for b in range(batch):
            t = pick[b][pick[b] >= 0].numpy()
            want = ora.values(now[b][t])
            assert np.array_equal(values[b].double().cpu().numpy()[pick[b].numpy() >= 0], want)
            check_request(q[b], want, SCALE, out[b], lse[b], (n, b))
            assert np.array_equal(now[b, int(pos[b]), :288], ora.pack(kv[b:b + 1, :512].float().cpu().numpy())[0])
        assert hs.hs_get_error(pool) == 0
    buf.close()


@pytest.mark.parametrize("batch,k", [(1, 200), (1, 3000), (20, 1100)])
def test_a_wait_that_runs_out(batch, k):
    """With the stall hook nothing is copied or multiplied: every role's wait runs out, the kernel returns, the error word says
    so, and the next call is right."""
    c = Case(batch, k, slots=300, seed=50)
    hs.hs_debug_attention(64, True)
    try:
        c.run()
        torch.cuda.synchronize()
    finally:
        hs.hs_debug_attention()
    assert hs.hs_get_error(c.pool, clear=True) == hs.HS_DEVERR_TIMEOUT
    c.check(*c.run(), requests=sorted({0, batch - 1}))
    c.close()


def test_captured_before_any_other_call():
    """Nothing has been called before in the process: the first call of each operator is captured, and replayed."""
    import os
    import subprocess
    import sys

    code = """
import sys
sys.path[:0] = [%r, %r]
import torch, hierarchical_sparse_attention_hs_gb300 as hs
import test_gpu_int4_decode as t, test_gpu_int4_rows as rows
cases = [t.Case(1, 2048, slots=2048, seed=60), t.Case(3, 40, slots=64, seed=61)]
outs = [[torch.zeros(c.batch, 128, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(c.batch, 128, device="cuda")] for c in cases]
vals = torch.zeros(3, 40, 576, device="cuda")
s = torch.cuda.Stream()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    for c, o in zip(cases, outs):
        c.run(out=o[0], lse=o[1])
    hs.hs_gather_values(cases[1].pool, 1, 3, cases[1].e, 40, None, 0, vals, hs.HS_TYPE_F32)
for _ in range(2):
    g.replay()
for c, o in zip(cases, outs):
    c.check(*o)
want = t.ora.values(cases[1].rows(2))
assert (vals[2].double().cpu().numpy() == want).all()
print("right")
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "right" in r.stdout, r.stderr[-2000:]


def test_back_to_back_calls_read_what_the_call_before_wrote():
    """Appends and attention by turns on one stream, without a pause: each attention sees the rows of the append before it."""
    batch, ctx = 3, 600
    buf = hs.PoolBuffers(1, batch, ctx, 16, 8, 416, noio=True)
    buf.host.numpy()[:] = model_rows(batch * ctx, 70).reshape(-1)
    buf.upload_noio()
    pool = buf.create()
    freq = torch.zeros(32, device="cuda")
    g = torch.Generator().manual_seed(7)
    steps = [torch.randn(batch * ctx, 576, generator=g).to(torch.bfloat16).cuda() for _ in range(4)]
    req = torch.arange(batch, dtype=torch.int32).repeat_interleave(ctx).cuda()
    pos = torch.arange(ctx, dtype=torch.int32).repeat(batch).cuda()
    topk = torch.stack([torch.randperm(ctx, generator=g) for _ in range(batch)]).int().cuda()
    q = torch.randn(batch, H, DQK, generator=g).to(torch.bfloat16).cuda()
    outs = [(torch.empty(batch, H, DV, device="cuda"), torch.empty(batch, H, device="cuda")) for _ in steps]
    descs = [hs.append_desc(kv, freq, pos, req_ids=req) for kv in steps]
    torch.cuda.synchronize()
    for d, (out, lse) in zip(descs, outs):
        hs.hs_append(pool, 0, batch * ctx, d, None, True)
        hs.hs_mla_decode_int4_history(pool, 0, batch, q, topk, ctx, SCALE, out, hs.HS_TYPE_F32, lse)
    torch.cuda.synchronize()
    for kv, (out, lse) in zip(steps, outs):
        kv = kv.float().cpu().numpy()
        for b in range(batch):
            mine = kv[b * ctx:(b + 1) * ctx]
            key = torch.from_numpy(mine[:, 512:]).to(torch.bfloat16).view(torch.uint8).numpy()
            rows = ora.values(np.concatenate([ora.pack(mine[:, :512]), key], 1))
            check_request(q[b], rows[topk[b].cpu().numpy()], SCALE, out[b], lse[b], b)
    buf.close()


def test_host_rows_rewritten_between_replays():
    """The history as the host leaves it before each replay, rows and list: nothing of the pass before is read again."""
    batch, k, ctx = 2, 900, 1000
    buf = hs.PoolBuffers(1, batch, ctx, 16, 8, 416)
    pool = buf.create()
    history = buf.host.numpy().reshape(batch, ctx, 416)
    mem = hs.HostBuffer(batch * k * 4)
    entries = np.ctypeslib.as_array((np.ctypeslib.ctypes.c_int32 * (batch * k)).from_address(mem.ptr)).reshape(batch, k)
    q = torch.randn(batch, H, DQK, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    out, lse = torch.empty(batch, H, DV, device="cuda"), torch.empty(batch, H, device="cuda")
    values = torch.empty(batch, k, 576, device="cuda")
    entries[:] = -1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_mla_decode_int4_history(pool, 0, batch, q, mem.ptr, k, SCALE, out, hs.HS_TYPE_F32, lse)
        hs.hs_gather_values_history(pool, 0, batch, mem.ptr, k, values, hs.HS_TYPE_F32)
    for seed in range(4):
        history[:] = model_rows(batch * ctx, 50 + seed).reshape(batch, ctx, 416)
        for b in range(batch):
            entries[b] = np.random.default_rng(seed + 9 * b).permutation(ctx)[:k]
        entries[1, 10 + 200 * seed:] = ctx + seed  # past the end: no row
        graph.replay()
        torch.cuda.synchronize()
        for b in range(batch):
            named = ora.values(history[b][entries[b][entries[b] < ctx]])
            check_request(q[b], named, SCALE, out[b], lse[b], (seed, b))
            assert np.array_equal(values[b, :len(named)].double().cpu().numpy(), named) and not values[b, len(named):].any()
    assert hs.hs_get_error(pool) == 0
    mem.close()
    buf.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,k", [(1, 65), (1, 700), (2, 2048), (1, 5000), (30, 1100), (77, 300), (80, 1300)])
def test_only_the_batch_is_written(batch, k, dtype):
    """Outputs beside the batch's, the rows and the list stay as they are, however a request is cut."""
    c = Case(batch, k, slots=700, seed=3, padded=0.1, max_batch=batch + 1)
    out, lse = torch.full((batch + 2, H, DV), 7.0, device="cuda", dtype=dtype), torch.full((batch + 2, H), 7.0, device="cuda")
    hot, e, q = c.buf.hot.clone(), c.e.clone(), c.q.clone()
    c.run(hs.HS_TYPE_F32 if dtype == torch.float32 else hs.HS_TYPE_BF16, out=out[1:-1], lse=lse[1:-1])
    c.check(out[1:-1], lse[1:-1], requests=sorted({0, batch - 1}))
    assert (out[[0, -1]] == 7).all() and (lse[[0, -1]] == 7).all()
    assert torch.equal(hot, c.buf.hot) and torch.equal(e, c.e) and torch.equal(q, c.q)
    c.close()


def test_a_large_batch_from_the_history():
    """More requests than the device holds at once, the last of them in a grid of their own: from the history as from hot slots."""
    batch, k, ctx = 80, 530, 600
    c = Case(batch, k, slots=ctx, seed=41, padded=0.02, garbage=False)
    buf = hs.PoolBuffers(2, batch, ctx, 16, 8, 416)
    pool = buf.create()
    buf.host.numpy().reshape(2, batch, ctx, 416)[1] = c.hot
    want = c.run()
    got = torch.empty_like(want[0]), torch.empty_like(want[1])
    hs.hs_mla_decode_int4_history(pool, 1, batch, c.q, c.e, k, SCALE, got[0], hs.HS_TYPE_BF16, got[1])
    c.check(*got, requests=[0, 1, 37, 75, 76, 77, 79])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and hs.hs_get_error(pool) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=got[0], lse=got[1])
    for seed in range(2):  # another list in the captured one's place
        c.entries = np.ascontiguousarray(np.roll(c.entries, 7, axis=0))
        c.e.copy_(torch.from_numpy(c.entries))
        graph.replay()
        c.check(*got, requests=[0, 74, 75, 76, 79])
    buf.close()
    c.close()
