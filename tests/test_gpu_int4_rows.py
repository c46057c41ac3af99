"""4-bit rows written by hs_append and read back, and rows of every format, by hs_gather_values.

Tolerance. Without a norm the latents are 32-bit numbers that the kernel has exactly, so the codes and scales are the
oracle's, bit for bit. With a norm a latent is off by less than e = 2^-14 of itself (512 additions of relative error 2^-24,
halved by the root, and a few more roundings): its block's scale is that of some largest magnitude within e, and its number
the nearest to a quotient off by e |z| / s, and by 2^-24 of itself for the division. Reading back: the product of a number
and its scale is exact in every type; of an e4m3 value and its scale it is rounded to 32 bits (2^-24) and to the type.
"""
import numpy as np
import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from oracle import append_rows as rows_of
from oracle import int4_rows as ora
from test_gpu_append import FREQ, TYPES, Setup

pytestmark = pytest.mark.gpu

E = 2.0 ** -14
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
CODES = {torch.bfloat16: hs.HS_TYPE_BF16, torch.float16: hs.HS_TYPE_F16, torch.float32: hs.HS_TYPE_F32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g

    g.build()


class Int4(Setup):
    """The setup of the append tests over 416-byte rows."""

    def __init__(self, n, **kw):
        super().__init__(n, 416, **kw)

    def check_rows(self, got):
        kv, want = self.expected()
        z, key = want[:, :512], want[:, 512:]
        pair = np.abs(kv[:, 512:])
        other = pair.reshape(-1, 32, 2)[..., ::-1].reshape(-1, 64) if self.interleaved else np.roll(pair, 32, axis=1)
        ktol = 2.0 ** -8 * np.abs(key) + 1.01 * 2.0 ** -20 * (pair + other) + 2.0 ** -133
        got = np.ascontiguousarray(got)
        q, codes, gkey = ora.unpack(got)
        assert (np.abs(gkey - key) <= ktol).all()
        if self.weight is None:
            assert np.array_equal(got[:, :288], ora.pack(z))
            return
        amax = np.abs(z.reshape(-1, 32, 16)).max(-1)
        assert ((codes >= ora.scale_code(amax * (1 - E))) & (codes <= ora.scale_code(amax * (1 + E)))).all()
        y = z / np.repeat(ora.scale_value(codes), 16, axis=1)
        assert (np.abs(q) <= 7).all()
        assert (np.abs(q - np.clip(y, -7, 7)) <= 0.5 + np.abs(y) * (E + 2.0 ** -23)).all()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_and_queries(dtype, interleaved, norm):
    s = Int4(37, dtype=TYPES[dtype], heads=5, norm=norm, interleaved=interleaved)
    s.run()
    s.check_all()
    assert hs.hs_get_error(s.pool) == 0


@pytest.mark.parametrize("n,heads,page", [(1, 128, 64), (1, 1, 1), (2, 16, 16), (33, 17, 128), (600, 31, 8)])
@pytest.mark.parametrize("norm", [False, True])
def test_sizes(n, heads, page, norm):
    s = Int4(n, heads=heads, page=page, requests=4, norm=norm)
    s.run()
    s.check_all()


def test_many_tokens():
    for dtype in TYPES.values():
        s = Int4(20000, dtype=dtype, requests=3, ctx=16384, page=64, norm=False)
        s.run(to_history=False)
        s.check_all(history=False)


@pytest.mark.parametrize("scale", [1e-7, 1e-5, 3e-4, 1.0, 900.0, 3e4, 1e30])
def test_magnitudes(scale):
    """Scales below the smallest, at the border of the format's two ranges, and cut off at the largest."""
    s = Int4(40, dtype=torch.float32, norm=False, scale=scale)
    s.run()
    s.check_all()


def test_ties_and_edges():
    """Latents at every half of a step, of scales with every fraction; whole blocks of zeros; equal largest magnitudes."""
    s = Int4(64, dtype=torch.bfloat16, norm=False)
    z = np.zeros((64, 32, 16), np.float32)
    for i in range(64):
        scale = (8 + i % 8) * 2.0 ** (i // 8 - 7)
        halves = np.arange(-6.5, 7.5, 1.0)  # 14 of them
        for b in range(32):
            z[i, b] = np.concatenate([halves, [7.0, -7.0]]) * scale if b % 4 else 0.0
    kv = torch.cat((torch.from_numpy(z.reshape(64, 512)), torch.randn(64, 64)), 1)
    assert torch.equal(kv[:, :512].to(torch.bfloat16).float(), kv[:, :512])
    s.kv = kv.to(torch.bfloat16).cuda()
    s.run()
    s.check_all()


def test_latents_that_are_not_finite():
    s = Int4(4, dtype=torch.float32, norm=False)
    s.kv[0, 5] = float("nan")
    s.kv[1, 40] = float("inf")
    s.kv[2, 511] = float("-inf")
    s.kv[3, 512] = float("inf")  # in the key: a value like any other
    s.run()
    i, at = s.live(), s.at()
    q, codes, key = ora.unpack(s.rows.cpu().numpy()[at])
    bad = np.zeros((4, 32), bool)
    bad[0, 0], bad[1, 2], bad[2, 31] = True, True, True
    assert np.array_equal(codes == 255, bad[i])
    fine = ~np.repeat(bad, 16, axis=1)
    want = ora.pack(np.where(fine, s.kv[:, :512].double().cpu().numpy(), 0.0))
    assert np.array_equal(codes[~bad[i]], want[:, 256:][i][~bad[i]])
    assert not np.isfinite(key[3]).all() and np.isfinite(key[:3]).all()
    v = read(s.pool, 1, 1, torch.from_numpy(-2 - at).int().view(1, -1).cuda(), s.rows)
    assert np.array_equal(np.isnan(v[0, :, :512].float().cpu().numpy()), ~fine)


def test_padding_ranges_and_missing_pages():
    s = Int4(50, heads=3)
    s.pos[::7] = -1
    s.pos[3], s.pos[10] = s.ctx, 1 << 30
    s.req[20] = 99
    s.run()
    assert hs.hs_get_error(s.pool, clear=True) == hs.HS_DEVERR_RANGE
    s.check_all()


def test_a_rewritten_token_reaches_its_hot_slot():
    s = Int4(6, requests=2, ctx=100)
    s.run(layer=0)
    topk = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    for r in range(2):
        mine = s.pos[s.req == r][:8]
        topk[r, : len(mine)] = mine.cuda()
    out = torch.empty_like(topk)
    hs.hs_step_begin(s.pool)
    hs.hs_resolve(s.pool, 0, 2, topk, 8, out)
    s.kv.mul_(-1.5)
    s.run(layer=0)
    v = read(s.pool, 0, 2, out)
    h = read(s.pool, 0, 2, topk, history=True)
    assert torch.equal(v, h)
    s.check_all(layer=0)


def test_another_stream_and_a_replayed_graph():
    s = Int4(20, heads=4, norm=False)
    d, p = s.desc(), s.paged()
    torch.cuda.synchronize()  # the inputs were made on the default stream
    side = torch.cuda.Stream()
    entries = torch.from_numpy(-2 - s.at()).int().cuda()
    got = torch.empty(20, 576, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        hs.hs_append(s.pool, 1, s.n, d, p, True)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            hs.hs_append(s.pool, 1, s.n, d, p, True)
            hs.hs_gather_values(s.pool, 1, 1, entries, 20, s.rows, s.rows.shape[0], got, hs.HS_TYPE_BF16)
    for seed in (1, 2):
        s.kv.copy_(torch.randn(20, 576, generator=torch.Generator().manual_seed(seed)))
        s.rows.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        s.check_all()
        assert np.array_equal(got.double().cpu().numpy(), ora.values(s.rows.cpu().numpy()[s.at()]))


# ---- reading back

def read(pool, layer, batch, entries, resident=None, dtype=torch.bfloat16, history=False, stream=None):
    k = entries.shape[1]
    dst = torch.full((batch, k, 576), float("nan"), dtype=dtype, device="cuda")
    if history:
        hs.hs_gather_values_history(pool, layer, batch, entries, k, dst, CODES[dtype], stream=stream)
    else:
        hs.hs_gather_values(pool, layer, batch, entries, k, resident, 0 if resident is None else resident.shape[0], dst,
                            CODES[dtype], stream=stream)
    return dst


def random_rows(n, row_bytes, seed):
    """Rows with every kind of content: codes and fp8 scales over their ranges, keys of any finite bf16 value."""
    g = np.random.default_rng(seed)
    key = g.integers(0, 1 << 16, (n, 64)).astype(np.uint16)
    key[(key >> 7 & 255) == 255] = 0x3F80
    key = key.view(np.uint8).reshape(n, 128)
    if row_bytes == 416:
        codes = g.integers(1, 16, (n, 256, 2))
        return np.concatenate([(codes[..., 0] | codes[..., 1] << 4).astype(np.uint8),
                               g.integers(1, ora.SCALE_CODES, (n, 32)).astype(np.uint8), key], 1)
    if row_bytes == 656:
        e = g.integers(0, 256, (n, 512)).astype(np.uint8)
        e[e & 127 == 127] = 0x38
        scale = (np.exp(g.standard_normal((n, 4)) * 3)).astype(np.float32)
        return np.concatenate([e, scale.view(np.uint8).reshape(n, 16), key], 1)
    lat = g.integers(0, 1 << 16, (n, 512)).astype(np.uint16)
    lat[(lat >> 7 & 255) == 255] = 0x3F80
    return np.concatenate([lat.view(np.uint8).reshape(n, 1024), key], 1)


def row_values(rows):
    rows = np.ascontiguousarray(rows)
    if rows.shape[1] == 416:
        return ora.values(rows)
    if rows.shape[1] == 656:
        s = np.ascontiguousarray(rows[:, 512:528]).view(np.float32).astype(np.float64)
        z = rows_of.e4m3_value(rows[:, :512]) * np.repeat(s, 128, axis=1)
        return np.concatenate([z, rows_of.bf16_value(np.ascontiguousarray(rows[:, 528:]).view(np.uint16))], 1)
    return rows_of.bf16_value(rows.view(np.uint16))


def check_values(got, want, row_bytes):
    """want: 64-bit values. Exact but for the rounding to the type (and, for fp8 rows, of the 32-bit product)."""
    dtype = got.dtype
    got = got.double().cpu().numpy().reshape(want.shape)
    with np.errstate(over="ignore"):
        if dtype == torch.float32 and row_bytes != 656:
            assert np.array_equal(got, want)
        elif dtype == torch.bfloat16 and row_bytes != 656:
            assert np.array_equal(got, want)
        else:
            rel = HALF_STEP[dtype] + (2.0 ** -24 if row_bytes == 656 else 0)
            tiny = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}[dtype]
            top = {torch.float16: 65520.0}.get(dtype, np.inf)
            inside = np.abs(want) * (1 + 2.0 ** -24) < top
            assert (np.abs(got - want)[inside] <= rel * np.abs(want[inside]) + tiny).all()
            assert (np.abs(got[~inside]) >= 65504).all()


@pytest.fixture(params=[416, 656, 1152])
def tiers(request):
    """A pool of two layers with random rows in the history, the hot buffer and rows beside them."""
    rb, layers, reqs, ctx, slots = request.param, 2, 3, 70, 24
    buf = hs.PoolBuffers(layers, reqs, ctx, slots, 16, rb)
    host = random_rows(layers * reqs * ctx, rb, 1)
    buf.host.numpy()[:] = host.reshape(-1)
    hot = random_rows(layers * reqs * slots, rb, 2)
    buf.hot.copy_(torch.from_numpy(hot.reshape(-1)))
    away = random_rows(11, rb, 3)
    yield dict(buf=buf, pool=buf.create(), rb=rb, ctx=ctx, slots=slots, reqs=reqs, host=host.reshape(layers, reqs, ctx, rb),
               hot=hot.reshape(layers, reqs, slots, rb), away=away, away_d=torch.from_numpy(away).cuda())
    torch.cuda.synchronize()
    buf.close()


def expected(t, layer, entries, history, away=True):
    out = np.zeros(entries.shape + (576,))
    src = (t["host"] if history else t["hot"])[layer]
    for b in range(entries.shape[0]):
        v = row_values(src[b])
        far = row_values(t["away"])
        for i, e in enumerate(entries[b]):
            if 0 <= e < len(v):
                out[b, i] = v[e]
            elif e <= -2 and not history and away and -2 - int(e) < len(far):
                out[b, i] = far[-2 - int(e)]
    return out


@pytest.mark.parametrize("dtype", list(CODES))
@pytest.mark.parametrize("k", [1, 3, 4, 5, 33, 200])
def test_read_back(tiers, dtype, k):
    t = tiers
    g = np.random.default_rng(k)
    for layer in (0, 1):
        for history in (False, True):
            n = t["ctx"] if history else t["slots"]
            e = g.integers(-14, n + 3, (t["reqs"], k)).astype(np.int32)
            e.flat[0] = [2 ** 31 - 1, -2 ** 31][layer]
            got = read(t["pool"], layer, t["reqs"], torch.from_numpy(e).cuda(), t["away_d"], dtype, history)
            check_values(got, expected(t, layer, e, history), t["rb"])
    e = g.integers(-14, t["slots"], (2, k)).astype(np.int32)  # fewer requests than the pool has, nothing resident
    check_values(read(t["pool"], 1, 2, torch.from_numpy(e).cuda(), None, dtype), expected(t, 1, e, False, False), t["rb"])
    assert hs.hs_get_error(t["pool"]) == 0


def test_lists_in_mapped_host_memory(tiers):
    t = tiers
    mem = hs.HostBuffer(3 * 40 * 4)
    e = np.ctypeslib.as_array((np.ctypeslib.ctypes.c_int32 * 120).from_address(mem.ptr)).reshape(3, 40)
    for seed in (1, 2):  # rewritten between calls
        e[:] = np.random.default_rng(seed).integers(-1, t["slots"], (3, 40))
        dst = torch.empty(3, 40, 576, dtype=torch.float32, device="cuda")
        hs.hs_gather_values(t["pool"], 0, 3, mem.ptr, 40, None, 0, dst, hs.HS_TYPE_F32)
        torch.cuda.synchronize()
        check_values(dst, expected(t, 0, e, False), t["rb"])
    mem.close()


def test_a_device_copy_of_the_history():
    buf = hs.PoolBuffers(1, 2, 50, 8, 8, 416, noio=True)
    host = random_rows(100, 416, 5)
    buf.host.numpy()[:] = host.reshape(-1)
    buf.upload_noio()
    buf.host.numpy()[:] = 0
    pool = buf.create()
    e = torch.randint(0, 50, (2, 77), dtype=torch.int32)
    got = read(pool, 0, 2, e.cuda(), history=True)
    want = ora.values(host).reshape(2, 50, 576)
    check_values(got, np.stack([want[b][e[b].numpy()] for b in range(2)]), 416)
    torch.cuda.synchronize()
    buf.close()


def test_rows_past_4_gb():
    """Resident rows whose bytes pass 32 bits, and outputs that do."""
    count = (1 << 32) // 416 + 100
    rows = torch.empty(count, 416, dtype=torch.uint8, device="cuda")
    some = random_rows(64, 416, 6)
    at = torch.cat((torch.arange(32), torch.arange(count - 32, count)))
    rows[at.cuda()] = torch.from_numpy(some).cuda()
    buf = hs.PoolBuffers(1, 1, 16, 8, 8, 416)
    pool = buf.create()
    e = (-2 - at).int().view(1, -1).cuda()
    check_values(read(pool, 0, 1, e, rows), ora.values(some)[None], 416)
    k = (1 << 32) // 1152 + 70
    long = e.repeat(1, -(-k // 64))[:, :k].contiguous()
    got = read(pool, 0, 1, long, rows)
    want = torch.from_numpy(ora.values(some)).cuda().to(torch.bfloat16)
    for lo in range(0, k, 1 << 20):
        m = min(1 << 20, k - lo)
        assert torch.equal(got[0, lo:lo + m], want[torch.arange(lo, lo + m, device="cuda") % 64])
    torch.cuda.synchronize()
    buf.close()
