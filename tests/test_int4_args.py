"""hs_gather_values, hs_mla_decode_int4, their history forms and 4-bit rows in hs_append: a good call reaches its launch and a
call that differs from it in one argument is refused, before anything is launched (the stand-in runtime of
test_args_fake_runtime.py); and what the binding refuses of tensors."""
import ctypes

import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from test_args_fake_runtime import under  # noqa: F401 (a fixture)

CALLS = """
def with_pool(f, p, **kw):
    block = p or pool(row_bytes=416)
    return code(lambda: f(ctypes.addressof(block), kw))


def values(p=None, history=False, **kw):
    a = {**dict(layer=0, batch=2, idx=A, k=5, rows=A, count=10, dst=A, type=hs.HS_TYPE_BF16), **kw}
    def call(block, _):
        lib = hs.load()
        rc = (lib.hs_gather_values_history(block, a["layer"], a["batch"], a["idx"], a["k"], a["dst"], a["type"], 0) if history else
              lib.hs_gather_values(block, a["layer"], a["batch"], a["idx"], a["k"], a["rows"], a["count"], a["dst"], a["type"], 0))
        if rc:
            raise hs.HsError(rc, "hs_gather_values")
    return with_pool(call, p)


def decode(p=None, history=False, **kw):
    a = {**dict(layer=0, batch=2, q=A, idx=A, k=5, rows=A, count=10, out=A, type=hs.HS_TYPE_BF16, lse=A), **kw}
    def call(block, _):
        lib = hs.load()
        rc = (lib.hs_mla_decode_int4_history(block, a["layer"], a["batch"], a["q"], a["idx"], a["k"], 0.1, a["out"], a["type"],
                                             a["lse"], 0) if history else
              lib.hs_mla_decode_int4(block, a["layer"], a["batch"], a["q"], a["idx"], a["k"], a["rows"], a["count"], 0.1,
                                     a["out"], a["type"], a["lse"], 0))
        if rc:
            raise hs.HsError(rc, "hs_mla_decode_int4")
    return with_pool(call, p)


def other_device(block):
    at = ctypes.addressof(block) + ctypes.sizeof(hs.hs_pool_desc) + ctypes.sizeof(hs.hs_meta_layout)
    ctypes.memmove(at, (ctypes.c_int32 * 2)(1, 152), 8)
    return block


def empty(f, **kw):  # a call with nothing to do: no launch, no error
    before = fake.fake_launches()
    block = pool(row_bytes=416)
    rc = f(ctypes.addressof(block), **kw)
    return [rc, fake.fake_launches() - before]
"""


def test_good_calls_and_refusals(under):  # noqa: F811
    got = under(CALLS + """
both = dict(values=values, decode=decode)
got = {}
for name, f in both.items():
    common = [dict(layer=-1), dict(layer=2), dict(batch=-1), dict(batch=5), dict(idx=None), dict(idx=A + 2), dict(k=-1), dict(type=-1),
              dict(type=3)]
    own = ([dict(dst=None), dict(dst=A + 8), dict(k=1 << 30)] if name == "values" else
           [dict(q=None), dict(q=A + 8), dict(out=None), dict(out=A + 8), dict(lse=None), dict(lse=A + 2), dict(k=(1 << 30) + 1),
            dict(type=hs.HS_TYPE_F16)])
    got[name] = dict(
        good=[f(), f(history=True), f(rows=None, count=0), f(layer=1), f(batch=4), f(batch=1, k=1), f(k=100000), f(idx=A + 4),
              f(type=hs.HS_TYPE_F32)],
        bad=[f(**kw) for kw in common + own] + [f(history=True, **kw) for kw in common + own],
        rows=[f(count=-1), f(rows=A + 8), f(rows=A + 16)],
        format=[f(p=pool(row_bytes=b)) for b in (1152, 656, 416, 1024, 288)],
        device=[f(p=other_device(pool(row_bytes=416))), f(p=other_device(pool(row_bytes=416)), history=True)])
got["values"]["most"] = [values(batch=1, k=1 << 30), values(batch=2, k=1 << 29), values(batch=3, k=1 << 29)]
got["decode"]["most"] = [decode(k=1 << 30), decode(batch=4, k=1 << 30)]
lib = hs.load()
got["null"] = [lib.hs_gather_values(0, 0, 1, A, 1, 0, 0, A, 0, 0), lib.hs_gather_values_history(0, 0, 1, A, 1, A, 0, 0),
               lib.hs_mla_decode_int4(0, 0, 1, A, A, 1, 0, 0, 0.1, A, 0, A, 0), lib.hs_mla_decode_int4_history(0, 0, 1, A, A, 1, 0.1, A, 0, A, 0)]
got["empty"] = [empty(lambda p: lib.hs_gather_values(p, 0, b, 0, k, 0, 0, 0, 0, 0)) for b, k in ((0, 3), (2, 0))]
got["empty"] += [empty(lambda p: lib.hs_mla_decode_int4(p, 0, b, 0, 0, k, 0, 0, 0.1, 0, 0, 0, 0)) for b, k in ((0, 3), (2, 0))]
fake.fake_fail(1)
got["fail"] = [values(), fake.fake_last_error(), decode(), fake.fake_last_error()]
fake.fake_fail(0)
got["append"] = [append(p=pool(row_bytes=416)), append(p=pool(row_bytes=416), paged=pages()), append(p=pool(row_bytes=400)),
                 append(p=pool(row_bytes=416), kv_stride=575), append(p=pool(row_bytes=416), inv_freq=A + 1)]
""")
    for name in ("values", "decode"):
        g = got[name]
        assert g["good"] == [0] * len(g["good"]), name
        assert g["bad"] == [-1] * len(g["bad"]), name
        assert g["rows"] == [-1, -1, 0], name
        assert g["format"] == ([0, 0, 0, -5, -5] if name == "values" else [-5, -5, 0, -5, -5])
        assert g["device"] == [-1, -1]
    assert got["values"]["most"] == [0, 0, -1] and got["decode"]["most"] == [0, 0]
    assert got["null"] == [-1] * 4
    assert got["empty"] == [[0, 0]] * 4
    assert got["fail"] == [-2, 0, -2, 0]
    assert got["append"] == [0, 0, -5, -1, -1]


def test_grids(under):  # noqa: F811
    """Rows read back: a warp for four entries, at most a device full of blocks. Attention: a cluster for each request, its list
    cut into splits and its value columns into halves while the device (76 clusters of any size) holds them all."""
    got = under(CALLS + """
def grid(f, *a, **kw):
    rc = f(*a, **kw)
    return [rc, fake.fake_grid(fake.fake_launches() - 1)[0]]
big = pool(row_bytes=416, max_batch=200)
got = dict(values=[grid(values, batch=1, k=k) for k in (1, 32, 33, 64, 65, 1 << 20)],
           f32=grid(values, batch=1, k=1 << 20, type=hs.HS_TYPE_F32),
           decode=[grid(decode, batch=1, k=k) for k in (1, 256, 257, 2048, 1 << 20)],
           many=[grid(decode, p=big, batch=b, k=2048) for b in (76, 77, 200)])
""")
    assert got["values"] == [[0, 1], [0, 1], [0, 2], [0, 2], [0, 3], [0, 152 * 16]] and got["f32"] == [0, 152 * 8]
    assert got["decode"] == [[0, 4], [0, 4], [0, 8], [0, 16], [0, 16]]  # halves of the columns for short lists
    assert [rc for rc, _ in got["many"]] == [0, 0, 0] and all(g % 2 == 0 and g // 2 % b == 0 for (_, g), b in
                                                              zip(got["many"], (76, 77, 200)))


def test_the_binding_refuses_tensors_of_another_type_or_size(monkeypatch):
    """Refused before the library is called; addresses pass, as nothing is known of them."""
    monkeypatch.setitem(hs._pool_row_bytes, 7, 416)
    monkeypatch.setattr(hs, "_lib", None)
    monkeypatch.setattr(hs, "load", lambda: (_ for _ in ()).throw(KeyError("called")))
    idx, rows = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(9, 416, dtype=torch.uint8)
    dst, q = torch.zeros(2, 3, 576, dtype=torch.bfloat16), torch.zeros(2, 128, 576, dtype=torch.bfloat16)
    out, lse = torch.zeros(2, 128, 512, dtype=torch.bfloat16), torch.zeros(2, 128)
    good_v = dict(idx=idx, rows=rows, count=9, dst=dst, type=hs.HS_TYPE_BF16)
    good_d = dict(idx=idx, rows=rows, count=9, q=q, out=out, type=hs.HS_TYPE_BF16, lse=lse)

    def values(**kw):
        a = {**good_v, **kw}
        hs.hs_gather_values(7, 0, 2, a["idx"], 3, a["rows"], a["count"], a["dst"], a["type"], 0)

    def values_history(**kw):
        a = {**good_v, **kw}
        hs.hs_gather_values_history(7, 0, 2, a["idx"], 3, a["dst"], a["type"], 0)

    def decode(**kw):
        a = {**good_d, **kw}
        hs.hs_mla_decode_int4(7, 0, 2, a["q"], a["idx"], 3, a["rows"], a["count"], 0.1, a["out"], a["type"], a["lse"], 0)

    def decode_history(**kw):
        a = {**good_d, **kw}
        hs.hs_mla_decode_int4_history(7, 0, 2, a["q"], a["idx"], 3, 0.1, a["out"], a["type"], a["lse"], 0)

    lists = [dict(idx=idx.long()), dict(idx=idx[:, :2]), dict(idx=torch.zeros(3, 2, dtype=torch.int32).t())]
    tables = [dict(count=10), dict(rows=rows[:8]), dict(rows=torch.zeros(9, 832, dtype=torch.uint8)[:, ::2])]
    dsts = [dict(dst=dst.float()), dict(dst=dst[:1]), dict(type=hs.HS_TYPE_F32), dict(dst=dst.half())]
    heads = [dict(q=q.float()), dict(q=q[:1]), dict(out=out.float()), dict(out=out[:1]), dict(lse=lse.double()), dict(lse=lse[:1]),
             dict(type=hs.HS_TYPE_F32), dict(q=q.transpose(0, 1))]
    for call, bad in ((values, lists + tables + dsts), (values_history, lists + dsts), (decode, lists + tables + heads),
                      (decode_history, lists + heads)):
        for kw in bad:
            with pytest.raises(ValueError):
                call(**kw)
        with pytest.raises(KeyError, match="called"):
            call()
        with pytest.raises(KeyError, match="called"):
            call(idx=1 << 20, rows=1 << 20, dst=1 << 20, q=1 << 20, out=1 << 20, lse=1 << 20)
    with pytest.raises(KeyError, match="called"):
        values(rows=None, count=0)
    with pytest.raises(KeyError, match="called"):
        values(type=hs.HS_TYPE_F16, dst=dst.half())


def test_paged_rows_of_416_bytes(monkeypatch):
    pages = torch.zeros(4, dtype=torch.int32)
    p = hs.paged_rows(torch.zeros(64, 416, dtype=torch.uint8), pages, 16)
    assert p.count == 64
    monkeypatch.setitem(hs._pool_row_bytes, 7, 416)
    monkeypatch.setattr(hs, "load", lambda: (_ for _ in ()).throw(KeyError("called")))
    with pytest.raises(KeyError, match="called"):
        hs.hs_append(7, 0, 1, hs.hs_append_desc(), p, False, 0)
    with pytest.raises(ValueError, match="bytes"):
        hs.hs_append(7, 0, 1, hs.hs_append_desc(), hs.paged_rows(torch.zeros(64, 656, dtype=torch.uint8), pages, 16), False, 0)


def test_stages_of_a_loader_are_close():
    """The attention's loaders wait for a place of the ring by its barrier's parity, which holds as long as the stages that a loader
    has a part in are no further apart than the ring has places (five): their order, as hs_decode4.cu walks it, with all value
    columns to a pair of CTAs or half of them."""
    def walk(n, half):
        t = p = 0
        while t <= n:
            yield t, p
            p += 1
            if p == 4 - half or (p == 2 and t == 0):
                t, p = t + 1, 0
            if p == 0 and t >= n:
                p = 2

    def stages(n, last, loader, half):
        v = 8 >> half
        grp, pair = loader >> 2, loader >> 1 & 1
        for t, p in walk(n, half):
            if p < 2:
                at = (t * (9 + v) - v if t else 0) + 5 * p + 2 * grp
                yield from (at, at + 1)
            else:
                segment = (loader >> 1 if half else grp) + 2 * (p - 2)
                if segment < (last if t == n else 4):
                    yield t * (9 + v) - v + (0 if t == n else 9) + (segment if half else 2 * segment + pair)

    for half in (0, 1):
        for n in range(1, 6):
            order = [(t, p) for t in range(n + 1) for p in range(4 - half) if (t < n if p < 2 else t > 0)]
            assert list(walk(n, half)) == order
            for last in range(1, 5):
                filled = [0] * (n * 9 + (n - 1) * (8 >> half) + (2 * last >> half))
                for loader in range(8):
                    of = list(stages(n, last, loader, half))
                    assert of == sorted(of) and of[0] < 5 and all(b - a <= 5 for a, b in zip(of, of[1:]))
                    for x in of:
                        filled[x] += 1
                keys = {(t * (9 + (8 >> half)) - (8 >> half) if t else 0) + 4 for t in range(n)}
                # four loaders of a CTA for a stage of K, two for one of V, none for the rotary keys
                assert all(c == 0 if x in keys else c in (2, 4) for x, c in enumerate(filled))
