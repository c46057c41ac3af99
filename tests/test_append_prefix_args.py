"""hs_append, hs_mla_prefix: arguments that are refused before any CUDA call, checked without a device.

The checks read the pool's descriptor, the first member of the opaque struct, so a zeroed block that starts with a
descriptor stands in for a pool here; every call below has to be refused before anything else of it is used.
"""
import ctypes

import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs
from hierarchical_sparse_attention_hs_gb300 import build as hs_build

INVALID, UNSUPPORTED = hs.HS_ERR_INVALID_ARG, hs.HS_ERR_UNSUPPORTED
A = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs_build.build()


def fake_pool(row_bytes=1152, max_batch=4, ctx=1000, layers=2):
    block = ctypes.create_string_buffer(4096)
    d = hs.hs_pool_desc(layers, max_batch, ctx, 64, 32, row_bytes, A, 0, 0, A, A, None)
    ctypes.memmove(block, ctypes.byref(d), ctypes.sizeof(d))
    # the device number lies behind the descriptor and the layout: no device has this one
    at = ctypes.sizeof(hs.hs_pool_desc) + ctypes.sizeof(hs.hs_meta_layout)
    ctypes.memmove(ctypes.addressof(block) + at, ctypes.byref(ctypes.c_int32(1 << 20)), 4)
    return block


def desc(**kw):
    d = dict(type=hs.HS_TYPE_BF16, interleaved=1, kv=A, kv_stride=576, norm_weight=A, inv_freq=A, req_ids=A, positions=A,
             q_rope=A, q_rope_token_stride=128 * 64, q_rope_head_stride=64, q=A, q_token_stride=128 * 576,
             q_head_stride=576, q_heads=128, norm_eps=1e-6)
    d.update(kw)
    out = hs.hs_append_desc()
    for k, v in d.items():
        setattr(out, k, v)
    return out


def pages(**kw):
    d = dict(rows=A, count=100, pages=A, page_stride=10, page_rows=16)
    d.update(kw)
    return hs.hs_paged_rows(*d.values())


def refused(code, call):
    with pytest.raises(hs.HsError) as e:
        call()
    assert e.value.code == code


def append(code, layer=0, ntok=3, d=None, paged=None, to_history=True, pool=None, **kw):
    block = fake_pool() if pool is None else pool
    refused(code, lambda: hs.hs_append(ctypes.addressof(block), layer, ntok, d or desc(**kw), paged, to_history, 0))


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(type=-1), dict(kv=None), dict(kv=A + 8), dict(kv_stride=575), dict(kv_stride=580),
    dict(kv_stride=1 << 62), dict(norm_weight=A + 4), dict(norm_eps=-1.0), dict(norm_eps=float("nan")), dict(inv_freq=None),
    dict(positions=None), dict(q=None), dict(q_rope=None), dict(q_heads=0), dict(q_heads=-1), dict(q_rope=A + 2),
    dict(q=A + 8), dict(q_rope_token_stride=60), dict(q_rope_head_stride=65), dict(q_token_stride=0),
    dict(q_head_stride=577), dict(q_head_stride=-576)])
def test_append_refuses(kw):
    append(INVALID, **kw)


def test_append_refuses_calls():
    append(INVALID, layer=-1)
    append(INVALID, layer=2)
    append(INVALID, ntok=-1)
    append(INVALID, ntok=(1 << 30) + 1)
    append(INVALID, ntok=1 << 28, q_heads=81)
    append(INVALID, ntok=5, req_ids=None)  # token i is request i: at most max_batch
    append(UNSUPPORTED, pool=fake_pool(row_bytes=1024))
    append(INVALID, to_history=False, q_rope=None, q=None, q_heads=0)  # nothing to do
    refused(INVALID, lambda: hs.hs_append(0, 0, 1, desc(), None, True, 0))
    refused(INVALID, lambda: hs.hs_append(ctypes.addressof(fake_pool()), 0, 1, None, None, True, 0))
    append(INVALID)  # every argument is good, but the pool belongs to another device than the current one


@pytest.mark.parametrize("kw", [dict(rows=None), dict(rows=A + 8), dict(count=-1), dict(count=1 << 31), dict(pages=None),
                                dict(pages=A + 2), dict(page_stride=0), dict(page_rows=0), dict(page_rows=24),
                                dict(page_rows=1 << 17), dict(page_rows=-16)])
def test_bad_paged_rows_are_refused(kw):
    append(INVALID, paged=pages(**kw))
    prefix(INVALID, paged=pages(**kw))


def prefix(code, pool=None, batch=2, q=A, paged=None, max_length=100, length=None, own_out=None, own_lse=None, out=A,
           out_type=hs.HS_TYPE_BF16, lse=A):
    block = fake_pool() if pool is None else pool
    refused(code, lambda: hs.hs_mla_prefix(ctypes.addressof(block), batch, q, paged or pages(), max_length, length, 0.1,
                                           own_out, own_lse, out, out_type, lse, None, 0))


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(batch=1 << 18), dict(q=None), dict(q=A + 8), dict(max_length=-1), dict(max_length=161),
    dict(own_out=A), dict(own_lse=A), dict(own_out=A + 4, own_lse=A), dict(out=None), dict(out=A + 8), dict(lse=None),
    dict(lse=A + 2), dict(out_type=hs.HS_TYPE_F16), dict(out_type=7), dict(length=A + 1)])
def test_prefix_refuses(kw):
    prefix(INVALID, **kw)


def test_prefix_refuses_calls():
    prefix(UNSUPPORTED, pool=fake_pool(row_bytes=656))
    prefix(INVALID)  # another device
    refused(INVALID, lambda: hs.hs_mla_prefix(0, 1, A, pages(), 16, None, 0.1, None, None, A, 0, A, None, 0))
    refused(INVALID, lambda: hs.hs_mla_prefix(ctypes.addressof(fake_pool()), 1, A, None, 16, None, 0.1, None, None, A, 0,
                                              A, None, 0))
    assert hs.hs_mla_prefix_workspace(0, 1, 100) == 0
    assert hs.hs_mla_prefix_workspace(ctypes.addressof(fake_pool()), 0, 100) == 0
    assert hs.hs_mla_prefix_workspace(ctypes.addressof(fake_pool()), 1, -1) == 0


def test_empty_calls_do_nothing():
    block = fake_pool()
    hs.hs_append(ctypes.addressof(block), 0, 0, desc(), None, True, 0)
    hs.hs_mla_prefix(ctypes.addressof(block), 0, None, pages(), 100, None, 0.1, None, None, None, 0, None, None, 0)


@pytest.mark.parametrize("stride, rows", [(1 << 48, 1 << 16), (1 << 47, 1 << 16), ((1 << 63) - 1, 1), ((1 << 63) - 1, 64)])
def test_prefix_takes_lists_of_any_stride(stride, rows):
    """A list longer than 2^63 tokens is longer than max_length (an empty batch ends the call behind that check)."""
    block = fake_pool()
    hs.hs_mla_prefix(ctypes.addressof(block), 0, None, pages(page_stride=stride, page_rows=rows), 100, None, 0.1, None,
                     None, None, 0, None, None, 0)


def test_helpers_check_shapes_and_types():
    kv, f, p = torch.zeros(3, 576, dtype=torch.bfloat16), torch.zeros(32), torch.zeros(3, dtype=torch.int32)
    q, qr = torch.zeros(3, 8, 576, dtype=torch.bfloat16), torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    d = hs.append_desc(kv, f, p, q_rope=qr, q=q)
    assert (d.type, d.kv_stride, d.q_heads, d.q_token_stride, d.q_head_stride) == (hs.HS_TYPE_BF16, 576, 8, 8 * 576, 576)
    assert ctypes.sizeof(hs.hs_append_desc) == 8 + 8 * 12 + 8 and ctypes.sizeof(hs.hs_paged_rows) == 40
    for bad in (dict(kv=kv.double()), dict(kv=kv[:, :512]), dict(f=f.double()), dict(p=p.long()), dict(qr=None),
                dict(qr=qr.float()), dict(q=q[..., :512]), dict(kv=torch.zeros(576, 3, dtype=torch.bfloat16).t())):
        a = dict(kv=kv, f=f, p=p, qr=qr, q=q)
        a.update(bad)
        with pytest.raises(ValueError):
            hs.append_desc(a["kv"], a["f"], a["p"], q_rope=a["qr"], q=a["q"])
    with pytest.raises(ValueError):
        hs.paged_rows(torch.zeros(4, 16)[:, ::2], p, 1)
