"""hs_append, hs_mla_prefix: a good call reaches its launches and a call that differs from it in one argument is refused.

The calls run in a process of their own, in which a stand-in for the CUDA runtime (fake_cudart.c) is loaded first, so that
the checks run to the end without a device and nothing is launched. Without it a good call is refused as well (its pool
belongs to no device), and a refusal would prove nothing about the argument.
"""
import json
import os
import subprocess
import sys

import pytest

from hierarchical_sparse_attention_hs_gb300 import build as hs_build

HERE = os.path.dirname(os.path.abspath(__file__))

PREAMBLE = """
import ctypes, json, sys
sys.path.insert(0, %r)
import hierarchical_sparse_attention_hs_gb300 as hs

A = 1 << 20  # an aligned address that is never dereferenced
fake = ctypes.CDLL(%r)
fake.fake_grid.restype = ctypes.POINTER(ctypes.c_uint)


def pool(row_bytes=1152, max_batch=4, ctx=1000, layers=2):
    block = ctypes.create_string_buffer(4096)
    d = hs.hs_pool_desc(layers, max_batch, ctx, 64, 32, row_bytes, A, 0, 0, A, A, None)
    ctypes.memmove(block, ctypes.byref(d), ctypes.sizeof(d))
    # behind the descriptor and the layout: the device's number, and its SMs
    at = ctypes.addressof(block) + ctypes.sizeof(hs.hs_pool_desc) + ctypes.sizeof(hs.hs_meta_layout)
    ctypes.memmove(at, (ctypes.c_int32 * 2)(0, 152), 8)
    return block


def desc(**kw):
    d = dict(type=hs.HS_TYPE_BF16, interleaved=1, kv=A, kv_stride=576, norm_weight=A, inv_freq=A, req_ids=A, positions=A,
             q_rope=A, q_rope_token_stride=128 * 64, q_rope_head_stride=64, q=A, q_token_stride=128 * 576,
             q_head_stride=576, q_heads=128, norm_eps=1e-6)
    out = hs.hs_append_desc()
    for k, v in {**d, **kw}.items():
        setattr(out, k, v)
    return out


def pages(**kw):
    out = hs.hs_paged_rows()
    for k, v in {**dict(rows=A, count=100, pages=A, page_stride=10, page_rows=16), **kw}.items():
        setattr(out, k, v)
    return out


def code(call):
    before = fake.fake_launches()
    try:
        call()
        rc = 0
    except hs.HsError as e:
        rc = e.code
    made = fake.fake_launches() - before
    assert rc == -2 or (made > 0) == (rc == 0), (rc, made)
    return rc


def append(ntok=3, p=None, paged=None, to_history=True, layer=0, **kw):
    block = p or pool()
    return code(lambda: hs.hs_append(ctypes.addressof(block), layer, ntok, desc(**kw), paged, to_history, 0))


def prefix(batch=2, q=A, paged=None, max_length=100, length=None, own_out=None, own_lse=None, out=A,
           out_type=hs.HS_TYPE_BF16, lse=A, p=None, work=A, nbytes=1 << 40):
    block = p or pool()
    # straight at the library: the binding takes a workspace's size from its tensor
    def call():
        rc = hs.load().hs_mla_prefix(ctypes.addressof(block), batch, q, paged or pages(), max_length, length, 0.1, own_out,
                                     own_lse, out, out_type, lse, work, nbytes, 0)
        if rc:
            raise hs.HsError(rc, "hs_mla_prefix")
    return code(call)


"""


@pytest.fixture(scope="module")
def under(tmp_path_factory):
    """Runs Python code with the stand-in loaded; what it leaves in `got` comes back."""
    hs_build.build()
    so = str(tmp_path_factory.mktemp("fake") / "fake_cudart.so")
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-O1", "-o", so, os.path.join(HERE, "fake_cudart.c")])

    def run(code):
        text = PREAMBLE % (os.path.dirname(HERE), so) + code + "\nprint(json.dumps(got))\n"
        r = subprocess.run([sys.executable, "-c", text], capture_output=True, text=True, timeout=300,
                           env=dict(os.environ, LD_PRELOAD=so))
        assert r.returncode == 0, r.stderr[-2000:]
        return json.loads(r.stdout.splitlines()[-1])

    return run


def test_append_refuses_misaligned_arrays(under):
    """inv_freq, positions and req_ids hold 4-byte values: an address that is not a multiple of 4 would fault."""
    got = under("""
got = {"good": append(), "no ids": append(req_ids=None)}
for name in ("inv_freq", "positions", "req_ids"):
    got[name] = [append(**{name: A + off}) for off in (1, 2, 3, 4)]
""")
    assert got["good"] == 0 and got["no ids"] == 0
    for name in ("inv_freq", "positions", "req_ids"):
        assert got[name] == [-1, -1, -1, 0], name


def test_append_counts_heads_in_64_bits(under):
    """The work items of a token's queries are ceil(q_heads / 16); the largest counts round up past 32 bits."""
    got = under("""
got = []
for heads in (128, (1 << 31) - 16, (1 << 31) - 15, (1 << 31) - 1):
    rc = append(ntok=1, q_heads=heads)
    got.append([rc, list(fake.fake_grid(fake.fake_launches() - 1)[:3])])
got.append([append(ntok=8, q_heads=(1 << 31) - 1), append(ntok=9, q_heads=(1 << 31) - 1)])
""")
    assert got[0] == [0, [1 + 2, 1, 1]]  # a block of rows; 8 items are the warps of 2 blocks
    assert got[1] == got[2] == got[3] == [0, [1 + 152 * 16, 1, 1]]
    assert got[4] == [0, -1]  # 8 * 2^27 items are the limit


def test_lists_of_pages(under):
    """A block table says how many lists it holds; fewer than none is refused, and none of them means one a request."""
    got = under("""
got = {str(n): [append(paged=pages(lists=n)), prefix(paged=pages(lists=n))] for n in (-1, -(1 << 31), 0, 1, 4, 9)}
""")
    assert got == {"-1": [-1, -1], str(-(1 << 31)): [-1, -1], "0": [0, 0], "1": [0, 0], "4": [0, 0], "9": [0, 0]}


def test_workspace_of_the_largest_call_serves_the_smaller_ones(under):
    """The workspace of one call is no bound for calls of fewer requests or tokens; the bound is, and no call of a sweep
    (76 pairs of CTAs) is refused with it."""
    got = under("""
block = pool()
p = ctypes.addressof(block)
need, bound = hs.hs_mla_prefix_workspace, hs.hs_mla_prefix_workspace_bound
tokens = [0, 1, 256, 257, 511, 513, 2047, 4096, 8192, 9001, 30000, 131072, 1 << 20, 1 << 30]
over, low, refused = [], 0, []
for B in list(range(1, 80)) + [100, 152, 153, 229, 1000, 131072]:
    for L in tokens:
        top = bound(p, B, L)
        low = max(low, top)
        smaller = [(b, l) for b in {1, 2, 3, B // 3, B // 2, B - 1, B} if 0 < b <= B for l in tokens if l <= L]
        over += [(B, L, b, l) for b, l in smaller if need(p, b, l) > top]
for b in (1, 2, 7, 40, 75, 76, 77, 100, 150, 153):
    for l in tokens:
        n = bound(p, 153, 1 << 30)
        if prefix(batch=b, max_length=l, paged=pages(page_stride=1 << 26), nbytes=n):
            refused.append((b, l))
        if need(p, b, l) and not prefix(batch=b, max_length=l, paged=pages(page_stride=1 << 26), nbytes=need(p, b, l) - 1):
            refused.append((b, l, "not"))
def rc(*a):
    try:
        return [0, bound(*a)]
    except hs.HsError as e:
        return [e.code, None]
got = dict(over=over[:5], refused=refused[:5], most=low, listed=[need(p, 76, 8192), need(p, 40, 8192), need(p, 1, 8192)],
           bad=[rc(0, 1, 1), rc(p, -1, 1), rc(p, 131073, 1), rc(p, 1, -1), rc(p, 1, (1 << 30) + 1)], none=[rc(p, 0, 100), rc(p, 5, 256)],
           null=hs.load().hs_mla_prefix_workspace_bound(p, 1, 1, None),
           batches=[prefix(batch=131072, max_length=1), prefix(batch=131073, max_length=1)])
""")
    assert got["over"] == [] and got["refused"] == []
    assert got["most"] == 4 * 76 * 128 * (512 * 4 + 8)
    assert got["listed"][0] < got["listed"][2] < got["listed"][1]
    assert [x[0] for x in got["bad"]] == [-1] * 5 and got["none"] == [[0, 0], [0, 0]] and got["null"] == -1
    assert got["batches"] == [0, -1]


def test_rows_of_many_tokens_are_one_wave(under):
    """A launch of many tokens has as many blocks of rows as the device holds of its kernel, asked once for each kernel:
    more would run as a second, partly filled wave."""
    got = under("""
got, held = [], 0
for rb in (1152, 656):
    for type in (hs.HS_TYPE_BF16, hs.HS_TYPE_F16, hs.HS_TYPE_F32):
        for interleaved in (0, 1):
            call = dict(p=pool(row_bytes=rb), type=type, interleaved=interleaved, q_rope=None, q=None, q_heads=0)
            fake.fake_hold(0)  # the question fails, and is asked again by the next call
            got.append([append(ntok=1, **call), -2, 0])
            held += 1
            fake.fake_hold(held)
            for ntok in (1, 127, 5000, 152 * held * 4, 152 * held * 4 + 1, 131071, 1 << 30):
                rc = append(ntok=ntok, **call)
                blocks = fake.fake_grid(fake.fake_launches() - 1)[0]
                per = -(-ntok // (152 * held * 4))  # a warp's tokens, the least that one wave can have
                got.append([rc, 0, blocks - -(-(-(-ntok // per)) // 4)])
                got.append([blocks > 152 * held, False, 0])
""")
    assert [x for x in got if x[0] != x[1] or x[2]] == []


def test_a_launch_that_fails_leaves_no_error_behind(under):
    """A refused launch is the call's own error: the runtime's last error, which the caller's next check of another launch
    would take for its own, is clear again."""
    got = under("""
fake.fake_fail(1)
got = [append(), fake.fake_last_error(), prefix(), fake.fake_last_error(), prefix(max_length=4096, paged=pages(page_stride=1 << 20)),
       fake.fake_last_error()]
fake.fake_fail(2)  # the second launch of a call: the one that joins splits
got += [prefix(batch=1, max_length=9001, paged=pages(page_stride=1 << 20)), fake.fake_last_error()]
fake.fake_fail(0)
got += [append(), prefix()]
""")
    assert got == [-2, 0, -2, 0, -2, 0, -2, 0, 0, 0]


def _cases(function):
    """The keyword dicts that a test of test_append_prefix_args.py is run with."""
    return [m.args[1] for m in function.pytestmark if m.name == "parametrize"][0]


def test_every_refusal_is_of_its_argument(under):
    """The refusals that test_append_prefix_args.py lists, each of a call that is good but for it."""
    import test_append_prefix_args as listed

    got = under("""
nan = float("nan")
got = dict(good=[append(), prefix(), append(paged=pages()), prefix(own_out=A, own_lse=A), prefix(length=A), prefix(work=None, nbytes=0)],
           append=[append(**kw) for kw in %r], prefix=[prefix(**kw) for kw in %r],
           paged=[[append(paged=pages(**kw)), prefix(paged=pages(**kw))] for kw in %r],
           calls=[append(layer=-1), append(layer=2), append(layer=1), append(ntok=-1), append(ntok=(1 << 30) + 1),
                  append(ntok=1 << 28, q_heads=81), append(ntok=1 << 28, q_heads=64), append(ntok=5, req_ids=None),
                  append(ntok=4, req_ids=None), append(to_history=False, q_rope=None, q=None, q_heads=0),
                  append(to_history=False), append(p=pool(row_bytes=1024)), append(p=pool(row_bytes=656)),
                  prefix(p=pool(row_bytes=656)), prefix(batch=131072), prefix(max_length=160), prefix(max_length=0)],
           space=[prefix(batch=1, max_length=9001, paged=pages(page_stride=1000), work=w, nbytes=n)
                  for w, n in ((None, 1 << 40), (A + 16, 1 << 40), (A, 36 * 128 * 2056 - 1), (A, 36 * 128 * 2056))])
""" % (_cases(listed.test_append_refuses), _cases(listed.test_prefix_refuses), _cases(listed.test_bad_paged_rows_are_refused)))
    assert got["good"] == [0] * 6
    assert got["append"] == [-1] * len(got["append"]) and got["prefix"] == [-1] * len(got["prefix"])
    assert got["paged"] == [[-1, -1]] * len(got["paged"])
    assert got["calls"] == [-1, -1, 0, -1, -1, -1, 0, -1, 0, -1, 0, -5, 0, -5, 0, 0, 0]
    assert got["space"] == [-1, -1, -1, 0]
