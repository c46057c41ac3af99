"""hs_mla_decode_int4 when the device cannot be asked what it holds: the call fails and is not remembered, so that equal calls are
cut alike before and after (the stand-in runtime of test_args_fake_runtime.py, with queries that fail when told to)."""
import json
import os
import subprocess
import sys

import pytest

from hierarchical_sparse_attention_hs_gb300 import build as hs_build
from test_args_fake_runtime import HERE, PREAMBLE

CALLS = """
q = ctypes.CDLL(%r)


def decode(batch=2, k=2048):
    block = pool(row_bytes=416, max_batch=200)
    return hs.load().hs_mla_decode_int4(ctypes.addressof(block), 0, batch, A, A, k, A, 10, 0.1, A, hs.HS_TYPE_BF16, A, 0)


def seen(f, *a):  # what a call returns, the grids that it launches, the queries that it makes, the error that it leaves
    launches, queries = fake.fake_launches(), q.fake_queries()
    rc = f(*a)
    return [rc, [fake.fake_grid(i)[0] for i in range(launches, fake.fake_launches())], q.fake_queries() - queries,
            q.fake_query_error()]
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    hs_build.build()
    at = tmp_path_factory.mktemp("fake")
    so = []
    for name in ("fake_queries", "fake_cudart"):
        so.append(str(at / (name + ".so")))
        subprocess.check_call(["gcc", "-shared", "-fPIC", "-O1", "-o", so[-1], os.path.join(HERE, name + ".c")])

    def run(code):
        text = PREAMBLE % (os.path.dirname(HERE), so[1]) + CALLS % so[0] + code + "\nprint(json.dumps(got))\n"
        r = subprocess.run([sys.executable, "-c", text], capture_output=True, text=True, timeout=300,
                           env=dict(os.environ, LD_PRELOAD=" ".join(so)))
        assert r.returncode == 0, r.stderr[-2000:]
        return json.loads(r.stdout.splitlines()[-1])

    return run


@pytest.mark.parametrize("batch,k", [(1, 65), (2, 2048), (80, 2048)])
def test_a_failed_query_is_an_error_of_its_call_alone(run, batch, k):
    good = run(f"got = [seen(decode, {batch}, {k}), seen(decode, {batch}, {k})]")
    assert good[0][0] == 0 and good[0][1] and good[0][2] > 0
    assert good[1] == [0, good[0][1], 0, 0]  # answers are kept
    for at in range(1, good[0][2] + 1):
        got = run(f"q.fake_fail_query({at}, 999)\ngot = [seen(decode, {batch}, {k}), seen(decode, {batch}, {k})]")
        assert got[0] == [-2, [], at, 0], at
        assert got[1][0] == 0 and got[1][1] == good[0][1], at


def test_cluster_sizes_that_the_device_does_not_take_are_remembered(run):
    """That is an answer, not a failure: other cuts are taken, and nothing is asked again."""
    got = run("q.fake_clusters(8, 76)\ngot = [seen(decode, 1, 2048), seen(decode, 1, 2048)]")
    assert got[0][0] == 0 and all(0 < g <= 8 for g in got[0][1]) and got[0][3] == 0
    assert got[1] == [0, got[0][1], 0, 0]


def test_a_device_that_holds_no_pair(run):
    got = run("q.fake_clusters(16, 0)\ngot = [seen(decode), seen(decode)]")
    assert got[0][:2] == got[1][:2] == [-5, []] and got[0][2] > 0 and got[1][2] == 0


BF16 = """
q.fake_ask_first(1)


def attend(batch=2):
    block = pool(row_bytes=1152, max_batch=200)
    return hs.load().hs_mla_decode(ctypes.addressof(block), 0, batch, A, A, 100, A, 10, 0.1, A, A, 0)


def debug():
    n = ctypes.c_int32(-1)
    rc = hs.load().hs_debug_attention(0, 0, ctypes.byref(n))
    return [rc, n.value] if rc == 0 else [rc]
"""


def test_debug_attention_before_any_attention(run):
    """What it says is what hs_mla_decode does, whichever is called first."""
    assert run(BF16 + "got = [debug(), seen(attend)[:2], debug()]") == [[0, 76], [0, [8]], [0, 76]]
    assert run(BF16 + "got = [seen(attend)[:2], debug()]") == [[0, [8]], [0, 76]]


def test_a_failed_query_does_not_change_how_later_bf16_calls_are_split(run):
    good = run(BF16 + "got = [seen(attend), seen(attend, 76), seen(attend, 77)]")
    assert [g[:2] for g in good] == [[0, [8]], [0, [304]], [0, [154]]]  # clusters of four CTAs, as many as fit, then pairs
    for at in range(1, good[0][2] + 1):
        got = run(BF16 + f"q.fake_fail_query({at}, 999)\ngot = [seen(attend), seen(attend)]")
        assert got[0][0] in (-2, -5) and got[0][1] == [] and got[0][3] == 0, at
        assert got[1][:2] == [0, [8]], at
    got = run(BF16 + "q.fake_fail_query(2, 999)\ngot = [debug(), debug(), seen(attend)[:2]]")
    assert got == [[-2], [0, 76], [0, [8]]]
