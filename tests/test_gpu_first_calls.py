"""What the first call of a process does not leave behind for the later ones."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.path.insert(0, %r)
import torch, hierarchical_sparse_attention_hs_gb300 as hs
torch.zeros(1, device="cuda")
said = [hs.hs_debug_attention()] if sys.argv[1] == "ask" else []
buf = hs.PoolBuffers(1, 2, 300, 300, 256, 1152)
g = torch.Generator().manual_seed(1)
buf.hot.copy_(torch.randn(600, 576, generator=g).to(torch.bfloat16).view(torch.uint8).flatten())
q = torch.randn(2, 128, 576, generator=g).to(torch.bfloat16).cuda()
e = torch.stack([torch.randperm(300, generator=g)[:256] for _ in range(2)]).int().cuda()
out, lse = torch.empty(2, 128, 512, device="cuda"), torch.empty(2, 128, device="cuda")
hs.hs_mla_decode(buf.create(), 0, 2, q, e, 256, None, 0, 0.07, out, lse)
torch.cuda.synchronize()
said.append(hs.hs_debug_attention())
print(*said, hash((out.cpu().numpy().tobytes(), lse.cpu().numpy().tobytes())))
buf.close()
"""


def test_asking_for_the_split_first_changes_nothing():
    """hs_debug_attention before any hs_mla_decode says what it says after one, and outputs keep their bits."""
    import __graft_entry__ as g

    g.build()
    got = []
    for first in ("ask", "attend"):
        r = subprocess.run([sys.executable, "-c", CODE % ROOT, first], capture_output=True, text=True, timeout=300,
                           env=dict(os.environ, PYTHONHASHSEED="0"))
        assert r.returncode == 0, r.stderr[-2000:]
        got.append(r.stdout.split())
    (before, after, bits), (other, same) = got
    assert int(before) == int(after) == int(other) > 0 and bits == same
