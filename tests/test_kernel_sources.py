"""Properties of the kernels' source text that no run can show reliably."""
import re

from hierarchical_sparse_attention_hs_gb300 import build as hs_build


def test_inline_loads_stay_behind_the_wait():
    """A kernel waits for the one before it with a volatile asm; a load written as asm that is not volatile has no order
    with it, and the compiler may place it ahead of the wait, where the array may still be in the making."""
    for path in hs_build.SOURCES + hs_build.HEADERS:
        text = open(path).read()
        for m in re.finditer(r'asm\s*(volatile)?\s*\(\s*"([^"]*)"', text):
            if re.search(r"\bld\.(global|volatile|relaxed|acquire)", m.group(2)):
                assert m.group(1) == "volatile", (path, m.group(0))
