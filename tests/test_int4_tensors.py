"""What the binding of the 4-bit operators refuses of tensors before the library is called (a stand-in for it, on the CPU)."""
import types

import pytest
import torch

import hierarchical_sparse_attention_hs_gb300 as hs

POOL = 7


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library."""
    made = []
    names = ("hs_gather_values", "hs_gather_values_history", "hs_mla_decode_int4", "hs_mla_decode_int4_history")
    lib = types.SimpleNamespace(**{n: (lambda *a, n=n: made.append((n, a)) or 0) for n in names})
    monkeypatch.setattr(hs, "_lib", lib)
    monkeypatch.setitem(hs._pool_row_bytes, POOL, 416)
    return made


def values(rows, count):
    hs.hs_gather_values(POOL, 0, 1, 1 << 20, 3, rows, count, 1 << 20, hs.HS_TYPE_BF16, 0)


def decode(rows, count):
    hs.hs_mla_decode_int4(POOL, 0, 1, 1 << 20, 1 << 20, 3, rows, count, 0.1, 1 << 20, hs.HS_TYPE_BF16, 1 << 20, 0)


def bytes_of(*shape):
    """A tensor that says it is on the GPU: only what the binding asks of it."""
    class OnGpu(torch.Tensor):
        is_cuda = True

    return torch.zeros(shape, dtype=torch.uint8).as_subclass(OnGpu)


@pytest.mark.parametrize("call", [values, decode])
def test_resident_rows_of_another_format(calls, call):
    """Rows of 656 or 1152 bytes have room for as many of 416, and would be read at the wrong stride."""
    for bad in (bytes_of(9, 656), bytes_of(9, 1152), bytes_of(9, 1152).view(torch.bfloat16), bytes_of(2, 16, 656), bytes_of(9, 3, 656),
                bytes_of(1, 26, 656), bytes_of(1, 13, 1152)):
        with pytest.raises(ValueError, match="416"):
            call(bad, 9)
    assert not calls
    good = [bytes_of(9, 416), bytes_of(9, 416).view(torch.int32), bytes_of(3, 4, 416), bytes_of(9, 26, 16), bytes_of(9 * 416),
            bytes_of(12, 416), bytes_of(1, 9, 2, 208), bytes_of(3, 4 * 416), bytes_of(9 * 416 + 64), bytes_of(9 * 416).view(torch.int32)]
    for rows in good:
        call(rows, 9)
    call(bytes_of(0, 416), 0)
    call(None, 0)
    call(1 << 20, 9)
    assert len(calls) == len(good) + 3


def test_resident_rows_of_a_pool_of_fp8_rows(calls, monkeypatch):
    monkeypatch.setitem(hs._pool_row_bytes, POOL, 656)
    for bad in (bytes_of(82, 416), bytes_of(41, 1152), bytes_of(9, 1152)):  # 82 rows of 416 bytes are 52 of 656
        with pytest.raises(ValueError, match="656"):
            values(bad, 9)
    for rows in (bytes_of(9, 656), bytes_of(9, 41, 16), bytes_of(2, 8, 656)):
        values(rows, 9)
    assert len(calls) == 3


def test_tensors_in_ordinary_host_memory(calls):
    """Their addresses would go to a kernel that reads device memory."""
    on = lambda t: bytes_of(t.nbytes).view(t.dtype).view(t.shape)  # noqa: E731
    idx = torch.zeros(2, 3, dtype=torch.int32)
    dst, q = torch.zeros(2, 3, 576, dtype=torch.bfloat16), torch.zeros(2, 128, 576, dtype=torch.bfloat16)
    out, lse, rows = torch.zeros(2, 128, 512, dtype=torch.bfloat16), torch.zeros(2, 128), torch.zeros(9, 416, dtype=torch.uint8)
    host = dict(idx=idx, rows=rows, dst=dst, q=q, out=out, lse=lse)
    fine = {n: on(t) for n, t in host.items()}
    forms = dict(
        values=(lambda a: hs.hs_gather_values(POOL, 0, 2, a["idx"], 3, a["rows"], 9, a["dst"], 0, 0), ("idx", "rows", "dst")),
        values_history=(lambda a: hs.hs_gather_values_history(POOL, 0, 2, a["idx"], 3, a["dst"], 0, 0), ("idx", "dst")),
        decode=(lambda a: hs.hs_mla_decode_int4(POOL, 0, 2, a["q"], a["idx"], 3, a["rows"], 9, 0.1, a["out"], 0, a["lse"], 0),
                ("idx", "rows", "q", "out", "lse")),
        decode_history=(lambda a: hs.hs_mla_decode_int4_history(POOL, 0, 2, a["q"], a["idx"], 3, 0.1, a["out"], 0, a["lse"], 0),
                        ("idx", "q", "out", "lse")))
    for name, (call, takes) in forms.items():
        call(fine)
        assert len(calls) == 1, name
        for t in takes:
            with pytest.raises(ValueError, match="memory"):
                call({**fine, t: host[t]})
        call({**fine, **{t: 1 << 20 for t in takes}})
        assert len(calls) == 2, name
        calls.clear()


def test_a_page_locked_list(calls):
    """A list may be page-locked host memory."""
    class Locked(torch.Tensor):
        def is_pinned(self):
            return True

    idx = torch.zeros(1, 3, dtype=torch.int32).as_subclass(Locked)
    hs.hs_gather_values(POOL, 0, 1, idx, 3, None, 0, 1 << 20, 0, 0)
    hs.hs_mla_decode_int4_history(POOL, 0, 1, 1 << 20, idx, 3, 0.1, 1 << 20, 0, 1 << 20, 0)
    assert [a[3] if n == "hs_gather_values" else a[4] for n, a in calls] == [idx.data_ptr()] * 2
