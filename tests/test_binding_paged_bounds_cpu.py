"""What the paged-tail calls' binding passes to the library for numbers that a C int does not hold (CPU: the library is a
record of its arguments)."""
import ctypes

import pytest
import torch

from prefix_cached_kv_gb300 import binding

i32 = torch.int32


class _Lib:
    """Takes every call and keeps its arguments, as the declared C types hold them."""

    def __init__(self):
        self.calls = {}

    def pck_paged_workspace(self, h, cache, batch, H_q, window, sinks, n):
        return binding.OK

    def pck_paged_attend(self, h, cache, batch, H_q, Q, q_row, q_head, window, sinks, *rest):
        b = batch._obj
        self.calls["attend"] = dict(window=ctypes.c_int(window).value, sinks=ctypes.c_int(sinks).value, max_rows=b.max_rows, T=b.T)
        return binding.OK


class _Stream:
    cuda_stream = 0


@pytest.fixture
def attend(monkeypatch):
    c = binding.Context.__new__(binding.Context)   # no device: never created in the library
    c.lib, c.h, c.device = _Lib(), ctypes.c_void_p(1), torch.device("cpu")
    k = binding.PagedCache.__new__(binding.PagedCache)
    k.dtype, k.device, k.H_kv, k.D, k.page_size, k.n_pages, k._ws, k.ref = torch.float16, c.device, 2, 64, 16, 5, {}, None
    monkeypatch.setattr(c, "_empty", lambda stream, shape, dtype: torch.empty(shape, dtype=dtype), raising=False)
    Q, tab, n = torch.zeros((3, 4, 64), dtype=torch.float16), torch.zeros((1, 4), dtype=i32), torch.zeros(1, dtype=i32)

    def call(**kw):
        c.paged_attend(k, kw.pop("tab", tab), n, kw.pop("Q", Q), cu_rows=torch.zeros(2, dtype=i32), stream=_Stream(), **kw)
        return c.lib.calls["attend"]
    call.ctx = c
    return call


def test_bounds_keep_their_meaning(attend):
    top = 2 ** 31 - 1
    assert attend(window=20, sinks=4, max_rows=2) == dict(window=20, sinks=4, max_rows=2, T=3)
    for big in (top, 2 ** 31, 2 ** 32, 2 ** 32 + 20, 2 ** 63):
        assert attend(window=big, sinks=big, max_rows=big) == dict(window=top, sinks=top, max_rows=top, T=3)
    for low in (-1, -2 ** 31 - 1, -2 ** 32, -2 ** 32 + 1):
        got = attend(window=low, sinks=low, max_rows=low)
        assert got["window"] < 0 and got["sinks"] < 0 and got["max_rows"] < 1      # (which the library refuses)


def test_sizes_beyond_32_bits_are_refused(attend):
    many = torch.zeros((1, 4, 64), dtype=torch.float16).expand(2 ** 32 + 3, 4, 64)
    wide = torch.zeros((1, 1), dtype=i32).expand(1, 2 ** 32 + 4)
    for fn in (lambda: attend(Q=many), lambda: attend(tab=wide),
               lambda: attend.ctx.qk_norm_rope(many, None, norm=True, Q_out=many)):
        with pytest.raises(ValueError) as e:
            fn()
        assert "2^31 - 1" in str(e.value)
