"""The ends of what fp32 and bf16 hold of the quantised cache's values, on the GPU."""
import math

import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_e4m3_ref as r8
from tests.test_gpu_paged import BF16, F32, ctx, i32   # noqa: F401
from tests.test_gpu_paged_e4m3 import U8, _cu, _empty_pages

pytestmark = pytest.mark.gpu


def test_rows_next_to_fp32s_end(ctx):   # noqa: F811
    """Up to 248 * 2^120 (a tie, to the even code 256) a row reads back finite; from there on its code stands for 2^128."""
    D = 16
    below, above = 248 * 2.0 ** 120 * (1 - 2.0 ** -20), torch.finfo(F32).max
    x = torch.zeros((3, 1, D), dtype=F32)
    x[0, 0, 2], x[1, 0, 2], x[2, 0, 2] = below, above, -248 * 2.0 ** 120
    x = x.cuda()
    k, v, ks, vs = _empty_pages(1, 1, 16, D)
    c = binding.QuantizedPagedCache(k, v, ks, vs)
    tab, ln = torch.zeros((1, 1), dtype=i32, device="cuda"), torch.tensor([3], dtype=i32, device="cuda")
    ctx.paged_append(c, tab, ln, x, x, cu_rows=_cu([3]))
    for dtype in (F32, BF16):
        for t in ctx.paged_read(c, tab, ln, T=3, cu_rows=_cu([3]), dtype=dtype):
            assert t[:, 0, 2].tolist() == [240 * 2.0 ** 120, math.inf, -math.inf]
            assert (t[:, 0, :2] == 0).all() and (t[:, 0, 3:] == 0).all()
    ctx.sync()


@pytest.mark.parametrize("byte", [1, 2, 3, 4, 60, 245, 246])
def test_where_bf16_is_exact(ctx, byte):   # noqa: F811
    """Every finite code at scales 2^(byte - 127): exact in fp32, and in bf16 from byte 3 on (below, to half its smallest step)."""
    codes = torch.arange(256, dtype=U8, device="cuda").view(1, 1, 16, 16)
    scale = torch.full((1, 1, 16), byte, dtype=U8, device="cuda")
    c = binding.QuantizedPagedCache(codes.view(r8.E4M3), codes.clone().view(r8.E4M3), scale, scale)
    tab, ln = torch.zeros((1, 1), dtype=i32, device="cuda"), torch.tensor([16], dtype=i32, device="cuda")
    want = r8.values(codes.view(r8.E4M3), scale)[0, 0].nan_to_num(0)
    for dtype in (F32, BF16):
        got = ctx.paged_read(c, tab, ln, T=16, cu_rows=_cu([16]), dtype=dtype)[0][:, 0].double().nan_to_num(0)
        if dtype == F32 or byte >= 3:
            assert torch.equal(got, want)
        else:
            assert ((got - want).abs() <= 2.0 ** -134).all() and not torch.equal(got, want)
    ctx.sync()
