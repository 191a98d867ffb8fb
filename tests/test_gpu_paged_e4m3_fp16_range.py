"""Values of the quantised cache that fp16 cannot hold, under rows with an fp16 q, on the GPU."""
import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_e4m3_ref as r8
from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F16, _rand, ctx, i32   # noqa: F401
from tests.test_gpu_paged_e4m3 import PAIR, _bits, _cu, _empty_pages

pytestmark = pytest.mark.gpu
LENS, NEWS = [300, 90], [150, 40]


def _pages(side, at, exponent, code=0x38):
    """Pages with one code (1.0) of a token of sequence 0 at 2^exponent, on one side."""
    pg = r8.Pages8(8, LENS, 2, 64, 16)
    codes, scale = (pg.k, pg.ks) if side == "k" else (pg.v, pg.vs)
    where = (pg.table[0, at // 16].long(), 1, at % 16)
    _bits(codes)[where] = 0
    _bits(codes)[where][5] = code
    scale[where] = 127 + exponent
    return pg


def _rows(ctx, pg, dtype, **kw):   # noqa: F811
    Q = _rand(9, sum(NEWS), 4, 64, dtype=dtype, scale=0.1)
    O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=_cu(NEWS), **kw)
    return Q, O, L


@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("exponent,code", [(17, 0x38), (17, 0xb8), (8, 0x79), (100, 0x38)])      # 2^17, -2^17, 288 * 2^8 = 73,728, 2^100
def test_a_value_beyond_fp16_is_reported(ctx, side, exponent, code):   # noqa: F811
    ctx.sync()
    pg = _pages(side, 250, exponent, code)
    _rows(ctx, pg, F16)
    with pytest.raises(binding.PckError) as e:
        ctx.sync()
    assert e.value.code == binding.ECUDA and "code 16" in str(e.value) and "fp16" in str(e.value)
    ctx.sync()                                             # reported once
    # bf16 holds it, and so does one-token attention with either type
    if exponent < 100:
        Q, O, L = _rows(ctx, pg, BF16)
        ref.check_attend(O, L, r8.attend(pg, LENS, NEWS, Q), BF16, ref.P_ONCE[BF16])
        for dtype in (F16, BF16):
            q = _rand(10, 2, 4, 64, dtype=dtype, scale=0.1)
            O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, q)
            want = r8.attend(pg, LENS, [1, 1], q)
            if want[0].abs().max() < 60000:
                ref.check_attend(O, L, want, dtype, PAIR)
    # so does the read-back, at its largest value
    kv = ctx.paged_read(pg.cache(), pg.table, pg.lens, T=390, cu_rows=_cu(LENS))
    assert kv[side == "v"][250, 1, 5].abs() == 65504
    ctx.sync()


def test_what_is_not_reported(ctx):   # noqa: F811
    """Values within fp16, or next to its end; NaN; values that no row sees."""
    ctx.sync()
    for pg in (_pages("v", 250, 16), _pages("k", 250, 8, 0x77), _pages("v", 250, 8, 0x78)):       # 2^16, 240 * 2^8, 256 * 2^8
        Q, O, L = _rows(ctx, pg, F16)
        # (65,536 is 65,504 there: 2^-11 of it, as much as a weight's rounding moves it)
        ref.check_attend(O, L, r8.attend(pg, LENS, NEWS, Q), F16, 2 * ref.P_ONCE[F16])
    for side, exponent, code in (("v", 100, 0x7f), ("k", 8, 0xff), ("v", 128, 0x38)):             # a NaN code; the scale that is NaN
        _rows(ctx, _pages(side, 250, exponent, code), F16)
    ctx.sync()
    for side in ("k", "v"):
        pg = _pages(side, 100, 30)                         # in front of the first row's window
        Q, O, L = _rows(ctx, pg, F16, window=20)
        ref.check_attend(O, L, r8.attend(pg, LENS, NEWS, Q, window=20), F16, ref.P_ONCE[F16])
    ctx.sync()


def test_fp16_rows_at_the_types_end(ctx):   # noqa: F811
    """fp16's largest values, appended as they are (their codes say 65,536) and attended to by rows."""
    n, D = 64, 64
    k, v, ks, vs = _empty_pages(4, 1, 16, D)
    c = binding.QuantizedPagedCache(k, v, ks, vs)
    x = torch.full((n, 1, D), 65504.0, dtype=F16, device="cuda")
    x[::2] = -65504.0
    tab, ln = torch.arange(4, device="cuda", dtype=i32)[None], torch.tensor([n], dtype=i32, device="cuda")
    ctx.paged_append(c, tab, ln, torch.zeros_like(x), x, cu_rows=_cu([n]))
    O, _ = ctx.paged_attend(c, tab, ln, torch.zeros((n, 32, D), dtype=F16, device="cuda"), cu_rows=_cu([n]))
    ctx.sync()
    # equal weights: the mean of the values seen, -65,504 where their number is odd, over it, else 0
    i = torch.arange(n, dtype=torch.float64, device="cuda")
    want = torch.where(i % 2 == 0, -65504 / (i + 1), 0)[:, None, None]
    assert ((O.double() - want).abs() <= 2 * ref.P_ONCE[F16] * 65504).all()
