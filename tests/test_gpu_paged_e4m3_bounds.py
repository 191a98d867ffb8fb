"""Attention over the quantised cache, on the GPU: the one-token kernel's own bound (a weight as an fp16 pair) where its special
arithmetic is at work, and row attention with a workspace that holds anything."""
import pytest
import torch

from tests import paged_e4m3_ref as r8
from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F16, _rand, ctx, i32   # noqa: F401
from tests.test_gpu_paged_e4m3 import PAIR, U8, _attend, _bits, _cu
from tests.test_gpu_paged_e4m3_edges import U8_of
from tests.test_gpu_paged_e4m3_parts import _workspace

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the pair's bound

@pytest.mark.parametrize("qe,ke,ve", [(60, -60, 0), (-60, 60, 0), (-100, 90, 0), (0, 0, 60), (0, 0, -25), (30, -30, 90)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 32)])
def test_exponents(ctx, qe, ke, ve, D, page):   # noqa: F811
    """bf16 queries and scales whose powers of two cancel."""
    lens = [300, 33]
    for news in ([1, 1], [2, 2]):
        pg = r8.Pages8(5, lens, 2, D, page)
        used = pg.ks != 255
        pg.ks[used] += U8_of(ke)
        pg.vs[used] += U8_of(ve)
        Q = (_rand(6, sum(news), 8, D) * 2.0 ** qe).to(BF16)
        O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=None if max(news) == 1 else _cu(news), max_rows=max(news))
        ref.check_attend(O, L, r8.attend(pg, lens, news, Q), BF16, PAIR, f"{news}")
    ctx.sync()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("spread,scale", [((1.0, 24.0), 1.0), ((0.0, 0.0), 30.0), ((6.0, 1.0), 1.0)])
@pytest.mark.parametrize("H_q,H_kv,D,page", [(8, 2, 128, 16), (8, 2, 64, 64), (4, 2, 256, 16)])
def test_magnitudes(ctx, dtype, spread, scale, H_q, H_kv, D, page):   # noqa: F811
    for news in (None, [2, 2, 2], [2, 1, 1]):
        _attend(ctx, [700, 70, 33], H_q, H_kv, D, page, dtype, news=news, spread=spread, scale=scale, max_rows=None if news is None else 2, p_err=PAIR)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("width", [None, 400])
@pytest.mark.parametrize("W", [0, 70])
def test_shared_pages(ctx, dtype, width, W):   # noqa: F811
    pg = r8.Pages8(11, [300, 200], 2, 64, 16, width=width)
    pg.table = torch.cat((pg.table, pg.table[:1], pg.table[:1]))
    lens = [300, 200, 256, 100]
    pg.lens = torch.tensor(lens, dtype=i32, device="cuda")
    for news in ([1] * 4, [2, 1, 2, 2]):
        Q = _rand(3, sum(news), 8, 64, dtype=dtype)
        O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=None if max(news) == 1 else _cu(news), max_rows=max(news), window=W, sinks=3 if W else 0)
        ref.check_attend(O, L, r8.attend(pg, lens, news, Q, window=W, sinks=3 if W else 0), dtype, PAIR)
    ctx.sync()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_k_and_v_laid_out_apart(ctx, dtype):   # noqa: F811
    a, b = r8.Pages8(9, [77, 150], 3, 64, 32), r8.Pages8(9, [77, 150], 3, 64, 32, nhd=True)
    big = torch.zeros((a.k.shape[0], 3, 32, 3 * 64), dtype=U8, device="cuda")
    big[..., 64:128] = _bits(a.k)
    a.k, a.v = big.view(r8.E4M3)[..., 64:128], b.v
    for news in ([1, 1], [2, 2]):
        Q = _rand(4, sum(news), 6, 64, dtype=dtype)
        O, L = ctx.paged_attend(a.cache(), a.table, a.lens, Q, cu_rows=None if max(news) == 1 else _cu(news), max_rows=max(news))
        ref.check_attend(O, L, r8.attend(b, [77, 150], news, Q), dtype, PAIR)
    ctx.sync()


# ------------------------------------------------------------------ a workspace that holds anything

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("width", [None, 900])             # pages numbered by the sequences, and at the cache's own numbers
@pytest.mark.parametrize("lens,news,H_q,H_kv,D,page,W,sinks", [
    ([2000, 500], [700, 500], 24, 8, 128, 64, 256, 4), ([1500, 40], [200, 40], 8, 8, 64, 16, 100, 20), ([900, 3], [300, 2], 6, 2, 64, 112, 1, 0),
    ([1999, 130, 0], [130, 130, 3], 8, 2, 128, 128, 200, 150), ([1000, 77], [333, 77], 12, 4, 128, 48, 90, 50), ([5000], [64], 32, 8, 128, 128, 0, 0),
    ([3001, 17], [33, 17], 8, 1, 64, 48, 700, 130)])
def test_what_the_workspace_held_does_not_matter(ctx, dtype, width, lens, news, H_q, H_kv, D, page, W, sinks):   # noqa: F811
    """All bits set (NaN in the 16-bit pages, -1 in the page map) or none: the same result, and nothing reported. The pages read
    back hold only tokens that some row sees; tiles begin and end among others, between the sinks and the window and behind the
    last token."""
    pg = r8.Pages8(6, lens, H_kv, D, page, width=width)
    c, T = pg.cache(), sum(news)
    Q = _rand(7, T, H_q, D, dtype=dtype)
    n = _workspace(ctx, c, pg.table, lens, news, T, H_q, dtype, W, sinks)
    got = []
    for fill in (0xff, 0, 0x7f):
        ws = torch.full((n,), fill, dtype=U8, device="cuda")
        got.append(ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=_cu(news), window=W, sinks=sinks, workspace=ws))
        ctx.sync()
    for O, L in got[1:]:
        assert torch.equal(O, got[0][0]) and torch.equal(L, got[0][1])
    ref.check_attend(*got[0], r8.attend(pg, lens, news, Q, window=W, sinks=sinks), dtype, ref.P_ONCE[dtype])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,H_q,H_kv,D,page,W", [([2000] * 20, 8, 8, 64, 16, 0), ([40000, 3], 8, 2, 128, 48, 0), ([3000, 0, 9000], 8, 2, 256, 32, 5000)])
def test_and_that_of_one_token(ctx, dtype, lens, H_q, H_kv, D, page, W):   # noqa: F811
    """The partials and join descriptors of split items: only what the call itself wrote is read."""
    pg = r8.Pages8(6, lens, H_kv, D, page)
    c = pg.cache()
    Q = _rand(7, len(lens), H_q, D, dtype=dtype)
    first = ctx.paged_attend(c, pg.table, pg.lens, Q, window=W)
    n = max(c._ws.values())
    assert n > 0
    for fill in (0xff, 0, 0x7f):
        O, L = ctx.paged_attend(c, pg.table, pg.lens, Q, window=W, workspace=torch.full((n,), fill, dtype=U8, device="cuda"))
        ctx.sync()
        assert torch.equal(O, first[0]) and torch.equal(L, first[1])
    ref.check_attend(*first, r8.attend(pg, lens, [1] * len(lens), Q, window=W), dtype, PAIR)
