"""Attention of ragged rows over a paged cache (causal, windows with sinks, few rows over long caches,
merged with a prior) on the GPU against the 64-bit form."""
import math

import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_paged import BF16, F16, _rand, ctx, i32   # noqa: F401

pytestmark = pytest.mark.gpu


def _cu(news):
    return torch.tensor([0] + torch.tensor(news).cumsum(0).tolist(), dtype=i32, device="cuda")


def _case(ctx, lens, news, H_q, H_kv, D, page, dtype, W=0, sinks=0, prior=False, nhd=False, seed=1, pad=0, scale=1.0, width=None,
          max_rows=None, split_p=False):
    need_gpu()
    pg = ref.Pages(seed, lens, H_kv, D, page, dtype, nhd=nhd, width=width)
    T = sum(news)
    big = _rand(seed + 1, T + pad, H_q + 3, D, dtype=dtype, scale=scale)
    Q = big[:, 2:H_q + 2]
    pr = None
    if prior:
        pr = _rand(seed + 2, T + pad, H_q, D), _rand(seed + 3, T + pad, H_q) + 3
        pr[1][0, 0] = -math.inf
        pr[0][0, 0] = math.nan
    c = binding.PagedCache(pg.k, pg.v)
    O = torch.full((T + pad, H_q, D), 5.0, dtype=dtype, device="cuda")
    L = torch.full((T + pad, H_q), 6.0, device="cuda")
    kw = dict(cu_rows=_cu(news), window=W, sinks=sinks, prior=pr, max_rows=max_rows)
    ctx.paged_attend(c, pg.table, pg.lens, Q, O=O, LSE=L, **kw)
    want = ref.attend(pg.k, pg.v, pg.table, lens, news, Q[:T], W, sinks, None if pr is None else (pr[0][:T], pr[1][:T]))
    ref.check_attend(O[:T], L[:T], want, dtype, (ref.P_SPLIT if split_p else ref.P_ONCE)[dtype], f"lens {lens[:4]} news {news[:4]} D {D} W {W}")
    assert (O[T:] == 5).all() and (L[T:] == 6).all()       # rows behind the last sequence, left as they were
    O2, L2 = ctx.paged_attend(c, pg.table, pg.lens, Q, **kw)
    assert torch.equal(O[:T], O2[:T]) and torch.equal(L[:T], L2[:T])
    ctx.sync()
    return pg, c, Q, O[:T], L[:T]


SHAPES = [
    ([1], [1], 1, 1, 64, 16), ([5], [5], 4, 2, 128, 16), ([128], [128], 2, 2, 128, 128), ([300], [300], 8, 2, 128, 64),
    ([129, 0, 17, 500, 64], [129, 0, 17, 100, 1], 6, 2, 64, 32), ([1000], [257], 7, 1, 128, 48), ([700, 900], [3, 600], 16, 1, 128, 16),
    ([200, 40], [150, 40], 40, 1, 64, 16), ([1500], [1400], 12, 12, 64, 128), ([260], [260], 128, 1, 64, 16), ([4], [9], 2, 1, 64, 16),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,news,H_q,H_kv,D,page", SHAPES)
def test_rows(ctx, dtype, lens, news, H_q, H_kv, D, page):   # noqa: F811
    _case(ctx, lens, news, H_q, H_kv, D, page, dtype)
    _case(ctx, lens, news, H_q, H_kv, D, page, dtype, prior=True, nhd=True, pad=7, seed=5, max_rows=max(news))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("W,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (128, 17), (200, 130), (513, 4), (700, 5000), (100000, 4)])
def test_rows_window(ctx, dtype, W, sinks):   # noqa: F811
    _case(ctx, [1100, 333, 0, 17], [1100, 90, 0, 17], 8, 2, 128, 16, dtype, W, sinks)
    _case(ctx, [900, 1300], [1, 700], 6, 2, 64, 64, dtype, W, sinks, prior=True, nhd=True, pad=3)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,news,H_q,H_kv,D,page,W,sinks", [
    ([9000], [4], 32, 8, 128, 16, 0, 0), ([20000, 100], [2, 3], 4, 1, 64, 64, 0, 0), ([5000, 0, 7000], [17, 2, 1], 8, 2, 128, 128, 4000, 4),
    ([12000], [300], 2, 2, 128, 32, 0, 0)])
def test_few_rows_over_a_long_cache(ctx, dtype, lens, news, H_q, H_kv, D, page, W, sinks):   # noqa: F811
    _case(ctx, lens, news, H_q, H_kv, D, page, dtype, W, sinks)
    _case(ctx, lens, news, H_q, H_kv, D, page, dtype, W, sinks, prior=True, max_rows=max(news), width=2000)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H_q,H_kv,D,rows", [(4, 1, 64, 4), (8, 2, 128, 2), (6, 2, 128, 5), (4, 1, 128, 1), (8, 8, 128, 16), (8, 2, 192, 2),
                                             (2, 1, 256, 4), (3, 3, 256, 7)])
def test_a_few_rows(ctx, dtype, H_q, H_kv, D, rows):   # noqa: F811
    """Rows that share the one-token kernel's columns: a CTA per item, a range per CTA, a range per warp."""
    few = [min(rows, n) for n in (1, 2, rows, rows, 0, rows)]
    for lens, news in (([1, 17, 500, 33, 0, 2], few), ([1, 17, 5000, 33, 9, 2], few), ([(31 * i * i) % 900 for i in range(330)], [i % (rows + 1) for i in range(330)])):
        lens = [max(n, m) if i % 3 else n for i, (n, m) in enumerate(zip(lens, news))]     # some rows in front of their cache
        for kw in (dict(), dict(W=40, sinks=5, prior=True, nhd=True, pad=2), dict(W=1, sinks=0)):
            _case(ctx, lens, news, H_q, H_kv, D, 16, dtype, max_rows=rows, split_p=True, **kw)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_large_scores(ctx, dtype):   # noqa: F811
    """Scores in the hundreds, and scores that grow along the cache so that every block moves the maximum."""
    _case(ctx, [700], [500], 4, 2, 128, 16, dtype, scale=20.0)
    for rows, width in ((1500, None), (5, 900)):
        pg = ref.Pages(3, [1500], 1, 64, 16, dtype, width=width)
        Q = torch.ones((rows, 2, 64), dtype=dtype, device="cuda")
        p = torch.arange(1500, device="cuda")
        pg.k[pg.table[0, p // 16].long(), :, p % 16] = (p / 20.0).to(dtype)[:, None, None]
        O, L = ctx.paged_attend(binding.PagedCache(pg.k, pg.v), pg.table, pg.lens, Q, cu_rows=_cu([rows]))
        ref.check_attend(O, L, ref.attend(pg.k, pg.v, pg.table, [1500], [rows], Q), dtype, ref.P_ONCE[dtype])


@pytest.mark.parametrize("rows,width,W,sinks", [(300, None, 0, 0), (20, 3000, 0, 0), (300, None, 60, 5), (20, 3000, 600, 2), (8, None, 0, 0),
                                                (8, None, 20, 5), (8, 3000, 700, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_value_that_is_not_finite_stays_with_the_rows_that_see_it(ctx, rows, width, W, sinks, bad):   # noqa: F811
    """V (or K) of one token is not finite: rows that do not see it are as if it were not there."""
    n, D, H_q, H_kv = 1300, 64, 4, 2
    pg = ref.Pages(7, [n], H_kv, D, 16, F16, width=width)
    Q = _rand(8, rows, H_q, D, dtype=F16)
    c = binding.PagedCache(pg.k, pg.v)
    at = torch.arange(n - rows, n, device="cuda")
    for which in ("v", "k"):
        for j in (max(n - rows, n - rows + 13 if rows > 13 else n - 3), n - 30, n - 7, 1):
            t = getattr(pg, which)
            page, slot = int(pg.table[0, j // 16]), j % 16
            old = t[page, :, slot].clone()
            t[page, :, slot, 3] = bad
            O, L = ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=_cu([rows]), max_rows=rows, window=W, sinks=sinks)
            t[page, :, slot] = old
            see = at >= j
            if W:
                see &= (at - W < j) | (j < sinks)
            want = ref.attend(pg.k, pg.v, pg.table, [n], [rows], Q, W, sinks)
            blind = [x[~see] for x in want]
            if (~see).any():
                ref.check_attend(O[~see], L[~see], blind, F16, ref.P_ONCE[F16], f"{which} {j}")
            if which == "v":
                assert not torch.isfinite(O[see][..., 3]).any()
                keep = [d for d in range(D) if d != 3]
                ref.check_attend(O[see][..., keep], L[see], [want[0][see][..., keep]] + [x[see] for x in want[1:]], F16, ref.P_ONCE[F16], f"{which} {j}")
    ctx.sync()


def test_hidden_pages_are_not_read(ctx):   # noqa: F811
    lens, news, W, sinks = [3000, 700], [50, 1], 300, 20
    pg, c, Q, O, L = _case(ctx, lens, news, 8, 2, 128, 16, F16, W, sinks)
    table = pg.table.clone()
    for b, (n, m) in enumerate(zip(lens, news)):
        first = n - m + 1 - W
        for i in range(table.shape[1]):
            if 16 * i >= n or (16 * i >= sinks and 16 * i + 15 < first):
                table[b, i] = -7
                if 16 * i < n:
                    pg.k[pg.table[b, i]], pg.v[pg.table[b, i]] = math.nan, math.nan
    O2, L2 = ctx.paged_attend(c, table, pg.lens, Q, cu_rows=_cu(news), window=W, sinks=sinks)
    assert torch.equal(O, O2) and torch.equal(L, L2)
    ctx.sync()


def test_rows_out_of_range_are_reported(ctx):   # noqa: F811
    pg, c, Q, O, L = _case(ctx, [400, 100], [300, 20], 4, 2, 64, 16, F16)
    cu = _cu([300, 20])

    def code(*a, **kw):
        ctx.paged_attend(*a, **kw)
        with pytest.raises(binding.PckError) as e:
            ctx.sync()
        ctx.sync()
        return str(e.value)

    for bad in (-1, c.n_pages):
        t = pg.table.clone()
        t[0, 3] = bad
        assert "code 8" in code(c, t, pg.lens, Q, cu_rows=cu)
    assert "code 10" in code(c, pg.table, pg.lens + 500, Q, cu_rows=cu)
    assert "code 10" in code(c, pg.table, pg.lens, Q, cu_rows=cu, max_rows=10)
    assert "code 10" in code(c, pg.table, pg.lens, Q, cu_rows=cu, max_rows=4)
    O2, L2 = ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=cu)
    assert torch.equal(O, O2) and torch.equal(L, L2)
    with pytest.raises(binding.PckError) as e:
        d = torch.zeros((3, 1, 16, 256), dtype=F16, device="cuda")
        ctx.paged_attend(binding.PagedCache(d, d), pg.table, pg.lens, _rand(1, 320, 2, 256, dtype=F16), cu_rows=cu, max_rows=5)
    assert e.value.code == binding.EUNSUPPORTED
    with pytest.raises(binding.PckError) as e:
        ctx.paged_attend(c, pg.table, pg.lens, _rand(1, 320, 2 * 129, 64, dtype=F16), cu_rows=cu)
    assert e.value.code == binding.EUNSUPPORTED
    with pytest.raises(binding.PckError) as e:
        ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=cu, max_rows=0)
    assert e.value.code == binding.EINVAL


def test_chunked_prompt_equals_the_whole_and_the_token_steps(ctx):   # noqa: F811
    """A prompt appended and attended in chunks gives the rows of one call, and its last row is a one-token call's."""
    H_q, H_kv, D, P, n = 8, 2, 128, 32, 700
    x = _rand(3, n, H_q + 2 * H_kv, D, dtype=BF16)
    cs = ref.angles(n, D, "cuda")
    table = torch.randperm(30, device="cuda")[:-(-n // P)].to(i32)[None].contiguous()
    k, v = (torch.full((30, H_kv, P, D), math.nan, dtype=BF16, device="cuda") for _ in range(2))
    c = binding.PagedCache(k, v)
    out, at = [], 0
    for m in (300, 1, 399):
        at += m
        s = x[at - m:at]
        ln = torch.tensor([at], dtype=i32, device="cuda")
        q = ctx.paged_append(c, table, ln, s[:, H_q:H_q + H_kv], s[:, H_q + H_kv:], Q=s[:, :H_q], cu_rows=_cu([m]), cos_sin=cs, norm=True)
        out.append((q, *ctx.paged_attend(c, table, ln, q, cu_rows=_cu([m]))))
    q, O, L = (torch.cat(t) for t in zip(*out))
    want = ref.attend(k, v, table, [n], [n], q)
    ref.check_attend(O, L, want, BF16, ref.P_ONCE[BF16])
    O1, L1 = ctx.paged_attend(c, table, ln, q[-1:])
    ref.check_attend(O1, L1, [t[-1:] for t in want], BF16, ref.P_SPLIT[BF16])
    ctx.sync()


def test_prompt_in_a_graph_with_other_lengths(ctx):   # noqa: F811
    """A captured call follows the lengths and row counts it finds at replay."""
    H_q, H_kv, D, P, T = 8, 2, 64, 16, 400
    for width, lens, news in ((60, [[300, 100], [50, 900], [0, 400]], [[300, 100], [50, 350], [0, 400]]),
                              (900, [[9000, 30], [14000, 2]], [[20, 5], [3, 2]])):
        pg = ref.Pages(4, [16 * width // 2 if b else min(16 * width, 14400) for b in range(2)], H_kv, D, P, F16, width=width)
        rows = T if width == 60 else 25
        Q = _rand(5, rows, H_q, D, dtype=F16)
        ln, cu = torch.zeros(2, dtype=i32, device="cuda"), torch.zeros(3, dtype=i32, device="cuda")
        c = binding.PagedCache(pg.k, pg.v)
        ctx.paged_attend(c, pg.table, ln, Q, cu_rows=cu)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            O, L = ctx.paged_attend(c, pg.table, ln, Q, cu_rows=cu)
        for a, m in zip(lens, news):
            a = [min(x, int((pg.lens[i]))) for i, x in enumerate(a)]
            ln.copy_(torch.tensor(a, dtype=i32))
            cu.copy_(_cu(m))
            g.replay()
            torch.cuda.synchronize()
            t = sum(m)
            ref.check_attend(O[:t], L[:t], ref.attend(pg.k, pg.v, pg.table, a, m, Q[:t]), F16, ref.P_ONCE[F16])
    ctx.sync()


def test_row_counts_that_make_no_sense(ctx):   # noqa: F811
    """cu_rows that does not ascend, points outside the rows, or wraps: nothing outside O and LSE is touched, and sound
    calls are right afterwards."""
    pg, c, Q, O, L = _case(ctx, [400, 100], [300, 20], 4, 2, 64, 16, F16)
    big = 2 ** 31 - 1
    buf = torch.full((3, 320, 4, 64), 3.0, dtype=F16, device="cuda")
    lse = torch.full((3, 320, 4), 4.0, device="cuda")
    kk = pg.k.clone()
    for cu in ([0, 320, 300], [300, 0, 320], [-5, 100, 320], [0, big, 20], [-big - 1, big, 320], [310, 320, 900], [big, big, big], [0, 5, -big]):
        t = torch.tensor(cu, dtype=i32, device="cuda")
        for mr in (None, 4):
            ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=t, max_rows=mr, O=buf[1], LSE=lse[1])
            ctx.paged_append(c, pg.table, pg.lens - 400, Q[:, :2], Q[:, 2:], cu_rows=t)
            try:
                ctx.sync()
            except binding.PckError:
                pass
    for ln in (-1, -big - 1, big):
        ctx.paged_attend(c, pg.table, torch.full_like(pg.lens, ln), Q, cu_rows=_cu([300, 20]), O=buf[1], LSE=lse[1])
        ctx.paged_attend(c, pg.table, torch.full_like(pg.lens, ln), Q[:2], O=buf[1, :2], LSE=lse[1, :2])
        ctx.paged_append(c, pg.table, torch.full_like(pg.lens, ln), Q[:2, :2], Q[:2, 2:])
        try:
            ctx.sync()
        except binding.PckError:
            pass
    assert (buf[0] == 3).all() and (buf[2] == 3).all() and (lse[0] == 4).all() and (lse[2] == 4).all()
    ctx.sync()
    pg.k.copy_(kk)
    O2, L2 = ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=_cu([300, 20]))
    assert torch.isfinite(O2.float()).all()


def test_widest_windows_and_rows_in_front_of_the_cache(ctx):   # noqa: F811
    for W, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (3, 2 ** 31 - 1)):
        _case(ctx, [5, 300], [40, 200], 4, 2, 64, 16, F16, W, sinks)
        _case(ctx, [5, 300], [4, 3], 4, 2, 64, 16, F16, W, sinks, max_rows=4, split_p=True)


def test_many_sequences(ctx):   # noqa: F811
    """Hundreds of sequences, empty ones among them, with rows enough for the row kernel."""
    lens = [(13 * i) % 90 + 40 for i in range(700)]
    news = [(0, 7, 33)[i % 3] if i % 5 else 1 for i in range(700)]
    _case(ctx, lens, news, 4, 1, 64, 16, F16)
    _case(ctx, lens, news, 6, 2, 64, 16, BF16, W=20, sinks=3, max_rows=33, pad=4)


@pytest.mark.parametrize("D,H_kv", [(128, 8), (64, 16)])
def test_pages_beyond_32_bits(ctx, D, H_kv):   # noqa: F811
    """Pages more than 2^31 elements (and 2^32 bytes) into the cache: append, one token, rows, and a value that is not
    finite among them."""
    P, n_pages = 64, 2 ** 31 // (H_kv * 64 * D) + 40
    k, v = (torch.empty((n_pages, H_kv, P, D), dtype=F16, device="cuda") for _ in range(2))
    n, m, H_q = 700, 200, 2 * H_kv
    table = (n_pages - 1 - torch.arange(11, device="cuda")).to(i32)[None].contiguous()
    x = _rand(5, n, H_q + 2 * H_kv, D, dtype=F16)
    c = binding.PagedCache(k, v)
    ln = torch.tensor([n], dtype=i32, device="cuda")
    q = ctx.paged_append(c, table, ln, x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:], Q=x[:, :H_q], cu_rows=_cu([n]), norm=True)
    assert torch.equal(v[table[0, 3].long(), :, 5], x[3 * P + 5, H_q + H_kv:])
    small = slice(n_pages - 11, n_pages)
    tab = table - (n_pages - 11)
    want = ref.attend(k[small], v[small], tab, [n], [m], q[n - m:])
    O, L = ctx.paged_attend(c, table, ln, q[n - m:], cu_rows=_cu([m]))
    ref.check_attend(O, L, want, F16, ref.P_ONCE[F16])
    O, L = ctx.paged_attend(c, table, ln, q[-1:])
    ref.check_attend(O, L, [t[-1:] for t in want], F16, ref.P_SPLIT[F16])
    v[table[0, (n - 50) // P].long(), :, (n - 50) % P] = math.nan
    O, L = ctx.paged_attend(c, table, ln, q[n - m:], cu_rows=_cu([m]))
    ref.check_attend(O[:m - 50], L[:m - 50], [t[:m - 50] for t in want], F16, ref.P_ONCE[F16])
    assert torch.isnan(O[m - 50:]).all()
    ctx.sync()
