"""The quantised paged cache on the GPU against its 64-bit form: the append that quantises, rows read back, attention of one
row, a few rows and ragged rows over the codes, and a run of them together."""
import math

import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_e4m3_ref as r8
from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F16, F32, _close, _rand, ctx, i32   # noqa: F401

pytestmark = pytest.mark.gpu
U8 = torch.uint8


def _cu(news):
    return torch.tensor([0] + list(torch.tensor(news).cumsum(0)), dtype=i32, device="cuda")


def _bits(x):
    return x.view(U8)


def _empty_pages(n_pages, H_kv, page, D, nhd=False):
    shape = (n_pages, page, H_kv, D) if nhd else (n_pages, H_kv, page, D)
    k, v = (torch.full(shape, 0x55, dtype=U8, device="cuda") for _ in range(2))
    if nhd:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    ks, vs = (torch.full((n_pages, H_kv, page), 0x33, dtype=U8, device="cuda") for _ in range(2))
    return k.view(r8.E4M3), v.view(r8.E4M3), ks, vs


# ------------------------------------------------------------------ append

def _check_rows(codes, byte, want, what):
    """Codes and bytes of rows whose 64-bit values are `want`. The kernel's fp32 row is off by at most `slip` (norm_rope_tol's
    arithmetic); the scale is the least that holds its largest value, and a code is off by half a step of that row's value."""
    big = want.abs().amax(-1)
    slip = 64 * 2.0 ** -24 * big
    e = byte.double() - 127
    assert (448 * torch.exp2(e) >= big - slip).all(), f"{what}: scale too small"
    assert ((448 * torch.exp2(e - 1) < big + slip) | (e == -126)).all(), f"{what}: scale too large"
    got = r8.values(codes, byte)
    tol = r8.HALF_STEP * want.abs() + (slip * (1 + r8.HALF_STEP) + 2.0 ** -10 * torch.exp2(e))[..., None]
    over = ((got - want).abs() - tol).max().item()
    assert over <= 0, f"{what}: {over:.3e} over its bound"


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("lens,news,H_q,H_kv,D,R,page,inter,nhd", [
    ([1], [1], 1, 1, 16, 16, 16, False, False), ([17, 1, 160, 33], [1, 1, 1, 1], 8, 2, 64, 64, 16, False, True),
    ([40, 0, 300, 16, 7], [40, 0, 123, 3, 7], 6, 2, 128, 64, 32, True, False),
    ([100, 257], [64, 1], 4, 4, 256, 256, 48, False, False), ([64] * 70, [2] * 70, 3, 1, 96, 96, 64, False, True),
    ([9, 33], [9, 20], 2, 3, 512, 128, 16, True, False), ([50], [31], 1, 5, 48, 32, 16, False, False)])
def test_append(ctx, dtype, lens, news, H_q, H_kv, D, R, page, inter, nhd):   # noqa: F811
    pg = ref.Pages(5, lens, 1, 16, page, F16)          # its table
    T, one = sum(news), all(m == 1 for m in news)
    pad = 0 if one else 5                              # rows behind the last sequence
    x = _rand(6, T + pad, H_q + 2 * H_kv, D, dtype=dtype)
    Q, K, V = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    wq, wk = 1 + _rand(1, D, dtype=dtype, scale=0.2), 1 + _rand(2, D, dtype=dtype, scale=0.2)
    cs = ref.angles(max(lens) + 50, R, "cuda")
    cu = None if one else _cu(news)
    at = ref.rows_of(lens, news)
    p = torch.tensor([q for _, q in at], device="cuda")
    b = torch.tensor([q for q, _ in at], device="cuda")
    pages, slots = pg.table[b, p // page].long(), p % page
    for positions in (None, (p + 50).to(i32)):
        k, v, ks, vs = _empty_pages(int(pg.table.max()) + 2, H_kv, page, D, nhd)
        Qo = torch.full((T + pad, H_q, D), 9.0, dtype=dtype, device="cuda")
        if positions is not None:
            positions = torch.cat((positions, torch.full((pad,), 1 << 30, dtype=i32, device="cuda")))
        c = binding.QuantizedPagedCache(k, v, ks, vs)
        ctx.paged_append(c, pg.table, pg.lens, K, V, Q=Q, cu_rows=cu, cos_sin=cs, positions=positions, q_weight=wq,
                         k_weight=wk, eps=1e-5, interleaved=inter, Q_out=Qo)
        at_pos = p if positions is None else positions[:T]
        _close(Qo[:T], ref.norm_rope(Q[:T], wq, 1e-5, cs, at_pos, inter), dtype, "q")
        assert (Qo[T:] == 9).all()
        _check_rows(_bits(k)[pages, :, slots].view(r8.E4M3), ks[pages, :, slots], ref.norm_rope(K[:T], wk, 1e-5, cs, at_pos, inter), "k")
        want, e = r8.quantize(V[:T])
        assert torch.equal(vs[pages, :, slots].long() - 127, e)
        assert torch.equal(r8.values(_bits(v)[pages, :, slots].view(r8.E4M3), torch.full_like(vs[pages, :, slots], 127)), want)
        for t, was in ((_bits(k), 0x55), (_bits(v), 0x55), (ks, 0x33), (vs, 0x33)):     # and nothing else was written
            t[pages, :, slots] = was
            assert (t == was).all()
    ctx.sync()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_append_values_at_the_ends(ctx, dtype):   # noqa: F811
    """Rows as they are (no norm, no rotation): zeros, the type's largest and smallest values, scales at their ends, values
    between two codes, infinities and NaN. Codes and scales are those of the 64-bit form."""
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    D = 32
    rows = torch.zeros((12, D), dtype=torch.float64)
    rows[1, 3], rows[1, 4] = top, -top / 2
    rows[2, 5], rows[2, 6] = low, 3 * low
    rows[3, :8] = torch.tensor([448.0, 432.0, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -17.0])
    rows[4, :3] = torch.tensor([449.0, 1.0, -0.01])
    rows[5, :3] = torch.tensor([math.inf, 1.0, -0.5])
    rows[6, :3] = torch.tensor([-math.inf, math.nan, 0.0])
    rows[7] = math.nan
    rows[8, 31] = 1e-5
    rows[9] = torch.linspace(-1.75, 1.75, D)
    rows[10] = torch.linspace(-1.76, 1.76, D)
    rows[11, 0], rows[11, 1:] = 60000.0, torch.logspace(-7, 4, D - 1)
    x = rows.to(dtype)[:, None].cuda().repeat(1, 3, 1)
    k, v, ks, vs = _empty_pages(2, 3, 16, D)
    tab, ln = torch.tensor([[1]], dtype=i32, device="cuda"), torch.tensor([12], dtype=i32, device="cuda")
    ctx.paged_append(binding.QuantizedPagedCache(k, v, ks, vs.view(r8.E8M0)), tab, ln, x, x, cu_rows=_cu([12]))
    want, e = r8.quantize(x)
    for codes, scale in ((k, ks), (v, vs)):
        got = r8.values(codes[1].transpose(0, 1)[:12].contiguous(), torch.full((12, 3), 127, dtype=U8, device="cuda"))
        assert torch.equal(scale[1].t()[:12].long() - 127, e)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
    ctx.sync()


def test_append_of_padded_sequences(ctx):   # noqa: F811
    """Rows at a negative cache position store nothing, and their Q is 0."""
    for lens, news in (([9, 0, 17, 0], [1, 1, 1, 1]), ([40, 2, 0], [3, 6, 4])):
        pg = r8.Pages8(2, lens, 2, 64, 16)
        T = sum(news)
        x = _rand(3, T, 9, 64, dtype=BF16)
        k0, s0 = _bits(pg.k).clone(), pg.ks.clone()
        Q = ctx.paged_append(pg.cache(), pg.table, pg.lens, x[:, 5:7], x[:, 7:], Q=x[:, :5], cu_rows=None if T == len(lens) else _cu(news))
        at = ref.rows_of(lens, news)
        for t, (b, p) in enumerate(at):
            assert torch.equal(Q[t], x[t, :5] if p >= 0 else torch.zeros_like(x[t, :5]))
            if p >= 0:
                k0[pg.table[b, p // 16], :, p % 16] = _bits(pg.k)[pg.table[b, p // 16], :, p % 16]
                s0[pg.table[b, p // 16], :, p % 16] = pg.ks[pg.table[b, p // 16], :, p % 16]
        assert torch.equal(k0, _bits(pg.k)) and torch.equal(s0, pg.ks)
    ctx.sync()


# ------------------------------------------------------------------ reading back

def _read_want(pg, lens, news, dtype):
    k, v = pg.kv()
    page = pg.k.shape[2]
    out = []
    for x in (k, v):
        rows = [x[pg.table[b, p // page].long(), :, p % page] if p >= 0 else torch.zeros_like(x[0, :, 0]) for b, p in ref.rows_of(lens, news)]
        y = torch.stack(rows)
        out.append((y.clamp(-65504, 65504) if dtype == F16 else y).to(dtype))
    return out


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("lens,news,H_kv,D,page,nhd", [
    ([1], None, 1, 16, 16, False), ([17, 0, 160, 33], None, 2, 64, 16, True), ([40, 300, 16, 7], [40, 123, 3, 0], 3, 128, 32, False),
    ([100, 257], [100, 257], 2, 48, 48, False), ([5, 0, 90], [9, 3, 33], 2, 256, 64, True), ([65, 31], [64, 31], 5, 80, 16, False),
    ([1000] * 3, [999, 1, 1000], 1, 512, 128, False), (list(range(1, 200)), list(range(1, 200)), 2, 64, 16, False)])
def test_read(ctx, dtype, lens, news, H_kv, D, page, nhd):   # noqa: F811
    pg = r8.Pages8(4, lens, H_kv, D, page, nhd=nhd, spread=(8.0, 40.0))
    one = news is None
    news = [1] * len(lens) if one else news
    T = sum(news)
    want = _read_want(pg, lens, news, dtype)
    cu = None if one else _cu(news)
    got = ctx.paged_read(pg.cache(), pg.table, pg.lens, T=None if one else T, cu_rows=cu, dtype=dtype)
    for x, w in zip(got, want):
        assert x.dtype == dtype and torch.equal(x, w)
    # heads first, behind and in front of other rows
    Ko = torch.full((H_kv, T + 3, D), 7.0, dtype=dtype, device="cuda")
    Vo = torch.full((T, H_kv + 1, D), 7.0, dtype=dtype, device="cuda")
    ctx.paged_read(pg.cache(), pg.table, pg.lens, cu_rows=cu, K_out=Ko.transpose(0, 1)[:T], V_out=Vo[:, :H_kv])
    assert torch.equal(Ko[:, :T].transpose(0, 1), want[0]) and torch.equal(Vo[:, :H_kv], want[1])
    assert (Ko[:, T:] == 7).all() and (Vo[:, H_kv] == 7).all()
    ctx.sync()


def test_read_every_code_and_leave_other_rows(ctx):   # noqa: F811
    k = torch.arange(256, dtype=U8, device="cuda").view(1, 1, 16, 16).repeat(1, 2, 1, 1)
    for dtype in (F32, BF16, F16):
        scale = torch.tensor([0, 1, 2, 50, 100, 120, 126, 127, 128, 134, 135, 136, 200, 247, 254, 255], dtype=U8, device="cuda").expand(1, 2, 16).contiguous()
        c = binding.QuantizedPagedCache(k.view(r8.E4M3), k.flip(3).contiguous().view(r8.E4M3), scale, scale)
        tab, ln = torch.zeros((1, 1), dtype=i32, device="cuda"), torch.tensor([16], dtype=i32, device="cuda")
        out = [torch.full((20, 2, 16), 3.0, dtype=dtype, device="cuda") for _ in range(2)]
        ctx.paged_read(c, tab, ln, cu_rows=torch.tensor([2, 18], dtype=i32, device="cuda"), K_out=out[0], V_out=out[1])
        for o, x in zip(out, (c.k, c.v)):
            assert (o[:2] == 3).all() and (o[18:] == 3).all()
            w = r8.values(x, scale)[0].transpose(0, 1)
            w = (torch.where(w.abs() > 65504, torch.copysign(torch.full_like(w, 65504), w), w) if dtype == F16 else w).to(dtype)
            big = 3.0e38 if dtype != F16 else 7e4          # (infinities as themselves)
            assert torch.equal(o[2:18].isnan(), w.isnan())
            assert torch.equal(o[2:18].nan_to_num(0, big, -big), w.nan_to_num(0, big, -big))
    ctx.sync()


# ------------------------------------------------------------------ attention

PAIR = 2.0 ** -22      # relative rounding of a weight of one-token attention: an fp16 hi + lo pair, whatever Q's type


def _attend(ctx, lens, H_q, H_kv, D, page, dtype, news=None, W=0, sinks=0, prior=False, nhd=False, seed=1, scale=1.0, width=None,   # noqa: F811
            max_rows=None, spread=(1.0, 6.0), p_err=None, **kw):
    pg = r8.Pages8(seed, lens, H_kv, D, page, nhd=nhd, width=width, spread=spread)
    one = news is None
    news = [1] * len(lens) if one else news
    T = sum(news)
    Q = _rand(seed + 1, T, H_q + 3, D, dtype=dtype, scale=scale)[:, 1:H_q + 1]
    pr = None
    if prior:
        pr = (_rand(seed + 2, T, H_q, D), _rand(seed + 3, T, H_q) + math.log(max(max(lens), 1)))
        pr[1][0, 0] = -math.inf
    want = r8.attend(pg, lens, news, Q, window=W, sinks=sinks, prior=pr)
    O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=None if one else _cu(news), max_rows=max_rows, window=W,
                            sinks=sinks, prior=pr, **kw)
    ctx.sync()
    assert O.dtype == dtype
    ref.check_attend(O, L, want, dtype, ref.P_ONCE[dtype] if p_err is None else p_err, f"{lens[:4]} {D} {W}")
    return pg, Q, O, L


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,H_q,H_kv,D,page", [
    ([1], 1, 1, 64, 16), ([300], 32, 8, 128, 16), ([15, 16, 17, 0, 31, 32, 33, 1], 8, 2, 64, 16), ([63, 64, 65, 127, 129], 8, 4, 128, 48),
    ([2000, 5, 0, 777], 10, 2, 192, 32), ([1025, 40], 8, 2, 256, 16), ([513, 1, 900], 16, 1, 128, 64), ([257], 20, 1, 64, 16),
    ([333, 70], 66, 3, 128, 112), ([100] * 40, 8, 8, 64, 16), ([9000, 33], 12, 12, 64, 128), ([4097], 17, 1, 256, 32),
    ([20000], 8, 2, 128, 64)])
def test_one_row(ctx, dtype, lens, H_q, H_kv, D, page):   # noqa: F811
    _attend(ctx, lens, H_q, H_kv, D, page, dtype, p_err=PAIR)
    _attend(ctx, lens, H_q, H_kv, D, page, dtype, prior=True, nhd=True, seed=5, p_err=PAIR)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("W,sinks", [(1, 0), (16, 0), (17, 3), (100, 4), (1000, 17), (5000, 4), (250, 400), (33, 40)])
def test_one_row_window(ctx, dtype, W, sinks):   # noqa: F811
    _attend(ctx, [1500, 16, 0, 101, 333], 8, 2, 128, 16, dtype, W=W, sinks=sinks, p_err=PAIR)
    _attend(ctx, [700, 48], 4, 4, 64, 48, dtype, W=W, sinks=sinks, prior=True, seed=3, p_err=PAIR)
    _attend(ctx, [1300, 31, 32], 4, 2, 256, 32, dtype, W=W, sinks=sinks, seed=4, p_err=PAIR)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,lo,hi,H_q,H_kv,D,page,W", [(300, 1, 400, 4, 4, 64, 16, 0), (64, 100, 3000, 8, 8, 128, 32, 0), (40, 1, 6000, 8, 2, 128, 16, 0),
                                                     (24, 2000, 2100, 16, 8, 128, 16, 0), (32, 10, 5000, 64, 8, 128, 16, 512), (16, 900, 4000, 8, 2, 256, 32, 0),
                                                     (200, 500, 1500, 8, 8, 64, 16, 300), (1200, 1, 40, 2, 1, 64, 16, 0)])
def test_one_row_ragged_batches(ctx, dtype, B, lo, hi, H_q, H_kv, D, page, W):   # noqa: F811
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(lo, hi + 1, (B,), generator=g).tolist()
    _attend(ctx, lens, H_q, H_kv, D, page, dtype, W=W, sinks=4 if W else 0, p_err=PAIR)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,news,H_q,H_kv,D,page,W,sinks", [
    ([300, 40, 5000], [4, 1, 3], 8, 2, 64, 16, 0, 0), ([100, 0, 33], [2, 3, 2], 8, 2, 128, 48, 0, 0), ([2100, 64], [8, 2], 2, 2, 128, 16, 200, 5),
    ([700, 90, 17], [4, 4, 4], 4, 2, 256, 32, 100, 0), ([1500, 2], [2, 2], 8, 2, 192, 16, 0, 0)])
def test_a_few_rows(ctx, dtype, lens, news, H_q, H_kv, D, page, W, sinks):   # noqa: F811
    _attend(ctx, lens, H_q, H_kv, D, page, dtype, news=news, W=W, sinks=sinks, max_rows=max(news), p_err=PAIR)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,news,H_q,H_kv,D,page,W,sinks,prior", [
    ([200], [200], 4, 1, 64, 16, 0, 0, False), ([129, 1, 300], [129, 1, 64], 8, 2, 128, 32, 0, 0, True),
    ([1000, 0, 77], [333, 5, 77], 12, 4, 128, 48, 0, 0, False), ([2000, 500], [700, 500], 24, 8, 128, 64, 256, 4, False),
    ([5000], [64], 32, 8, 128, 128, 0, 0, False), ([1500, 40], [200, 40], 8, 8, 64, 16, 100, 20, True), ([900, 3], [300, 2], 6, 2, 64, 112, 1, 0, False)])
def test_rows(ctx, dtype, lens, news, H_q, H_kv, D, page, W, sinks, prior):   # noqa: F811
    _attend(ctx, lens, H_q, H_kv, D, page, dtype, news=news, W=W, sinks=sinks, prior=prior)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("spread,scale", [((1.0, 24.0), 1.0), ((0.0, 0.0), 30.0), ((6.0, 1.0), 1.0)])
def test_magnitudes(ctx, dtype, spread, scale):   # noqa: F811
    """Tokens whose values differ by 2^24, queries that pick one key, keys of very different size."""
    for news in (None, [3, 2, 3], [200, 70, 1]):
        _attend(ctx, [700, 70, 33], 8, 2, 128, 16, dtype, news=news, spread=spread, scale=scale, max_rows=None if news is None else max(news))


def test_hidden_and_visible_values_that_are_not_finite(ctx):   # noqa: F811
    """A NaN code of V, or a NaN scale, spoils the rows that see the token and no other; a NaN in K too."""
    for news, D in ((None, 64), ([3, 2], 128), ([4, 3], 64), ([2, 2], 256), ([150, 9], 128)):
        lens = [403, 90]
        rows = [1, 1] if news is None else news
        for dtype in (F16, BF16):
            base = r8.Pages8(8, lens, 2, D, 16)
            Q = _rand(9, sum(rows), 4, D, dtype=dtype)
            call = lambda pg, **kw: ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=None if news is None else _cu(news),   # noqa: E731
                                                     max_rows=max(rows), **kw)
            want, _ = call(base)
            exact = r8.attend(base, lens, rows, Q, window=100)
            for what in ("v", "k", "vs"):
                pg = r8.Pages8(8, lens, 2, D, 16)
                last, first = 402, 200                     # the last token of sequence 0, and one behind a window of 100
                for p in (last, first):
                    at = (pg.table[0, p // 16].long(), 1, p % 16)
                    if what == "vs":
                        pg.vs[at] = 255
                    else:
                        _bits(pg.v if what == "v" else pg.k)[at][5] = 0x7f
                O, L = call(pg, window=100)
                bad = O.float().isfinite().logical_not()
                clean = []
                for t, (b, p) in enumerate(ref.rows_of(lens, rows)):
                    if any(b == 0 and p - 100 < q <= p for q in (last, first)):
                        assert bad[t, 2:].any(-1).all() and not bad[t, :2].any(), (what, t)
                        if what == "v":
                            assert bad[t, 2:, 5].all() and not bad[t, 2:, :5].any() and not bad[t, 2:, 6:].any()
                    else:
                        clean.append(t)
                ref.check_attend(O[clean], L[clean], [x[clean] for x in exact], dtype, ref.P_ONCE[dtype], what)
            assert torch.equal(call(base)[0], want)
    ctx.sync()


def test_rows_behind_the_sequences_and_table_entries_unused(ctx):   # noqa: F811
    for news, mr in (([3, 2], 3), ([300, 20], None)):
        pg = r8.Pages8(4, [400, 90], 2, 64, 16, width=60)
        T = 2 + sum(news) + 3
        Q = _rand(5, T, 4, 64, dtype=F16)
        cu = torch.tensor([2, 2 + news[0], 2 + sum(news)], dtype=i32, device="cuda")
        O, L = torch.full((T, 4, 64), 5.0, dtype=F16, device="cuda"), torch.full((T, 4), 6.0, device="cuda")
        ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=cu, max_rows=mr, O=O, LSE=L)
        ref.check_attend(O[2:-3], L[2:-3], r8.attend(pg, [400, 90], news, Q[2:-3]), F16, ref.P_ONCE[F16])
        for x, y in ((O[:2], L[:2]), (O[-3:], L[-3:])):
            assert (x == 5).all() and (y == 6).all()
        ctx.sync()


# ------------------------------------------------------------------ what is refused, and what is reported

def _code(ctx, fn):   # noqa: F811
    """The device error code that a call leaves behind (0: none)."""
    ctx.sync()
    fn()
    try:
        ctx.sync()
    except binding.PckError as e:
        assert e.code == binding.ECUDA
        return next(n for n in (8, 9, 10) if f"code {n}" in str(e))
    return 0


def test_values_out_of_range_are_reported(ctx):   # noqa: F811
    pg = r8.Pages8(4, [40, 400], 2, 64, 16)
    c, Q = pg.cache(), _rand(5, 2, 4, 64, dtype=F16)
    big = pg.lens + 100000
    bad = pg.table.clone()
    bad[1, 3] = 1 << 20
    neg = pg.table.clone()
    neg[1, 24] = -5
    KV = Q[:, :2]
    cu = torch.tensor([0, 40, 440], dtype=i32, device="cuda")
    rows = _rand(6, 440, 4, 64, dtype=F16)
    for tab, ln, code in ((pg.table, pg.lens, 0), (bad, pg.lens, 8), (neg, pg.lens, 8), (pg.table, big, 10)):
        codes = (8, 10) if ln is big else (code,)          # (a length cut to the table's width meets its unused entries)
        assert _code(ctx, lambda: ctx.paged_attend(c, tab, ln, Q)) in codes
        assert _code(ctx, lambda: ctx.paged_attend(c, tab, ln, rows, cu_rows=cu)) in codes
        assert _code(ctx, lambda: ctx.paged_read(c, tab, ln, T=440, cu_rows=cu)) in codes
        if tab is not bad:
            assert _code(ctx, lambda: ctx.paged_append(c, tab, ln, KV, KV)) == code
    for cu in ((0, 41, 442), (0, 3, 2), (-1, 2, 4), (3, 2, 5), (0, 2 ** 31 - 1, 4)):
        t = torch.tensor(cu, dtype=i32, device="cuda")
        assert _code(ctx, lambda: ctx.paged_read(c, pg.table, pg.lens, T=4, cu_rows=t)) == 10
        assert _code(ctx, lambda: ctx.paged_attend(c, pg.table, pg.lens, rows[:4], cu_rows=t, max_rows=4)) == 10
        assert _code(ctx, lambda: ctx.paged_attend(c, pg.table, pg.lens, rows[:4], cu_rows=t, max_rows=400)) == 10
        assert _code(ctx, lambda: ctx.paged_append(c, pg.table, pg.lens, rows[:4, :2], rows[:4, :2], cu_rows=t)) == 10
    assert _code(ctx, lambda: ctx.paged_append(c, pg.table, pg.lens, KV, KV, cos_sin=ref.angles(50, 64, "cuda"))) == 9
    t = torch.tensor((0, 3, 4), dtype=i32, device="cuda")
    assert _code(ctx, lambda: ctx.paged_attend(c, pg.table, pg.lens, rows[:4], cu_rows=t, max_rows=2)) == 10
    assert _code(ctx, lambda: ctx.paged_attend(c, pg.table, pg.lens, Q)) == 0      # and the next call is quiet


def test_refusals(ctx):   # noqa: F811
    pg = r8.Pages8(4, [40, 4000], 2, 64, 16)
    c, Q = pg.cache(), _rand(5, 2, 4, 64, dtype=F16)

    def no(fn, code, text):
        with pytest.raises(binding.PckError) as e:
            fn()
        assert e.value.code == code and text in str(e.value), str(e.value)
    EINVAL, EUNS = binding.EINVAL, binding.EUNSUPPORTED
    no(lambda: ctx.paged_attend(c, pg.table, pg.lens, Q[:, :3]), EINVAL, "multiple of H_kv")
    no(lambda: ctx.paged_attend(c, pg.table, pg.lens, Q, window=-1), EINVAL, "window")
    no(lambda: ctx.paged_attend(c, pg.table, pg.lens, Q, workspace=torch.empty(16, dtype=U8, device="cuda")), EINVAL, "workspace")
    odd = r8.Pages8(4, [40], 2, 80, 16)
    no(lambda: ctx.paged_attend(odd.cache(), odd.table, odd.lens, _rand(5, 1, 4, 80, dtype=F16)), EUNS, "D=80")
    wide = r8.Pages8(4, [40], 2, 256, 16)
    no(lambda: ctx.paged_attend(wide.cache(), wide.table, wide.lens, _rand(5, 30, 4, 256, dtype=F16), cu_rows=_cu([30])), EUNS, "D=256")
    k = torch.zeros((3, 2, 24, 64), dtype=U8, device="cuda").view(r8.E4M3)
    s = torch.zeros((3, 2, 24), dtype=U8, device="cuda")
    no(lambda: ctx.paged_attend(binding.QuantizedPagedCache(k, k, s, s), pg.table, pg.lens, Q), EUNS, "page_size")
    k = torch.zeros((3, 2, 16, 72), dtype=U8, device="cuda").view(r8.E4M3)[..., :64]
    s = torch.zeros((3, 2, 16), dtype=U8, device="cuda")
    no(lambda: ctx.paged_attend(binding.QuantizedPagedCache(k, k, s, s), pg.table, pg.lens, Q), EINVAL, "multiples of 16")
    no(lambda: ctx.paged_read(binding.QuantizedPagedCache(k, k, s, s), pg.table, pg.lens), EINVAL, "multiples of 16")
    k = torch.zeros(3 * 2 * 16 * 64 + 8, dtype=U8, device="cuda")[8:].view(3, 2, 16, 64).view(r8.E4M3)
    no(lambda: ctx.paged_append(binding.QuantizedPagedCache(k, k, s, s), pg.table, pg.lens, Q[:, :2], Q[:, :2]), EINVAL, "16-byte aligned")
    o = torch.zeros((2, 2, 68), dtype=F16, device="cuda")[..., :64]
    no(lambda: ctx.paged_read(c, pg.table, pg.lens, K_out=o, V_out=o), EINVAL, "multiples of 8")
    ctx.sync()


def test_nothing_to_do(ctx):   # noqa: F811
    pg = r8.Pages8(4, [40, 400], 2, 64, 16)
    c = pg.cache()
    none, cu = torch.zeros((0, 4, 64), dtype=F16, device="cuda"), torch.zeros(3, dtype=i32, device="cuda")
    O, L = ctx.paged_attend(c, pg.table, pg.lens, none, cu_rows=cu)
    assert O.shape == (0, 4, 64) and L.shape == (0, 4)
    ctx.paged_append(c, pg.table, pg.lens, none[:, :2], none[:, :2], cu_rows=cu)
    assert ctx.paged_read(c, pg.table, pg.lens, T=0, cu_rows=cu)[0].shape == (0, 2, 64)
    O, _ = ctx.paged_attend(c, pg.table[:0], pg.lens[:0], none)
    assert O.shape == (0, 4, 64)
    ctx.sync()


# ------------------------------------------------------------------ streams and graphs

def test_other_streams_and_two_graphs(ctx):   # noqa: F811
    """A captured step (append, attention, reading back) replayed with other lengths and inputs, two such graphs side by
    side on two streams with a workspace each; and calls on a stream of their own."""
    H_q, H_kv, D, page, B = 8, 2, 128, 16, 3
    steps, kept = [], []
    for i, dtype in enumerate((F16, BF16)):
        pg = r8.Pages8(20 + i, [700, 41, 300], H_kv, D, page, width=60)
        pg.table.clamp_(min=0)
        c = pg.cache()
        x = _rand(30 + i, B, H_q + 2 * H_kv, D, dtype=dtype)
        cs = ref.angles(1000, D, "cuda")
        st = torch.cuda.Stream()

        def step(pg=pg, c=c, x=x, cs=cs):
            q = ctx.paged_append(c, pg.table, pg.lens, x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:], Q=x[:, :H_q], cos_sin=cs)
            O, L = ctx.paged_attend(c, pg.table, pg.lens, q)
            return q, O, L, ctx.paged_read(c, pg.table, pg.lens, dtype=torch.float32)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            step()
            st.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                out = step()
        steps.append((pg, x, g, st, out, dtype))
        kept.append(step)                                  # its cache and rotary table are read by every replay
    for round_ in range(3):
        for pg, x, g, st, out, dtype in steps:
            pg.lens -= 1 + round_
            x.copy_(_rand(50 + round_, *x.shape, dtype=dtype))
        torch.cuda.synchronize()
        for _ in range(5):
            for pg, x, g, st, out, dtype in steps:
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for pg, x, g, st, (q, O, L, (kr, vr)), dtype in steps:
            lens = pg.lens.tolist()
            ref.check_attend(O, L, r8.attend(pg, lens, [1] * B, q), dtype, ref.P_ONCE[dtype], "replayed")
            wk, wv = _read_want(pg, lens, [1] * B, torch.float32)
            assert torch.equal(kr, wk) and torch.equal(vr, wv)
            v = x[:, H_q + H_kv:].double()
            assert ((vr.double() - v).abs() <= r8.HALF_STEP * v.abs() + 2.0 ** -17 * v.abs().amax(-1, keepdim=True)).all()
    ctx.sync()
    side = torch.cuda.Stream()
    pg, x, _, _, _, dtype = steps[0]
    Q = x[:, :H_q].contiguous()
    torch.cuda.synchronize()
    O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, stream=side)
    kr, _ = ctx.paged_read(pg.cache(), pg.table, pg.lens, stream=side)
    side.synchronize()
    ref.check_attend(O, L, r8.attend(pg, pg.lens.tolist(), [1] * B, Q), dtype, ref.P_ONCE[dtype], "side stream")
    assert torch.equal(kr, _read_want(pg, pg.lens.tolist(), [1] * B, F16)[0])
    assert len(kept) == 2


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_session_from_prompt_to_resident_prefix(ctx, dtype):   # noqa: F811
    """Prompts appended and attended in two chunks, then tokens one by one, against attention over the values that the cache
    holds; the cache read back is stored as a resident prefix, and the next token's attention over that prefix is the one
    over the pages; with the prefix resident, new tokens go to fresh pages and are merged with it."""
    H_q, H_kv, D, page = 8, 2, 64, 16
    B = 2
    cs = ref.angles(200, D, "cuda")
    k, v, ks, vs = _empty_pages(20, H_kv, page, D)
    c = binding.QuantizedPagedCache(k, v, ks, vs.view(r8.E8M0))
    order = torch.randperm(20, generator=torch.Generator().manual_seed(1)).to(i32)
    table, free = order[:16].view(2, 8).cuda(), order[16:17].view(1, 1).cuda()
    wq, wk = (1 + _rand(i, D, dtype=dtype, scale=0.1) for i in (1, 2))

    class _Pg:   # as r8.attend wants it
        def kv(self):
            return r8.values(k, ks), r8.values(v, vs)
    _Pg.table = table
    lens = [0, 0]
    seen = [[], []]       # the rows' original v
    for news in ([50, 20], [20, 13], [1, 1], [1, 1], [1, 1]):
        T = sum(news)
        lens = [a + b for a, b in zip(lens, news)]
        ln = torch.tensor(lens, dtype=i32, device="cuda")
        x = _rand(100 + sum(lens), T, H_q + 2 * H_kv, D, dtype=dtype)
        cu = None if T == B else _cu(news)
        q = ctx.paged_append(c, table, ln, x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:], Q=x[:, :H_q], cu_rows=cu, cos_sin=cs, q_weight=wq, k_weight=wk)
        O, L = ctx.paged_attend(c, table, ln, q, cu_rows=cu)
        ref.check_attend(O, L, r8.attend(_Pg(), lens, news, q), dtype, ref.P_ONCE[dtype], f"{lens}")
        for b, r in ((0, slice(0, news[0])), (1, slice(news[0], T))):
            seen[b].append(x[r, H_q + H_kv:].double())
    assert lens == [73, 36]
    T = sum(lens)
    kr, vr = ctx.paged_read(c, table, ln, T=T, cu_rows=_cu(lens), dtype=F16)
    v0 = torch.cat(seen[0] + seen[1])
    big = v0.abs().amax(-1, keepdim=True)      # the scale is below big / 224
    assert ((vr.double() - v0).abs() <= r8.HALF_STEP * v0.abs() + 2.0 ** -17 * big).all()
    # sequence 0 becomes a resident prefix
    n0 = lens[0]
    Kp, Vp = (t[:n0].transpose(0, 1).contiguous() for t in (kr, vr))
    ctx.store("tail", 0, Kp, Vp)
    q1 = _rand(7, 1, H_q, D, dtype=F16)
    O_paged, L_paged = ctx.paged_attend(c, table[:1], ln[:1], q1)
    Op, Lp = ctx.query("tail", 0, q1.transpose(0, 1).contiguous())
    assert (Op.view(H_q, D).double() - O_paged[0].double()).abs().max() < 4e-3 and (Lp.view(-1) - L_paged[0]).abs().max() < 1e-3
    # behind it: a fresh page
    x = _rand(8, 1, 2 * H_kv, D, dtype=F16)
    one = torch.ones(1, dtype=i32, device="cuda")
    ctx.paged_append(c, free, one, x[:, :H_kv], x[:, H_kv:])
    O2, L2 = ctx.paged_attend(c, free, one, q1, prior=(Op.view(1, H_q, D), Lp.view(1, H_q)))
    kk, vv = (t[free[0, 0].long(), :, :1] for t in _Pg().kv())
    K = torch.cat((Kp.double(), kk), 1)
    V = torch.cat((Vp.double(), vv), 1)
    s = torch.einsum("hgd,hnd->hgn", q1[0].double().view(H_kv, -1, D), K) / math.sqrt(D)
    w = torch.einsum("hgn,hnd->hgd", torch.softmax(s, -1), V).reshape(H_q, D)
    assert (O2[0].double() - w).abs().max() < 4e-3 and (L2[0].double() - torch.logsumexp(s, -1).reshape(-1)).abs().max() < 2e-3
    ctx.drop("tail")
    ctx.sync()
