"""The paged-tail operators on the GPU against their 64-bit forms: head norms with the rotation, the
append, attention of one row per sequence, and a run of them together behind a resident prefix."""
import ctypes
import math
import os

import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_ref as ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
i32 = torch.int32


@pytest.fixture(scope="module")
def ctx():
    need_gpu()
    c = binding.Context(0, max_slots=4)
    yield c
    c.sync()       # no kernel of this module left an error behind
    c.close()


def _rand(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _close(x, want, dtype, what):
    tol = ref.norm_rope_tol(want, dtype)
    over = ((x.double() - want).abs() - tol).max().item()
    assert over <= 0, f"{what}: {over:.3e} over its bound"


# ------------------------------------------------------------------ head norms and rotation

@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,H_q,H_kv,D,R,inter", [(1, 1, 1, 16, 16, False), (1, 32, 8, 128, 128, False), (3, 5, 1, 96, 48, False),
                                                  (67, 24, 8, 128, 64, True), (33, 8, 2, 256, 256, False), (130, 7, 7, 64, 32, True),
                                                  (5, 2, 2, 512, 128, False), (1000, 3, 1, 32, 32, False), (19, 10, 2, 192, 96, False),
                                                  (2, 3, 3, 48, 16, True), (5000, 2, 1, 64, 64, False)])
def test_norm_rope(ctx, dtype, T, H_q, H_kv, D, R, inter):
    x = _rand(T + D, T, H_q + 2 * H_kv, D, dtype=dtype, scale=3.0)
    Q, K = x[:, :H_q], x[:, H_q:H_q + H_kv]
    keep = x.clone()
    cs = ref.angles(4000, R, "cuda")
    pos = torch.randint(0, 4000, (T,), device="cuda", dtype=i32)
    wq, wk = 1 + _rand(1, D, dtype=dtype, scale=0.2), 1 + _rand(2, D, dtype=dtype, scale=0.2)
    q, k = ctx.qk_norm_rope(Q, K, pos, cs, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=inter)
    _close(q, ref.norm_rope(Q, wq, 1e-5, cs, pos, inter), dtype, "q")
    _close(k, ref.norm_rope(K, wk, 1e-5, cs, pos, inter), dtype, "k")
    assert torch.equal(x, keep)
    # rotation alone, norm alone (no weight), one side alone, in place
    q, _ = ctx.qk_norm_rope(Q, None, pos, cs, interleaved=inter)
    _close(q, ref.norm_rope(Q, None, None, cs, pos, inter), dtype, "rotation")
    _, k = ctx.qk_norm_rope(None, K, norm=True, eps=1e-3)
    _close(k, ref.norm_rope(K, None, 1e-3), dtype, "norm")
    wantq, wantk = ref.norm_rope(Q, wq, 1e-5, cs, pos, inter), ref.norm_rope(K, None, 1e-5, cs, pos, inter)
    ctx.qk_norm_rope(Q, K, pos, cs, q_weight=wq, eps=1e-5, interleaved=inter, Q_out=Q, K_out=K)
    _close(Q, wantq, dtype, "q in place")
    _close(K, wantk, dtype, "k in place, no weight")
    assert torch.equal(x[:, H_q + H_kv:], keep[:, H_q + H_kv:])


def test_norm_rope_into_the_fused_query(ctx):
    """Its outputs, written with the strides of pck_query_fused's Q and suffix, give attention over prefix + suffix."""
    H_q, H_kv, N, S, D = 8, 2, 300, 40, 64
    Kp, Vp = _rand(1, H_kv, N, D, dtype=F16), _rand(2, H_kv, N, D, dtype=F16)
    x = _rand(3, S, H_q + 2 * H_kv, D, dtype=F16)
    cs = ref.angles(N + S, D, "cuda")
    pos = torch.arange(N, N + S, device="cuda", dtype=i32)
    Q = torch.empty((H_q, S, D), dtype=F16, device="cuda")
    Ks = torch.empty((H_kv, S, D), dtype=F16, device="cuda")
    ctx.qk_norm_rope(x[:, :H_q], x[:, H_q:H_q + H_kv], pos, cs, norm=True, Q_out=Q.transpose(0, 1), K_out=Ks.transpose(0, 1))
    Vs = x[:, H_q + H_kv:].transpose(0, 1).contiguous()
    ctx.store("fused", 0, Kp, Vp)
    O, L = ctx.query_fused("fused", 0, Q, Ks, Vs)
    _close(Q.transpose(0, 1), ref.norm_rope(x[:, :H_q], None, 1e-6, cs, pos), F16, "q")
    # the same through the 64-bit form: one sequence whose cache is prefix + suffix
    K, V = torch.cat((Kp, Ks), 1), torch.cat((Vp, Vs), 1)
    n = -(-(N + S) // 16)
    pad = torch.zeros((H_kv, n * 16 - N - S, D), dtype=F16, device="cuda")
    k, v = (torch.cat((t, pad), 1).view(H_kv, n, 16, D).transpose(0, 1) for t in (K, V))
    want = ref.attend(k, v, torch.arange(n, device="cuda")[None], [N + S], [S], Q.transpose(0, 1))
    assert (O.transpose(0, 1).double() - want[0]).abs().max() < 2e-3 and (L.t().double() - want[1]).abs().max() < 1e-3


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F32, F16), (F32, BF16)])
@pytest.mark.parametrize("lens,news,H_q,H_kv,D,R,page,inter,nhd", [
    ([1], [1], 1, 1, 16, 16, 16, False, False), ([17, 1, 160, 33], [1, 1, 1, 1], 8, 2, 64, 64, 16, False, True),
    ([40, 0, 300, 16, 7], [40, 0, 123, 3, 7], 6, 2, 128, 64, 32, True, False),
    ([100, 257], [64, 1], 4, 4, 256, 256, 48, False, False), ([64] * 70, [2] * 70, 3, 1, 96, 96, 64, False, True)])
def test_append(ctx, dtype, cache, lens, news, H_q, H_kv, D, R, page, inter, nhd):
    pg = ref.Pages(5, lens, H_kv, D, page, cache, fill=7.0, nhd=nhd)
    T = sum(news)
    one = all(m == 1 for m in news)
    pad = 0 if one else 5          # rows behind the last sequence
    x = _rand(6, T + pad, H_q + 2 * H_kv, D, dtype=dtype)
    Q, K, V = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    wq, wk = 1 + _rand(1, D, dtype=dtype, scale=0.2), 1 + _rand(2, D, dtype=dtype, scale=0.2)
    cs = ref.angles(max(lens) + 50, R, "cuda")
    cu = None if one else torch.tensor([0] + list(torch.tensor(news).cumsum(0)), dtype=i32, device="cuda")
    at = ref.rows_of(lens, news)
    p = torch.tensor([q for _, q in at], device="cuda")
    b = torch.tensor([q for q, _ in at], device="cuda")
    for positions in (None, (p + 50).to(i32)):
        k0, v0 = pg.k.clone(), pg.v.clone()
        Qo = torch.full((T + pad, H_q, D), 9.0, dtype=dtype, device="cuda")
        if positions is not None:
            positions = torch.cat((positions, torch.full((pad,), 1 << 30, dtype=i32, device="cuda")))
        c = binding.PagedCache(pg.k, pg.v)
        ctx.paged_append(c, pg.table, pg.lens, K, V, Q=Q, cu_rows=cu, cos_sin=cs, positions=positions, q_weight=wq,
                         k_weight=wk, eps=1e-5, interleaved=inter, Q_out=Qo)
        at_pos = p if positions is None else positions[:T]
        _close(Qo[:T], ref.norm_rope(Q[:T], wq, 1e-5, cs, at_pos, inter), dtype, "q")
        assert (Qo[T:] == 9).all()
        pages = pg.table[b, p // page].long()
        _close(pg.k[pages, :, p % page], ref.norm_rope(K[:T], wk, 1e-5, cs, at_pos, inter), cache, "k")
        assert torch.equal(pg.v[pages, :, p % page], V[:T].to(cache))
        k0[pages, :, p % page], v0[pages, :, p % page] = pg.k[pages, :, p % page], pg.v[pages, :, p % page]
        assert torch.equal(k0, pg.k) and torch.equal(v0, pg.v)      # and nothing else was written
    # as they are: neither norm nor rotation
    ctx.paged_append(binding.PagedCache(pg.k, pg.v), pg.table, pg.lens, K, V, cu_rows=cu)
    assert torch.equal(pg.k[pages, :, p % page], K[:T].to(cache)) and torch.equal(pg.v[pages, :, p % page], V[:T].to(cache))


# ------------------------------------------------------------------ attention, one row per sequence

def _attend_case(ctx, lens, H_q, H_kv, D, page, dtype, W=0, sinks=0, prior=False, nhd=False, seed=1, scale=1.0, fill=float("nan"), width=None):
    pg = ref.Pages(seed, lens, H_kv, D, page, dtype, nhd=nhd, fill=fill, width=width)
    B = len(lens)
    big = _rand(seed + 1, B, H_q + 3, D, dtype=dtype, scale=scale)
    Q = big[:, 1:H_q + 1]
    pr = None
    if prior:
        pr = _rand(seed + 2, B, H_q, D), _rand(seed + 3, B, H_q) + 3
        pr[1][0, 0] = -math.inf
        pr[0][0, 0] = math.nan
    c = binding.PagedCache(pg.k, pg.v)
    O, L = ctx.paged_attend(c, pg.table, pg.lens, Q, window=W, sinks=sinks, prior=pr)
    news = [1] * B
    want = ref.attend(pg.k, pg.v, pg.table, lens, news, Q, W, sinks, pr)
    ref.check_attend(O, L, want, dtype, ref.P_SPLIT[dtype], f"lens {lens[:4]} D {D} W {W}")
    O2, L2 = ctx.paged_attend(c, pg.table, pg.lens, Q, window=W, sinks=sinks, prior=pr)
    assert torch.equal(O, O2) and torch.equal(L, L2)      # the same bits again
    return pg, Q, O, L


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,H_q,H_kv,D,page", [
    ([1], 1, 1, 64, 16), ([0, 1, 2, 15, 16, 17, 31, 33], 4, 2, 128, 16), ([300], 32, 8, 128, 16), ([511, 512, 513, 5], 8, 2, 256, 32),
    ([777, 0, 4096, 100], 12, 4, 64, 48), ([2000] * 3, 10, 2, 192, 64), ([1, 9000], 28, 4, 128, 128), ([1000, 3], 16, 1, 128, 16),
    ([1200, 50], 40, 1, 64, 16), ([600, 700], 24, 1, 256, 16), ([30000], 8, 8, 128, 64), ([70001], 2, 1, 64, 256),
    (list(range(0, 1400, 7)), 8, 4, 64, 16)])
def test_token(ctx, dtype, lens, H_q, H_kv, D, page):
    _attend_case(ctx, lens, H_q, H_kv, D, page, dtype)
    _attend_case(ctx, lens, H_q, H_kv, D, page, dtype, prior=True, nhd=True, seed=11)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("W,sinks", [(1, 0), (1, 1), (16, 4), (17, 33), (100, 0), (255, 16), (512, 17), (1000, 5000), (100000, 4)])
def test_token_window(ctx, dtype, W, sinks):
    lens = [0, 1, 15, 16, 17, 99, 100, 101, 513, 1025, 5000]
    _attend_case(ctx, lens, 8, 2, 128, 16, dtype, W, sinks)
    _attend_case(ctx, lens, 7, 1, 64, 32, dtype, W, sinks, prior=True, nhd=True)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 64), (32, 2, 64), (16, 4, 128), (64, 4, 128), (20, 4, 192), (9, 3, 256), (128, 4, 128)])
def test_token_many_items(ctx, dtype, H_q, H_kv, D):
    """More items than a few per SM: a range per warp, with whole items, items cut once and items over many ranges."""
    lens = [(37 * i * i) % 700 for i in range(180)] + [9000, 0, 1, 2500]
    _attend_case(ctx, lens, H_q, H_kv, D, 16, dtype)
    _attend_case(ctx, lens, H_q, H_kv, D, 32, dtype, W=300, sinks=5, prior=True, nhd=True, seed=4, width=600)


@pytest.mark.parametrize("B", [1, 19, 20, 40, 77, 160, 310, 700])
@pytest.mark.parametrize("H_q,H_kv,D", [(8, 8, 128), (12, 3, 64), (32, 2, 128), (16, 4, 256)])
def test_token_short_caches(ctx, B, H_q, H_kv, D):
    """An item per CTA, per CTA of half the warps, and ranges per warp once the items are many."""
    lens = [(61 * i * i + 7 * B) % 300 for i in range(B)]
    _attend_case(ctx, lens, H_q, H_kv, D, 16, F16 if B % 2 else BF16, prior=B % 3 == 0)
    _attend_case(ctx, lens, H_q, H_kv, D, 32, BF16, W=50, sinks=3, seed=3)


@pytest.mark.parametrize("B,H_q,H_kv,D", [(19, 8, 8, 128), (20, 32, 8, 128), (77, 12, 3, 64), (40, 16, 4, 192), (70, 24, 8, 256), (912, 1, 1, 64), (913, 1, 1, 64)])
def test_token_ranges_of_ragged_caches(ctx, B, H_q, H_kv, D):
    """One item per SM and just above, up to six: ranges per CTA and per CTA of half the warps, then per warp."""
    lens = [(61 * i * i + 7 * B) % (1700 if i % 5 == 0 else 90) for i in range(B)]
    _attend_case(ctx, lens, H_q, H_kv, D, 16, BF16 if B % 2 else F16, prior=B % 4 == 0, width=2000)
    _attend_case(ctx, lens, H_q, H_kv, D, 16, BF16, W=1100, sinks=20, width=2000, seed=2)


@pytest.mark.parametrize("B,n", [(14, 1100), (16, 1500), (20, 1200), (38, 1100), (39, 1100), (64, 1050)])
@pytest.mark.parametrize("spread", [0, 0.2])
def test_token_caches_of_one_length(ctx, B, n, spread):
    """Items that stay whole because they have nearly one length, and those that just do not."""
    lens = [n - int(spread * n * ((7 * i) % 10) / 10) for i in range(B)]
    _attend_case(ctx, lens, 16, 8, 64, 16, BF16, prior=B % 2 == 0)
    if not spread:
        _attend_case(ctx, [3000 - 100 * (i % 2) for i in range(B)], 8, 8, 64, 32, F16, W=n, sinks=5, seed=2)


@pytest.mark.parametrize("W,sinks", [(1023, 0), (1024, 0), (1024, 17), (1025, 0), (1100, 300)])
def test_token_windows_of_a_cta(ctx, W, sinks):
    lens = [0, 1, 15, 16, 17, 1000, 1023, 1024, 1025, 1040, 1337, 2000, 4999]
    _attend_case(ctx, lens, 8, 2, 128, 16, BF16, W=W, sinks=sinks)
    _attend_case(ctx, lens * 10, 8, 2, 64, 16, F16, W=W, sinks=sinks, seed=2)


def test_token_hidden_keys_hold_anything(ctx):
    """Behind the window, in front of the last token and in unneeded pages: NaN, infinities, the lowest value, and table
    entries that are no pages."""
    for fill in (math.inf, -math.inf, torch.finfo(F16).min):
        lens, W, sinks = [700, 33, 4097], 37, 3
        pg, Q, O, L = _attend_case(ctx, lens, 8, 2, 128, 16, F16, W, sinks, fill=fill)
        for b, n in enumerate(lens):
            for p in range(n):
                if n - W > p >= sinks:
                    pg.k[pg.table[b, p // 16], :, p % 16] = math.nan
                    pg.v[pg.table[b, p // 16], :, p % 16] = fill
        table = pg.table.clone()
        for b, n in enumerate(lens):
            for i in range(table.shape[1]):
                if 16 * i >= n or (16 * i >= sinks and 16 * i + 15 < n - W):
                    table[b, i] = 1 << 30
        O2, L2 = ctx.paged_attend(binding.PagedCache(pg.k, pg.v), table, pg.lens, Q, window=W, sinks=sinks)
        assert torch.equal(O, O2) and torch.equal(L, L2)
    ctx.sync()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_token_large_scores(ctx, dtype):
    """Scores in the hundreds, and growing along the cache so that every tile moves the maximum."""
    _attend_case(ctx, [900, 2000], 8, 2, 128, 16, dtype, scale=20.0)
    lens = [1500]
    pg = ref.Pages(3, lens, 1, 64, 16, dtype)
    Q = torch.ones((1, 2, 64), dtype=dtype, device="cuda")
    p = torch.arange(1500, device="cuda")
    pg.k[pg.table[0, p // 16].long(), :, p % 16] = (p / 20.0).to(dtype)[:, None, None]
    O, L = ctx.paged_attend(binding.PagedCache(pg.k, pg.v), pg.table, pg.lens, Q)
    ref.check_attend(O, L, ref.attend(pg.k, pg.v, pg.table, lens, [1], Q), dtype, ref.P_SPLIT[dtype])


def test_token_nan_in_a_visible_key_shows(ctx):
    pg = ref.Pages(3, [40, 40], 1, 64, 16, F16)
    pg.k[pg.table[1, 1], 0, 3] = math.nan
    Q = _rand(1, 2, 2, 64, dtype=F16)
    for width in (3, 100):      # one CTA per item, and split ranges
        tab = torch.full((2, width), -1, dtype=i32, device="cuda")
        tab[:, :3] = pg.table
        O, L = ctx.paged_attend(binding.PagedCache(pg.k, pg.v), tab, pg.lens, Q)
        assert torch.isfinite(O[0]).all() and torch.isnan(O[1]).all() and torch.isnan(L[1]).all()


def test_token_split_widths_agree(ctx):
    """A wide table (ranges over all SMs, joined) and a narrow one (a CTA per item) hold the same bound."""
    for width in (32, 64, 65, 4000):
        _attend_case(ctx, [500, 0, 1, 512, 77], 8, 2, 128, 16, F16, width=width, prior=True)


def test_values_out_of_range_are_reported_and_not_followed(ctx):
    lens = [40, 100]
    pg = ref.Pages(3, lens, 2, 64, 16, F16)
    Q = _rand(1, 2, 4, 64, dtype=F16)
    c = binding.PagedCache(pg.k, pg.v)
    good = ctx.paged_attend(c, pg.table, pg.lens, Q)

    def code(fn):
        ctx.sync()
        fn()
        with pytest.raises(binding.PckError) as e:
            ctx.sync()
        assert e.value.code == binding.ECUDA
        ctx.sync()
        return str(e.value)

    for bad in (-1, c.n_pages, 1 << 30):
        t = pg.table.clone()
        t[1, 2] = bad
        assert "code 8" in code(lambda: ctx.paged_attend(c, t, pg.lens, Q))
        k0, v0 = pg.k.clone(), pg.v.clone()
        at = torch.tensor([40, 33], dtype=i32, device="cuda")
        assert "code 8" in code(lambda: ctx.paged_append(c, t, at, Q[:, :2], Q[:, 2:]))
        k0[pg.table[0, 2], :, 7], v0[pg.table[0, 2], :, 7] = Q[0, :2], Q[0, 2:]
        assert torch.equal(k0.nan_to_num(), pg.k.nan_to_num()) and torch.equal(v0.nan_to_num(), pg.v.nan_to_num())
    long = pg.lens + 100
    assert "code 10" in code(lambda: ctx.paged_attend(c, pg.table, long, Q))
    assert "code 10" in code(lambda: ctx.paged_append(c, pg.table, long, Q[:, :2], Q[:, 2:]))
    cs = ref.angles(39, 32, "cuda")
    assert "code 9" in code(lambda: ctx.paged_append(c, pg.table, pg.lens, Q[:, :2], Q[:, 2:], cos_sin=cs))
    assert "code 9" in code(lambda: ctx.qk_norm_rope(Q, None, torch.tensor([-1, 5], dtype=i32, device="cuda"), cs))
    pg2 = ref.Pages(3, lens, 2, 64, 16, F16)
    again = ctx.paged_attend(binding.PagedCache(pg2.k, pg2.v), pg2.table, pg2.lens, Q)
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


# ------------------------------------------------------------------ refusals: nothing is launched

def test_refusals(ctx):
    pg = ref.Pages(3, [40, 100], 2, 64, 16, F16)
    Q = _rand(1, 2, 4, 64, dtype=F16)
    c = binding.PagedCache(pg.k, pg.v)

    def code(fn):
        with pytest.raises(binding.PckError) as e:
            fn()
        return e.value.code

    at = lambda cache=c, Q=Q, tab=pg.table, **kw: code(lambda: ctx.paged_attend(cache, tab, pg.lens, Q, **kw))   # noqa: E731
    assert at(window=-1) == binding.EINVAL and at(sinks=-1) == binding.EINVAL
    assert at(Q=Q[:, :3]) == binding.EINVAL                                       # 3 q heads on 2 kv heads
    assert at(Q=_rand(1, 2, 4, 68, dtype=F16)[..., 1:65]) == binding.EINVAL         # alignment
    assert at(Q=_rand(1, 2, 4, 68, dtype=F16)[..., :64]) == binding.EINVAL          # strides of 68 elements
    assert at(tab=torch.zeros((2, 0), dtype=i32, device="cuda")) == binding.EINVAL
    odd = torch.zeros((3, 2, 24, 64), dtype=F16, device="cuda")
    assert at(cache=binding.PagedCache(odd, odd)) == binding.EUNSUPPORTED           # page_size 24
    d96 = torch.zeros((3, 2, 16, 96), dtype=F16, device="cuda")
    assert at(cache=binding.PagedCache(d96, d96), Q=_rand(1, 2, 4, 96, dtype=F16)) == binding.EUNSUPPORTED
    same = torch.zeros((1, 2, 16, 64), dtype=F16, device="cuda").expand(3, 2, 16, 64)
    assert at(cache=binding.PagedCache(same, same)) == binding.EINVAL               # stride 0
    lib, vp = ctx.lib, ctypes.c_void_p
    batch = ctx._batch(c, pg.table, pg.lens, None, 2, None)
    O = torch.empty_like(Q)
    call = lambda ws, n, Op=None, Lp=None: lib.pck_paged_attend(   # noqa: E731
        ctx.h, ctypes.byref(c.c), ctypes.byref(batch), 4, Q.data_ptr(), 256, 64, 0, 0, Op, Lp, O.data_ptr(), None, ws, n, None)
    assert call(None, 0) == binding.OK                                            # 7 pages: a CTA per item, no workspace
    assert call(None, 0, Op=O.data_ptr()) == binding.EINVAL                       # a prior without its LSE
    batch.max_pages = 100                                                         # (not launched: refused first)
    assert call(None, 0) == binding.EINVAL and call(vp(O.data_ptr()), 64) == binding.EINVAL
    n = ctypes.c_size_t()
    assert lib.pck_paged_workspace(ctx.h, ctypes.byref(c.c), ctypes.byref(batch), 4, 0, 0, ctypes.byref(n)) == binding.OK and n.value > 64
    batch.T = 3
    assert call(None, 0) == binding.EINVAL                                        # three rows, two sequences
    assert lib.pck_paged_attend(None, ctypes.byref(c.c), ctypes.byref(batch), 4, Q.data_ptr(), 256, 64, 0, 0, None, None,
                                O.data_ptr(), None, None, 0, None) == binding.EINVAL
    K = Q[:, :2]
    ap = lambda **kw: code(lambda: ctx.paged_append(c, pg.table, pg.lens, K, Q[:, 2:], **kw))   # noqa: E731
    assert ap(cos_sin=ref.angles(200, 40, "cuda")) == binding.EUNSUPPORTED         # R = 40
    assert ap(cos_sin=ref.angles(200, 128, "cuda")) == binding.EUNSUPPORTED        # R > D
    assert ap(norm=True, eps=-1.0) == binding.EINVAL
    nr = lambda Q=Q, **kw: code(lambda: ctx.qk_norm_rope(Q, None, **kw))   # noqa: E731
    assert nr() == binding.EINVAL                                                  # neither norm nor rotation
    assert nr(Q=_rand(1, 2, 4, 72, dtype=F16), norm=True) == binding.EUNSUPPORTED  # D = 72
    assert nr(Q=_rand(1, 2, 4, 68, dtype=F16)[..., :64], norm=True) == binding.EINVAL
    ctx.sync()


def test_nothing_to_do(ctx):
    pg = ref.Pages(3, [5], 2, 64, 16, F16)
    c = binding.PagedCache(pg.k, pg.v)
    none = torch.empty((0, 4, 64), dtype=F16, device="cuda")
    tab, n = torch.empty((0, 3), dtype=i32, device="cuda"), torch.empty(0, dtype=i32, device="cuda")
    O, L = ctx.paged_attend(c, tab, n, none)
    assert O.shape == (0, 4, 64) and L.shape == (0, 4)
    ctx.paged_append(c, tab, n, none[:, :2], none[:, :2])
    assert ctx.qk_norm_rope(none, None, norm=True)[0].shape == (0, 4, 64)
    ctx.sync()


# ------------------------------------------------------------------ together, streams, graphs

def test_decode_steps_behind_a_resident_prefix(ctx):
    """Prefix slots in the context, tails in pages: each step norms, rotates and appends, asks the prefix for (O, LSE) and
    merges it into the tail's attention. Against one 64-bit attention over prefix and tail end to end."""
    H_q, H_kv, D, N, B, P = 8, 2, 64, 200, 3, 16
    sess = [(_rand(20 + b, H_kv, N, D, dtype=F16), _rand(30 + b, H_kv, N, D, dtype=F16)) for b in range(B)]
    for b, (Kp, Vp) in enumerate(sess):
        ctx.store(f"tail{b}", 0, Kp, Vp)
    lens = [0, 15, 40]
    pg = ref.Pages(9, [n + 6 for n in lens], H_kv, D, P, F16)
    c = binding.PagedCache(pg.k, pg.v)
    cs = ref.angles(N + 64, D, "cuda")
    wq = 1 + _rand(1, D, dtype=F16, scale=0.1)
    n = torch.tensor(lens, dtype=i32, device="cuda")
    for step in range(6):
        n += 1
        x = _rand(100 + step, B, H_q + 2 * H_kv, D, dtype=F16)
        q = ctx.paged_append(c, pg.table, n, x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:], Q=x[:, :H_q], cos_sin=cs,
                             positions=n + (N - 1), q_weight=wq)
        Op, Lp = torch.empty((B, H_q, D), device="cuda"), torch.empty((B, H_q), device="cuda")
        ctx.query_batch([dict(sid=f"tail{b}", layer=0, Q=q[b], O=Op[b], LSE=Lp[b]) for b in range(B)], H_q, H_kv, D, q_dtype=binding.DT_F16)
        O, L = ctx.paged_attend(c, pg.table, n, q, prior=(Op, Lp))
        _close(q, ref.norm_rope(x[:, :H_q], wq, 1e-6, cs, n + (N - 1)), F16, "q")
        for b in range(B):
            nb = int(n[b])
            rows = [(pg.k[pg.table[b, p // P], :, p % P], pg.v[pg.table[b, p // P], :, p % P]) for p in range(nb)]
            K = torch.cat((sess[b][0], torch.stack([r[0] for r in rows], 1)), 1)
            V = torch.cat((sess[b][1], torch.stack([r[1] for r in rows], 1)), 1)
            tot = N + nb
            pad = torch.zeros((H_kv, -tot % 16, D), dtype=F16, device="cuda")
            k, v = (torch.cat((t, pad), 1).view(H_kv, -1, 16, D).transpose(0, 1) for t in (K, V))
            want = ref.attend(k, v, torch.arange(k.shape[0], device="cuda")[None], [tot], [1], q[b:b + 1])
            assert (O[b:b + 1].double() - want[0]).abs().max() < 2e-3 and (L[b:b + 1].double() - want[1]).abs().max() < 1e-3
    ctx.sync()


def test_other_streams_and_two_graphs_at_once(ctx):
    """Calls on a stream of their own, and two captured steps replayed side by side on two streams, with lengths that grow
    between replays: each holds its own workspace."""
    H_q, H_kv, D, P = 8, 2, 128, 16
    cases = []
    for seed, lens in ((1, [900, 30, 2000]), (2, [100, 3000])):
        pg = ref.Pages(seed, [n + 4 for n in lens], H_kv, D, P, BF16)
        cases.append(dict(lens=lens, pg=pg, c=binding.PagedCache(pg.k, pg.v), n=torch.tensor(lens, dtype=i32, device="cuda"),
                          x=_rand(seed, len(lens), H_q + 2 * H_kv, D, dtype=BF16), s=torch.cuda.Stream()))
    torch.cuda.synchronize()

    def step(k, stream=None):
        k["n"] += 1
        x = k["x"]
        q = ctx.paged_append(k["c"], k["pg"].table, k["n"], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:], Q=x[:, :H_q], norm=True)
        return q, *ctx.paged_attend(k["c"], k["pg"].table, k["n"], q)

    for k in cases:
        with torch.cuda.stream(k["s"]):
            step(k)                       # warm-up
            k["n"] -= 1
    torch.cuda.synchronize()
    for k in cases:
        k["g"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(k["g"], stream=k["s"]):
            k["out"] = step(k)
    for rep in range(3):
        for _ in range(1):
            for k in cases:
                with torch.cuda.stream(k["s"]):
                    k["g"].replay()
        torch.cuda.synchronize()
        for k in cases:
            q, O, L = k["out"]
            lens = [n + rep + 1 for n in k["lens"]]
            assert k["n"].tolist() == lens
            ref.check_attend(O, L, ref.attend(k["pg"].k, k["pg"].v, k["pg"].table, lens, [1] * len(lens), q), BF16, ref.P_SPLIT[BF16])
    # the stream argument: the work is queued there, behind what was queued before it
    k = cases[0]
    side = torch.cuda.Stream()
    lens = k["n"].tolist()
    q = k["out"][0].clone()
    torch.cuda.synchronize()
    O, L = ctx.paged_attend(k["c"], k["pg"].table, k["n"], q, stream=side)
    side.synchronize()
    ref.check_attend(O, L, ref.attend(k["pg"].k, k["pg"].v, k["pg"].table, lens, [1] * len(lens), q), BF16, ref.P_SPLIT[BF16])


def test_first_calls_inside_a_capture():
    """A process whose very first paged calls are captured (their kernels are loaded then), replayed against eager ones."""
    import subprocess
    import sys
    need_gpu()
    code = """
import torch
from prefix_cached_kv_gb300 import binding
ctx = binding.Context(0)
k, v = (torch.randn((9, 2, 16, 64), device="cuda").half() for _ in range(2))
c = binding.PagedCache(k, v)
x = torch.randn((3, 8, 64), device="cuda").half()
tab = torch.arange(9, device="cuda", dtype=torch.int32).view(1, 9).expand(3, 9).contiguous()
n = torch.tensor([100, 17, 140], dtype=torch.int32, device="cuda")
wide = torch.cat((tab, tab.new_full((3, 200), -1)), 1)
cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
def calls():
    q, _ = ctx.qk_norm_rope(x[:, :4], None, norm=True)
    return [q] + [t for w in (tab, wide) for kw in (dict(), dict(cu_rows=cu, max_rows=1), dict(cu_rows=cu)) for t in ctx.paged_attend(c, w, n, q, **kw)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = calls()
g.replay()
torch.cuda.synchronize()
for a, b in zip(out, calls()):
    assert torch.equal(a, b)
ctx.sync()
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr[-2000:]
