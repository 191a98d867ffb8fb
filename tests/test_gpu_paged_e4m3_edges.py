"""Calls of the quantised paged tail at the edges of what its interface allows, on the GPU."""
import math

import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_e4m3_ref as r8
from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F16, F32, _rand, ctx, i32   # noqa: F401
from tests.test_gpu_paged_e4m3 import PAIR, U8, _bits, _cu, _read_want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,H_kv,P", [(128, 8, 64), (64, 16, 48), (256, 4, 32)])
def test_pages_beyond_32_bits(ctx, D, H_kv, P):   # noqa: F811
    """Pages more than 2^31 codes into the cache: append, one token, rows (D up to 128), reading back."""
    n_pages = 2 ** 31 // (H_kv * P * D) + 40
    k, v = (torch.empty((n_pages, H_kv, P, D), dtype=U8, device="cuda").view(r8.E4M3) for _ in range(2))
    ks, vs = (torch.empty((n_pages, H_kv, P), dtype=U8, device="cuda") for _ in range(2))
    n, m, H_q, used = 500, 200, 2 * H_kv, 500 // P + 1
    table = (n_pages - 1 - torch.arange(used, device="cuda")).to(i32)[None].contiguous()
    x = _rand(5, n, H_q + 2 * H_kv, D, dtype=F16)
    c = binding.QuantizedPagedCache(k, v, ks, vs)
    ln = torch.tensor([n], dtype=i32, device="cuda")
    q = ctx.paged_append(c, table, ln, x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:], Q=x[:, :H_q], cu_rows=_cu([n]), norm=True)
    small = slice(n_pages - used, n_pages)
    _bits(k)[n_pages - used, :, n % P:], _bits(v)[n_pages - used, :, n % P:] = 0x7f, 0x7f       # behind the last token

    class Pg:
        def kv(self):
            return r8.values(k[small], ks[small]), r8.values(v[small], vs[small])
    Pg.k, Pg.table = k[small], table - (n_pages - used)
    want = r8.attend(Pg(), [n], [m], q[n - m:])
    if D <= 128:
        O, L = ctx.paged_attend(c, table, ln, q[n - m:], cu_rows=_cu([m]))
        ref.check_attend(O, L, want, F16, ref.P_ONCE[F16])
    O, L = ctx.paged_attend(c, table, ln, q[-1:])
    ref.check_attend(O, L, [t[-1:] for t in want], F16, PAIR)
    got = ctx.paged_read(c, table, ln, T=m, cu_rows=_cu([m]), dtype=BF16)
    for g, w in zip(got, _read_want(Pg(), [n], [m], BF16)):
        assert torch.equal(g, w)
    ctx.sync()


@pytest.mark.parametrize("width", [None, 400])
@pytest.mark.parametrize("W", [0, 70])
def test_sequences_that_share_pages(ctx, width, W):   # noqa: F811
    """The same pages in several tables (a common beginning), narrow tables and ones much wider than the cache."""
    H_q, H_kv, D, P = 8, 2, 64, 16
    pg = r8.Pages8(11, [300, 200], H_kv, D, P, width=width)
    pg.table = torch.cat((pg.table, pg.table[:1], pg.table[:1]))
    lens = [300, 200, 256, 100]
    pg.lens = torch.tensor(lens, dtype=i32, device="cuda")
    for dtype in (F16, BF16):
        for news in ([1] * 4, [2, 1, 2, 2], [200, 1, 90, 100]):
            Q = _rand(3, sum(news), H_q, D, dtype=dtype)
            one = max(news) == 1
            O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=None if one else _cu(news), max_rows=max(news), window=W, sinks=3 if W else 0)
            ref.check_attend(O, L, r8.attend(pg, lens, news, Q, window=W, sinks=3 if W else 0), dtype, ref.P_ONCE[dtype])
    got = ctx.paged_read(pg.cache(), pg.table, pg.lens, T=sum(lens), cu_rows=_cu(lens), dtype=F32)
    for g, w in zip(got, _read_want(pg, lens, lens, F32)):
        assert torch.equal(g, w)
    ctx.sync()


@pytest.mark.parametrize("qe,ke,ve", [(60, -60, 0), (-60, 60, 0), (-100, 90, 0), (0, 0, 60), (0, 0, -40), (30, -30, 90)])
def test_exponents_far_from_zero(ctx, qe, ke, ve):   # noqa: F811
    """bf16 queries and scales of K whose powers of two cancel, and V far from 1: within the bounds of ordinary ones."""
    for news in ([1, 1], [3, 2], [64, 33]):
        pg = r8.Pages8(5, [300, 33], 2, 64, 16)
        used = pg.ks != 255
        pg.ks[used] += U8_of(ke)
        pg.vs[used] += U8_of(ve)
        one = max(news) == 1
        Q = (_rand(6, sum(news), 8, 64) * 2.0 ** qe).to(BF16)
        O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=None if one else _cu(news), max_rows=max(news))
        ref.check_attend(O, L, r8.attend(pg, [300, 33], news, Q), BF16, ref.P_ONCE[BF16], f"{news}")
    ctx.sync()


def U8_of(n):
    return torch.tensor(n % 256, dtype=U8, device="cuda")       # (added modulo 256)


def test_queries_of_zeros_and_of_one_large_element(ctx):   # noqa: F811
    pg = r8.Pages8(7, [90, 300], 2, 128, 32)
    for dtype in (F16, BF16):
        Q = _rand(8, 2, 8, 128, dtype=dtype)
        Q[0, 0] = 0
        Q[1, 1] *= 1e-4
        Q[1, 1, 3] = 300.0
        Q[0, 5, 7] = torch.finfo(dtype).smallest_normal
        Q[1, 6] = torch.finfo(dtype).smallest_normal
        O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q)
        ref.check_attend(O, L, r8.attend(pg, [90, 300], [1, 1], Q), dtype, PAIR)
    ctx.sync()


def test_k_and_v_laid_out_apart(ctx):   # noqa: F811
    """K stored head by head and V token by token, both as parts of larger tensors."""
    a, b = r8.Pages8(9, [77, 150], 3, 64, 32), r8.Pages8(9, [77, 150], 3, 64, 32, nhd=True)
    big = torch.zeros((a.k.shape[0], 3, 32, 3 * 64), dtype=U8, device="cuda")
    big[..., 64:128] = _bits(a.k)
    a.k, a.v = big.view(r8.E4M3)[..., 64:128], b.v
    for news in ([1, 1], [2, 2], [40, 100]):
        Q = _rand(4, sum(news), 6, 64, dtype=BF16)
        O, L = ctx.paged_attend(a.cache(), a.table, a.lens, Q, cu_rows=None if max(news) == 1 else _cu(news), max_rows=max(news))
        ref.check_attend(O, L, r8.attend(b, [77, 150], news, Q), BF16, ref.P_ONCE[BF16])
    for g, w in zip(ctx.paged_read(a.cache(), a.table, a.lens, dtype=F32), _read_want(b, [77, 150], [1, 1], F32)):
        assert torch.equal(g, w)
    x = _rand(5, 2, 6, 64, dtype=F16)
    k0 = big.clone()
    ctx.paged_append(a.cache(), a.table, a.lens, x[:, :3], x[:, 3:])
    assert torch.equal(k0[..., :64], big[..., :64]) and torch.equal(k0[..., 128:], big[..., 128:])
    for g, w in zip(ctx.paged_read(a.cache(), a.table, a.lens, dtype=F32), (x[:, :3], x[:, 3:])):
        c, e = r8.quantize(w)
        assert torch.equal(g.double(), c * torch.exp2(e.double())[..., None])
    ctx.sync()


def test_bounds_beyond_32_bits_and_the_same_bits_again(ctx):   # noqa: F811
    pg = r8.Pages8(4, [400, 90, 2500], 2, 128, 16)
    for news in ([1, 1, 1], [3, 2, 3], [300, 20, 64]):
        Q = _rand(5, sum(news), 8, 128, dtype=F16)
        kw = dict(cu_rows=None if max(news) == 1 else _cu(news), max_rows=max(news))
        O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, **kw)
        for more in ({}, dict(window=2 ** 32 + 20), dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(window=20, sinks=2 ** 32 + 1)):
            O2, L2 = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, **kw, **more)
            if "window" in more:
                ref.check_attend(O2, L2, r8.attend(pg, [400, 90, 2500], news, Q), F16, ref.P_ONCE[F16])
            else:
                assert torch.equal(O, O2) and torch.equal(L, L2)
        if max(news) > 1:
            O2, L2 = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=kw["cu_rows"], max_rows=2 ** 40)
            ref.check_attend(O2, L2, r8.attend(pg, [400, 90, 2500], news, Q), F16, ref.P_ONCE[F16])
    ctx.sync()


def test_many_sequences(ctx):   # noqa: F811
    """The batch limit, most of them empty or short, through every operator."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (binding_limit(),), generator=g).tolist()
    pg = r8.Pages8(3, lens, 1, 64, 16)
    B = len(lens)
    x = _rand(2, B, 4, 64, dtype=F16)
    live = [b for b in range(B) if lens[b]]
    q = ctx.paged_append(pg.cache(), pg.table, pg.lens, x[:, 2:3], x[:, 3:], Q=x[:, :2])
    O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, q)
    ref.check_attend(O, L, r8.attend(pg, lens, [1] * B, q), F16, PAIR)
    got = ctx.paged_read(pg.cache(), pg.table, pg.lens, dtype=F32)
    for y, w in zip(got, _read_want(pg, lens, [1] * B, F32)):
        assert torch.equal(y, w)
    c, e = r8.quantize(x[live, 3:])
    assert torch.equal(got[1][live].double(), c * torch.exp2(e.double())[..., None])
    with pytest.raises(binding.PckError):
        more = torch.cat((pg.lens, pg.lens[:1]))
        ctx.paged_attend(pg.cache(), torch.cat((pg.table, pg.table[:1])), more, torch.cat((q, q[:1])))
    ctx.sync()


def binding_limit():
    return 2048      # PCK_PAGED_MAX_BATCH


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_dominant_token_leaves_the_others_their_bits(ctx, dtype):   # noqa: F811
    """40,000 tokens whose weights are 2^-14 .. 2^-30 of the first one's, or whose values are: their sum keeps its place in O."""
    n, D = 40000, 64
    for down in (14, 22, 26, 30):
        for values_too in (False, True):
            pages = n // 16
            k = torch.zeros((pages, 1, 16, D), dtype=F32, device="cuda")
            k[0, 0, 0, 0] = 1.0
            v = torch.ones((pages, 1, 16, D), dtype=F32, device="cuda")
            v[0, 0, 0] = 0 if not values_too else -(2.0 ** 20)
            c = [torch.zeros((pages, 1, 16, D), dtype=U8, device="cuda").view(r8.E4M3) for _ in range(2)]
            s = [torch.zeros((pages, 1, 16), dtype=U8, device="cuda") for _ in range(2)]
            cache = binding.QuantizedPagedCache(*c, *s)
            tab, ln = torch.arange(pages, device="cuda", dtype=i32)[None], torch.tensor([n], dtype=i32, device="cuda")
            ctx.paged_append(cache, tab, ln, k.view(n, 1, D), v.view(n, 1, D), cu_rows=_cu([n]))
            Q = torch.zeros((1, 2, D), dtype=dtype, device="cuda")
            Q[..., 0] = down * math.log(2) * 8                   # tau = 1/8: the first score is `down` (log2) above the others

            class Pg:
                table = tab

                def kv(self):
                    return r8.values(c[0], s[0]), r8.values(c[1], s[1])
            O, L = ctx.paged_attend(cache, tab, ln, Q)
            want = r8.attend(Pg(), [n], [1], Q)
            if values_too and dtype == F16:      # O is below -2^18 in every case: nearer to fp16's -infinity than to -65,504
                assert (want[0] < -2.0 ** 18).all() and (O == -math.inf).all()
                assert ((L.double() - want[1]).abs() <= want[2] + 2.0 ** -20 + 2.0 ** -22 * (want[1].abs() + 8)).all()
            elif values_too:
                ref.check_attend(O, L, want, dtype, PAIR, f"{down}")
            else:       # the first token's value is 0: O is the others' share alone, to O's own rounding and a score's error
                tol = (ref.HALF_STEP[dtype] + 2 * want[2][..., None] + 2.0 ** -18) * want[0] + torch.finfo(dtype).smallest_normal
                assert ((O.double() - want[0]).abs() <= tol).all(), f"{down}"
    ctx.sync()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,H_kv,P", [(64, 2, 64), (64, 2, 16), (128, 2, 32), (256, 1, 16)])
def test_long_windows(ctx, dtype, D, H_kv, P):   # noqa: F811
    """Windows longer than a CTA takes whole, with sinks that end inside a page, at caches shorter and longer than they are."""
    lens = [9000, 4000, 20, 5071]
    pg = r8.Pages8(6, lens, H_kv, D, P)
    for news in ([1] * 4, [2, 1, 2, 2]):
        Q = _rand(3, sum(news), 2 * H_kv, D, dtype=dtype)
        for W, sinks in ((3000, 0), (5000, 70), (4097, 33), (65, 4000)):
            O, L = ctx.paged_attend(pg.cache(), pg.table, pg.lens, Q, cu_rows=None if max(news) == 1 else _cu(news), max_rows=max(news),
                                    window=W, sinks=sinks)
            ref.check_attend(O, L, r8.attend(pg, lens, news, Q, window=W, sinks=sinks), dtype, PAIR, f"{W} {sinks}")
    ctx.sync()
