"""Calls of the paged tail at the edges of what its interface allows, on the GPU."""
import math

import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F16, F32, _close, _rand, ctx, i32   # noqa: F401

pytestmark = pytest.mark.gpu


def _cu(*at):
    return torch.tensor(at, dtype=i32, device="cuda")


def _reports(ctx, fn):
    """Whether the call sets the device error of a length or row count out of range (and no other)."""
    ctx.sync()
    fn()
    try:
        ctx.sync()
    except binding.PckError as e:
        assert e.code == binding.ECUDA and "code 10" in str(e), str(e)
        return True
    return False


@pytest.mark.parametrize("max_rows", [2, 3, 4, 300])
@pytest.mark.parametrize("cu,sound", [((0, 2, 4), True), ((0, 0, 4), True), ((0, 3, 4), True), ((0, 1, 2), True), ((1, 2, 3), True),
                                      ((0, 3, 5), False), ((0, 4, 2), False), ((2, 0, 4), False), ((-1, 2, 4), False), ((0, 0, -3), False),
                                      ((0, 2 ** 31 - 1, 4), False), ((-2 ** 31, 2 ** 31 - 1, 4), False), ((5, 5, 6), False)])
def test_row_counts_that_make_no_sense_are_reported(ctx, cu, sound, max_rows):   # noqa: F811
    """cu_rows that descends or points outside the call's rows is reported by the append and by either attention, and so
    are more rows than max_rows; sound ones are not."""
    pg = ref.Pages(4, [400, 400], 1, 64, 16, F16)
    c = binding.PagedCache(pg.k, pg.v)
    T = 4 if max_rows < 300 else 400
    if T == 400 and not sound and max(cu) <= 6:
        cu = tuple(x if x in (0, -1) else x * 100 for x in cu)
    Q = _rand(5, T, 4, 64, dtype=F16)
    t = _cu(*cu)
    few = sound and all(b - a <= max_rows for a, b in zip(cu, cu[1:]))
    assert _reports(ctx, lambda: ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=t, max_rows=max_rows)) is not few
    k0, v0 = pg.k.clone(), pg.v.clone()
    assert _reports(ctx, lambda: ctx.paged_append(c, pg.table, pg.lens - 50, Q[:, :1], Q[:, 1:2], cu_rows=t)) is not sound
    if not sound:      # no token behind the sequences' own was written
        for b in range(2):
            for p in range(350, 400):
                at = (pg.table[b, p // 16].long(), slice(None), p % 16)
                assert torch.equal(k0[at], pg.k[at]) and torch.equal(v0[at], pg.v[at])


def test_rows_in_front_of_and_behind_the_sequences(ctx):   # noqa: F811
    """Rows that belong to no sequence, before the first or behind the last, are left as they were."""
    pg = ref.Pages(4, [400, 90], 2, 64, 16, F16)
    c = binding.PagedCache(pg.k, pg.v)
    for news, mr in (([3, 2], 3), ([300, 20], None)):
        T = 2 + sum(news) + 3
        Q = _rand(5, T, 4, 64, dtype=F16)
        cu = _cu(2, 2 + news[0], 2 + sum(news))
        O, L = torch.full((T, 4, 64), 5.0, dtype=F16, device="cuda"), torch.full((T, 4), 6.0, device="cuda")
        ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=cu, max_rows=mr, O=O, LSE=L)
        want = ref.attend(pg.k, pg.v, pg.table, [400, 90], news, Q[2:-3])
        ref.check_attend(O[2:-3], L[2:-3], want, F16, ref.P_ONCE[F16])
        for x, y in ((O[:2], L[:2]), (O[-3:], L[-3:])):
            assert (x == 5).all() and (y == 6).all()
    ctx.sync()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rope", [False, True])
def test_append_of_padded_sequences_gives_q_zero(ctx, dtype, rope):   # noqa: F811
    """Rows at a negative cache position store nothing; their Q comes out as zeros, not as it lay in memory."""
    cache = F16 if dtype == F32 else dtype
    H_q, H_kv, D = 5, 2, 64
    for lens, news in (([9, 0, 17, 0], [1, 1, 1, 1]), ([40, 2, 0], [3, 6, 4])):
        pg = ref.Pages(2, lens, H_kv, D, 16, cache)
        T = sum(news)
        x = _rand(3, T + 2, H_q + 2 * H_kv, D, dtype=dtype)
        one = all(m == 1 for m in news)
        cu = None if one else _cu(0, *torch.tensor(news).cumsum(0).tolist())
        n = T if one else T + 2
        cs = ref.angles(50, 32, "cuda") if rope else None
        p = torch.tensor([q for _, q in ref.rows_of(lens, news)], device="cuda")
        for positions in (None, torch.cat((p, p.new_full((2,), 9))).to(i32)[:n] if rope else None):
            Qo = torch.full((n, H_q, D), math.nan, dtype=dtype, device="cuda")
            Q = x[:n, :H_q].clone()
            for out in (Qo, Q):     # of its own, and in place
                ctx.paged_append(binding.PagedCache(pg.k, pg.v), pg.table, pg.lens, x[:n, H_q:H_q + H_kv], x[:n, H_q + H_kv:], Q=Q,
                                 cu_rows=cu, cos_sin=cs, positions=positions, norm=True, Q_out=out)
                assert (out[:T][p < 0] == 0).all()
                good = p >= 0
                _close(out[:T][good], ref.norm_rope(x[:T, :H_q][good], None, 1e-6, cs, p[good]), dtype, "q")
            assert torch.isnan(Qo[T:]).all() and torch.equal(Q[T:], x[T:n, :H_q])    # of no sequence: left as they were
    ctx.sync()


def test_max_rows_beyond_the_rows(ctx):   # noqa: F811
    """max_rows is a bound: one far above the rows that there are decides nothing that the rows themselves do not."""
    for D, G, T in ((192, 4, 2), (256, 2, 4), (256, 8, 1), (128, 4, 4), (64, 3, 5)):
        pg = ref.Pages(6, [300], 2, D, 16, F16)
        Q = _rand(7, T, 2 * G, D, dtype=F16)
        c = binding.PagedCache(pg.k, pg.v)
        want = ref.attend(pg.k, pg.v, pg.table, [300], [T], Q)
        for mr in (T, 100, 2 ** 31 - 1):
            O, L = ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=_cu(0, T), max_rows=mr)
            ref.check_attend(O, L, want, F16, ref.P_SPLIT[F16])
    ctx.sync()


def test_bounds_wider_than_32_bits(ctx):   # noqa: F811
    """Windows, sinks and row bounds beyond int32 are as good as the widest, and never wrap to a narrow one."""
    pg = ref.Pages(6, [300], 2, 64, 16, F16)
    Q = _rand(7, 3, 4, 64, dtype=F16)
    c = binding.PagedCache(pg.k, pg.v)
    at = lambda **kw: ctx.paged_attend(c, pg.table, pg.lens, Q, cu_rows=_cu(0, 3), **kw)   # noqa: E731
    want = at()
    for kw in (dict(window=2 ** 32 + 20), dict(window=2 ** 31 + 5), dict(window=20, sinks=2 ** 32 + 1), dict(max_rows=2 ** 32 + 1), dict(window=2 ** 63 - 1)):
        for a, b in zip(at(**kw), want):
            assert torch.equal(a, b), kw
    for kw in (dict(window=-2 ** 32), dict(sinks=-2 ** 32 - 1), dict(max_rows=-2 ** 32 + 1), dict(max_rows=2 ** 32 * -1)):
        with pytest.raises(binding.PckError) as e:
            at(**kw)
        assert e.value.code == binding.EINVAL
    ctx.sync()
