"""Rows that an append to the quantised cache leaves out, beside rows that it stores, and Q written back in place; on the GPU."""
import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_e4m3_ref as r8
from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F16, F32, _close, _rand, ctx, i32   # noqa: F401
from tests.test_gpu_paged_e4m3 import _bits, _check_rows, _empty_pages

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("B,H_q,H_kv,D,R", [(90, 8, 2, 128, 64), (300, 3, 1, 64, 64), (24, 32, 8, 128, 128), (40, 2, 3, 512, 128), (7, 1, 1, 16, 16)])
def test_append_beside_rows_left_out(ctx, dtype, B, H_q, H_kv, D, R):   # noqa: F811
    """Every third sequence is padded (all its rows, or the first of them, at negative positions), and rows lie in front of the
    first sequence and behind the last: they store nothing; the others' codes are theirs. Q out of place and back into the
    projection that Q, K and V are parts of: the same bits."""
    page, lens, news = 16, [], []
    for b in range(B):
        news.append(1 + b % 5)
        lens.append(0 if b % 6 == 2 else 1 if b % 6 == 5 else news[-1] + 7 * (b % 11))
    front, back = 6, 11
    T = front + sum(news) + back
    pg = ref.Pages(3, lens, 1, 16, page, F16)              # its table
    x = _rand(4, T, H_q + 2 * H_kv, D, dtype=dtype)
    wq, wk = 1 + _rand(1, D, dtype=dtype, scale=0.2), 1 + _rand(2, D, dtype=dtype, scale=0.2)
    cs = ref.angles(200, R, "cuda")
    cu = torch.tensor([front] + [front + n for n in torch.tensor(news).cumsum(0).tolist()], dtype=i32, device="cuda")
    at = ref.rows_of(lens, news)
    live = torch.tensor([front + i for i, (_, p) in enumerate(at) if p >= 0], device="cuda")
    none = torch.tensor([front + i for i, (_, p) in enumerate(at) if p < 0], device="cuda")
    p = torch.tensor([q for _, q in at if q >= 0], device="cuda")
    b = torch.tensor([s for s, q in at if q >= 0], device="cuda")
    pages, slots = pg.table[b, p // page].long(), p % page
    outer = [t for t in range(T) if t < front or t >= T - back]
    got = []
    for place in ("out", "in"):
        k, v, ks, vs = _empty_pages(int(pg.table.max()) + 2, H_kv, page, D)
        y = x.clone()
        Q = y[:, :H_q]
        Qo = Q if place == "in" else torch.full((T, H_q, D), 9.0, dtype=dtype, device="cuda")
        ctx.paged_append(binding.QuantizedPagedCache(k, v, ks, vs), pg.table, pg.lens, y[:, H_q:H_q + H_kv], y[:, H_q + H_kv:], Q=Q, cu_rows=cu,
                         cos_sin=cs, q_weight=wq, k_weight=wk, Q_out=Qo)
        _close(Qo[live], ref.norm_rope(x[live, :H_q], wq, 1e-6, cs, p, False), dtype, "q")
        assert (Qo[none] == 0).all()
        assert torch.equal(Qo[outer], x[outer, :H_q] if place == "in" else torch.full_like(Qo[outer], 9.0))
        assert torch.equal(y[:, H_q:], x[:, H_q:])
        _check_rows(_bits(k)[pages, :, slots].view(r8.E4M3), ks[pages, :, slots],
                    ref.norm_rope(x[live, H_q:H_q + H_kv], wk, 1e-6, cs, p, False), "k")
        want, e = r8.quantize(x[live, H_q + H_kv:])
        assert torch.equal(vs[pages, :, slots].long() - 127, e)
        assert torch.equal(r8.values(_bits(v)[pages, :, slots].view(r8.E4M3), torch.full_like(vs[pages, :, slots], 127)), want)
        got.append([t.clone() for t in (Qo[live], _bits(k), _bits(v), ks, vs)])
        for t, was in ((_bits(k), 0x55), (_bits(v), 0x55), (ks, 0x33), (vs, 0x33)):     # and nothing else was written
            t[pages, :, slots] = was
            assert (t == was).all()
    for one, other in zip(*got):
        assert torch.equal(one, other)
    ctx.sync()


def test_rows_that_cu_rows_names_again_and_again(ctx):   # noqa: F811
    """A cu_rows that goes up to T and back to 0 for every sequence names 1024 T rows: reported, and no more work than T rows can be."""
    T, B = 1 << 22, 2048
    pg = r8.Pages8(2, [40] * 2, 1, 16, 16)
    table, lens = pg.table[:1].expand(B, -1).contiguous(), torch.full((B,), 40, dtype=i32, device="cuda")
    cu = torch.zeros(B + 1, dtype=i32, device="cuda")
    cu[1::2] = T
    ctx.sync()
    a, z = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    ctx.paged_read(pg.cache(), table, lens, T=T, cu_rows=cu)
    z.record()
    z.synchronize()
    with pytest.raises(binding.PckError) as e:
        ctx.sync()
    assert "code 10" in str(e.value)
    # T rows of 16 + 16 fp16 values: 268 MB. A thousand times as many would take a second.
    assert a.elapsed_time(z) < 200
    K, V = ctx.paged_read(pg.cache(), pg.table, pg.lens, T=80, cu_rows=torch.tensor([0, 40, 80], dtype=i32, device="cuda"))     # the next call is quiet
    for got, x in zip((K, V), pg.kv()):
        assert torch.equal(got[:40], x[pg.table[0].long()].transpose(1, 2).reshape(-1, 1, 16)[:40].half())
    ctx.sync()


@pytest.mark.parametrize("cu,stored", [((3, 0, 9, 1, 9), []), ((4, 0, 9, 0, 9), []), ((0, 9, 2, 9, 4), [(0, 0, 31), (1, 0, 32)])])
def test_rows_that_only_a_senseless_cu_rows_places(ctx, cu, stored):   # noqa: F811
    """Reported; and a row outside [cu_rows[0], cu_rows[B]), which is not copied, is not stored where a descending cu_rows seems to
    place it. stored: (row, sequence, position) of those that are."""
    pg = ref.Pages(3, [40] * 4, 1, 16, 16, F16)            # its table
    k, v, ks, vs = _empty_pages(int(pg.table.max()) + 2, 2, 16, 64)
    x = _rand(4, 9, 4, 64, dtype=F16)
    ctx.sync()
    ctx.paged_append(binding.QuantizedPagedCache(k, v, ks, vs), pg.table, pg.lens, x[:, :2], x[:, 2:], cu_rows=torch.tensor(cu, dtype=i32, device="cuda"))
    with pytest.raises(binding.PckError) as e:
        ctx.sync()
    assert "code 10" in str(e.value)
    for t, b, p in stored:
        at = (pg.table[b, p // 16].long(), slice(None), p % 16)
        for codes, scale, y in ((k, ks, x[t, :2]), (v, vs, x[t, 2:])):
            want, exp = r8.quantize(y)
            assert torch.equal(scale[at].long() - 127, exp)
            assert torch.equal(r8.values(_bits(codes)[at].view(r8.E4M3), torch.full_like(scale[at], 127)), want)
            _bits(codes)[at], scale[at] = 0x55, 0x33
    assert (_bits(k) == 0x55).all() and (_bits(v) == 0x55).all() and (ks == 0x33).all() and (vs == 0x33).all()
