"""Row attention over the quantised cache whose tables could name more pages than the call may read back at once, on the GPU:
it goes through its kv heads, and then its sequences, some at a time."""
import ctypes
import math

import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_e4m3_ref as r8
from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F16, _rand, ctx, i32   # noqa: F401
from tests.test_gpu_paged_e4m3 import U8, _bits, _cu

pytestmark = pytest.mark.gpu
GIB = 1 << 30


def _spread_out(pg, n_pages, width):
    """The pages of pg at random places of a cache of n_pages pages (NaN elsewhere), in tables of that width."""
    H, page, D = pg.k.shape[1:]
    g = torch.Generator().manual_seed(7)
    at = torch.randperm(n_pages, generator=g)[:pg.k.shape[0]].cuda()
    out = []
    for t, none in ((pg.k, 0x7f), (pg.v, 0x7f), (pg.ks, 255), (pg.vs, 255)):
        t = _bits(t)
        big = torch.full((n_pages, *t.shape[1:]), none, dtype=U8, device="cuda")
        big[at] = t
        out.append(big)
    table = torch.full((pg.table.shape[0], width), -1, dtype=i32, device="cuda")
    table[:, :pg.table.shape[1]] = torch.where(pg.table >= 0, at[pg.table.long()].to(i32), -1)
    return binding.QuantizedPagedCache(out[0].view(r8.E4M3), out[1].view(r8.E4M3), out[2], out[3]), table


def _workspace(ctx, c, table, lens, news, T, H_q, dtype, window, sinks):   # noqa: F811
    batch = binding.PagedBatchT(len(lens), T, 1, 1, 1, table.shape[1], T)      # (sizes only are looked at)
    n = ctypes.c_size_t()
    ctx._rc(ctx.lib.pck_paged_workspace_e4m3(ctx.h, c.ref, ctypes.byref(batch), binding._PAGED_DT[dtype], H_q, window, sinks, ctypes.byref(n)))
    return n.value


def _check(ctx, dtype, lens, news, G, H_kv, D, page, n_pages, width, W=0, sinks=0, prior=False, whole=0):   # noqa: F811
    pg = r8.Pages8(3, lens, H_kv, D, page)
    c, table = _spread_out(pg, n_pages, width)
    H_q, front, back = G * H_kv, 3, 5
    T = front + sum(news) + back
    Q = _rand(4, T, H_q + 1, D, dtype=dtype)[:, 1:]
    cu = _cu(news) + front
    pr = None
    if prior:
        pr = (_rand(5, T, H_q, D), _rand(6, T, H_q) + math.log(max(lens)))
        pr[1][front, 0] = -math.inf
    # what a call of this kind may take: 4 GiB or half of the codes (or one sequence's pages of one kv head), the page map, the
    # partials of 152 splits
    codes = 2 * n_pages * H_kv * page * D
    most = max(4 * GIB, codes // 2, min(n_pages, width) * page * D * 4)
    need = _workspace(ctx, c, table, lens, news, T, H_q, dtype, W, sinks)
    assert need <= most + len(lens) * width * 4 + 256 + (64 << 20), f"{need / GIB:.2f} GiB"
    assert whole > most
    O, L = torch.full((T, H_q, D), 5.0, dtype=dtype, device="cuda"), torch.full((T, H_q), 6.0, device="cuda")
    ctx.paged_attend(c, table, pg.lens, Q, cu_rows=cu, window=W, sinks=sinks, prior=pr, O=O, LSE=L)
    ctx.sync()
    at = slice(front, T - back)
    want = r8.attend(pg, lens, news, Q[at], window=W, sinks=sinks, prior=None if pr is None else (pr[0][at], pr[1][at]))
    ref.check_attend(O[at], L[at], want, dtype, ref.P_ONCE[dtype])
    for s in (slice(0, front), slice(T - back, T)):
        assert (O[s] == 5).all() and (L[s] == 6).all()
    return ctx, c, table, pg, Q, cu, O, L


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("G,H_kv,D,prior", [(4, 7, 64, False), (3, 4, 128, True), (1, 5, 64, False)])
def test_kv_heads_some_at_a_time(ctx, dtype, G, H_kv, D, prior):   # noqa: F811
    """Wide tables over a large cache: the pages at the cache's own numbers, a few kv heads at a time."""
    page, n_pages, lens, news = 64, 90000, [700, 33, 64, 257, 0], [300, 33, 40, 129, 2]
    _check(ctx, dtype, lens, news, G, H_kv, D, page, n_pages, 20000, prior=prior, whole=n_pages * page * D * H_kv * 4)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_sequences_some_at_a_time(ctx, dtype):   # noqa: F811
    """Tables so wide that one head's pages are too many: some sequences at a time, one kv head each; the same bits again, and from
    a captured graph."""
    page, n_pages, width, D, H_kv = 16, 2500000, 200000, 64, 2
    lens, news = [400, 90, 17, 800, 129, 300, 64], [300, 20, 17, 64, 100, 1, 64]
    ctx_, c, table, pg, Q, cu, O, L = _check(ctx, dtype, lens, news, 4, H_kv, D, page, n_pages, width, whole=len(lens) * width * page * D * H_kv * 4)
    st = torch.cuda.Stream()
    ws = torch.empty(_workspace(ctx, c, table, lens, news, Q.shape[0], Q.shape[1], dtype, 0, 0), dtype=U8, device="cuda")
    O2, L2 = torch.full_like(O, 5.0), torch.full_like(L, 6.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        ctx.paged_attend(c, table, pg.lens, Q, cu_rows=cu, O=O2, LSE=L2, workspace=ws)
    for _ in range(3):
        ws.fill_(0xff)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, O2) and torch.equal(L, L2)
    ctx.sync()


def test_windows_and_counts(ctx):   # noqa: F811
    """Long windows over wide tables; and a call is one query, however many parts it takes."""
    before = ctx.info()["queries_served"]
    _check(ctx, BF16, [700, 33, 5000], [300, 33, 200], 4, 8, 128, 64, 40000, 12000, W=700000, sinks=5, whole=3 * 700000 * 128 * 8 * 4)
    assert ctx.info()["queries_served"] == before + 1
