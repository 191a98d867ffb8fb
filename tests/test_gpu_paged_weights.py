"""Softmax weights far below the largest one (a strong first token over a long cache of near-equal keys) on the GPU:
their sum is a visible share of O however small each of them is."""
import math

import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F16, ctx, i32   # noqa: F401

pytestmark = pytest.mark.gpu


def _check(ctx, n, rows, B, H_kv, G, D, dtype, p_err, at, adds):
    """B sequences over the same n tokens: token `at` scores 17 to 33 (log2) above all others, which score 0; V is 0
    there and 256 elsewhere, so with x keys beside it O = 256 x / (2^gap + x). adds: fp32 additions of one running sum."""
    page = 64
    n_pages = -(-n // page)
    k = torch.full((n_pages + 1, H_kv, page, D), math.nan, dtype=dtype, device="cuda")
    v = k.clone()
    for t, x in ((k, 0), (v, 256)):
        t[:n // page], t[n // page, :, :n % page] = x, x
    k[at // page, :, at % page, 0], v[at // page, :, at % page] = 16, 0
    table = torch.arange(n_pages, dtype=i32, device="cuda").expand(B, n_pages).contiguous()
    T, H_q = B * rows, H_kv * G
    gap = 17 + 16 * torch.arange(T * H_q, device="cuda").double().view(T, H_q) / (T * H_q)
    Q = torch.zeros((T, H_q, D), dtype=dtype, device="cuda")
    Q[..., 0] = (gap * math.sqrt(D) * math.log(2) / 16).to(dtype)
    lens = torch.full((B,), n, dtype=i32, device="cuda")
    cu = None if rows == 1 else torch.arange(0, T + 1, rows, dtype=i32, device="cuda")
    O, L = ctx.paged_attend(binding.PagedCache(k, v), table, lens, Q, cu_rows=cu, max_rows=rows)
    s = Q[..., 0].double() * 16 / math.sqrt(D)                       # the row's one score that is not 0
    x = (n - rows + torch.arange(rows, device="cuda").repeat(B)).double()[:, None]   # keys beside that one
    z = torch.logaddexp(s, x.log())
    want = (256 * torch.exp(x.log() - z))[..., None].expand(T, H_q, D)
    # a score is one product, exact in fp32; its scaling and the subtraction of the maximum round it by half a step
    # each. Each addition to a sum rounds it by half a step.
    ds = (2 * s + adds) * 2.0 ** -24
    ref.check_attend(O, L, (want, z, ds, torch.full_like(s, 256)), dtype, p_err, f"n {n} rows {rows} B {B} D {D}")
    ctx.sync()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,rows,B,H_kv,G,D", [
    (1000, 1, 3, 2, 4, 128), (900, 1, 90, 2, 4, 64),                                       # an item per CTA, per half CTA
    (131070, 1, 1, 2, 8, 128), (131070, 1, 2, 1, 16, 64), (131070, 1, 1, 2, 4, 256),       # ranges per CTA
    (40000, 1, 40, 4, 4, 128), (40000, 1, 230, 4, 4, 64), (40000, 1, 240, 4, 2, 192),      # per half CTA, per warp
    (131070, 4, 1, 2, 4, 128), (60000, 2, 100, 2, 4, 64)])                                 # a few rows of a sequence
@pytest.mark.parametrize("at", [0, 777])
def test_token_weights_behind_a_dominant_key(ctx, dtype, n, rows, B, H_kv, G, D, at):   # noqa: F811
    # tiles of 16 tokens that one of the card's warps takes (twice an even share, and what a CTA's own item may have),
    # two additions to a lane's sum for each
    tiles = min(n // 16 + 1, 64 + 2 * B * H_kv * (n // 16) // (152 * (8 if D <= 128 else 4)))
    _check(ctx, n, rows, B, H_kv, G, D, dtype, ref.P_SPLIT[dtype], at, 2 * tiles)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,rows,B,H_kv,G,D", [(131070, 20, 1, 2, 4, 128), (131070, 40, 1, 1, 4, 64),     # keys split
                                               (131070, 300, 1, 64, 1, 64), (100000, 300, 2, 20, 2, 128)])   # whole
@pytest.mark.parametrize("at", [0, 777])
def test_rows_weights_behind_a_dominant_key(ctx, dtype, n, rows, B, H_kv, G, D, at):   # noqa: F811
    _check(ctx, n, rows, B, H_kv, G, D, dtype, ref.P_ONCE[dtype], at, n // 128 + 1)     # one addition a block of 128 keys
