"""What the arithmetic of one-token attention over the quantised cache is stated to keep, on the GPU."""
import math

import pytest
import torch

from prefix_cached_kv_gb300 import binding
from tests import paged_e4m3_ref as r8
from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, ctx, i32   # noqa: F401
from tests.test_gpu_paged_e4m3 import U8, _cu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ve", [10, -39, -45, -50, -60])
def test_weights_of_small_v_scales(ctx, D, ve, rows):   # noqa: F811
    """One token without a value (its codes are 0) and 40,000 others whose weights are 2^-down of its own, all with V scales 2^ve:
    O is the others' share. The kernel holds a weight to 22 bits or, as a share of the largest one, to 2^-37, for V scales of
    2^(-40 - b) to 2^(-37 + b): n equal weights off by that much move O by n times it."""
    n = 40000
    page = 16 if D != 128 else 64
    k = torch.zeros((n // page, 1, page, D), dtype=U8, device="cuda")
    k[0, 0, 0, 0] = 0x38                                   # 1.0
    v = torch.full_like(k, 0x38)
    v[0, 0, 0] = 0
    ks = torch.full(k.shape[:3], 127, dtype=U8, device="cuda")
    vs = torch.full_like(ks, 127 + ve)
    cache = binding.QuantizedPagedCache(k.view(r8.E4M3), v.view(r8.E4M3), ks, vs)
    tab, ln = torch.arange(n // page, device="cuda", dtype=i32)[None], torch.tensor([n], dtype=i32, device="cuda")

    class Pg:
        table = tab

        def kv(self):
            return r8.values(k.view(r8.E4M3), ks), r8.values(v.view(r8.E4M3), vs)
    share = 2.0 ** (-37 + max(0, -40 - ve))
    for down in (8, 14, 20, 26):
        Q = torch.zeros((rows, 2, D), dtype=BF16, device="cuda")
        Q[..., 0] = down * math.log(2) * math.sqrt(D)      # the first score is about `down` (log2) above the others
        O, L = ctx.paged_attend(cache, tab, ln, Q, cu_rows=None if rows == 1 else _cu([rows]), max_rows=rows)
        Or, Lr, ds, _ = r8.attend(Pg(), [n], [rows], Q)
        tol = (ref.HALF_STEP[BF16] + 2 * ds[..., None] + 2.0 ** -18) * Or + 1.01 * n * share * 2.0 ** ve
        assert ((O.double() - Or).abs() <= tol).all(), f"{down}: {((O.double() - Or).abs() / Or).max().item():.3e}"
        # a scores' difference of up to 2^6 in fp32 (m lies up to 52 below the largest): 2^-19 of 2^x and of the LSE
        assert ((L.double() - Lr).abs() <= ds + 2.0 ** -18).all()
    ctx.sync()
