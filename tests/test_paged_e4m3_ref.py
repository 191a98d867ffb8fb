"""The 64-bit form of the quantised cache against hand-worked values and torch's own e4m3, on the CPU."""
import math

import torch

from tests import paged_e4m3_ref as r8


def test_exponents():
    a = torch.tensor([448.0, 448.0 * (1 + 2.0 ** -20), 224.0, 225.0, 1.0, 1.75, 1.76, 0.0, 2.0 ** -140, 3.0e38], dtype=torch.float64)
    assert r8.scale_exponents(a).tolist() == [0, 1, -1, 0, -8, -8, -7, -126, -126, 120]


def test_codes():
    x = torch.tensor([448.0, 432.0, 440.0, 1.0, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, -0.3], dtype=torch.float64)
    want = [448.0, 448.0, 448.0, 1.0, 1.0, 1.25, 2.0 ** -9, 0.0, 2.0 ** -8, 0.0, -0.3125]
    assert r8.round_codes(x).tolist() == want        # 432 and 1.0625 lie between two codes: the even one
    g = torch.Generator().manual_seed(1)
    y = (torch.rand(20000, generator=g) * 2 - 1) * 448 * torch.exp2(-12 * torch.rand(20000, generator=g))
    assert torch.equal(r8.round_codes(y.double()), y.to(r8.E4M3).double())
    every = torch.arange(256, dtype=torch.uint8).view(r8.E4M3).double()
    fine = every[every.isfinite()]
    assert torch.equal(r8.round_codes(fine), fine)


def test_quantize_and_values():
    y = torch.tensor([[3.0, -448.0, 0.1], [0.0, 0.0, 0.0], [math.inf, 2.0, math.nan]])
    c, e = r8.quantize(y)
    assert e.tolist() == [0, -126, -7]
    assert c[0].tolist() == [3.0, -448.0, 0.1015625] and c[1].tolist() == [0.0, 0.0, 0.0]
    assert c[2, 0].isnan() and c[2, 2].isnan() and c[2, 1] == 256.0
    v = r8.values(c.float().to(r8.E4M3), (e + 127).to(torch.uint8))
    assert v[0].tolist() == c[0].tolist() and v[2, 1] == 2.0
    got = r8.values(torch.ones((3, 2)).to(r8.E4M3), torch.tensor([0, 255, 128], dtype=torch.uint8))
    assert got[0].tolist() == [2.0 ** -127] * 2 and got[1].isnan().all() and got[2].tolist() == [2.0, 2.0]


def test_pages():
    pg = r8.Pages8(3, [5, 0, 40], 2, 16, 16, device="cpu", nhd=True)
    k, v = pg.kv()
    assert k.shape == (3 + 4, 2, 16, 16) and pg.k.stride()[1] == 16
    used = torch.isfinite(k).all(-1)
    assert int(used.sum()) == 2 * 45 and torch.equal(used, torch.isfinite(v).all(-1))
    q = torch.randn((1, 2, 16))
    one = r8.attend(pg, [5], [1], q)[0]
    page = pg.table[0, 0]
    for h in range(2):
        s = (k[page, h, :5] @ q[0, h].double()) / 4
        assert torch.allclose(one[0, h], torch.softmax(s, 0) @ v[page, h, :5])
