"""The 64-bit forms of the paged-tail operators against hand-made values and loops (CPU)."""
import math

import pytest
import torch

from tests import paged_ref as ref


def test_rotation_by_hand():
    # one pair set of 16: position 1 turns pair i by its angle; quarter turns map (a, b) to (-b, a)
    cs = torch.cat((torch.zeros(1, 8), torch.ones(1, 8)), 1)
    x = torch.arange(1.0, 17.0).view(1, 1, 16)
    half = ref.norm_rope(x, cos_sin=cs, pos=torch.zeros(1))[0, 0]
    assert half[:8].tolist() == [-9., -10., -11., -12., -13., -14., -15., -16.]
    assert half[8:].tolist() == [1., 2., 3., 4., 5., 6., 7., 8.]
    adj = ref.norm_rope(x, cos_sin=cs, pos=torch.zeros(1), interleaved=True)[0, 0]
    assert adj.tolist() == [-2., 1., -4., 3., -6., 5., -8., 7., -10., 9., -12., 11., -14., 13., -16., 15.]


def test_norm_and_partial_rotation():
    torch.manual_seed(0)
    x, w = torch.randn(3, 2, 48), torch.rand(48) + 0.5
    y = ref.norm_rope(x, w, 1e-5, ref.angles(10, 32), torch.tensor([0, 3, 9]))
    n = x.double() / (x.double().pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * w.double()
    assert torch.allclose(y[..., 32:], n[..., 32:], rtol=1e-12)
    assert torch.allclose(y[0], n[0], rtol=1e-12)                                     # position 0 turns nothing
    assert torch.allclose(y[..., :32].norm(dim=-1), n[..., :32].norm(dim=-1), rtol=1e-6)   # rotations keep lengths


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (5, 2), (1, 1), (100, 3)])
def test_attend_by_loops(window, sinks):
    lens, news = [7, 0, 33, 16], [3, 0, 33, 1]
    pg = ref.Pages(3, lens, 2, 16, 16, torch.float32, device="cpu")
    torch.manual_seed(1)
    Q = torch.randn(sum(news), 4, 16)
    prior = torch.randn(sum(news), 4, 16), torch.randn(sum(news), 4)
    O, L, _, _ = ref.attend(pg.k, pg.v, pg.table, lens, news, Q, window, sinks)
    Om, Lm, _, _ = ref.attend(pg.k, pg.v, pg.table, lens, news, Q, window, sinks, prior)
    for r, (b, p) in enumerate(ref.rows_of(lens, news)):
        for h in range(4):
            keys = [j for j in range(p + 1) if window == 0 or j > p - window or j < sinks]
            kv = [(pg.k[pg.table[b, j // 16], h // 2, j % 16].double(), pg.v[pg.table[b, j // 16], h // 2, j % 16].double())
                  for j in keys]
            s = [float(Q[r, h].double() @ k) / 4.0 for k, _ in kv]
            z = math.log(sum(math.exp(x) for x in s))
            o = sum(math.exp(x - z) * v for x, (_, v) in zip(s, kv))
            assert abs(L[r, h].item() - z) < 1e-12 and (O[r, h] - o).abs().max() < 1e-12
            w = 1 / (1 + math.exp(prior[1][r, h].item() - z))
            assert (Om[r, h] - (w * o + (1 - w) * prior[0][r, h].double())).abs().max() < 1e-12
            assert abs(Lm[r, h].item() - math.log(math.exp(z) + math.exp(prior[1][r, h].item()))) < 1e-12


def test_attend_empty_rows():
    pg = ref.Pages(4, [0, 5], 1, 16, 16, torch.float32, device="cpu")
    Q = torch.ones(2, 2, 16)
    O, L, _, _ = ref.attend(pg.k, pg.v, pg.table, [0, 5], [1, 1], Q)
    assert (O[0] == 0).all() and (L[0] == -math.inf).all() and torch.isfinite(O[1]).all()
    prior = torch.full((2, 2, 16), 3.0), torch.tensor([[1.0, -math.inf], [-math.inf, -math.inf]])
    Om, Lm, _, _ = ref.attend(pg.k, pg.v, pg.table, [0, 5], [1, 1], Q, prior=prior)
    assert (Om[0, 0] == 3).all() and Lm[0, 0] == 1 and (Om[0, 1] == 0).all() and torch.equal(Om[1], O[1])


def test_a_planted_mistake_is_seen():
    """The comparison fails for an off-by-one window, a missing sink, a dropped scale and bf16-rounded weights."""
    lens, news = [200], [4]
    pg = ref.Pages(5, lens, 1, 64, 16, torch.float16, device="cpu")
    torch.manual_seed(2)
    Q = torch.randn(4, 2, 64).half()
    good = ref.attend(pg.k, pg.v, pg.table, lens, news, Q, 50, 4)
    ref.check_attend(good[0].half(), good[1].float(), good, torch.float16, ref.P_SPLIT[torch.float16])
    for bad in (ref.attend(pg.k, pg.v, pg.table, lens, news, Q, 51, 4), ref.attend(pg.k, pg.v, pg.table, lens, news, Q, 50, 3),
                ref.attend(pg.k, pg.v, pg.table, lens, news, Q * 8, 50, 4)):
        with pytest.raises(AssertionError):
            ref.check_attend(bad[0].half(), bad[1].float(), good, torch.float16, ref.P_SPLIT[torch.float16])
    with pytest.raises(AssertionError):
        ref.check_attend(good[0].half() * (1 + 2.0 ** -8), good[1].float(), good, torch.float16, ref.P_SPLIT[torch.float16])
