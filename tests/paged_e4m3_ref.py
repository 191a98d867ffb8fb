"""The quantised paged cache in 64 bits, from its definition, and the tolerances that its arithmetic allows. Plain torch on any
device; used by the tests only."""
import torch

from tests import paged_ref as ref

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
HALF_STEP = 2.0 ** -4          # of a code, relative to its value; 2^-10 in units of the scale below the normal range


def scale_exponents(a):
    """Least e with a 2^-e <= 448, held to -126 .. 120, for magnitudes a (64 bits, finite): by search from above."""
    e = torch.full(a.shape, 120, dtype=torch.int64, device=a.device)
    for cand in range(119, -127, -1):
        e = torch.where(a <= 448.0 * 2.0 ** cand, cand, e)
    return e


def round_codes(x):
    """64-bit values (at most 448 in magnitude) to the nearest e4m3 value, ties to the even code."""
    a = x.abs()
    _, e = torch.frexp(a)
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def quantize(y):
    """fp64 rows [..., D] -> (values of the codes, exponents): what is not finite becomes NaN."""
    y = y.double()
    ok = torch.isfinite(y)
    e = scale_exponents(torch.where(ok, y.abs(), 0).amax(-1))
    c = round_codes(torch.where(ok, y, 0) * torch.exp2(-e.double())[..., None])
    return torch.where(ok, c, torch.nan), e


def values(codes, scale):
    """codes [..., D] (e4m3) and scales [...] (exponent bytes) -> 64-bit values, as the format says."""
    b = scale.view(torch.uint8).double()
    f = torch.exp2(b - 127).masked_fill(b == 255, torch.nan)
    return codes.view(torch.uint8).cpu().view(E4M3).double().to(codes.device) * f[..., None]


class Pages8:
    """Random quantised pages and tables for sequences of the given lengths; unused slots hold NaN codes and NaN
    scales, unused table entries -1. spread: (log2) range of the tokens' magnitudes in k and in v."""

    def __init__(self, seed, lens, H_kv, D, page, device="cuda", nhd=False, extra=3, width=None, spread=(1.0, 6.0)):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(n, 0) // page) for n in lens]
        n_pages = sum(need) + extra
        order = torch.randperm(n_pages, generator=g)
        width = max(1, max(need)) if width is None else width
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        used = torch.zeros((n_pages, page), dtype=torch.bool)
        at = 0
        for b, n in enumerate(lens):
            for i in range(need[b]):
                table[b, i] = order[at]
                used[order[at], :min(page, n - i * page)] = True
                at += 1

        def side(sp):
            x = torch.randn((n_pages, H_kv, page, D), generator=g)
            x = x * torch.exp2(sp * (torch.rand((n_pages, H_kv, page, 1), generator=g) - 0.5))
            m, e = torch.frexp(x.abs().amax(-1))
            e = e - 9 + (m > 0.875).int()
            codes = (x * torch.exp2(-e.float())[..., None]).to(E4M3).view(torch.uint8)
            codes = torch.where(used[:, None, :, None], codes, 0x7f).to(torch.uint8).to(device)
            scale = torch.where(used[:, None], e + 127, 255).to(torch.uint8).to(device).contiguous()
            if nhd:
                codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
            return codes.view(E4M3), scale
        self.k, self.ks = side(spread[0])
        self.v, self.vs = side(spread[1])
        self.table = table.to(device)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)

    def cache(self):
        from prefix_cached_kv_gb300 import binding
        return binding.QuantizedPagedCache(self.k, self.v, self.ks, self.vs)

    def kv(self):
        """64-bit values of the pages [n_pages, H_kv, page, D]."""
        return values(self.k, self.ks), values(self.v, self.vs)


def attend(pg, lens, news, Q, **kw):
    k, v = pg.kv()
    return ref.attend(k, v, pg.table, lens, news, Q, **kw)
