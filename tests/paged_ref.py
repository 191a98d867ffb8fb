"""The paged-tail operators in 64 bits, from their definitions, and the tolerances that the kernels'
arithmetic allows. Plain torch on any device; used by the tests only."""
import math

import torch

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float16, torch.bfloat16, torch.float32)}


def norm_rope(x, weight=None, eps=None, cos_sin=None, pos=None, interleaved=False):
    """x [T, H, D] -> 64 bits: RMS norm (eps None: none) and rotation by rows pos [T] of cos_sin [n, R]."""
    y = x.double()
    if eps is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.double()
    if cos_sin is None:
        return y
    R = cos_sin.shape[1]
    c, s = (t[:, None] for t in cos_sin[pos.long()].double().split(R // 2, 1))
    out = y.clone()
    i = torch.arange(R // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    out[..., ia] = y[..., ia] * c - y[..., ib] * s
    out[..., ib] = y[..., ib] * c + y[..., ia] * s
    return out


def norm_rope_tol(ref, dtype):
    """fp32 arithmetic on values of at most |y|: the sum of squares (D terms, its error halved by the root), the
    root, two products, the rotation's two products and sum: under 32 roundings of 2^-24, relative to the head's
    largest value; then the rounding to dtype (and, below the normal range, half its smallest step)."""
    big = ref.abs().amax(-1, keepdim=True)
    return HALF_STEP[dtype] * ref.abs() + 64 * 2.0 ** -24 * big + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def angles(n, R, device="cpu", base=10000.0):
    inv = base ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)
    a = torch.arange(n, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float().contiguous()


def rows_of(lens, news):
    """(sequence, cache position) of each row, in order."""
    return [(b, n - m + i) for b, (n, m) in enumerate(zip(lens, news)) for i in range(m)]


def attend(k, v, table, lens, news, Q, window=0, sinks=0, prior=None):
    """64-bit O [T, H_q, D], LSE [T, H_q] and a bound on each row's error of a score and largest |v|.
    k, v [n_pages, H_kv, P, D]; keys that no row of a sequence sees never enter."""
    H_kv, P, D = k.shape[1:]
    T, H_q, _ = Q.shape
    G = H_q // H_kv
    O = torch.zeros((T, H_q, D), dtype=torch.float64, device=Q.device)
    L = torch.full((T, H_q), -math.inf, dtype=torch.float64, device=Q.device)
    ds = torch.zeros((T, H_q), dtype=torch.float64, device=Q.device)
    vm = torch.zeros((T, H_q), dtype=torch.float64, device=Q.device)
    r = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        if m == 0:
            continue
        at = torch.arange(n - m, n, device=Q.device)
        j = torch.arange(max(n, 0), device=Q.device)
        see = j[None] <= at[:, None]
        if window > 0:
            see &= (j[None] > at[:, None] - window) | (j[None] < sinks)
        used = see.any(0)
        if n > 0 and bool(used.any()):
            jj = j[used]
            pages = table[b].long()[jj // P]
            K, V = (x[pages, :, jj % P].double() for x in (k, v))       # [n', H_kv, D]
            q = Q[r:r + m].double().view(m, H_kv, G, D)
            S = torch.einsum("mhgd,nhd->hgmn", q, K) / math.sqrt(D)
            mag = torch.einsum("mhgd,nhd->hgmn", q.abs(), K.abs()) / math.sqrt(D)
            hid = ~see[:, used]
            S = S.masked_fill(hid, -math.inf)
            z = torch.logsumexp(S, -1)
            p = torch.exp(S - z[..., None].clamp(min=-1e300))
            O[r:r + m] = torch.einsum("hgmn,nhd->mhgd", p, V).reshape(m, H_q, D)
            L[r:r + m] = z.permute(2, 0, 1).reshape(m, H_q)
            # a score: D fp32 additions of products whose magnitudes sum to mag, the scaling and the maximum's
            # subtraction (half a step each of at most mag)
            ds[r:r + m] = (mag.masked_fill(hid, 0).amax(-1) * (D + 4) * 2.0 ** -23).permute(2, 0, 1).reshape(m, H_q)
            vm[r:r + m] = torch.where(hid[None, None, ..., None], 0, V.permute(1, 0, 2).abs()[:, None, None]).amax((-1, -2)) \
                .permute(2, 0, 1).expand(m, H_kv, G).reshape(m, H_q) if m * n * D * H_kv <= 1 << 26 else V.abs().max()
        r += m
    if prior is not None:
        Op, Lp = (x.double() for x in prior)
        both = torch.logaddexp(L, Lp)
        none = both == -math.inf
        a, c = torch.exp(L - both), torch.exp(Lp - both)
        a, c = a.masked_fill(none, 0), c.masked_fill(none, 0)
        O = O * a[..., None] + torch.where((Lp == -math.inf)[..., None], 0, Op * c[..., None])
        vm = torch.maximum(vm, torch.where(Lp == -math.inf, 0, Op.abs().amax(-1)))
        L = both
    return O, L, ds, vm


def check_attend(O, LSE, ref, dtype, p_err, what=""):
    """p_err: relative rounding of the softmax weights as the kernel multiplies them. Weights off by a score's error
    ds, twice (numerator and sum), by p_err, and by 2^-20 (2^x, the sums, the division) move O by that share of the
    largest |v|; O is then rounded to dtype. The LSE moves by ds, its sum's 2^-20 and fp32 rounding of its terms."""
    Or, Lr, ds, vm = ref
    rel = 2 * ds + p_err + 2.0 ** -20
    tol = HALF_STEP[dtype] * Or.abs() + (rel * vm)[..., None] + torch.finfo(dtype).smallest_normal
    assert torch.isfinite(O.float()).all(), f"{what}: O not finite"
    over = ((O.double() - Or).abs() - tol).max().item() if O.numel() else -1
    assert over <= 0, f"{what}: O off by {(O.double() - Or).abs().max().item():.3e}, {over:.3e} over its bound"
    empty = Lr == -math.inf
    assert torch.equal(LSE == -math.inf, empty), f"{what}: rows without keys"
    tl = ds + 2.0 ** -20 + 4 * 2.0 ** -24 * (Lr.abs() + 8)
    off = (LSE.double() - Lr).abs().masked_fill(empty, 0) - tl.masked_fill(empty, 0)
    assert not off.numel() or off.max().item() <= 0, f"{what}: LSE over its bound by {off.max().item():.3e}"


# relative rounding of p in the kernels: a 16-bit hi + lo pair (half a step of the lo part), or one rounding
P_SPLIT = {torch.float16: 2.0 ** -22, torch.bfloat16: 2.0 ** -17}
P_ONCE = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


class Pages:
    """Random pages and tables for sequences of the given lengths; unused slots and pages hold `fill`, unused
    table entries -1."""

    def __init__(self, seed, lens, H_kv, D, page, dtype, device="cuda", fill=float("nan"), nhd=False, extra=3, width=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(n, 0) // page) for n in lens]
        n_pages = sum(need) + extra
        shape = (n_pages, page, H_kv, D) if nhd else (n_pages, H_kv, page, D)
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
        u = (used[:, :, None, None] if nhd else used[:, None, :, None])
        mk = lambda: torch.where(u, torch.randn(shape, generator=g), torch.tensor(fill)).to(dtype).to(device)  # noqa: E731
        self.k, self.v = mk(), mk()
        if nhd:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.table = table.to(device)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)
