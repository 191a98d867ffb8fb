"""Cases of the paged tail held in 8 bits: the append that quantises, attention over the codes (one new token per sequence,
ragged prompts, windows with sinks), and rows of the cache read back.

The cache: codes k, v [n_pages, H_kv, page, D] in e4m3 and one scale per token and kv head, a power of two 2^e held as its
exponent byte e + 127. A head row y with a = max |y| has the least e with a 2^-e <= 448 (held to -126 .. 120), and its
codes are y 2^-e rounded to e4m3.

A case's "kind" says which operator it runs:
  append  Q, K, V rows of a ragged batch -> rotated Q, and the cache with the new rows in it
  attend  Q rows over the cache -> O, LSE
  read    the last rows of each sequence out of the cache -> K, V
Sequence lengths follow from the case alone (log-spread between "lo" and "hi"); page orders and values come from the seed.
"""
import math

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_EPS = 1e-6
_context = None


def _ctx():
    """The framework's context, one for the process."""
    global _context
    if _context is None:
        from prefix_cached_kv_gb300 import binding
        _context = binding.Context(0)
    return _context


# ---------------------------------------------------------------- cases

def listed():
    ap = lambda name, B, rows, lo, hi, H_q, H_kv, D, R, dtype, norm, inter, page: dict(  # noqa: E731
        name=name, kind="append", B=B, rows=rows, lo=lo, hi=hi, H_q=H_q, H_kv=H_kv, D=D, R=R, dtype=dtype,
        interleaved=inter, norm=norm, page=page)
    rd = lambda name, B, rows, lo, hi, H_kv, D, dtype, page: dict(  # noqa: E731
        name=name, kind="read", B=B, rows=rows, lo=lo, hi=hi, H_q=H_kv, H_kv=H_kv, D=D, dtype=dtype, page=page)
    at = lambda name, B, rows, lo, hi, H_q, H_kv, D, dtype, page, W, sinks, prior: dict(  # noqa: E731
        name=name, kind="attend", B=B, rows=rows, lo=lo, hi=hi, H_q=H_q, H_kv=H_kv, D=D, dtype=dtype, page=page,
        window=W, sinks=sinks, prior=prior)
    return [
        # one decode step of 64 sessions: latency
        ap("append decode step", 64, 1, 100, 8192, 32, 8, 64, 64, "fp16", False, False, 16),
        # an odd chunk of one session, projections in 32 bits, half of each head rotated, adjacent pairs
        ap("append odd chunk", 1, 1037, 1500, 1500, 24, 8, 128, 64, "fp32", True, True, 16),
        # prompts of eight sessions prefilled together, head norms on the way
        ap("append ragged prompts", 8, 4096, 300, 4096, 32, 8, 128, 128, "bf16", True, False, 32),
        # a short session taken out of the cache
        rd("read a short session", 1, 300, 300, 300, 8, 128, "fp16", 16),
        # long sessions taken out, to become resident prefixes
        rd("read long sessions", 16, 32768, 1000, 32768, 8, 128, "bf16", 64),
        # the first tokens of a chat: latency
        at("token, short cache", 1, 1, 300, 300, 32, 8, 128, "fp16", 16, 0, 0, False),
        # one long document: all SMs have to share one sequence
        at("token, one long cache", 1, 1, 131071, 131071, 32, 8, 128, "bf16", 64, 0, 0, False),
        # the decode step of 64 sessions behind a resident prefix
        at("token, ragged batch, prefix", 64, 1, 100, 16384, 32, 8, 64, "fp16", 16, 0, 0, True),
        # wide heads, few kv heads, long caches
        at("token, wide heads", 16, 1, 30000, 65536, 8, 2, 256, "bf16", 32, 0, 0, False),
        # a windowed layer's decode step
        at("token, window and sinks", 32, 1, 500, 32768, 64, 8, 128, "bf16", 16, 2048, 4, False),
        # ragged prompts through a windowed layer, three q heads per kv head
        at("prompts, window and sinks", 6, 4096, 700, 4096, 24, 8, 128, "bf16", 64, 1024, 4, False),
        # a chunk of a long prompt over what is already cached
        at("prompt chunk, long cache", 1, 4096, 16384, 16384, 32, 8, 128, "fp16", 128, 0, 0, False),
    ]


_HEADS = ((32, 8, 64), (24, 8, 128), (8, 2, 256), (8, 8, 128), (32, 8, 128), (64, 8, 128), (28, 4, 128), (16, 1, 128),
          (40, 8, 128), (12, 12, 64), (10, 2, 192))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("append", "append", "read", "attend", "attend", "attend", "attend"))
    H_q, H_kv, D = rng.choice(_HEADS)
    dtype = rng.choice(("fp16", "bf16"))
    page = rng.choice((16, 32, 48, 64, 128))
    if kind == "append":
        B = _log(rng, 1, 128)
        rows = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 4096 * 8 // B))
        lo = _log(rng, 1, max(2, 4096 * 4 // B))
        return dict(kind=kind, B=B, rows=rows, lo=lo, hi=max(lo, rows, _log(rng, 1, max(2, 4096 * 16 // B))), H_q=H_q, H_kv=H_kv, D=D,
                    R=rng.choice([r for r in (32, 64, D // 2, D) if r <= D]), dtype=rng.choice(("fp16", "bf16", "bf16", "fp32")),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.6, page=page)
    if kind == "read":
        B = _log(rng, 1, 64)
        hi = _log(rng, 16, max(32, min(131072, (1 << 27) // (B * H_kv * D))))
        return dict(kind=kind, B=B, rows=_log(rng, 1, hi), lo=_log(rng, 1, hi), hi=hi, H_q=H_kv, H_kv=H_kv, D=D, dtype=dtype, page=page)
    W, sinks = (_log(rng, 16, 4096), rng.choice((0, 1, 4, 17))) if rng.random() < 0.5 else (0, 0)
    if rng.random() < 0.65:    # one new token of each sequence
        B = _log(rng, 1, 128)
        hi = _log(rng, 16, max(32, min(131072, (1 << 29) // (B * H_kv * D))))
        return dict(kind=kind, B=B, rows=1, lo=_log(rng, 1, hi), hi=hi, H_q=H_q, H_kv=H_kv, D=D, dtype=dtype, page=page,
                    window=W, sinks=sinks, prior=rng.random() < 0.3)
    H_q, H_kv, D = rng.choice([h for h in _HEADS if h[2] <= 128])
    B = _log(rng, 1, 16)
    rows = _log(rng, 2, 2048)
    hi = max(rows, _log(rng, rows, max(rows + 1, min(32768, (1 << 29) // (B * rows * H_q)))))
    rows = max(1, min(rows, (1 << 29) // (B * H_q * hi)))
    return dict(kind=kind, B=B, rows=rows, lo=_log(rng, 1, hi), hi=hi, H_q=H_q, H_kv=H_kv, D=D, dtype=dtype, page=page,
                window=W, sinks=sinks, prior=rng.random() < 0.3)


def _lengths(c):
    """Cache lengths and rows of each sequence: the last one is as long as any, the others spread in the logarithm."""
    B, lo, hi = c["B"], min(c["lo"], c["hi"]), c["hi"]
    lens = [max(1, int(round(lo * (hi / lo) ** ((b + 1) * 0.6180339887498949 % 1.0)))) for b in range(B - 1)] + [hi]
    return lens, [min(n, c["rows"]) for n in lens]


def _visible(c, p):
    """Keys that a row at position p sees."""
    if c["window"] <= 0:
        return p + 1
    first = max(0, p + 1 - c["window"])
    return p + 1 - first + min(first, c["sinks"])


def work(c):
    H_q, H_kv, D = c["H_q"], c["H_kv"], c["D"]
    size = 4 if c["dtype"] == "fp32" else 2
    lens, news = _lengths(c)
    T = sum(news)
    if c["kind"] == "append":
        return {"bytes": T * ((2 * H_q + 2 * H_kv) * D * size + 2 * H_kv * (D + 1) + c["R"] * 4 + 4) + 8 * c["B"],
                "flops": T * ((H_q + H_kv) * (3 * c["R"] + (4 * D if c["norm"] else 0)) + 2 * H_kv * 2 * D)}
    if c["kind"] == "read":
        return {"bytes": T * 2 * H_kv * (D + 1 + D * size) + T // c["page"] * 4 + 8 * c["B"], "flops": T * 2 * H_kv * D}
    keys = pairs = 0
    for n, m in zip(lens, news):
        first = _visible(c, n - m)       # the first row's keys, and for each later row at most one more that is new
        keys += min(n, first + m - 1)
        if c["window"] <= 0:
            pairs += m * (2 * n - m + 1) // 2
        else:
            pairs += sum(_visible(c, p) for p in range(n - m, n))
    b = keys * H_kv * 2 * (D + 1) + 2 * T * H_q * D * size + T * H_q * 4 + sum(-(-n // c["page"]) for n in lens) * 4
    return {"bytes": b + (T * H_q * (D + 1) * 4 if c["prior"] else 0), "flops": 4 * pairs * H_q * D}


# ---------------------------------------------------------------- the format, in plain torch

def _quantize(y):
    """fp32 rows [..., D] -> codes (e4m3) and exponent bytes [...]."""
    a = y.abs().masked_fill(~torch.isfinite(y), 0).amax(-1)
    m, e = torch.frexp(a)                        # a = m 2^e with m in [1/2, 1), and 448 = 7/8 2^9
    e = torch.where(a > 0, e - 9 + (m > 0.875).to(torch.int32), -126).clamp(-126, 120)
    down = ((127 - e) << 23).view(torch.float32)                    # 2^-e
    return (y * down[..., None]).to(_E4M3), (e + 127).to(torch.uint8)


def _scale(byte):
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _take(x, *at):
    """x[at] of an 8-bit tensor, as fp32 values (codes) or scales (exponent bytes)."""
    y = x.view(torch.uint8)[at]
    return y.view(_E4M3).float() if x.dtype == _E4M3 else _scale(y)


# ---------------------------------------------------------------- inputs

def _angles(n, R, dev):
    """The rotary table of n positions: R/2 cosines and R/2 sines a row, fp32 (angles in 64 bits)."""
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[c["dtype"]]
    H_q, H_kv, D = c["H_q"], c["H_kv"], c["D"]

    def rand(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale

    s = dict(c=c)
    lens, news = _lengths(c)
    P, T = c["page"], sum(news)
    width = -(-max(lens) // P)
    need = [-(-n // P) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    row = torch.tensor(need, device=dev)
    cols = torch.arange(width, device=dev)[None]
    at = (row.cumsum(0) - row)[:, None] + cols
    tab = torch.where(cols < row[:, None], order[at.clamp(max=n_pages - 1)], torch.zeros((), dtype=torch.int32, device=dev))
    cu = [0]
    for m in news:
        cu.append(cu[-1] + m)
    channels = torch.exp(rand(H_kv, 1, D, scale=0.5))      # keys have channels that stand out
    k, ks = _quantize(rand(n_pages, H_kv, P, D) * channels)
    v, vs = _quantize(rand(n_pages, H_kv, P, D))
    s.update(k=k, v=v, ks=ks.view(_E8M0), vs=vs.view(_E8M0), tab=tab.contiguous(), T=T, max_rows=max(news),
             len=torch.tensor(lens, dtype=torch.int32, device=dev), cu=torch.tensor(cu, dtype=torch.int32, device=dev))
    if c["kind"] == "append":
        qkv = rand(T, H_q + 2 * H_kv, D).to(dt)            # the projection's output: q, k and v side by side
        weights = [(1 + rand(D, scale=0.1)).to(dt) if c["norm"] else None for _ in range(2)]
        s.update(Q=qkv[:, :H_q], K=qkv[:, H_q:H_q + H_kv], V=qkv[:, H_q + H_kv:], table=_angles(max(lens), c["R"], dev),
                 wq=weights[0], wk=weights[1])
    elif c["kind"] == "attend":
        s.update(Q=rand(T, H_q, D).to(dt), prior=None)
        if c["prior"]:
            s["prior"] = (rand(T, H_q, D, scale=0.1), rand(T, H_q) + math.log(4000.0))
    if own:   # the cache object that a user's program makes once, beside its pages
        from prefix_cached_kv_gb300 import binding
        s["cache"] = binding.QuantizedPagedCache(s["k"], s["v"], s["ks"], s["vs"])
    return s


# ---------------------------------------------------------------- plain forms

def _norm_rope(x, w, pos, table, R, inter):
    """fp32 rows [T, H, D]: RMS norm with weight w (None: none), then the rotation of the first R elements."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w.float()
    cs = table[pos.long()][:, None]
    co, si = cs[..., :R // 2], cs[..., R // 2:]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    ra, rb = a * co - b * si, b * co + a * si
    rot = torch.stack((ra, rb), -1).flatten(-2) if inter else torch.cat((ra, rb), -1)
    return torch.cat((rot, x[..., R:]), -1)


def _rows_of(s, T):
    """Sequence and cache position of each row."""
    r = torch.arange(T, device=s["cu"].device)
    b = torch.searchsorted(s["cu"].long(), r, right=True) - 1
    return b, s["len"].long()[b] - (s["cu"].long()[b + 1] - r)


def _plain(s):
    c = s["c"]
    dt = _DT[c["dtype"]]
    H_q, H_kv, D = c["H_q"], c["H_kv"], c["D"]
    P, T = c["page"], s["T"]
    seq, p = _rows_of(s, T)
    page, slot = s["tab"][seq, p // P].long(), p % P
    if c["kind"] == "append":
        y = _norm_rope(s["K"], s["wk"], p, s["table"], c["R"], c["interleaved"])
        for x, codes, scale in ((y, s["k"], s["ks"]), (s["V"].float(), s["v"], s["vs"])):
            q, e = _quantize(x)
            codes.view(torch.uint8)[page, :, slot] = q.view(torch.uint8)
            scale.view(torch.uint8)[page, :, slot] = e
        return _norm_rope(s["Q"], s["wq"], p, s["table"], c["R"], c["interleaved"]).to(dt), s["k"], s["v"], s["ks"], s["vs"]
    if c["kind"] == "read":
        heads = slice(None)
        return tuple((_take(x, page, heads, slot) * _take(e, page, heads, slot)[..., None]).to(dt)
                     for x, e in ((s["k"], s["ks"]), (s["v"], s["vs"])))
    G, M = H_q // H_kv, s["max_rows"]
    B, L = s["tab"].shape[0], s["tab"].shape[1] * P
    j = torch.arange(L, device=p.device)
    tab = s["tab"].long()
    K, V = ((_take(x, tab) * _take(e, tab)[..., None]).transpose(1, 2).reshape(B, H_kv, L, D)
            for x, e in ((s["k"], s["ks"]), (s["v"], s["vs"])))
    i = torch.arange(T, device=p.device) - s["cu"].long()[seq]
    Q = torch.zeros((B, M, H_kv, G, D), device=p.device)
    Q[seq, i] = s["Q"].float().view(T, H_kv, G, D)
    pos = torch.full((B, M), -1, device=p.device)
    pos[seq, i] = p
    S = torch.matmul(Q.permute(0, 2, 3, 1, 4).reshape(B, H_kv, G * M, D), K.transpose(-1, -2)).view(B, H_kv, G, M, L)
    S *= D ** -0.5
    seen = j <= pos[..., None]
    if c["window"] > 0:
        seen &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    S.masked_fill_(~seen[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True).clamp(min=-1e30)
    S.sub_(m).exp_()
    l = S.sum(-1, keepdim=True)
    O = torch.matmul(S.view(B, H_kv, G * M, L), V).view(B, H_kv, G, M, D) / l.clamp(min=1e-30)
    O = O.permute(0, 3, 1, 2, 4)[seq, i].reshape(T, H_q, D)
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2)[seq, i].reshape(T, H_q)
    if s["prior"] is not None:
        Op, Lp = s["prior"]
        both = torch.logaddexp(lse, Lp)
        O = O * (lse - both).exp()[..., None] + Op * (Lp - both).exp()[..., None]
        lse = both
    return O.to(dt), lse


def run(s):
    if not own:
        return _plain(s)
    c, ctx = s["c"], _ctx()
    cu = s["cu"] if s["max_rows"] > 1 else None
    if c["kind"] == "append":
        Q = ctx.paged_append(s["cache"], s["tab"], s["len"], s["K"], s["V"], Q=s["Q"], cu_rows=cu, cos_sin=s["table"],
                             q_weight=s["wq"], k_weight=s["wk"], eps=_EPS, interleaved=c["interleaved"])
        return Q, s["k"], s["v"], s["ks"], s["vs"]
    if c["kind"] == "read":
        return ctx.paged_read(s["cache"], s["tab"], s["len"], T=s["T"], cu_rows=cu, dtype=_DT[c["dtype"]])
    return ctx.paged_attend(s["cache"], s["tab"], s["len"], s["Q"], cu_rows=cu, max_rows=s["max_rows"],
                            window=c["window"], sinks=c["sinks"], prior=s["prior"])


# ---------------------------------------------------------------- 64 bits, from the definitions

def _exact_rotated(x, w, at, table, R, inter):
    """Tokens' heads [m, H, D] (64 bits) at positions `at`: norm, then each pair as a complex number times c + i s."""
    x = x.double()
    if w is not None:
        x = x / ((x.square().sum(-1, keepdim=True) / x.shape[-1]) + _EPS).sqrt() * w.double()
    turn = torch.complex(table[at, :R // 2].double(), table[at, R // 2:].double())[..., None, :]
    y = x.clone()
    pairs = x[..., :R].unflatten(-1, (R // 2, 2)) if inter else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y[..., :R] = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
    return y


def _exact_codes(y):
    """Head rows over their scale: what the codes round (64 bits)."""
    e = torch.ceil(torch.log2(y.abs().amax(-1, keepdim=True) / 448)).clamp(-126, 120)
    return y * torch.exp2(-e)


def _exact_values(codes, scale):
    return codes.double() * torch.exp2(scale.view(torch.uint8).double() - 127)[..., None]


def exact(c, seed):
    """Codes are compared with the values that they round; a scale is a step of its row's maximum and has no such value."""
    s = prepare(c, seed)
    P = c["page"]
    lens, news = _lengths(c)
    H_q, H_kv, D = c["H_q"], c["H_kv"], c["D"]
    G = H_q // H_kv
    if c["kind"] == "append":
        Qo, k, v, r = [], s["k"].double(), s["v"].double(), 0
        for b, (n, m) in enumerate(zip(lens, news)):
            at = torch.arange(n - m, n, device=k.device)
            page = s["tab"][b].long()[torch.div(at, P, rounding_mode="floor")]
            k[page, :, at % P] = _exact_codes(_exact_rotated(s["K"][r:r + m], s["wk"], at, s["table"], c["R"], c["interleaved"]))
            v[page, :, at % P] = _exact_codes(s["V"][r:r + m].double())
            Qo.append(_exact_rotated(s["Q"][r:r + m], s["wq"], at, s["table"], c["R"], c["interleaved"]))
            r += m
        return torch.cat(Qo), k, v, None, None
    if c["kind"] == "read":
        out = [], []
        for b, (n, m) in enumerate(zip(lens, news)):
            pages = s["tab"][b, (n - m) // P:-(-n // P)].long()
            first = (n - m) % P
            for o, x, e in ((out[0], s["k"], s["ks"]), (out[1], s["v"], s["vs"])):
                y = _exact_values(x.view(torch.uint8)[pages].view(_E4M3), e.view(torch.uint8)[pages])
                o.append(y.transpose(1, 2).reshape(-1, H_kv, D)[first:first + m])
        return tuple(torch.cat(o) for o in out)
    T = sum(news)
    O = torch.zeros((T, H_q, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H_q), -math.inf, dtype=torch.float64, device="cuda")
    r = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        pages = s["tab"][b, :-(-n // P)].long()
        at = torch.arange(n - m, n, device="cuda")
        j = torch.arange(n, device="cuda")
        hidden = j[None] > at[:, None]
        if c["window"] > 0:
            hidden |= (j[None] <= at[:, None] - c["window"]) & (j[None] >= c["sinks"])
        for h in range(H_kv):
            k, v = (_exact_values(x.view(torch.uint8)[pages, h].view(_E4M3), e.view(torch.uint8)[pages, h]).reshape(-1, D)[:n]
                    for x, e in ((s["k"], s["ks"]), (s["v"], s["vs"])))
            step = max(1, (1 << 28) // (m * n))
            for g0 in range(0, G, step):   # q heads at once: 2 GB of scores at most
                heads = slice(h * G + g0, h * G + min(G, g0 + step))
                x = torch.einsum("mgd,nd->gmn", s["Q"][r:r + m, heads].double(), k) / math.sqrt(D)
                x.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[r:r + m, heads] = z.T
                O[r:r + m, heads] = torch.einsum("gmn,nd->mgd", (x - z[..., None]).exp_(), v)
        r += m
    if s["prior"] is not None:
        Op, Lp = (x.double() for x in s["prior"])
        w = torch.sigmoid(Lp - lse)[..., None]      # the prior's share
        O = O * (1 - w) + Op * w
        lse = torch.logsumexp(torch.stack((lse, Lp)), 0)
    return O, lse
