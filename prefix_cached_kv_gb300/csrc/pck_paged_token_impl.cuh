// pck_paged_token_impl.cuh -- attention of one new token (or a few) per sequence over a paged KV cache, split
// over the cache's length and joined.
//
// Per sequence b (n = kv_len[b] keys, the new token's own among them) and q head h of kv head g:
//   s_j = tau q_h . k_j,  O = sum_j 2^(s_j' - m) v_j / l,  LSE = (m + log2 l) ln 2   (s' = s log2 e)
// over the visible keys: all n, or with a window W the last W and the first `sinks`.
//
// Every K and V byte is read once and used for G = H_q / H_kv heads (above 16 of them, 8 at D > 128, once for each 16
// or 8: they are items of their own): 4 G flop per 4 bytes, so HBM bounds it and the kernel's business is to keep loads
// in flight on every SM whatever the lengths:
//  * A unit is a cache tile of 16 tokens of one kv head (a page is a multiple of 16, so a unit never
//    leaves its page). The units of all items (sequence, kv head, group of q heads) laid end to end
//    are cut into equal ranges from the lengths on the device (one block scan per CTA), so a ragged
//    batch, one long sequence and many short ones all load every SM evenly, and a captured graph
//    follows the lengths it finds. A range is a CTA's, whose warps take every NW-th unit and join through
//    shared memory: neighbouring warps then read neighbouring tiles, and an item has few pieces. With more
//    items than SMs the CTAs have half the warps, two to an SM, so that a change of item (its q, its end) stalls
//    half of the SM's streams; with many more a range is a warp's, and it stalls one of them. Items of nearly
//    one length (a batch behind one window, say) stay whole where they fill the CTAs: 32 windows of 2048 tokens
//    46.3 us against 49.2, 24 x 4000 tokens 65 against 72, 16 x 32,000 314 against 319 (8 kv heads of 128).
//  * One or two CTAs per SM; each warp streams its units through a ring of its own (two TMA tile loads a unit,
//    128-byte swizzle, evict-first). Lane i of a warp resolves the i-th of its next 32 units
//    (sequence, tile, page number) at once, so page-table latency is paid once in 32 units and off the
//    critical path; rings run on across items.
//  * S^T = K q^T with the 16 tokens as MMA rows and up to 8 (16) q heads, or rows x q heads, as columns. m stands TOP
//    (log2) below the running maximum and moves only when a score passes m by CAP, so every p <= 2^CAP; p goes into
//    O^T += V^T p^T as a 16-bit hi + lo pair (two MMAs into one accumulator), which keeps 22 bits of p (fp16, of a p
//    above 2^-15 of the largest one; below that it is held to 2^-37 of the largest) or 16 (bf16, of any p): the
//    result's own rounding is then the only visible one, and these MMAs are hidden behind the loads.
//  * An item that lies within one range is finished there; one that crosses ranges leaves a partial [m, l, O]
//    per range, at most two per range, and a second, programmatically launched kernel joins them.
//  * When no sequence can have more than TK_DIRECT_UNITS units and the items are not many, each item gets a CTA
//    whose warps take its units in turn and join through shared memory: one launch. With more items than SMs
//    these CTAs too have half the warps (24 sequences of 100 tokens, 8 kv heads: 6.9 us against 11.0; 64 of 500
//    tokens 27.9 against 36.3).
// Measured: one cache of 131,071 tokens (8 kv heads of 128, 4 q heads each) 88 us, 6.1 TB/s; 16 caches of 30-65k tokens
// (2 kv heads of 256) 232 us, 6.5 TB/s; 64 ragged sequences (8 kv heads of 64) 83.5 us, 5.5 TB/s; 32 windows of 2048
// tokens (8 kv heads of 128, 8 q heads each) 46 us, 5.0 TB/s.
#pragma once

#include "pck_paged.cuh"

namespace pck {
namespace {

// Units of an item up to which it gets a CTA (1024 tokens): one sequence of 300 tokens 7.1 us against 10.0 cut into
// ranges, of 1000 tokens 10.8 against 10.4, of 2000 tokens 15.3 against 10.2 (8 kv heads of 128). Items of equal length
// gain up to 4000 tokens (24 x 2000: 35.6 against 41.2), but ragged ones lose twice that (24 x 1-2000: 26.1 against 17.2).
constexpr int TK_DIRECT_UNITS = 64;
// Items per SM above which a range is a warp's. 64 ragged sequences (3.4 per SM) 83 us with a range per half CTA, 86 with
// one per warp, 101 with one per whole CTA; 200 x 1-1000 tokens (10.5) 45 against 43, 600 x 100 (32) 85 against 58. Items
// that could have a CTA each: 100 x 500 tokens (5.3) 41 us with one, 52 with a range per warp; 200 x 1-1000 47 against 43.
constexpr int TK_FEW_ITEMS = 6;
// How a call is cut: an item per CTA, per CTA of half the warps; a range per CTA, per CTA of half the warps, per warp.
// At one item per SM or less, CTAs are whole: one cache of 131k tokens 87 us (halves 89), 16 caches of 30-65k 230 (234).
enum { TK_ITEM, TK_ITEM_HALF, TK_CTA, TK_CTA_HALF, TK_WARP };
__host__ __device__ constexpr bool is_split(int mode) { return mode >= TK_CTA; }
__host__ __device__ constexpr int per_sm(int mode) { return mode == TK_ITEM_HALF || mode == TK_CTA_HALF ? 2 : 1; }   // CTAs
// Warps per SM. At D = 64 a unit is 4 KB and its warp's chain of MMAs bounds it: where an item or a range is short, 16
// warps with 3 stages each beat 8 with 6 (600 x 1-1000 tokens 58 us against 78, 64 of them 16 against 20, one sequence of
// 1000 tokens 8.6 against 9.9), but a CTA's long ranges then have more to join (64 ragged sequences 91 against 83).
__host__ __device__ constexpr int warps_sm(int D, int mode) {
    return D > 128 ? 4 : D == 64 && mode != TK_CTA && mode != TK_CTA_HALF ? 16 : 8;
}
// Units per range at least (one per warp, or what a warp's start is worth): 2000 tokens 10.2 us, with twice as many
// 10.5, with four times 11.9.
__host__ __device__ constexpr int tk_min_units(int mode) { return mode == TK_WARP ? 4 : 8; }
// What an item costs beside its units (its q, its end), in units: ranges are cut by units + this per item, so that a
// range of many short items does not take long after the others (64 ragged sequences, ranges per CTA: 132 us with 0, 122
// with 8, 101 with 24; ranges per warp: 122 with 4, 101 with 8, 85 with 16, 87 with 32).
__host__ __device__ constexpr int tk_item_units(int mode) { return mode == TK_WARP ? 16 : 24; }
constexpr int TK_MAX_B = PCK_PAGED_MAX_BATCH;

template <int D, int MODE>
struct TCfg {
    static constexpr int NW = warps_sm(D, MODE) / per_sm(MODE);   // warps per CTA
    static constexpr int UNIT = PG_SUB * D * 2;                   // bytes of a K (or V) unit
    static constexpr int STAGE = 2 * UNIT;
    static constexpr int ST = D <= 64 ? 48 / warps_sm(D, MODE) : D == 192 ? 4 : 3;      // stages of a warp's ring
    static constexpr int RING = NW * ST * STAGE;
    static constexpr int JROW = D / 2 + 4;                        // floats of a join row (half of D, padded)
    static constexpr int JOIN = NW * 8 * JROW * 4;
    static constexpr int OFF_JOIN = RING;
    static constexpr int OFF_ML = OFF_JOIN + JOIN;                // [NW][16] m, then l
    static constexpr int OFF_BAR = OFF_ML + NW * 16 * 2 * 4;
    static constexpr int OFF_SCAN = OFF_BAR + NW * ST * 8 + 8;
    static constexpr int OFF_PRE = OFF_SCAN + 64 * 4;             // prefix of units per sequence [B + 1]
    static constexpr int SMEM_BASE = OFF_PRE + 1024;              // + alignment slack; + 4 (B + 1)
};

template <typename T> struct Elem;
template <> struct Elem<__half> {
    // fp16 has no step below 2^-24, so p = 2^-20 would have five bits and 2^-26 none, however many keys have it: the
    // maximum stands at 2^12 when it moves and may rise to 2^15.9 (65,504 is the largest value). A weight is then
    // within 2^-37 of the largest one. At 2^0, 40,000 equal keys behind one 24 to 26 (log2) above them moved O by 3e-4 of
    // the largest |v|. Costs nothing: one cache of 131k tokens 87.8 us as with 2^0, the ragged batch 83.5 against 83.0
    // (2^7 83.6, 2^14 84.0).
    static constexpr float TOP = 12.f, CAP = 15.9f;
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        mma16816(c, a, b0, b1);
    }
    static __device__ __forceinline__ void split(float x0, float x1, uint32_t& hi, uint32_t& lo) { split_hi_lo(x0, x1, hi, lo); }
    static __device__ __forceinline__ uint32_t pack(float x0, float x1) { return h2_as_u32(__floats2half2_rn(x0, x1)); }
    static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
    static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
    // x * 0 is NaN where x is infinite or NaN
    static __device__ __forceinline__ bool not_finite8(uint4 x) {
        const __half2 z = __float2half2_rn(0.f);
        const __half2 a = __hfma2(u32_as_h2(x.x), z, __hmul2(u32_as_h2(x.y), z)), b = __hfma2(u32_as_h2(x.z), z, __hmul2(u32_as_h2(x.w), z));
        return (h2_as_u32(__hadd2(a, b)) & 0x7fff7fffu) != 0;
    }
};
template <> struct Elem<__nv_bfloat16> {
    static constexpr float TOP = 0.f, CAP = 8.f;      // p keeps its bits at any size
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float x0, float x1) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ bool not_finite8(uint4 x) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
        return bad;
    }
    static __device__ __forceinline__ void split(float x0, float x1, uint32_t& hi, uint32_t& lo) {
        hi = pack(x0, x1);
        lo = pack(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u));
    }
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap* tm, int tok, int head, int page, uint32_t bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;"
        ::"r"(dst), "l"(tm), "r"(0), "r"(tok), "r"(0), "r"(head), "r"(page), "r"(bar), "l"(pol) : "memory");
}

// The units (cache tiles of SUB tokens) that one sequence's rows read: tiles [0, ns) hold the sinks, then come tiles
// [w0, w0 + n - ns). `rows` of len tokens: the first row sees len - rows + 1 keys. A sequence without keys (or rows)
// has one unit with nothing visible.
struct Span {
    int n, ns, w0;
};
template <int SUB = PG_SUB>
__device__ __forceinline__ Span span_of(int len, int rows, int window, int sinks) {
    Span s;
    const int end = rows > 0 ? (len + SUB - 1) / SUB : 0, first = len - rows + 1;
    s.ns = 0;
    s.w0 = 0;
    if (window > 0 && rows > 0 && first > window) {
        s.w0 = (first - window) / SUB;
        s.ns = min((min(sinks, len) + SUB - 1) / SUB, s.w0);
    }
    s.n = max(1, s.ns + end - s.w0);
    return s;
}

// Sequence b's rows: the first one's index and their number (at most max_rows; none where cu_rows makes no sense).
struct RowSpan {
    int r0, n;
};
template <bool ROWS>
__device__ __forceinline__ RowSpan rows_of(const PagedAttn& P, int b, bool report) {
    if (!ROWS) return RowSpan{b, 1};
    const int r0 = P.cu_rows[b], r1 = P.cu_rows[b + 1];
    const bool ok = rows_sound(r0, r1, P.T);
    if (report && !(ok && r1 - r0 <= P.max_rows)) set_err(P.err, ERR_KV_LEN);
    return RowSpan{r0, ok ? min(r1 - r0, P.max_rows) : 0};
}

__device__ __forceinline__ int clamp_len(const PagedAttn& P, int b, bool report) {
    int len = P.kv_len[b];
    const int64_t most = (int64_t)P.max_pages * P.page;
    if (len > most) {
        if (report) set_err(P.err, ERR_KV_LEN);
        len = static_cast<int>(most);
    }
    return max(len, 0);
}

// Weight of a part with maximum m in a join at M. A part without a visible key has m = -inf and sums of 0 (or
// NaN, from a NaN score), which weight 1 passes on.
__device__ __forceinline__ float join_weight(float m, float M) { return m > -INFINITY ? ex2_approx(m - M) : 1.f; }

// Weights of a row's own attention and of the prior in the result, and the LSE of both.
struct RowEnd {
    float wo, wp, lse;
    bool prior;
};
__device__ __forceinline__ RowEnd row_end(const PagedAttn& P, int64_t row, float m, float l) {
    RowEnd r;
    const bool none = l == 0.f;
    r.wo = none ? 0.f : 1.0f / l;
    r.wp = 0.f;
    r.lse = none ? -INFINITY : (m + log2f(l)) * PG_LN2;
    r.prior = false;
    if (P.O_prior) {
        const float lp = P.LSE_prior[row];
        if (lp != -INFINITY) {
            const float mx = fmaxf(r.lse, lp);
            const float wn = expf(r.lse - mx), wp = expf(lp - mx), sum = wn + wp;
            r.wo *= wn / sum;
            r.wp = wp / sum;
            r.lse = mx + logf(sum);
            r.prior = true;
        }
    }
    return r;
}

// Elements d, d + 1 of a row of O (token x H_q + head), and (first) its LSE.
template <typename T>
__device__ __forceinline__ void finish2(const PagedAttn& P, int64_t row, int D, int d, float a0, float a1, float m, float l,
                                        bool first) {
    const RowEnd r = row_end(P, row, m, l);
    a0 *= r.wo;
    a1 *= r.wo;
    if (r.prior) {
        const float2 op = *reinterpret_cast<const float2*>(P.O_prior + row * D + d);
        a0 = fmaf(op.x, r.wp, a0);
        a1 = fmaf(op.y, r.wp, a1);
    }
    *reinterpret_cast<uint32_t*>(static_cast<T*>(P.O) + row * D + d) = Elem<T>::pack(a0, a1);
    if (first && P.LSE) P.LSE[row] = r.lse;
}

// Partial of a range (two slots per range): [heads][D + 4] floats: m, l, -, -, O (not normalised).
__host__ __device__ constexpr int slot_floats(int D, int heads) { return heads * (D + 4); }

// A split item's descriptor, written by the range in which it begins (pieces = 0: none).
struct JoinDesc {
    int r0, x, pieces, rows;
};

// a / b for a >= 0, b > 0: most quotients here need no 64-bit division, which takes some 100 instructions one after another.
__device__ __forceinline__ int64_t div_pos(int64_t a, int b) {
    return (a >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// The range of a worker (a warp of a TK_WARP call, else the CTA) among the units of all items laid end to end: [u0, u1). pre
// gets the units before each sequence (of the CTA's one sequence when nothing is split). idle: more workers than ranges.
struct Cut {
    int64_t u0, u1, U;       // U: the items' whole weight
    int workers, b_first;
    bool idle;
};
template <int NW, int MODE, bool ROWS, int SUB, int TK_ITEM_UNITS>
__device__ __forceinline__ Cut cut_units(const PagedAttn& P, int worker, int workers, int* s_scan, int* pre) {
    constexpr int NT = NW * 32, TK_MIN_UNITS = tk_min_units(MODE);
    constexpr bool SPLIT = is_split(MODE), BY_WARP = MODE == TK_WARP;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hg = P.H_kv * P.n_groups, B = P.B;
    Cut c;
    c.U = 0;
    c.b_first = 0;
    c.workers = workers;
    c.idle = false;
    if (SPLIT) {
        // units before each sequence (per kv head and group): a scan over the lengths
        const int per = (B + NT - 1) / NT;
        int sum = 0, top = 0, n = 0;          // (one sequence a thread, most often: its n is not looked up again)
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < B) {
                n = span_of<SUB>(clamp_len(P, b, blockIdx.x == 0), rows_of<ROWS>(P, b, blockIdx.x == 0).n, P.window, P.sinks).n;
                sum += n;
                top = max(top, n);
            }
        }
        if (!BY_WARP) top = __reduce_max_sync(0xffffffffu, top);
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) {
            s_scan[warp] = inc;
            s_scan[32 + warp] = top;
        }
        __syncthreads();
        int base = 0;
        for (int w = 0; w < warp; ++w) base += s_scan[w];
        int run = base + inc - sum;
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < B) {
                pre[b] = run;
                run += per == 1 ? n : span_of<SUB>(clamp_len(P, b, false), rows_of<ROWS>(P, b, false).n, P.window, P.sinks).n;
            }
        }
        if (tid == NT - 1) pre[B] = run;      // the last thread's sum is the total (later b's are empty)
        __syncthreads();
        c.U = ((int64_t)pre[B] + (int64_t)TK_ITEM_UNITS * B) * Hg;      // the items' whole weight
        const int64_t most = div_pos(c.U + TK_MIN_UNITS - 1, TK_MIN_UNITS);
        if (most < workers) workers = static_cast<int>(most);
        c.workers = workers;
        c.idle = worker >= workers;
        if (c.idle) return c;
        // the unit at which weight w falls; weights behind an item's units fall on its end
        auto unit_at = [&](int64_t w) -> int64_t {
            const int v = static_cast<int>(div_pos(w, Hg));
            int lo = 0, hi = B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pre[mid] + TK_ITEM_UNITS * mid <= v) lo = mid;
                else hi = mid - 1;
            }
            const int n = pre[lo + 1] - pre[lo], nw = n + TK_ITEM_UNITS;
            const int64_t rem = w - ((int64_t)pre[lo] + (int64_t)TK_ITEM_UNITS * lo) * Hg;
            const int64_t x = div_pos(rem, nw);
            return (int64_t)pre[lo] * Hg + x * n + min((int64_t)n, rem - x * nw);
        };
        // Items of nearly one length (the longest at most 6/5 of the mean) that fill the ranges, or the last round of
        // them, to a half (three quarters where an SM has one) stay whole: nothing is left to join.
        bool even = false;
        const int64_t items = (int64_t)B * Hg;
        if (!BY_WARP) {
            for (int w = 0; w < NW; ++w) top = max(top, s_scan[32 + w]);
            const int64_t left = items - div_pos(items, workers) * workers;
            even = (int64_t)5 * top * B <= (int64_t)6 * pre[B]
                   && (items < workers ? items * 4 >= workers * (MODE == TK_CTA ? 3 : 2) : left == 0 || left * 2 >= workers);
        }
        auto unit_of = [&](int64_t item) -> int64_t {
            const int b = static_cast<int>(div_pos(item, Hg));
            return b < B ? (int64_t)pre[b] * Hg + (item - (int64_t)b * Hg) * (pre[b + 1] - pre[b]) : (int64_t)pre[B] * Hg;
        };
        // both ends at once: even lanes the first, odd lanes the last
        const int at = worker + (lane & 1);
        const int64_t end = even ? unit_of(div_pos(items * at, workers))
                            : at < workers ? unit_at(div_pos(c.U * at, workers)) : (int64_t)pre[B] * Hg;
        c.u0 = __shfl_sync(0xffffffffu, end, 0);
        c.u1 = __shfl_sync(0xffffffffu, end, 1);
    } else {
        c.b_first = blockIdx.x / Hg;
        const int n = span_of<SUB>(clamp_len(P, c.b_first, true), rows_of<ROWS>(P, c.b_first, true).n, P.window, P.sinks).n;
        if (tid == 0) {
            pre[0] = 0;
            pre[1] = n;
        }
        __syncthreads();
        c.u0 = (int64_t)(blockIdx.x - c.b_first * Hg) * n;
        c.u1 = c.u0 + n;
    }
    return c;
}

// ROWS: a sequence may have several rows (cu_rows); else it has one.
template <typename T, int D, int NB, int MODE, bool ROWS>
__global__ void __launch_bounds__(TCfg<D, MODE>::NW * 32, per_sm(MODE)) paged_token_kernel(const __grid_constant__ PagedAttn P) {
    using C = TCfg<D, MODE>;
    constexpr int NW = C::NW, ST = C::ST, KS = D / 16, NT = NW * 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_base = smem_u32(smem);
    float* jbuf = reinterpret_cast<float*>(smem + C::OFF_JOIN);
    float* s_m = reinterpret_cast<float*>(smem + C::OFF_ML);
    float* s_l = s_m + NW * 16;
    int* s_scan = reinterpret_cast<int*>(smem + C::OFF_SCAN);
    int* pre = reinterpret_cast<int*>(smem + C::OFF_PRE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = s_base + warp * ST * C::STAGE;
    const uint32_t bar = s_base + C::OFF_BAR + warp * ST * 8;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(bar + 8 * i, 1);
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.tm_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.tm_v) : "memory");
    }
    pdl_wait();
    pdl_release();
    fence_proxy_async_all();     // the pages may have been written by the kernel before, and are read by TMA

    // ---- the range of units of this warp (BY_WARP) or CTA
    const int Hg = P.H_kv * P.n_groups;
    const int B = P.B;
    const int heads = P.heads_per_group, cols = P.cols;
    constexpr bool SPLIT = is_split(MODE), BY_WARP = MODE == TK_WARP;
    constexpr int TK_ITEM_UNITS = tk_item_units(MODE);
    const int worker = BY_WARP ? warp * gridDim.x + blockIdx.x : blockIdx.x;    // few workers spread over the SMs
    int workers = BY_WARP ? gridDim.x * NW : gridDim.x;
    JoinDesc* jd = reinterpret_cast<JoinDesc*>(P.ws + (size_t)2 * workers * slot_floats(D, cols));
    const Cut cut = cut_units<NW, MODE, ROWS, PG_SUB, tk_item_units(MODE)>(P, worker, workers, s_scan, pre);
    if (SPLIT && cut.idle) {
        if (BY_WARP ? lane == 0 : tid == 0) jd[worker].pieces = 0;
        return;
    }
    const int64_t u0 = cut.u0, u1 = cut.u1, U = cut.U;
    workers = cut.workers;
    const int b_first = cut.b_first;
    const int nseq = SPLIT ? B : 1;     // sequences in pre[]

    // ---- a warp's units: u0 + k of its own range, u0 + warp + k NW of its CTA's. Lane i resolves unit k0 + i: coordinates of its
    // loads.
    const int64_t uf = BY_WARP ? u0 : u0 + warp;
    constexpr int STEP = BY_WARP ? 1 : NW;
    const uint64_t pol = l2_evict_first();
    int pl_tok = 0, pl_head = 0, pl_page = 0;
    auto resolve = [&](int k0) {
        const int64_t u = uf + (int64_t)(k0 + lane) * STEP;
        if (u < u1) {
            const int v = static_cast<int>(u / Hg);
            int lo = 0, hi = nseq - 1;      // the sequence with pre[b] <= v < pre[b + 1]
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pre[mid] <= v) lo = mid;
                else hi = mid - 1;
            }
            const int b = b_first + lo;
            const int n = pre[lo + 1] - pre[lo];
            const int64_t rem = u - (int64_t)pre[lo] * Hg;
            const int x = static_cast<int>(rem / n), j = static_cast<int>(rem - (int64_t)x * n);
            const int len = clamp_len(P, b, false);
            const int rows = rows_of<ROWS>(P, b, false).n;
            const Span s = span_of(len, rows, P.window, P.sinks);
            const int tile = j < s.ns ? j : j - s.ns + s.w0;
            const int tok = tile * PG_SUB;
            const int pi = tok / P.page;
            pl_tok = tok - pi * P.page;
            pl_head = x / P.n_groups;
            pl_page = 0;
            if (len > 0 && rows > 0 && pi < P.max_pages) {
                const int pg = P.table[(int64_t)b * P.max_pages + pi];
                if (pg < 0 || pg >= P.n_pages) set_err(P.err, ERR_PAGE_ID);   // and page 0 is read instead
                else pl_page = pg;
            }
        }
    };
    const int nk = static_cast<int>(u1 > uf ? (u1 - uf + STEP - 1) / STEP : 0);   // units of this warp
    int kp = 0;                          // next unit to load
    auto produce = [&]() {
        if (kp >= nk) return;
        if ((kp & 31) == 0) resolve(kp);
        const int tok = __shfl_sync(0xffffffffu, pl_tok, kp & 31);
        const int head = __shfl_sync(0xffffffffu, pl_head, kp & 31);
        const int page = __shfl_sync(0xffffffffu, pl_page, kp & 31);
        const int st = kp % ST;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar + 8 * st, C::STAGE);
            tma_5d(ring + st * C::STAGE, &P.tm_k, tok, head, page, bar + 8 * st, pol);
            tma_5d(ring + st * C::STAGE + C::UNIT, &P.tm_v, tok, head, page, bar + 8 * st, pol);
        }
        ++kp;
    };
    for (int i = 0; i < ST; ++i) produce();

    // ---- items of the range, in order
    bool failed = false;
    int k_failed = 0;                    // the unit whose copy never landed
    int k = 0;                           // next unit to consume
    int64_t u = u0;                      // first unit of the current piece
    int bi = 0;                          // index into pre[] of the current sequence
    {
        const int v = static_cast<int>(u0 / Hg);
        int hi = nseq - 1;
        while (bi < hi) {
            const int mid = (bi + hi + 1) >> 1;
            if (pre[mid] <= v) bi = mid;
            else hi = mid - 1;
        }
    }
    bool crosses = false;                // an item begins here and goes on in the next range
    while (u < u1) {
        while ((int64_t)pre[bi + 1] * Hg <= u) ++bi;
        const int b = b_first + bi;
        const int n = pre[bi + 1] - pre[bi];
        const int64_t first_of_b = (int64_t)pre[bi] * Hg;
        const int x = static_cast<int>((u - first_of_b) / n);
        const int64_t a = first_of_b + (int64_t)x * n, e = a + n;   // the item's units
        const int64_t pe = e < u1 ? e : u1;                         // end of this range's piece
        const int g = x / P.n_groups, grp = x - g * P.n_groups;
        const int hq0 = g * P.G + grp * heads;
        const int nh = min(heads, P.G - grp * heads);                 // heads of a row
        const RowSpan rs = rows_of<ROWS>(P, b, false);
        const int nq = nh * rs.n;                                     // columns: row i, head h in column i nh + h
        const int len = clamp_len(P, b, false);
        const Span sp = span_of(len, rs.n, P.window, P.sinks);
        const int p0 = len - rs.n;                                    // position of the first row
        const int lo0 = P.window > 0 ? max(0, p0 + 1 - P.window) : 0; // first key of its window, and of the last row's
        const int lo1 = P.window > 0 ? max(0, len - P.window) : 0;
        const auto row_i = [&](int col) { return ROWS ? col / nh : 0; };       // a column's row, and its head
        const auto row_h = [&](int col) { return ROWS ? col % nh : col; };
        const auto row_of = [&](int col) { return (int64_t)(rs.r0 + row_i(col)) * P.H_q + hq0 + row_h(col); };   // of O
        int pos[NB][2];                                               // positions of the lane's columns
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = nb * 8 + 2 * (lane & 3) + i;
                pos[nb][i] = !ROWS ? p0 : col < nq ? p0 + row_i(col) : -1;
            }

        // q as the B operand: column lane / 4, elements 16 s + 2 (lane % 4) and + 8
        uint32_t qf[NB][KS][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int col = nb * 8 + (lane >> 2);
            const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const T*>(P.Q) + (int64_t)(rs.r0 + row_i(col)) * P.q_row +
                                                                  (int64_t)(hq0 + row_h(col)) * P.q_head) + (lane & 3);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qf[nb][s][0] = col < nq ? q[8 * s] : 0u;
                qf[nb][s][1] = col < nq ? q[8 * s + 4] : 0u;
            }
        }
        float o[NB][KS][4];
        float m[NB][2], l[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb][0] = m[nb][1] = -INFINITY;
            l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nb][s][i] = 0.f;
        }
        for (; k < nk; ++k) {
            const int64_t uk = uf + (int64_t)k * STEP;
            if (uk >= pe) break;
            const int j = static_cast<int>(uk - a);
            const int tile = j < sp.ns ? j : j - sp.ns + sp.w0;
            const int st = k % ST;
            const uint32_t ks = ring + st * C::STAGE, vs = ks + C::UNIT;
            if (!failed && !__all_sync(0xffffffffu, mbar_wait_bounded(bar + 8 * st, (k / ST) & 1))) {
                failed = true;
                k_failed = k;
            }
            if (failed) continue;
            // visible keys of the tile: token t of it is key key0 + t
            const int key0 = tile * PG_SUB;
            const bool full = key0 + PG_SUB - 1 <= p0 && (key0 >= lo1 || key0 + PG_SUB <= P.sinks);
            bool spoilt = false;
            if (!full) {
                // V rows hidden from every column may hold anything (also NaN, which 0 * v would keep): zero them
                for (int t = 0; t < PG_SUB; ++t)
                    if (key0 + t >= len || (key0 + t < lo0 && key0 + t >= P.sinks))
                        for (int c = lane; c < D / 8; c += 32)
                            *reinterpret_cast<uint4*>(smem + (vs - s_base) + (c >> 3) * (PG_SUB * 128) + t * 128 + (c & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                // one that some rows see and others do not, and that is not finite, must not reach those others
                if (ROWS && rs.n > 1) {
                    bool bad = false;
                    for (int c = lane; c < PG_SUB * D / 8; c += 32)
                        bad |= Elem<T>::not_finite8(*reinterpret_cast<const uint4*>(smem + (vs - s_base) + c * 16));
                    spoilt = __any_sync(0xffffffffu, bad);
                }
            }
            // S^T = K q^T
            float s4[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) s4[nb][i] = 0.f;
            {
                const int r = lane & 15, half = lane >> 4;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int c = 2 * s + half;
                    uint32_t af[4];
                    ldsm_x4(ks + (c >> 3) * (PG_SUB * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), af);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) Elem<T>::mma(s4[nb], af, qf[nb][s][0], qf[nb][s][1]);
                }
            }
            // lane: tokens lane / 4 and + 8, heads 2 (lane % 4) and + 1 of each column block
            const int t0 = lane >> 2;
            bool up = false;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = s4[nb][i] * P.scale_log2;
                    if (!full) {
                        const int key = key0 + t0 + (i >> 1) * 8, p = pos[nb][i & 1];
                        if (key > p || (P.window > 0 && key <= p - P.window && key >= P.sinks)) v = -INFINITY;
                    }
                    s4[nb][i] = v;
                    up |= !(v <= m[nb][i & 1] + Elem<T>::CAP);   // (a NaN too)
                }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mx = fmaxf(s4[nb][i], s4[nb][i + 2]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        mx = fmaxf(mx - Elem<T>::TOP, m[nb][i]);
                        const float al = m[nb][i] > -INFINITY ? ex2_approx(m[nb][i] - mx) : 0.f;
                        m[nb][i] = mx;
                        l[nb][i] *= al;
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            o[nb][s][i] *= al;
                            o[nb][s][i + 2] *= al;
                        }
                    }
            }
            // p, its sum, and its transpose (tokens as k) as hi + lo B fragments
            uint32_t ph[NB][2], plo[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float e0 = ex2_approx(s4[nb][2 * r] - (m[nb][0] > -INFINITY ? m[nb][0] : 0.f));
                    const float e1 = ex2_approx(s4[nb][2 * r + 1] - (m[nb][1] > -INFINITY ? m[nb][1] : 0.f));
                    l[nb][0] += e0;
                    l[nb][1] += e1;
                    if (ROWS && spoilt) {
                        s4[nb][2 * r] = e0;
                        s4[nb][2 * r + 1] = e1;
                    }
                    uint32_t hi, lo;
                    Elem<T>::split(e0, e1, hi, lo);
                    ph[nb][r] = movmatrix_trans(hi);
                    plo[nb][r] = movmatrix_trans(lo);
                }
            if (ROWS && spoilt) {
                // token by token, each column only those that it sees. Lane: elements lane / 4 + 8 q, its columns' p in the
                // lane of token t with the same columns.
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll 1
                    for (int t8 = 0; t8 < 8; ++t8) {
                        const int t = 8 * r + t8, key = key0 + t;
                        float v[KS][2];
#pragma unroll
                        for (int s = 0; s < KS; ++s)
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const int c = 2 * s + q;
                                v[s][q] = Elem<T>::to_float(*reinterpret_cast<const T*>(
                                    smem + (vs - s_base) + (c >> 3) * (PG_SUB * 128) + t * 128 + (((c & 7) ^ t8) << 4) + (lane >> 2) * 2));
                            }
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float pt = __shfl_sync(0xffffffffu, s4[nb][2 * r + i], t8 * 4 + (lane & 3));
                                const int p = pos[nb][i];
                                if (key > p || (P.window > 0 && key <= p - P.window && key >= P.sinks)) continue;
#pragma unroll
                                for (int s = 0; s < KS; ++s)
#pragma unroll
                                    for (int q = 0; q < 2; ++q) o[nb][s][2 * q + i] = fmaf(pt, v[s][q], o[nb][s][2 * q + i]);
                            }
                    }
            } else
            // O^T += V^T p^T
            {
                const int r = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int c = 2 * s + half;
                    uint32_t af[4];
                    ldsm_x4_t(vs + (c >> 3) * (PG_SUB * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), af);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        Elem<T>::mma(o[nb][s], af, ph[nb][0], ph[nb][1]);
                        Elem<T>::mma(o[nb][s], af, plo[nb][0], plo[nb][1]);
                    }
                }
            }
            __syncwarp();
            produce();
        }
        // the rows' sums, in every lane of a head's eight
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], 4);
                l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], 8);
                l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], 16);
            }
        const bool whole = a >= u0 && e <= u1;
        float* part = P.ws + (size_t)(a < u0 ? 2 * worker : 2 * worker + 1) * slot_floats(D, cols);
        if (SPLIT && a >= u0 && e > u1) {
            crosses = true;
            // the item's last unit, of weight w, lies in the last range that begins at w or before
            const int64_t w = e - 1 + (int64_t)TK_ITEM_UNITS * ((int64_t)bi * Hg + x);
            const int last = static_cast<int>(((w + 1) * workers - 1) / U);
            if (BY_WARP ? lane == 0 : tid == 0) jd[worker] = JoinDesc{rs.r0, x, last - worker + 1, rs.n};
        }
        if (BY_WARP) {
            // the warp's own: the result, or a partial. Lane: heads 2 (lane % 4) + i, elements lane / 4 + 8 q.
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int lh = nb * 8 + 2 * (lane & 3) + i;
                    if (lh >= nq) continue;
                    if (whole) {
                        const int64_t row = row_of(lh);
                        const RowEnd r = row_end(P, row, m[nb][i], l[nb][i]);
                        T* out = static_cast<T*>(P.O) + row * D + (lane >> 2);
                        const float* op = P.O_prior + row * D + (lane >> 2);
#pragma unroll
                        for (int s = 0; s < KS; ++s)
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                float v = o[nb][s][2 * q + i] * r.wo;
                                if (r.prior) v = fmaf(op[16 * s + 8 * q], r.wp, v);
                                out[16 * s + 8 * q] = Elem<T>::from(v);
                            }
                        if (lane < 4 && P.LSE) P.LSE[row] = r.lse;
                    } else {
                        float* pr = part + lh * (D + 4);
#pragma unroll
                        for (int s = 0; s < KS; ++s)
#pragma unroll
                            for (int q = 0; q < 2; ++q) pr[4 + 16 * s + 8 * q + (lane >> 2)] = o[nb][s][2 * q + i];
                        if (lane < 4) *reinterpret_cast<float2*>(pr) = make_float2(m[nb][i], l[nb][i]);
                    }
                }
        } else {
            // the CTA's warps join: maxima and sums first, then O in two halves of D per column block
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (lane < 4) {
                        s_m[warp * 16 + nb * 8 + 2 * lane + i] = m[nb][i];
                        s_l[warp * 16 + nb * 8 + 2 * lane + i] = l[nb][i];
                    }
            __syncthreads();
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float al[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float M = -INFINITY;
#pragma unroll
                    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * 16 + nb * 8 + 2 * (lane & 3) + i]);
                    al[i] = join_weight(m[nb][i], M);
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float* row = jbuf + (warp * 8 + 2 * (lane & 3)) * C::JROW + (lane >> 2);
#pragma unroll
                    for (int s = 0; s < KS / 2; ++s) {
                        const float (&v)[4] = o[nb][hf * (KS / 2) + s];
                        row[16 * s] = v[0] * al[0];
                        row[C::JROW + 16 * s] = v[1] * al[1];
                        row[16 * s + 8] = v[2] * al[0];
                        row[C::JROW + 16 * s + 8] = v[3] * al[1];
                    }
                    __syncthreads();
                    for (int i = tid; i < 8 * (D / 4); i += NT) {   // (head, pair of elements)
                        const int h = i / (D / 4), d = 2 * (i - h * (D / 4));
                        const int lh = nb * 8 + h;
                        if (lh < nq) {
                            float M = -INFINITY, L = 0.f;
#pragma unroll
                            for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * 16 + lh]);
                            float a0 = 0.f, a1 = 0.f;
#pragma unroll
                            for (int w = 0; w < NW; ++w) {
                                const float mw = s_m[w * 16 + lh];
                                L += s_l[w * 16 + lh] * join_weight(mw, M);
                                const float2 f = *reinterpret_cast<const float2*>(jbuf + (w * 8 + h) * C::JROW + d);
                                a0 += f.x;
                                a1 += f.y;
                            }
                            const int dd = hf * (D / 2) + d;
                            if (!SPLIT || whole) {
                                finish2<T>(P, row_of(lh), D, dd, a0, a1, M, L, dd == 0);
                            } else {
                                float* pr = part + lh * (D + 4);
                                *reinterpret_cast<float2*>(pr + 4 + dd) = make_float2(a0, a1);
                                if (dd == 0) *reinterpret_cast<float2*>(pr) = make_float2(M, L);
                            }
                        }
                    }
                    __syncthreads();
                }
            }
        }
        u = pe;
    }
    if (SPLIT && !crosses && (BY_WARP ? lane == 0 : tid == 0)) jd[worker].pieces = 0;
    if (failed) {
        set_err(P.err, ERR_PAGED_TOKEN);
        for (k = k_failed; k < kp; ++k)   // copies still in flight, waited for with the same limit
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar + 8 * (k % ST), (k / ST) & 1))) break;
    }
}

// Joins the partials of a split item: CTA (c, h, w) takes the one that begins in range w gridDim.x + c, if any, column h
// (row and q head) of it; 256 / (D/4) pieces at a time, one float4 of the row a thread.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_token_join_kernel(const __grid_constant__ PagedAttn P) {
    constexpr int LP = D / 4, NP = 256 / LP;
    __shared__ float4 s_acc[NP][LP];
    pdl_wait();
    pdl_release();
    const int h = blockIdx.y, c = blockIdx.z * gridDim.x + blockIdx.x;
    const int heads = P.heads_per_group, cols = P.cols;
    const JoinDesc d = reinterpret_cast<const JoinDesc*>(P.ws + (size_t)2 * gridDim.x * gridDim.z * slot_floats(D, cols))[c];
    if (d.pieces == 0) return;
    const int g = d.x / P.n_groups, grp = d.x - g * P.n_groups;
    const int nh = min(heads, P.G - grp * heads);
    if (h >= nh * d.rows) return;
    const int64_t row = (int64_t)(d.r0 + h / nh) * P.H_q + g * P.G + grp * heads + h % nh;
    const int tid = threadIdx.x, pp = tid / LP, q = tid - pp * LP;
    // piece i: slot 2 c + 1 for the first, 2 (c + i) for the others
    auto part = [&](int i) { return P.ws + (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * slot_floats(D, cols) + h * (D + 4); };
    float M = -INFINITY;
    for (int i = tid & 31; i < d.pieces; i += 32) M = fmaxf(M, part(i)[0]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    for (int i = tid & 31; i < d.pieces; i += 32) {
        const float2 ml = *reinterpret_cast<const float2*>(part(i));
        L += ml.y * join_weight(ml.x, M);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pp < NP) {
#pragma unroll 4
        for (int i = pp; i < d.pieces; i += NP) {
            const float* p = part(i);
            const float4 v = *reinterpret_cast<const float4*>(p + 4 + 4 * q);
            const float w = join_weight(p[0], M);
            acc.x = fmaf(w, v.x, acc.x);
            acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z);
            acc.w = fmaf(w, v.w, acc.w);
        }
        s_acc[pp][q] = acc;
    }
    __syncthreads();
    if (tid < LP) {
        float4 a = s_acc[0][tid];
#pragma unroll
        for (int i = 1; i < NP; ++i) {
            const float4 v = s_acc[i][tid];
            a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
        }
        finish2<T>(P, row, D, 4 * tid, a.x, a.y, M, L, tid == 0);
        finish2<T>(P, row, D, 4 * tid + 2, a.z, a.w, M, L, false);
    }
}

template <typename T, int D, int NB, int MODE, bool ROWS>
cudaError_t launch_t(PagedAttn& p, cudaStream_t st) {
    using C = TCfg<D, MODE>;
    constexpr bool SPLIT = is_split(MODE);
    static_assert(C::SMEM_BASE + 4 * (TK_MAX_B + 1) <= 232448, "one CTA's shared memory");
    const cudaError_t e0 = allow_smem<paged_token_kernel<T, D, NB, MODE, ROWS>>(C::SMEM_BASE + 4 * (TK_MAX_B + 1), p.device);
    if (e0 != cudaSuccess) return e0;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.n_ctas);
    cfg.blockDim = dim3(C::NW * 32);
    cfg.dynamicSmemBytes = C::SMEM_BASE + 4 * ((SPLIT ? p.B : 1) + 1);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_token_kernel<T, D, NB, MODE, ROWS>, p);
    if (e != cudaSuccess || !SPLIT) return e;
    cfg.gridDim = dim3(p.n_ctas, p.cols, MODE == TK_WARP ? C::NW : 1);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, paged_token_join_kernel<T, D>, p);
}

template <typename T, int D, int NB, bool ROWS>
cudaError_t launch_m(PagedAttn& p, cudaStream_t st) {
    return p.mode == TK_WARP  ? launch_t<T, D, NB, TK_WARP, ROWS>(p, st)
           : p.mode == TK_CTA_HALF ? launch_t<T, D, NB, TK_CTA_HALF, ROWS>(p, st)
           : p.mode == TK_CTA ? launch_t<T, D, NB, TK_CTA, ROWS>(p, st)
           : p.mode == TK_ITEM_HALF ? launch_t<T, D, NB, TK_ITEM_HALF, ROWS>(p, st)
                              : launch_t<T, D, NB, TK_ITEM, ROWS>(p, st);
}
template <typename T, int D, int NB>
cudaError_t launch_s(PagedAttn& p, cudaStream_t st) {
    return p.cu_rows ? launch_m<T, D, NB, true>(p, st) : launch_m<T, D, NB, false>(p, st);
}

template <typename T>
cudaError_t launch_d(PagedAttn& p, int D, cudaStream_t st) {
    const bool two = p.cols > 8;
    switch (D) {
        case 64: return two ? launch_s<T, 64, 2>(p, st) : launch_s<T, 64, 1>(p, st);
        case 128: return two ? launch_s<T, 128, 2>(p, st) : launch_s<T, 128, 1>(p, st);
        case 192: return launch_s<T, 192, 1>(p, st);
        case 256: return launch_s<T, 256, 1>(p, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace
}  // namespace pck
