// pck_paged_token_e4m3_impl.cuh -- attention of one new token (or a few) per sequence over a quantised paged cache.
//
// With codes c and scales 2^ek, 2^ev of each token and kv head (pck_paged_e4m3.cuh), tau' = tau log2 e:
//   s_j = 2^ek_j tau' (q . c_j),  O = sum_j 2^(s_j - m) 2^ev_j c'_j / l,  l = sum_j 2^(s_j - m),  LSE = (m + log2 l) ln 2.
// Codes are exact in fp16, so both products run on fp16 MMAs with fp32 sums and the scales never touch the operands: 2^ek
// multiplies a token's finished scores and 2^ev its weights. D + 1 bytes a head row are read once: half of a 16-bit
// cache's, so HBM still bounds it, with half the time a byte for everything else. How a call is cut into ranges of units, and
// the kernel that joins them, are the 16-bit cache's (pck_paged_token_impl.cuh); here is what differs:
//  * A unit is 32 tokens of a kv head (16 at D > 128, 64 in long ranges at D = 64), so its two code tiles are as large as the
//    16-bit kernel's. Pages that hold whole units give one TMA box of K and one of V; from other pages (multiples of 16) the lanes
//    copy 16-byte pieces, each 16 tokens' from their own page (boxes of 16 tokens took as long: 89.6 us against 87.7 on 64 ragged
//    sequences, 43.0 against 43.6 on windows). Scales come by 4-byte copies of the lanes. All of them arrive on one mbarrier.
//  * Operands: a 16-byte row piece of a code tile holds 16 elements, so one ldmatrix.x4 fetches 16 tokens x 32 elements. Lane
//    (g, c) gets elements 4c .. 4c+3 of token g; as the MMA's k index only pairs K with q, they are its k = 2c, 2c+1, 2c+8,
//    2c+9, and q is loaded in that order. V comes through the transposing ldmatrix in pairs of elements: bytes (2g, 2g+1) of
//    tokens 2c and 2c+1, which one byte permutation turns into (tokens 2c, 2c+1) of element 2g and of 2g+1: rows g and g+8
//    of an MMA whose rows are elements in that order. One conversion makes two fp16 values.
//  * q: fp16 as it is; a bf16 row is moved by a power of two so that its largest element is 2^14 .. 2^15 and then exact in fp16
//    but for elements 2^-29 of that one and less, which are held to 2^-39 of it.
//  * Weights: w = 2^(s - m) 2^ev enters the second MMA as an fp16 pair hi + lo, held to 22 bits or to 2^-25, whichever is more. m stands
//    so that the largest of s + ev (a token's largest share of O) is TOP, and moves only when a weight passes W_TOP: that is seen on
//    the weights themselves, not on the scores. So a weight is held to 2^-37 of the largest one. ev counts from EV_LOW up in m, which
//    keeps l within fp32: where the token that counts most has a V scale 2^-b below 2^EV_LOW, the largest weight is 2^(TOP - b).
//  * Up to 4 columns (4 q heads per kv head): the weights' lo parts take columns 4-7 of the MMA's 8, one MMA instead of two.
// Measured (graph replays): one cache of 131,071 tokens (8 kv heads of 128, 4 q heads each) 48-49 us, 5.5 TB/s; 16 caches of 30-65k
// tokens (2 kv heads of 256) 125 us, 6.0 TB/s; 64 ragged sequences (8 kv heads of 64, prior) 57 us, 4.1 TB/s; 32 windows of up to
// 2048 tokens (8 kv heads of 128, 8 q heads each) 32 us, 3.6 TB/s; 300 tokens 6.6 us; a few rows on four caches of 20-32k tokens
// (8 kv heads of 128, 4 q heads each) 44 us with 2 rows, 57 with 4 (0.71 and 0.55 of HBM: two column blocks, hi and lo). What is
// left: the start (lengths, page table and first loads one after another, 5-8 us), the slowest range's end and the join (3-5 us); in
// between the loads run at 5.5-6.3 TB/s.
#pragma once

#include "pck_paged_e4m3.cuh"
#include "pck_paged_token_impl.cuh"

namespace pck {
namespace {

constexpr float EV_LOW = -40.f;      // weights of V scales of 2^(-40 - b) are held to 2^(-37 + b) of the largest
constexpr float M_NONE = -1e30f;     // m before a visible key: finite, so that a hidden one's 2^(-inf - m) is 0
constexpr float W_TOP = 61440.f, L_TOP = 1e30f;      // the largest weight (fp16 ends at 65,504), and sum of a unit's p
// What an item costs beside its units, in units (as tk_item_units). Ranges per half CTA, 24 x 1-4000 tokens: 19.3 us with 12, 19.4 with 16, 21.9
// with 24; ranges per warp, 600 x 1-1000 tokens 39 with 3, 45 with 5, 49 with 8, and 64 ragged sequences 57, 58, 59.
__host__ __device__ constexpr int item_units8(int mode) { return mode == TK_WARP ? 3 : 16; }
// Tokens of a unit. At D = 64 what a unit costs whatever its size (its loads' addresses, its scales, votes) is a visible share:
// 16 caches of 30,000 tokens 135 us with 32, 91 with 64; but short items then end in half-empty units (600 x 100 tokens 44 us
// with 32, 56 with 64).
__host__ __device__ constexpr int sub8(int D, int mode) {
    return D > 128 ? 16 : D == 64 && (mode == TK_CTA || mode == TK_CTA_HALF) ? 64 : 32;
}
// Warps per SM: 192 KB of ring, 3 stages each (4 at D = 192). 12 warps of 2 stages: one cache of 131k tokens 49.7 us against
// 48.0, 4 rows on 20-32k tokens 90 against 63 (registers). At D = 64 units of 32 tokens have 16 warps of 3 stages: 64 ragged sequences
// 57 us, 600 x 1-1000 tokens 39; with 8 of 6 stages 69 and 48, with 12 of 4 57 and 40.
__host__ __device__ constexpr int warps_sm8(int D, int mode) { return D == 64 && sub8(D, mode) == 32 ? 16 : 8; }

template <int D, int MODE, bool QUAD>
struct TCfg8 {
    static constexpr int SUB = sub8(D, MODE);
    static constexpr int CHB = D % 128 == 0 ? 128 : 64;           // bytes of a row that lie together: the swizzle's width
    static constexpr int NW = warps_sm8(D, MODE) / per_sm(MODE);  // warps per CTA
    static constexpr int UNIT = SUB * D;                          // bytes of a K (or V) unit
    static constexpr int STAGE = 2 * UNIT;
    static constexpr int ST = 196608 / warps_sm8(D, MODE) / STAGE;
    static constexpr int RING = NW * ST * STAGE;
    static constexpr int SCB = SUB > 32 ? SUB : 32;
    static constexpr int JC = QUAD ? 4 : 8;                       // columns that are joined at a time
    static constexpr int JP = (D > 128 ? 2 : 1) * (QUAD ? 1 : 2); // parts in which O is joined
    static constexpr int JROW = D / JP + 4;                       // floats of a join row (padded)
    static constexpr int OFF_SC = RING;                           // [NW][ST][2 SCB]: scale bytes of K, then of V
    static constexpr int OFF_JOIN = OFF_SC + NW * ST * 2 * SCB;
    static constexpr int OFF_ML = OFF_JOIN + NW * JC * JROW * 4;   // [NW][16] m, then l
    static constexpr int OFF_BAR = OFF_ML + NW * 16 * 2 * 4;
    static constexpr int OFF_SCAN = OFF_BAR + NW * ST * 8 + 8;
    static constexpr int OFF_PRE = OFF_SCAN + 64 * 4;             // prefix of units per sequence [B + 1]
    static constexpr int SMEM_BASE = OFF_PRE + 1024;              // + alignment slack; + 4 (B + 1)
};

// Where the 16-byte piece c16 of a token's row lies in a code tile of SUB tokens.
template <int SUB, int CHB>
__device__ __forceinline__ uint32_t piece_at(int token, int c16) {
    constexpr int PC = CHB / 16;
    const int swz = CHB == 128 ? token & 7 : (token >> 1) & 3;
    return (c16 / PC) * (SUB * CHB) + token * CHB + (((c16 % PC) ^ swz) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint64_t pol) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(pol) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// 2^e for a score or a weight: NaN for byte 255, and 0 for byte 0 (2^-127: nothing that a sum would notice).
__device__ __forceinline__ float quick_scale(uint32_t byte) {
    const float x = __uint_as_float(byte << 23);
    return fmaf(x, 0.f, x);
}

__device__ __forceinline__ bool nan_codes(uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
    return bad;
}

__device__ __forceinline__ uint32_t pack_out(int dtype, float a, float b) {
    return dtype == PCK_DT_F16 ? Elem<__half>::pack(a, b) : Elem<__nv_bfloat16>::pack(a, b);
}

// Elements d, d + 1 of a row of O (token x H_q + head), and (first) its LSE.
__device__ __forceinline__ void finish8(const PagedAttn& P, int64_t row, int D, int d, float a0, float a1, float m, float l, bool first) {
    const RowEnd r = row_end(P, row, m, l);
    a0 *= r.wo;
    a1 *= r.wo;
    if (r.prior) {
        const float2 op = *reinterpret_cast<const float2*>(P.O_prior + row * D + d);
        a0 = fmaf(op.x, r.wp, a0);
        a1 = fmaf(op.y, r.wp, a1);
    }
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(P.O) + (row * D + d) * 2) = pack_out(P.dtype, a0, a1);
    if (first && P.LSE) P.LSE[row] = r.lse;
}

// NBQ: column blocks of 8, or 0: at most 4 columns, whose weights' lo parts take the other 4 of one block.
template <int D, int NBQ, int MODE, bool ROWS>
__global__ void __launch_bounds__(TCfg8<D, MODE, NBQ == 0>::NW * 32, per_sm(MODE)) paged_token8_kernel(const __grid_constant__ PagedAttn P) {
    using C = TCfg8<D, MODE, NBQ == 0>;
    constexpr int NW = C::NW, ST = C::ST, KS = D / 16, NT = NW * 32, SUB = C::SUB, NS = SUB / 16, NB = NBQ ? NBQ : 1;
    constexpr bool QUAD = NBQ == 0;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_base = smem_u32(smem);
    float* jbuf = reinterpret_cast<float*>(smem + C::OFF_JOIN);
    float* s_m = reinterpret_cast<float*>(smem + C::OFF_ML);
    float* s_l = s_m + NW * 16;
    int* s_scan = reinterpret_cast<int*>(smem + C::OFF_SCAN);
    int* pre = reinterpret_cast<int*>(smem + C::OFF_PRE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lg = lane >> 2, lc = lane & 3;
    const uint32_t ring = s_base + warp * ST * C::STAGE;
    const uint32_t bar = s_base + C::OFF_BAR + warp * ST * 8;
    constexpr int SC_LANES = SUB / 2;    // lanes that copy scales: 4 of a token each, K's and then V's
    const uint8_t* s_sc = smem + C::OFF_SC + warp * ST * 2 * C::SCB;
    if (lane == 0) {
        // arrivals of a phase: the lanes' (all that copy pieces; those of the scales) and, with tile loads, that of their bytes
        for (int i = 0; i < ST; ++i) mbar_init(bar + 8 * i, P.pieces ? 32 : SC_LANES + 1);
        fence_mbar_init();
        if (!P.pieces) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(&P.tm_k) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(&P.tm_v) : "memory");
        }
    }
    pdl_wait();
    pdl_release();
    fence_proxy_async_all();     // the pages may have been written by the kernel before, and are read by TMA

    const int Hg = P.H_kv * P.n_groups;
    const int heads = P.heads_per_group, cols = P.cols;
    constexpr bool SPLIT = is_split(MODE), BY_WARP = MODE == TK_WARP;
    constexpr int TK_ITEM_UNITS = item_units8(MODE);
    const int worker = BY_WARP ? warp * gridDim.x + blockIdx.x : blockIdx.x;    // few workers spread over the SMs
    int workers = BY_WARP ? gridDim.x * NW : gridDim.x;
    JoinDesc* jd = reinterpret_cast<JoinDesc*>(P.ws + (size_t)2 * workers * slot_floats(D, cols));
    const Cut cut = cut_units<NW, MODE, ROWS, SUB, item_units8(MODE)>(P, worker, workers, s_scan, pre);
    if (SPLIT && cut.idle) {
        if (BY_WARP ? lane == 0 : tid == 0) jd[worker].pieces = 0;
        return;
    }
    const int64_t u0 = cut.u0, u1 = cut.u1, U = cut.U;
    workers = cut.workers;
    const int b_first = cut.b_first;
    const int nseq = SPLIT ? P.B : 1;     // sequences in pre[]

    // ---- a warp's units: u0 + k of its own range, u0 + warp + k NW of its CTA's. Lane i resolves unit k0 + i: coordinates of
    // its loads (of each 16 tokens where pages are no multiples of a unit)
    const int64_t uf = BY_WARP ? u0 : u0 + warp;
    constexpr int STEP = BY_WARP ? 1 : NW;
    const uint64_t pol = l2_evict_first();
    auto seq_of = [&](int64_t u) {      // the sequence (of pre[]) whose units u is one of
        int lo = 0, hi = nseq - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)pre[mid] * Hg <= u) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    int pl_head = 0, pl_tok[NS] = {}, pl_page[NS] = {};
    auto resolve = [&](int k0) {
        const int64_t u = uf + (int64_t)(k0 + lane) * STEP;
        if (u < u1) {
            const int lo = seq_of(u);
            const int b = b_first + lo;
            const int n = pre[lo + 1] - pre[lo];
            const int64_t rem = u - (int64_t)pre[lo] * Hg;
            const int x = static_cast<int>(div_pos(rem, n)), j = static_cast<int>(rem - (int64_t)x * n);
            const int len = clamp_len(P, b, false);
            const int rows = rows_of<ROWS>(P, b, false).n;
            const Span s = span_of<SUB>(len, rows, P.window, P.sinks);
            const int tok0 = (j < s.ns ? j : j - s.ns + s.w0) * SUB;
            const int lo0 = P.window > 0 ? len - rows + 1 - P.window : 0;    // first key of the first row's window
            pl_head = x / P.n_groups;
#pragma unroll
            for (int h = 0; h < NS; ++h) {
                if (h > 0 && !P.pieces) break;
                const int tok = tok0 + 16 * h, pi = tok / P.page;
                pl_tok[h] = tok - pi * P.page;
                pl_page[h] = 0;
                // 16 tokens that no row sees are not looked up (their page may not exist): the first page is read in their place
                const bool seen = !P.pieces || (tok < len && (tok + 16 > lo0 || tok < P.sinks));
                if (len > 0 && rows > 0 && pi < P.max_pages && seen) {
                    const int pg = P.table[(int64_t)b * P.max_pages + pi];
                    if (pg < 0 || pg >= P.n_pages) set_err(P.err, ERR_PAGE_ID);   // and page 0 is read instead
                    else pl_page[h] = pg;
                }
            }
        }
    };
    const int nk = static_cast<int>(u1 > uf ? (u1 - uf + STEP - 1) / STEP : 0);   // units of this warp
    int kp = 0, pst = 0;                 // next unit to load, and its stage
    auto produce = [&]() {
        if (kp >= nk) return;
        if ((kp & 31) == 0) resolve(kp);
        const int head = __shfl_sync(0xffffffffu, pl_head, kp & 31);
        const int st = pst;
        pst = st + 1 == ST ? 0 : st + 1;
        const uint32_t b = bar + 8 * st, dst = ring + st * C::STAGE;
        int tok[NS], page[NS];
#pragma unroll
        for (int h = 0; h < NS; ++h) {
            tok[h] = __shfl_sync(0xffffffffu, pl_tok[h], kp & 31);
            page[h] = __shfl_sync(0xffffffffu, pl_page[h], kp & 31);
        }
        if (P.pieces) {
            const uint8_t *kc[NS], *vc[NS];
#pragma unroll
            for (int h = 0; h < NS; ++h) {
                kc[h] = static_cast<const uint8_t*>(P.k_base) + page[h] * P.kv_stride[0] + head * P.kv_stride[1] + tok[h] * P.kv_stride[2];
                vc[h] = static_cast<const uint8_t*>(P.v_base) + page[h] * P.kv_stride[3] + head * P.kv_stride[4] + tok[h] * P.kv_stride[5];
            }
#pragma unroll
            for (int i = 0; i < SUB * KS / 32; ++i) {
                const int t = (lane + 32 * i) / KS, c = (lane + 32 * i) % KS, h = 32 * i / KS / 16;     // (a step stays in one 16)
                const uint32_t at = dst + piece_at<SUB, C::CHB>(t, c);
                cp_async16(at, kc[h] + (t & 15) * P.kv_stride[2] + 16 * c, pol);
                cp_async16(at + C::UNIT, vc[h] + (t & 15) * P.kv_stride[5] + 16 * c, pol);
            }
        } else if (lane == 0) {
            mbar_arrive_expect_tx(b, C::STAGE);
            tma_5d(dst, &P.tm_k, tok[0], head, page[0], b, pol);
            tma_5d(dst + C::UNIT, &P.tm_v, tok[0], head, page[0], b, pol);
        }
        if (lane < SC_LANES) {
            const int t = (lane % (SUB / 4)) * 4;
            int pg = page[0], at = tok[0] + t;
#pragma unroll
            for (int h = 1; h < NS; ++h)
                if (P.pieces && t >= 16 * h) {
                    pg = page[h];
                    at = tok[h] + t - 16 * h;
                }
            const int64_t so = ((int64_t)pg * P.H_kv + head) * P.page + at;
            cp_async4(s_base + C::OFF_SC + (warp * ST + st) * 2 * C::SCB + (lane < SUB / 4 ? 0 : C::SCB) + t,
                      (lane < SUB / 4 ? P.k_scale : P.v_scale) + so);
        }
        if (P.pieces || lane < SC_LANES) cp_async_arrive(b);
        ++kp;
    };
#pragma unroll 1
    for (int i = 0; i < ST; ++i) produce();

    // ---- items of the range, in order
    bool failed = false;
    int k_failed = 0;                    // the unit whose copy never landed
    int k = 0, st = 0, phase = 0;        // next unit to consume, its stage and that stage's phase
    int64_t u = u0;                      // first unit of the current piece
    int bi = seq_of(u0);                 // index into pre[] of the current sequence
    bool crosses = false;                // an item begins here and goes on in the next range
    while (u < u1) {
        while ((int64_t)pre[bi + 1] * Hg <= u) ++bi;
        const int b = b_first + bi;
        const int n = pre[bi + 1] - pre[bi];
        const int64_t first_of_b = (int64_t)pre[bi] * Hg;
        const int x = static_cast<int>(div_pos(u - first_of_b, n));
        const int64_t a = first_of_b + (int64_t)x * n, e = a + n;   // the item's units
        const int64_t pe = e < u1 ? e : u1;                         // end of this range's piece
        const int g = x / P.n_groups, grp = x - g * P.n_groups;
        const int hq0 = g * P.G + grp * heads;
        const int nh = min(heads, P.G - grp * heads);                 // heads of a row
        const RowSpan rs = rows_of<ROWS>(P, b, false);
        const int nq = nh * rs.n;                                     // columns: row i, head h in column i nh + h
        const int len = clamp_len(P, b, false);
        const Span sp = span_of<SUB>(len, rs.n, P.window, P.sinks);
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
                const int col = nb * 8 + 2 * lc + i;
                pos[nb][i] = !ROWS ? p0 : col < nq ? p0 + row_i(col) : -1;
            }

        // q as the B operand: column lg, elements 16 s + 4 lc .. + 3; qs: what a finished score of the lane's columns is worth
        uint32_t qf[NB][KS][2];
        float qs[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int col = nb * 8 + lg;
            const __half* q = static_cast<const __half*>(P.Q) + (int64_t)(rs.r0 + row_i(col)) * P.q_row + (int64_t)(hq0 + row_h(col)) * P.q_head + 4 * lc;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint2 w = col < nq ? *reinterpret_cast<const uint2*>(q + 16 * s) : make_uint2(0u, 0u);
                qf[nb][s][0] = w.x;
                qf[nb][s][1] = w.y;
            }
            qs[nb][0] = qs[nb][1] = P.scale_log2;
            if (P.dtype == PCK_DT_BF16) {
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[nb][s][i] << 16)), fabsf(__uint_as_float(qf[nb][s][i] & 0xffff0000u))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ex = min(static_cast<int>(__float_as_uint(top) >> 23), 254);
                const int up = min(268 - ex, 253);                    // biased exponent of the factor: 2^(14 + 127 - ex)
                const float f = __uint_as_float(static_cast<uint32_t>(up) << 23);
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qf[nb][s][i] = Elem<__half>::pack(__uint_as_float(qf[nb][s][i] << 16) * f, __uint_as_float(qf[nb][s][i] & 0xffff0000u) * f);
                const float down = P.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
#pragma unroll
                for (int i = 0; i < 2; ++i) qs[nb][i] = __shfl_sync(0xffffffffu, down, (2 * lc + i) * 4);
            }
        }
        float o[NB][KS][4];
        float m[NB][2], l[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb][0] = m[nb][1] = M_NONE;
            l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nb][s][i] = 0.f;
        }
        const int kend = pe > uf ? static_cast<int>((pe - uf + STEP - 1) / STEP) : 0;      // (pe <= u1: at most nk)
        int j = static_cast<int>(uf + (int64_t)k * STEP - a);
        for (; k < kend; ++k, j += STEP) {
            const int tile = j < sp.ns ? j : j - sp.ns + sp.w0;
            const uint32_t ks = ring + st * C::STAGE, vs = ks + C::UNIT;
            const uint8_t* scale = s_sc + st * 2 * C::SCB + lg;
            if (!failed && !__all_sync(0xffffffffu, mbar_wait_bounded(bar + 8 * st, phase))) {
                failed = true;
                k_failed = k;
            }
            st = st + 1 == ST ? 0 : st + 1;
            phase ^= st == 0;
            if (failed) continue;
            // visible keys of the tile: token t of it is key key0 + t
            const int key0 = tile * SUB;
            const bool full = key0 + SUB - 1 <= p0 && (key0 >= lo1 || key0 + SUB <= P.sinks);
            // the scales of the lane's tokens 8 r + lg
            float sk[2 * NS], sv[2 * NS];
#pragma unroll
            for (int r = 0; r < 2 * NS; ++r) {
                sk[r] = quick_scale(scale[8 * r]);
                sv[r] = quick_scale(scale[C::SCB + 8 * r]);
            }
            // V rows hidden from every column may hold anything (also NaN, which 0 * v would keep): the permutation that pairs tokens
            // 8 r + 2 lc and + 1 takes zeros for them. (Zeroing them in shared memory, with the fence that the next tile load
            // then needs, took 2.7 us a unit, and every item ends in such a unit.)
            uint32_t pick[2 * NS];
            bool spoilt = false;
            const auto hidden = [&](int t) { return key0 + t >= len || (key0 + t < lo0 && key0 + t >= P.sinks); };
#pragma unroll
            for (int r = 0; r < 2 * NS; ++r) pick[r] = 0x3120;
            if (!full) {
                bool bad = false;
#pragma unroll
                for (int r = 0; r < 2 * NS; ++r) {
                    if (hidden(8 * r + 2 * lc)) pick[r] = 0x3424;
                    if (hidden(8 * r + 2 * lc + 1)) pick[r] = pick[r] & 0x0f0f | 0x4040;
                    if (hidden(8 * r + lg)) sv[r] = 0.f;
                    bad |= sv[r] != sv[r];
                }
                // one that some rows see and others do not, and that is NaN (a code, or its scale), must not reach those others
                if (ROWS && rs.n > 1) {
                    for (int c = lane; c < SUB * KS; c += 32)
                        if (!hidden(c / (C::CHB / 16) % SUB)) bad |= nan_codes(*reinterpret_cast<const uint4*>(smem + (vs - s_base) + c * 16));
                    spoilt = __any_sync(0xffffffffu, bad);
                }
            }
            // S^T = K q^T
            const int r16 = lane & 15, half = lane >> 4;
            float s4[NS][NB][4], t4[NS][NB][4];       // sums over the even and the odd k steps: short chains, all side by side
#pragma unroll
            for (int sb = 0; sb < NS; ++sb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s4[sb][nb][i] = t4[sb][nb][i] = 0.f;
#pragma unroll
            for (int s = 0; s < KS; s += 2)
#pragma unroll
                for (int sb = 0; sb < NS; ++sb) {
                    uint32_t w[4], af[4];
                    ldsm_x4(ks + piece_at<SUB, C::CHB>(16 * sb + r16, s + half), w);
                    half_codes(w[0], af[0], af[2]);
                    half_codes(w[1], af[1], af[3]);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma16816(s4[sb][nb], af, qf[nb][s][0], qf[nb][s][1]);
                    half_codes(w[2], af[0], af[2]);
                    half_codes(w[3], af[1], af[3]);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma16816(t4[sb][nb], af, qf[nb][s + 1][0], qf[nb][s + 1][1]);
                }
            // lane: tokens 8 r + lg, columns 2 lc and + 1 of each column block
#pragma unroll
            for (int sb = 0; sb < NS; ++sb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s4[sb][nb][i] = (s4[sb][nb][i] + t4[sb][nb][i]) * (sk[2 * sb + (i >> 1)] * qs[nb][i & 1]);
            if (!full) {
#pragma unroll
                for (int sb = 0; sb < NS; ++sb)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = key0 + 8 * (2 * sb + (i >> 1)) + lg, p = pos[nb][i & 1];
                            if (key > p || (P.window > 0 && key <= p - P.window && key >= P.sinks)) s4[sb][nb][i] = -INFINITY;
                        }
            }
            // p = 2^(s - m), the weights w = p 2^ev and p's sums over the lane's tokens; m moves when a weight would not fit fp16
            // (or l grow too large: where every ev is far below 0). The first unit's m is M_NONE, which nothing visible fits.
            float sum[NB][2], w4[NS][NB][4];
#pragma unroll 1
            for (int pass = 0;; ++pass) {
                bool up = false;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) sum[nb][0] = sum[nb][1] = 0.f;
#pragma unroll
                for (int sb = 0; sb < NS; ++sb)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p = ex2_approx(s4[sb][nb][i] - m[nb][i & 1]);
                            sum[nb][i & 1] += p;
                            w4[sb][nb][i] = p * sv[2 * sb + (i >> 1)];
                            up |= !(w4[sb][nb][i] <= W_TOP);             // (a NaN too)
                        }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) up |= !(fmaxf(sum[nb][0], sum[nb][1]) <= L_TOP);
                if (pass || !__any_sync(0xffffffffu, up)) break;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int r = 0; r < 2 * NS; ++r) {
                            const float ev = fmaxf(static_cast<float>(static_cast<int>(__float_as_uint(sv[r]) >> 23) - 127), EV_LOW);
                            mx = fmaxf(mx, s4[r >> 1][nb][2 * (r & 1) + i] + ev);
                        }
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        mx = fmaxf(mx - Elem<__half>::TOP, m[nb][i]);
                        float al = ex2_approx(m[nb][i] - mx);
                        m[nb][i] = mx;
                        l[nb][i] *= al;
                        if (QUAD) {                      // O of columns 4 .. 7 belongs to 0 .. 3
                            const float other = __shfl_up_sync(0xffffffffu, al, 2);
                            if (lc >= 2) al = other;
                        }
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            o[nb][s][i] *= al;
                            o[nb][s][i + 2] *= al;
                        }
                    }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                l[nb][0] += sum[nb][0];
                l[nb][1] += sum[nb][1];
            }
            // the weights' transpose (tokens as k) as hi + lo B fragments
            uint32_t ph[NS][NB][2], plo[NS][NB][2];
#pragma unroll
            for (int sb = 0; sb < NS; ++sb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        uint32_t hi, lo;
                        split_hi_lo(w4[sb][nb][2 * r], w4[sb][nb][2 * r + 1], hi, lo);
                        if (QUAD) {
                            const uint32_t other = __shfl_up_sync(0xffffffffu, lo, 2);
                            ph[sb][nb][r] = movmatrix_trans(lc < 2 ? hi : other);
                        } else {
                            ph[sb][nb][r] = movmatrix_trans(hi);
                            plo[sb][nb][r] = movmatrix_trans(lo);
                        }
                    }
            if (ROWS && spoilt) {
                // token by token, each column only those that it sees. Lane: elements 16 s + 2 lg and + 1, its columns' weights in the
                // lane of the token with the same columns.
#pragma unroll
                for (int r = 0; r < 2 * NS; ++r)
#pragma unroll 1
                    for (int t8 = 0; t8 < 8; ++t8) {
                        const int t = 8 * r + t8, key = key0 + t;
                        float w[NB][2];
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int i = 0; i < 2; ++i) w[nb][i] = __shfl_sync(0xffffffffu, w4[r >> 1][nb][2 * (r & 1) + i], t8 * 4 + lc);
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            const uint32_t two = *reinterpret_cast<const uint16_t*>(smem + (vs - s_base) + piece_at<SUB, C::CHB>(t, s) + 2 * lg);
                            uint32_t h2, none;
                            half_codes(two, h2, none);
                            const float2 v = __half22float2(u32_as_h2(h2));
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const int p = pos[nb][i];
                                    if (QUAD && lc >= 2) continue;
                                    if (key > p || (P.window > 0 && key <= p - P.window && key >= P.sinks)) continue;
                                    o[nb][s][i] = fmaf(w[nb][i], v.x, o[nb][s][i]);
                                    o[nb][s][2 + i] = fmaf(w[nb][i], v.y, o[nb][s][2 + i]);
                                }
                        }
                    }
            } else
            // O^T += V^T p^T
            {
#pragma unroll
                for (int sb = 0; sb < NS; ++sb)
#pragma unroll
                    for (int s = 0; s < KS; s += 2) {
                        uint32_t w[4];
                        ldsm_x4_t(vs + piece_at<SUB, C::CHB>(16 * sb + r16, s + half), w);
                        uint32_t af[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            half_codes(__byte_perm(w[2 * h], 0, pick[2 * sb]), af[h][0], af[h][1]);
                            half_codes(__byte_perm(w[2 * h + 1], 0, pick[2 * sb + 1]), af[h][2], af[h][3]);
                        }
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) mma16816(o[nb][s + h], af[h], ph[sb][nb][0], ph[sb][nb][1]);
                            if (!QUAD) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) mma16816(o[nb][s + h], af[h], plo[sb][nb][0], plo[sb][nb][1]);
                            }
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
        if (QUAD) {
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[0][s][i] += __shfl_xor_sync(0xffffffffu, o[0][s][i], 2);
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
            // the warp's own: the result, or a partial. Lane: columns 2 lc + i, elements 16 s + 2 lg and + 1.
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int lh = nb * 8 + 2 * lc + i;
                    if (lh >= nq) continue;
                    if (whole) {
                        const int64_t row = row_of(lh);
                        const RowEnd r = row_end(P, row, m[nb][i], l[nb][i]);
                        uint32_t* out = static_cast<uint32_t*>(P.O) + (row * D >> 1) + lg;
                        const float* op = P.O_prior + row * D + 2 * lg;
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            float a0 = o[nb][s][i] * r.wo, a1 = o[nb][s][2 + i] * r.wo;
                            if (r.prior) {
                                const float2 f = *reinterpret_cast<const float2*>(op + 16 * s);
                                a0 = fmaf(f.x, r.wp, a0);
                                a1 = fmaf(f.y, r.wp, a1);
                            }
                            out[8 * s] = pack_out(P.dtype, a0, a1);
                        }
                        if (lane < 4 && P.LSE) P.LSE[row] = r.lse;
                    } else {
                        float* pr = part + lh * (D + 4);
#pragma unroll
                        for (int s = 0; s < KS; ++s)
                            *reinterpret_cast<float2*>(pr + 4 + 16 * s + 2 * lg) = make_float2(o[nb][s][i], o[nb][s][2 + i]);
                        if (lane < 4) *reinterpret_cast<float2*>(pr) = make_float2(m[nb][i], l[nb][i]);
                    }
                }
        } else {
            // the CTA's warps join: maxima and sums first, then O in JP parts of D per column block (one copy of the code that sums:
            // a call on a short cache runs it once, and spends its time fetching it)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (lane < 4) {
                        s_m[warp * 16 + nb * 8 + 2 * lane + i] = m[nb][i];
                        s_l[warp * 16 + nb * 8 + 2 * lane + i] = l[nb][i];
                    }
            __syncthreads();
            constexpr int DP = D / C::JP, KP = KS / C::JP;
            constexpr int COPIES = NB == 1 ? 1 : NB * C::JP;         // (rolled up, two column blocks of O would go through memory)
#pragma unroll COPIES
            for (int part_i = 0; part_i < NB * C::JP; ++part_i) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if (part_i / C::JP != nb || (QUAD && lc >= 2)) continue;
                    float al[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float M = M_NONE;
#pragma unroll
                        for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * 16 + nb * 8 + 2 * lc + i]);
                        al[i] = ex2_approx(m[nb][i] - M);
                    }
                    float* row = jbuf + (warp * C::JC + 2 * lc) * C::JROW + 2 * lg;
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        if (part_i % C::JP != s / KP) continue;
                        const float (&v)[4] = o[nb][s];
                        *reinterpret_cast<float2*>(row + 16 * (s % KP)) = make_float2(v[0] * al[0], v[2] * al[0]);
                        *reinterpret_cast<float2*>(row + C::JROW + 16 * (s % KP)) = make_float2(v[1] * al[1], v[3] * al[1]);
                    }
                }
                __syncthreads();
#pragma unroll 1
                for (int i = tid; i < C::JC * (DP / 2); i += NT) {   // (column, pair of elements)
                    const int h = i / (DP / 2), d = 2 * (i - h * (DP / 2));
                    const int lh = part_i / C::JP * 8 + h;
                    if (lh < nq) {
                        float M = M_NONE, L = 0.f;
#pragma unroll
                        for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * 16 + lh]);
                        float a0 = 0.f, a1 = 0.f;
#pragma unroll
                        for (int w = 0; w < NW; ++w) {
                            L += s_l[w * 16 + lh] * ex2_approx(s_m[w * 16 + lh] - M);
                            const float2 f = *reinterpret_cast<const float2*>(jbuf + (w * C::JC + h) * C::JROW + d);
                            a0 += f.x;
                            a1 += f.y;
                        }
                        const int dd = part_i % C::JP * DP + d;
                        if (!SPLIT || whole) {
                            finish8(P, row_of(lh), D, dd, a0, a1, M, L, dd == 0);
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
        u = pe;
    }
    if (SPLIT && !crosses && (BY_WARP ? lane == 0 : tid == 0)) jd[worker].pieces = 0;
    if (failed) {
        set_err(P.err, ERR_PAGED_TOKEN);
        for (k = k_failed; k < kp; ++k)   // copies still in flight, waited for with the same limit
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar + 8 * (k % ST), (k / ST) & 1))) break;
    }
}

// Joins the partials of split items: a warp per (range in which one begins, column). Most ranges of a ragged batch begin
// none or one of two or three pieces, so a CTA for each (the 16-bit kernel's way) is mostly CTAs that look and leave: 64 ragged sequences in
// 2,432 ranges of 4 columns took 12 us from the last range's end to the next call.
template <int D>
__global__ void __launch_bounds__(256) paged_token8_join_kernel(const __grid_constant__ PagedAttn P, int ranges) {
    constexpr int V = D >= 128 ? 4 : 2, NV = (D + 32 * V - 1) / (32 * V);   // floats of a lane's load, and loads of a row
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31, cols = P.cols, heads = P.heads_per_group;
    const int id = blockIdx.x * 8 + (threadIdx.x >> 5), c = id / cols, h = id - c * cols;
    if (c >= ranges) return;
    const JoinDesc d = reinterpret_cast<const JoinDesc*>(P.ws + (size_t)2 * ranges * slot_floats(D, cols))[c];
    if (d.pieces == 0) return;
    const int g = d.x / P.n_groups, grp = d.x - g * P.n_groups;
    const int nh = min(heads, P.G - grp * heads);
    if (h >= nh * d.rows) return;
    const int64_t row = (int64_t)(d.r0 + h / nh) * P.H_q + g * P.G + grp * heads + h % nh;
    // piece i: slot 2 c + 1 for the first, 2 (c + i) for the others
    auto part = [&](int i) { return P.ws + (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * slot_floats(D, cols) + h * (D + 4); };
    float M = M_NONE;
    for (int i = lane; i < d.pieces; i += 32) M = fmaxf(M, part(i)[0]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    for (int i = lane; i < d.pieces; i += 32) {
        const float2 ml = *reinterpret_cast<const float2*>(part(i));
        L += ml.y * ex2_approx(ml.x - M);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float acc[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[j][i] = 0.f;
#pragma unroll 4
    for (int i = 0; i < d.pieces; ++i) {
        const float* p = part(i);
        const float w = ex2_approx(p[0] - M);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = (j * 32 + lane) * V;
            if (D % (32 * V) && at >= D) continue;
#pragma unroll
            for (int q = 0; q < V; q += 2) {
                const float2 v = *reinterpret_cast<const float2*>(p + 4 + at + q);
                acc[j][q] = fmaf(w, v.x, acc[j][q]);
                acc[j][q + 1] = fmaf(w, v.y, acc[j][q + 1]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int at = (j * 32 + lane) * V;
        if (D % (32 * V) && at >= D) continue;
#pragma unroll
        for (int q = 0; q < V; q += 2) finish8(P, row, D, at + q, acc[j][q], acc[j][q + 1], M, L, at + q == 0);
    }
}

template <int D, int NBQ, int MODE, bool ROWS>
cudaError_t launch8_t(PagedAttn& p, cudaStream_t st) {
    using C = TCfg8<D, MODE, NBQ == 0>;
    constexpr bool SPLIT = is_split(MODE);
    static_assert(C::SMEM_BASE + 4 * (TK_MAX_B + 1) <= 232448, "one CTA's shared memory");
    const cudaError_t e0 = allow_smem<paged_token8_kernel<D, NBQ, MODE, ROWS>>(C::SMEM_BASE + 4 * (TK_MAX_B + 1), p.device);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_token8_kernel<D, NBQ, MODE, ROWS>, p);
    if (e != cudaSuccess || !SPLIT) return e;
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    if (MODE != TK_CTA) {
        const int ranges = p.n_ctas * (MODE == TK_WARP ? C::NW : 1);
        cfg.gridDim = dim3((ranges * p.cols + 7) / 8);
        return cudaLaunchKernelEx(&cfg, paged_token8_join_kernel<D>, p, ranges);
    }
    // few items, each in many pieces: a CTA per (range, column), its threads over the pieces (one cache of 131k tokens 48.4 us, with a
    // warp per range and column 51.2; 2000 tokens 10.8 against 11.4)
    cfg.gridDim = dim3(p.n_ctas, p.cols, 1);
    return p.dtype == PCK_DT_F16 ? cudaLaunchKernelEx(&cfg, paged_token_join_kernel<__half, D>, p)
                                 : cudaLaunchKernelEx(&cfg, paged_token_join_kernel<__nv_bfloat16, D>, p);
}

template <int D, int NBQ, bool ROWS>
cudaError_t launch8_m(PagedAttn& p, cudaStream_t st) {
    return p.mode == TK_WARP  ? launch8_t<D, NBQ, TK_WARP, ROWS>(p, st)
           : p.mode == TK_CTA_HALF ? launch8_t<D, NBQ, TK_CTA_HALF, ROWS>(p, st)
           : p.mode == TK_CTA ? launch8_t<D, NBQ, TK_CTA, ROWS>(p, st)
           : p.mode == TK_ITEM_HALF ? launch8_t<D, NBQ, TK_ITEM_HALF, ROWS>(p, st)
                              : launch8_t<D, NBQ, TK_ITEM, ROWS>(p, st);
}
template <int D, int NBQ>
cudaError_t launch8_s(PagedAttn& p, cudaStream_t st) {
    return p.cu_rows ? launch8_m<D, NBQ, true>(p, st) : launch8_m<D, NBQ, false>(p, st);
}

template <int D>
cudaError_t launch8_d(PagedAttn& p, cudaStream_t st) {
    if (p.cols <= 4) return launch8_s<D, 0>(p, st);
    if constexpr (D <= 128)
        if (p.cols > 8) return launch8_s<D, 2>(p, st);
    return launch8_s<D, 1>(p, st);
}

}  // namespace
}  // namespace pck
