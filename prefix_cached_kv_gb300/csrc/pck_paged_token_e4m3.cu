// pck_paged_token_e4m3.cu -- attention of one new token (or a few) per sequence over a quantised paged cache.
//
// With codes c and scales 2^ek, 2^ev of each token and kv head (pck_paged_e4m3.cuh), tau' = tau log2 e:
//   s_j = 2^ek_j tau' (q . c_j),  O = sum_j 2^(s_j - m) 2^ev_j c'_j / l,  l = sum_j 2^(s_j - m),  LSE = (m + log2 l) ln 2.
// Codes are exact in fp16, so both products run on fp16 MMAs with fp32 sums and the scales never touch the operands: 2^ek
// multiplies a token's finished scores and 2^ev its weights. D + 1 bytes a head row are read once: half of a 16-bit
// cache's, so HBM still bounds it, with half the time a byte for everything else. How a call is cut into ranges of units, and
// the kernel that joins them, are the 16-bit cache's (pck_paged_token_impl.cuh); here is what differs:
//  * A unit is 32 tokens of a kv head (16 at D > 128), so its two code tiles are as large as the 16-bit kernel's and a copy
//    moves as much. Pages that are multiples of 32 give a unit with one box of K, one of V and two short copies of scales;
//    other pages (multiples of 16) with two of each, which may lie in different pages.
//  * Operands: a 16-byte row piece of a code tile holds 16 elements, so one ldmatrix.x4 fetches 16 tokens x 32 elements. Lane
//    (g, c) gets elements 4c .. 4c+3 of token g; as the MMA's k index only pairs K with q, they are its k = 2c, 2c+1, 2c+8,
//    2c+9, and q is loaded in that order. V comes through the transposing ldmatrix in pairs of elements: bytes (2g, 2g+1) of
//    tokens 2c and 2c+1, which one byte permutation turns into (tokens 2c, 2c+1) of element 2g and of 2g+1: rows g and g+8
//    of an MMA whose rows are elements in that order. One conversion makes two fp16 values.
//  * q: fp16 as it is; a bf16 row is moved by a power of two so that its largest element is 2^14 .. 2^15 and then exact in fp16
//    but for elements 2^-29 of that one and less, which are held to 2^-39 of it.
//  * The maximum is that of s + ev (a token's largest possible share of O), so that a weight times its scale fits fp16: it
//    enters the second MMA as a pair hi + lo, held to 2^-37 of the largest. ev counts from EV_LOW up in this, which keeps
//    l within fp32.
#include "pck_paged_e4m3.cuh"
#include "pck_paged_token_impl.cuh"

namespace pck {
namespace {

constexpr float EV_LOW = -40.f;      // values of V below 2^-40 * 448 lose bits where no larger ones are seen
__host__ __device__ constexpr int warps_sm8(int D, int mode) { return D == 64 && mode != TK_CTA && mode != TK_CTA_HALF ? 16 : 8; }
// Units of an item up to which it gets a CTA (1024 tokens).
__host__ __device__ constexpr int sub8(int D) { return D <= 128 ? 32 : 16; }     // tokens of a unit
__host__ __device__ constexpr int direct_units8(int D) { return 1024 / sub8(D); }

template <int D, int MODE>
struct TCfg8 {
    static constexpr int SUB = sub8(D);
    static constexpr int CHB = D % 128 == 0 ? 128 : 64;           // bytes of a row that lie together: the swizzle's width
    static constexpr int NW = warps_sm8(D, MODE) / per_sm(MODE);  // warps per CTA
    static constexpr int UNIT = SUB * D;                          // bytes of a K (or V) unit
    static constexpr int STAGE = 2 * UNIT;
    static constexpr int ST = 196608 / warps_sm8(D, MODE) / STAGE;
    static constexpr int RING = NW * ST * STAGE;
    static constexpr int JP = D > 128 ? 4 : 2;                    // parts in which O is joined
    static constexpr int JROW = D / JP + 4;                       // floats of a join row (padded)
    static constexpr int OFF_SC = RING;                           // [NW][ST][64]: scale bytes of K, then of V
    static constexpr int OFF_JOIN = OFF_SC + NW * ST * 64;
    static constexpr int OFF_ML = OFF_JOIN + NW * 8 * JROW * 4;   // [NW][16] m, then l
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

template <int D, int NB, int MODE, bool ROWS>
__global__ void __launch_bounds__(TCfg8<D, MODE>::NW * 32, per_sm(MODE)) paged_token8_kernel(const __grid_constant__ PagedAttn P) {
    using C = TCfg8<D, MODE>;
    constexpr int NW = C::NW, ST = C::ST, KS = D / 16, NT = NW * 32, SUB = C::SUB, NS = SUB / 16;
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
    const uint8_t* s_sc = smem + C::OFF_SC + warp * ST * 64;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(bar + 8 * i, 1);
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.tm_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.tm_v) : "memory");
    }
    pdl_wait();
    pdl_release();
    fence_proxy_async_all();     // the pages may have been written by the kernel before, and are read by TMA

    const int Hg = P.H_kv * P.n_groups;
    const int heads = P.heads_per_group, cols = P.cols;
    constexpr bool SPLIT = is_split(MODE), BY_WARP = MODE == TK_WARP;
    constexpr int TK_ITEM_UNITS = tk_item_units(MODE);
    const int worker = BY_WARP ? warp * gridDim.x + blockIdx.x : blockIdx.x;    // few workers spread over the SMs
    int workers = BY_WARP ? gridDim.x * NW : gridDim.x;
    JoinDesc* jd = reinterpret_cast<JoinDesc*>(P.ws + (size_t)2 * workers * slot_floats(D, cols));
    const Cut cut = cut_units<NW, MODE, ROWS, SUB>(P, worker, workers, s_scan, pre);
    if (SPLIT && cut.idle) {
        if (BY_WARP ? lane == 0 : tid == 0) jd[worker].pieces = 0;
        return;
    }
    const int64_t u0 = cut.u0, u1 = cut.u1, U = cut.U;
    workers = cut.workers;
    const int b_first = cut.b_first;
    const int nseq = SPLIT ? P.B : 1;     // sequences in pre[]

    // ---- a warp's units: u0 + k of its own range, u0 + warp + k NW of its CTA's. Lane i resolves unit k0 + i: coordinates of
    // its loads (of both halves of 16 tokens where pages are no multiples of a unit)
    const int64_t uf = BY_WARP ? u0 : u0 + warp;
    constexpr int STEP = BY_WARP ? 1 : NW;
    const uint64_t pol = l2_evict_first();
    int pl_head = 0, pl_tok[NS] = {}, pl_page[NS] = {};
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
            const Span s = span_of<SUB>(len, rows, P.window, P.sinks);
            const int tok0 = (j < s.ns ? j : j - s.ns + s.w0) * SUB;
            const int lo0 = P.window > 0 ? len - rows + 1 - P.window : 0;    // first key of the first row's window
            pl_head = x / P.n_groups;
#pragma unroll
            for (int h = 0; h < NS; ++h) {
                if (h > 0 && !P.halves) break;
                const int tok = tok0 + 16 * h, pi = tok / P.page;
                pl_tok[h] = tok - pi * P.page;
                pl_page[h] = 0;
                // a half that no row sees is not looked up (its page may not exist): the first page is read in its place
                const bool seen = !P.halves || (tok < len && (tok + 16 > lo0 || tok < P.sinks));
                if (len > 0 && rows > 0 && pi < P.max_pages && seen) {
                    const int pg = P.table[(int64_t)b * P.max_pages + pi];
                    if (pg < 0 || pg >= P.n_pages) set_err(P.err, ERR_PAGE_ID);   // and page 0 is read instead
                    else pl_page[h] = pg;
                }
            }
        }
    };
    const int nk = static_cast<int>(u1 > uf ? (u1 - uf + STEP - 1) / STEP : 0);   // units of this warp
    int kp = 0;                          // next unit to load
    auto produce = [&]() {
        if (kp >= nk) return;
        if ((kp & 31) == 0) resolve(kp);
        const int head = __shfl_sync(0xffffffffu, pl_head, kp & 31);
        const int st = kp % ST;
        const uint32_t b = bar + 8 * st, dst = ring + st * C::STAGE, sc = s_base + C::OFF_SC + (warp * ST + st) * 64;
        if (lane == 0) mbar_arrive_expect_tx(b, C::STAGE + 2 * SUB);
#pragma unroll
        for (int h = 0; h < NS; ++h) {
            if (h > 0 && !P.halves) break;
            const int tok = __shfl_sync(0xffffffffu, pl_tok[h], kp & 31);
            const int page = __shfl_sync(0xffffffffu, pl_page[h], kp & 31);
            if (lane == 0) {
                const uint32_t at = h * 16 * C::CHB;       // (a unit of two halves has one chunk: D <= 128)
                tma_5d(dst + at, &P.tm_k, tok, head, page, b, pol);
                tma_5d(dst + C::UNIT + at, &P.tm_v, tok, head, page, b, pol);
                const int64_t so = ((int64_t)page * P.H_kv + head) * P.page + tok;
                const uint32_t bytes = P.halves ? 16 : SUB;
                bulk_g2s(sc + 16 * h, P.k_scale + so, bytes, b);
                bulk_g2s(sc + 32 + 16 * h, P.v_scale + so, bytes, b);
            }
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
            const int key0 = tile * SUB;
            const bool full = key0 + SUB - 1 <= p0 && (key0 >= lo1 || key0 + SUB <= P.sinks);
            bool spoilt = false;
            if (!full) {
                // V rows hidden from every column may hold anything (also NaN, which 0 * v would keep): zero them
                for (int t = 0; t < SUB; ++t)
                    if (key0 + t >= len || (key0 + t < lo0 && key0 + t >= P.sinks))
                        for (int c = lane; c < KS; c += 32)
                            *reinterpret_cast<uint4*>(smem + (vs - s_base) + piece_at<SUB, C::CHB>(t, c)) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                // one that some rows see and others do not, and that holds a NaN, must not reach those others
                if (ROWS && rs.n > 1) {
                    bool bad = false;
                    for (int c = lane; c < SUB * KS; c += 32) bad |= nan_codes(*reinterpret_cast<const uint4*>(smem + (vs - s_base) + c * 16));
                    spoilt = __any_sync(0xffffffffu, bad);
                }
            }
            // the scales of the lane's tokens 8 r + lg
            float sk[2 * NS], sv[2 * NS], ev[2 * NS];
#pragma unroll
            for (int r = 0; r < 2 * NS; ++r) {
                sk[r] = scale_up(s_sc[st * 64 + 8 * r + lg]);
                const uint32_t v = s_sc[st * 64 + 32 + 8 * r + lg];
                sv[r] = scale_up(v);
                ev[r] = fmaxf(static_cast<float>(static_cast<int>(v) - 127), EV_LOW);
            }
            // S^T = K q^T
            const int r16 = lane & 15, half = lane >> 4;
            float s4[NS][NB][4];
#pragma unroll
            for (int sb = 0; sb < NS; ++sb) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s4[sb][nb][i] = 0.f;
#pragma unroll
                for (int s = 0; s < KS; s += 2) {
                    uint32_t w[4];
                    ldsm_x4(ks + piece_at<SUB, C::CHB>(16 * sb + r16, s + half), w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t af[4];
                        half_codes(w[2 * h], af[0], af[2]);
                        half_codes(w[2 * h + 1], af[1], af[3]);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma16816(s4[sb][nb], af, qf[nb][s + h][0], qf[nb][s + h][1]);
                    }
                }
            }
            // lane: tokens 8 r + lg, columns 2 lc and + 1 of each column block
            bool up = false;
#pragma unroll
            for (int sb = 0; sb < NS; ++sb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 2 * sb + (i >> 1);
                        float v = s4[sb][nb][i] * (sk[r] * qs[nb][i & 1]);
                        if (!full) {
                            const int key = key0 + 8 * r + lg, p = pos[nb][i & 1];
                            if (key > p || (P.window > 0 && key <= p - P.window && key >= P.sinks)) v = -INFINITY;
                        }
                        s4[sb][nb][i] = v;
                        up |= !(v + ev[r] <= m[nb][i & 1] + Elem<__half>::CAP);   // (a NaN too)
                    }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int r = 0; r < 2 * NS; ++r) mx = fmaxf(mx, s4[r >> 1][nb][2 * (r & 1) + i] + ev[r]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        mx = fmaxf(mx - Elem<__half>::TOP, m[nb][i]);
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
            // p, its sum, and the weights' transpose (tokens as k) as hi + lo B fragments
            uint32_t ph[NS][NB][2], plo[NS][NB][2];
#pragma unroll
            for (int sb = 0; sb < NS; ++sb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float v = s4[sb][nb][2 * r + i];
                            const float p = ex2_approx(v - (m[nb][i] > -INFINITY ? m[nb][i] : 0.f));
                            l[nb][i] += p;
                            w[i] = p * sv[2 * sb + r];
                            if (!full && v == -INFINITY) w[i] = 0.f;     // (the scale of a hidden token may be anything)
                            if (ROWS && spoilt) s4[sb][nb][2 * r + i] = w[i];
                        }
                        uint32_t hi, lo;
                        split_hi_lo(w[0], w[1], hi, lo);
                        ph[sb][nb][r] = movmatrix_trans(hi);
                        plo[sb][nb][r] = movmatrix_trans(lo);
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
                            for (int i = 0; i < 2; ++i) w[nb][i] = __shfl_sync(0xffffffffu, s4[r >> 1][nb][2 * (r & 1) + i], t8 * 4 + lc);
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
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t af[4];
                            half_codes(__byte_perm(w[2 * h], 0, 0x3120), af[0], af[1]);
                            half_codes(__byte_perm(w[2 * h + 1], 0, 0x3120), af[2], af[3]);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                mma16816(o[nb][s + h], af, ph[sb][nb][0], ph[sb][nb][1]);
                                mma16816(o[nb][s + h], af, plo[sb][nb][0], plo[sb][nb][1]);
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
            // the CTA's warps join: maxima and sums first, then O in JP parts of D per column block
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
                    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * 16 + nb * 8 + 2 * lc + i]);
                    al[i] = join_weight(m[nb][i], M);
                }
                constexpr int DP = D / C::JP, KP = KS / C::JP;
#pragma unroll
                for (int hf = 0; hf < C::JP; ++hf) {
                    float* row = jbuf + (warp * 8 + 2 * lc) * C::JROW + 2 * lg;
#pragma unroll
                    for (int s = 0; s < KP; ++s) {
                        const float (&v)[4] = o[nb][hf * KP + s];
                        *reinterpret_cast<float2*>(row + 16 * s) = make_float2(v[0] * al[0], v[2] * al[0]);
                        *reinterpret_cast<float2*>(row + C::JROW + 16 * s) = make_float2(v[1] * al[1], v[3] * al[1]);
                    }
                    __syncthreads();
                    for (int i = tid; i < 8 * (DP / 2); i += NT) {   // (column, pair of elements)
                        const int h = i / (DP / 2), d = 2 * (i - h * (DP / 2));
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
                            const int dd = hf * DP + d;
                            if (!SPLIT || whole) {
                                if (P.dtype == PCK_DT_F16) finish2<__half>(P, row_of(lh), D, dd, a0, a1, M, L, dd == 0);
                                else finish2<__nv_bfloat16>(P, row_of(lh), D, dd, a0, a1, M, L, dd == 0);
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

template <int D, int NB, int MODE, bool ROWS>
cudaError_t launch8_t(PagedAttn& p, cudaStream_t st) {
    using C = TCfg8<D, MODE>;
    constexpr bool SPLIT = is_split(MODE);
    static_assert(C::SMEM_BASE + 4 * (TK_MAX_B + 1) <= 232448, "one CTA's shared memory");
    const cudaError_t e0 = allow_smem<paged_token8_kernel<D, NB, MODE, ROWS>>(C::SMEM_BASE + 4 * (TK_MAX_B + 1), p.device);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_token8_kernel<D, NB, MODE, ROWS>, p);
    if (e != cudaSuccess || !SPLIT) return e;
    cfg.gridDim = dim3(p.n_ctas, p.cols, MODE == TK_WARP ? C::NW : 1);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return p.dtype == PCK_DT_F16 ? cudaLaunchKernelEx(&cfg, paged_token_join_kernel<__half, D>, p)
                                 : cudaLaunchKernelEx(&cfg, paged_token_join_kernel<__nv_bfloat16, D>, p);
}

template <int D, int NB, bool ROWS>
cudaError_t launch8_m(PagedAttn& p, cudaStream_t st) {
    return p.mode == TK_WARP  ? launch8_t<D, NB, TK_WARP, ROWS>(p, st)
           : p.mode == TK_CTA_HALF ? launch8_t<D, NB, TK_CTA_HALF, ROWS>(p, st)
           : p.mode == TK_CTA ? launch8_t<D, NB, TK_CTA, ROWS>(p, st)
           : p.mode == TK_ITEM_HALF ? launch8_t<D, NB, TK_ITEM_HALF, ROWS>(p, st)
                              : launch8_t<D, NB, TK_ITEM, ROWS>(p, st);
}
template <int D, int NB>
cudaError_t launch8_s(PagedAttn& p, cudaStream_t st) {
    return p.cu_rows ? launch8_m<D, NB, true>(p, st) : launch8_m<D, NB, false>(p, st);
}

}  // namespace

bool paged_token_e4m3_halves(int D, int page) { return page % sub8(D) != 0; }
int paged_token_e4m3_box(int D, int page) { return paged_token_e4m3_halves(D, page) ? 16 : sub8(D); }

// How a call is cut: as the 16-bit cache's (paged_token_plan), in this kernel's units.
size_t paged_token_e4m3_plan(PagedAttn& p, int D, int sms) {
    const int most = paged_token_cols(D), sub = sub8(D);
    const int rows = p.cu_rows ? p.max_rows : 1;
    p.n_groups = (p.G * rows + most - 1) / most;       // 1 with more than one row
    p.heads_per_group = (p.G + p.n_groups - 1) / p.n_groups;
    p.cols = p.heads_per_group * rows;
    p.halves = paged_token_e4m3_halves(D, p.page);
    int64_t bound = ((int64_t)p.max_pages * p.page + sub - 1) / sub;       // units of one item
    int64_t direct = direct_units8(D);
    if (p.window > 0) {
        const int64_t edges = 1 + ((int64_t)p.sinks + sub - 1) / sub;      // units beside the window's own
        const int64_t w = ((int64_t)p.window + rows + sub - 1) / sub + edges;
        if (w < bound) {
            bound = w;
            direct += 1 + (edges < 8 ? edges : 8);      // (a window of 1024 tokens has as many units in the middle)
        }
    }
    const int64_t items = (int64_t)p.B * p.H_kv * p.n_groups;
    const bool spread = items > sms;                    // more than one item per SM
    p.mode = items > (int64_t)TK_FEW_ITEMS * sms ? TK_WARP
             : bound <= direct                   ? (spread ? TK_ITEM_HALF : TK_ITEM)
                                                 : (spread ? TK_CTA_HALF : TK_CTA);
    p.n_ctas = is_split(p.mode) ? sms * per_sm(p.mode) : static_cast<int>(items);
    const size_t ranges = is_split(p.mode) ? (size_t)p.n_ctas * (p.mode == TK_WARP ? warps_sm8(D, TK_WARP) : 1) : 0;
    return ranges * (2 * slot_floats(D, p.cols) * sizeof(float) + sizeof(JoinDesc));
}

cudaError_t launch_paged_token_e4m3(PagedAttn& p, int D, cudaStream_t st) {
    const bool two = p.cols > 8;
    switch (D) {
        case 64: return two ? launch8_s<64, 2>(p, st) : launch8_s<64, 1>(p, st);
        case 128: return two ? launch8_s<128, 2>(p, st) : launch8_s<128, 1>(p, st);
        case 192: return launch8_s<192, 1>(p, st);
        case 256: return launch8_s<256, 1>(p, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pck
