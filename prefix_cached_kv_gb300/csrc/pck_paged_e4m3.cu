// pck_paged_e4m3.cu -- the append to a quantised paged cache, and rows of that cache read back.
//
// The append: y = rope(x * rsqrt(mean(x^2) + eps) * w) for q and k, v as it is (pck_paged_rope_impl.cuh), all in fp32; q is rounded
// to its type; a k or v head row becomes codes and one exponent byte: with a = max |y| over the finite elements, the least e with
// a 2^-e <= 448 (e held to -126 .. 120) and codes rn(y 2^-e). A shift of exponents rounds nothing, so a code is y's one
// rounding. HBM bounds it. Rows are held as in the 16-bit append (D/16 lanes, two vectors of 8), with a loop of its own per kind of
// head, packed fp32 arithmetic, and each lane's next heads on their way into shared memory by asynchronous copies: a thread goes
// through a dozen heads, each a round trip to memory, and more of them in registers cost the warps that would hide them. 8
// ragged prompts, 32 + 8 + 8 heads of 128: 61.5 us as the 16-bit kernel with another store (two heads in registers, 65 % of the issue slots),
// 61.4 with a loop per kind and packed arithmetic, 50.5 with the copies, at three blocks an SM; four blocks spill (62), two 57.
//
// Reading back: out = code * 2^e, rounded once to the output's type (fp32 holds it exactly below 2^128, bf16 for e of -124 .. 119; in fp16
// what is beyond 65,504 becomes 65,504). D + 1 bytes in and 2 D or 4 D out per row, so HBM bounds it. A warp takes tiles of 16 tokens of one kv
// head, K and V: 8 codes a lane, so that its 16-byte stores lie side by side, with DEPTH loads of K and of V in flight before the
// first is used: 6.1 TB/s read and written on the long sessions (0.90 of a copy).
// The tiles of all sequences laid end to end are dealt to the warps from the lengths on the device (one block scan), so
// one long session and many short ones fill the GPU alike.
#include <type_traits>

#include "pck_paged_e4m3.cuh"
#include "pck_paged_rope_impl.cuh"

namespace pck {
namespace {

// ---------------------------------------------------------------- append

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{ .reg .b64 x, y, w, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 w, {%6, %7}; fma.rn.f32x2 z, x, y, w; mov.b64 {%0, %1}, z; }"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Codes of 8 values times `down`.
__device__ __forceinline__ void store_codes(uint8_t* p, const float2 (&x)[4], float2 down) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = mul2(x[i], down);
        w[i] = codes2(y.x, y.y);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

template <typename TI>
__device__ __forceinline__ void unpack8(const typename Vec8<TI>::Raw& r, float2 (&x)[4]) {
    float f[8];
    Vec8<TI>::unpack(r, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(f[2 * i], f[2 * i + 1]);
}

// Blocks per SM, and heads whose copies a lane has in flight.
constexpr int A8_BLOCKS = 3;
template <typename TI> __host__ __device__ constexpr int a8_depth() { return sizeof(TI) == 4 ? 2 : 3; }

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <typename TI, int L>
__global__ void __launch_bounds__(NR_THREADS, A8_BLOCKS) append8_kernel(const __grid_constant__ RopeParams P) {
    typedef typename Vec8<TI>::Raw Raw;
    constexpr int SUBS = NR_THREADS / L;
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    const int64_t t64 = (int64_t)blockIdx.x * (SUBS / P.spt) + sub / P.spt;
    const uint32_t mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31) / L * L);
    if (t64 >= P.T) return;
    const int t = static_cast<int>(t64), h0 = sub % P.spt;
    if (h0 >= P.q.H + P.k.H + P.v.H) return;
    // rows in front of the first sequence and behind the last are not read: they need not exist
    const bool owned = !P.cu_rows || (t >= P.cu_rows[0] && t < P.cu_rows[P.B]);
    const bool active = lane < P.D / 16;
    const int rv = P.R / 16;
    const bool rot = lane < rv;
    const int s0 = rot ? lane : P.R / 8 + (lane - rv);            // the lane's two vectors
    const int s1 = rot ? lane + rv : s0 + (P.D - P.R) / 16;
    // The thread's heads, those of all kinds one behind the other: its n-th is h0 + n spt. Each lane copies its two vectors of the
    // next DEPTH of them into shared memory, the first while the row's sequence, page and angles are looked up one after another.
    constexpr int DEPTH = a8_depth<TI>();
    __shared__ __align__(16) Raw ring[NR_THREADS / 32][DEPTH][2][32];
    Raw(*mine)[2][32] = ring[threadIdx.x >> 5];
    const int in_warp = threadIdx.x & 31, Hqk = P.q.H + P.k.H, Ht = Hqk + P.v.H;
    int next = owned ? h0 : Ht, put = 0, get = 0;
    const auto fetch = [&]() {
        if (next < Ht && active) {
            const RowsArg& A = next < P.q.H ? P.q : next < Hqk ? P.k : P.v;
            const int h = next - (next < P.q.H ? 0 : next < Hqk ? P.q.H : Hqk);
            const TI* src = static_cast<const TI*>(A.in) + (int64_t)t * A.in_row + (int64_t)h * A.in_head;
#pragma unroll
            for (int i = 0; i < (int)sizeof(Raw); i += 16) {
                copy16(reinterpret_cast<uint8_t*>(&mine[put][0][in_warp]) + i, reinterpret_cast<const uint8_t*>(src + 8 * s0) + i);
                copy16(reinterpret_cast<uint8_t*>(&mine[put][1][in_warp]) + i, reinterpret_cast<const uint8_t*>(src + 8 * s1) + i);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        next += P.spt;
        put = put + 1 == DEPTH ? 0 : put + 1;
    };
#pragma unroll 1
    for (int i = 0; i < DEPTH; ++i) fetch();
    RowPlace at = {};
    float co[8], si[8];
    // (a cu_rows that makes no sense, which place_row reports, may place a row that is not owned)
    if (!place_row<TI, L>(P, t, lane, mask, h0, at) || !owned || (P.R > 0 && !load_angles(P, t, lane, at.pos, rot, s0, s1, co, si))) {
        asm volatile("cp.async.wait_all;" ::: "memory");         // the copies land before the block can end
        return;
    }

    // KIND 0: q, 1: k, 2: v. The heads of all kinds one behind the other are dealt to the token's subwarps in turn.
    const auto heads = [&](auto kind, const RowsArg& A, int first) {
        constexpr int KIND = decltype(kind)::value;
        Raw w0 = Raw{}, w1 = Raw{};
        const bool norm = KIND != 2 && A.norm, weight = norm && A.w;
        if (weight && active && first < A.H) {
            w0 = *reinterpret_cast<const Raw*>(static_cast<const TI*>(A.w) + 8 * s0);
            w1 = *reinterpret_cast<const Raw*>(static_cast<const TI*>(A.w) + 8 * s1);
        }
#pragma unroll 1
        for (int h = first; h < A.H; h += P.spt) {
            float2 x[4], y[4];
            asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
            unpack8<TI>(active ? mine[get][0][in_warp] : Raw{}, x);
            unpack8<TI>(active ? mine[get][1][in_warp] : Raw{}, y);
            get = get + 1 == DEPTH ? 0 : get + 1;
            fetch();          // into the place just read
            if (norm) {
                float2 ss = mul2(x[0], x[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) ss = fma2(x[i], x[i], ss);
#pragma unroll
                for (int i = 0; i < 4; ++i) ss = fma2(y[i], y[i], ss);
                float sum = ss.x + ss.y;
#pragma unroll
                for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(mask, sum, o, L);
                const float r = rsqrtf(sum * P.inv_d + P.eps);
                const float2 rr = make_float2(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = mul2(x[i], rr);
                    y[i] = mul2(y[i], rr);
                }
                if (weight) {
                    float2 u[4], v[4];
                    unpack8<TI>(w0, u);
                    unpack8<TI>(w1, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = mul2(x[i], u[i]);
                        y[i] = mul2(y[i], v[i]);
                    }
                }
            }
            if (KIND != 2 && rot) {
                if (P.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 a = x[i], b = y[i];
                        x[i] = make_float2(a.x * co[i] - a.y * si[i], a.y * co[i] + a.x * si[i]);
                        y[i] = make_float2(b.x * co[4 + i] - b.y * si[4 + i], b.y * co[4 + i] + b.x * si[4 + i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 c = make_float2(co[2 * i], co[2 * i + 1]), s = make_float2(si[2 * i], si[2 * i + 1]);
                        const float2 a = x[i], b = y[i], nb = make_float2(-b.x, -b.y);
                        x[i] = fma2(nb, s, mul2(a, c));
                        y[i] = fma2(a, s, mul2(b, c));
                    }
                }
            }
            if (KIND == 0) {
                if (!active) continue;
                float f[8], g[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = x[i].x;
                    f[2 * i + 1] = x[i].y;
                    g[2 * i] = y[i].x;
                    g[2 * i + 1] = y[i].y;
                }
                TI* dst = static_cast<TI*>(A.out) + (int64_t)t * A.out_row + (int64_t)h * A.out_head;
                Vec8<TI>::store(dst + 8 * s0, f);
                Vec8<TI>::store(dst + 8 * s1, g);
                continue;
            }
            const auto largest = [&]() {               // (fmaxf passes over NaN)
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a = fmaxf(a, fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(y[i].x), fabsf(y[i].y))));
#pragma unroll
                for (int o = L / 2; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(mask, a, o, L));
                return a;
            };
            float a = largest();
            if (a == INFINITY) {                       // e4m3 has no infinity: those elements become NaN, the scale is the others'
                const auto finite = [](float v) { return fabsf(v) == INFINITY ? NAN : v; };
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = make_float2(finite(x[i].x), finite(x[i].y));
                    y[i] = make_float2(finite(y[i].x), finite(y[i].y));
                }
                a = largest();
            }
            const int e = scale_byte(a);
            if (active) {
                const float down = scale_down(e);
                const float2 d2 = make_float2(down, down);
                uint8_t* dst = static_cast<uint8_t*>(A.out) + (KIND == 1 ? at.k : at.v) + (int64_t)h * A.out_head;
                store_codes(dst + 8 * s0, x, d2);
                store_codes(dst + 8 * s1, y, d2);
            }
            if (lane == 0) (KIND == 1 ? P.k_scale : P.v_scale)[at.s + (int64_t)h * P.page] = static_cast<uint8_t>(e);
        }
    };
    heads(std::integral_constant<int, 0>{}, P.q, h0);
    heads(std::integral_constant<int, 1>{}, P.k, (h0 - P.q.H) & (P.spt - 1));                  // (spt is a power of two)
    heads(std::integral_constant<int, 2>{}, P.v, (h0 - P.q.H - P.k.H) & (P.spt - 1));
}

template <typename TI, int L>
cudaError_t launch_append_l(RopeParams p, int sms, cudaStream_t st) {
    constexpr int SUBS = NR_THREADS / L;
    const int Ht = p.q.H + p.k.H + p.v.H;
    int spt = 32 / L;                    // as the 16-bit append's
    while (spt < SUBS && spt < Ht && (int64_t)p.T * spt < (int64_t)sms * (2048 / L)) spt *= 2;
    p.spt = spt;
    p.inv_d = 1.0f / p.D;
    const int tpb = SUBS / spt;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.T + tpb - 1) / tpb);
    cfg.blockDim = dim3(NR_THREADS);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append8_kernel<TI, L>, p);
}

template <typename TI>
cudaError_t launch_append_t(const RopeParams& p, int sms, cudaStream_t st) {
    const int l = p.D / 16;
    if (l <= 2) return launch_append_l<TI, 2>(p, sms, st);
    if (l <= 4) return launch_append_l<TI, 4>(p, sms, st);
    if (l <= 8) return launch_append_l<TI, 8>(p, sms, st);
    if (l <= 16) return launch_append_l<TI, 16>(p, sms, st);
    return launch_append_l<TI, 32>(p, sms, st);
}

// ---------------------------------------------------------------- reading back

constexpr int RD_THREADS = 256;
// Pieces of 8 codes of K, and of V, that a lane has in flight (DEPTH), and blocks per SM.
// Few blocks with many loads each: 16 sessions of 1000-32,768 tokens (8 heads of 128, bf16 out) 156 us with two blocks of 8 loads, 170 with
// three, 184 with four; heads of 64, of which 4 loads a lane are a tile, 90 us with four blocks, 92 with three, 104 with six.
__host__ __device__ constexpr int rd_blocks(int depth) { return depth == 4 ? 4 : 2; }

// 8 codes times 2^e, stored as 8 values.
__device__ __forceinline__ float held(float x) { return x > 65504.f ? 65504.f : x < -65504.f ? -65504.f : x; }   // (NaN stays)
template <typename TO>
__device__ __forceinline__ void put8(TO* p, const uint2& c, float s) {
    const uint32_t w[2] = {c.x, c.y};
    float x[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t a, b;
        half_codes(w[i], a, b);
        const float2 f = __half22float2(u32_as_h2(a)), g = __half22float2(u32_as_h2(b));
        x[4 * i] = f.x * s;
        x[4 * i + 1] = f.y * s;
        x[4 * i + 2] = g.x * s;
        x[4 * i + 3] = g.y * s;
    }
    if constexpr (std::is_same<TO, __half>::value) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = held(x[i]);
    }
    Vec8<TO>::store(p, x);
}

// What a call reads of a sequence: tokens [lo, len) and, where a window hides what lies between, [0, sinks); in tiles of 16
// tokens: [0, ns) and then [w0, w0 + n - ns).
struct ReadSpan {
    int lo, len, sinks, ns, w0, n;
    int r0;                          // the first row's index (rows)
};
__device__ __forceinline__ ReadSpan read_span(const ReadParams& P, int b, bool report) {
    ReadSpan s = {};
    int rows = 1;
    s.r0 = b;
    if (P.cu_rows) {
        const int r0 = P.cu_rows[b], r1 = P.cu_rows[b + 1];
        const bool ok = rows_sound(r0, r1, P.T);
        if (report && !(ok && r1 - r0 <= P.max_rows)) set_err(P.err, ERR_KV_LEN);
        rows = ok ? min(r1 - r0, P.max_rows) : 0;
        s.r0 = r0;
    }
    const int64_t most = (int64_t)P.max_pages * P.page;
    int len = P.kv_len[b];
    if (len > most) {
        if (report) set_err(P.err, ERR_KV_LEN);
        len = static_cast<int>(most);
    }
    s.len = len = max(len, 0);
    if (rows <= 0) return s;
    s.lo = len - rows;
    if (P.pages) {
        if (len == 0) return s;
        s.lo = P.window > 0 ? max(0, len - rows + 1 - P.window) : 0;
        s.sinks = P.window > 0 ? min(P.sinks, len) : 0;
        s.w0 = s.lo / 16;
        s.ns = min((s.sinks + 15) / 16, s.w0);
    } else {
        s.w0 = s.lo >= 0 ? s.lo / 16 : -((-s.lo + 15) / 16);       // rows at negative positions are written too, as zeros
    }
    s.n = s.ns + (s.len + 15) / 16 - s.w0;
    return s;
}

template <typename TO, int DEPTH>
__global__ void __launch_bounds__(RD_THREADS, rd_blocks(DEPTH)) paged_read_kernel(const __grid_constant__ ReadParams P) {
    extern __shared__ int pre[];         // tiles before each sequence [B + 1]
    __shared__ int s_scan[RD_THREADS / 32];
    pdl_wait();
    pdl_release();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    {
        const int per = (P.B + RD_THREADS - 1) / RD_THREADS;
        int sum = 0;
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < P.B) sum += read_span(P, b, blockIdx.x == 0).n;
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int run = inc - sum;
        for (int w = 0; w < warp; ++w) run += s_scan[w];
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < P.B) {
                pre[b] = run;
                run += read_span(P, b, false).n;
            }
        }
        if (tid == RD_THREADS - 1) pre[P.B] = run;
        __syncthreads();
    }
    // (rows that cu_rows names more than once, which is reported, take no more tiles than T rows can)
    const int tiles = P.pages ? pre[P.B] : static_cast<int>(min((int64_t)pre[P.B], (int64_t)P.T / 16 + 2 * P.B));
    const int64_t total = (int64_t)tiles * P.H, stride = (int64_t)gridDim.x * (RD_THREADS / 32);
    const int lpr = P.D / 8, pieces = 16 * lpr;       // pieces of 8 codes of a row, and of a tile
    const int t_lane = lane / lpr, c_lane = lane - t_lane * lpr, t_step = 32 / lpr, c_step = 32 - t_step * lpr;
    // Lane i looks up the warp's next tile but i at once: its head, tokens, page and place in the output.
    int head = 0, first = 0, page = 0, lo = 0, len = 0, sinks = 0, out = -1;      // out -1: nothing to do
    const auto look_up = [&](int64_t it) {
        out = -1;
        if (it >= total) return;
        const int v = (total >> 32) == 0 ? static_cast<uint32_t>(it) / static_cast<uint32_t>(P.H) : static_cast<int>(it / P.H);
        head = static_cast<int>(it - (int64_t)v * P.H);
        int b = 0, hi = P.B - 1;
        while (b < hi) {
            const int mid = (b + hi + 1) >> 1;
            if (pre[mid] <= v) b = mid;
            else hi = mid - 1;
        }
        const ReadSpan s = read_span(P, b, false);
        const int j = v - pre[b];
        if (j < 0 || j >= s.n) return;                      // (only where cu_rows made no sense)
        first = (j < s.ns ? j : j - s.ns + s.w0) * 16;
        lo = s.lo;
        len = s.len;
        sinks = s.sinks;
        // a tile in front of the cache (padded rows) has no page
        page = 0;
        const int pi = first >= 0 ? first / P.page : 0;
        if (first >= 0) {
            page = P.table[(int64_t)b * P.max_pages + pi];
            if (page < 0 || page >= P.n_pages) {
                set_err(P.err, ERR_PAGE_ID);
                page = 0;                                   // read instead: the call's results are invalid
            }
        }
        if (P.pages) {
            const int sp = (s.sinks + P.page - 1) / P.page, wp = s.lo / P.page;
            const int os = wp > sp && pi >= wp ? pi - wp + sp : pi;
            if (!P.by_page && os >= P.slots) return;        // (only where kv_len or cu_rows made no sense)
            out = P.by_page ? page : b * P.slots + os;
            if (head == 0) P.page_map[(int64_t)b * P.max_pages + pi] = out;
        } else {
            out = s.r0;
        }
    };
    int left = 0;                        // tiles that lanes have looked up
    for (int64_t it = (int64_t)blockIdx.x * (RD_THREADS / 32) + warp; it < total; it += stride) {
        if (left == 0) {
            look_up(it + lane * stride);
            left = 32;
        }
        const int from = 32 - left--;
        const int o = __shfl_sync(0xffffffffu, out, from), h = __shfl_sync(0xffffffffu, head, from), tok = __shfl_sync(0xffffffffu, first, from);
        const int64_t pg = __shfl_sync(0xffffffffu, page, from);
        const int t_lo = __shfl_sync(0xffffffffu, lo, from), t_len = __shfl_sync(0xffffffffu, len, from), t_sinks = __shfl_sync(0xffffffffu, sinks, from);
        if (o < 0) continue;
        const auto taken = [&](int p) { return p < t_len && (p >= t_lo || static_cast<uint32_t>(p) < static_cast<uint32_t>(t_sinks)); };
        const int slot = tok >= 0 ? tok % P.page : 0;
        TO *ko = static_cast<TO*>(P.Ko), *vo = static_cast<TO*>(P.Vo);
        if (P.pages) {
            const int64_t off = (((int64_t)o * P.H + h) * P.page + slot) * P.D;
            ko += off;
            vo += off;
        } else {
            const int64_t row = o + ((int64_t)tok - t_lo);
            ko += row * P.ko_row + h * P.ko_head;
            vo += row * P.vo_row + h * P.vo_head;
        }
        const int64_t ors = P.pages ? P.D : P.ko_row, vrs = P.pages ? P.D : P.vo_row;
        const uint8_t* kc = P.K + pg * P.k_page + h * P.k_head + slot * P.k_token;
        const uint8_t* vc = P.V + pg * P.v_page + h * P.v_head + slot * P.v_token;
        const int64_t sc = (pg * P.scale_heads + h) * P.page + slot;
        const uint32_t scale = tok >= 0 ? (lane < 16 ? P.k_scale : P.v_scale)[sc + (lane & 15)] : 0;    // of token lane % 16
        if constexpr (std::is_same<TO, __half>::value) {
            // Attention would take 65,504 for what fp16 cannot hold: reported. Only rows whose scale allows it are looked at (448 * 2^7 is
            // within fp16): 16 tokens' K and V in one vote. 65,536, the code next to 65,504, is held to fp16's own half step.
            // (Checked at each value instead, 300 tokens took 8.3 us where they take 7.6.)
            uint32_t look = P.pages ? __ballot_sync(0xffffffffu, scale > 134 && scale < 255 && taken(tok + (lane & 15))) : 0;
            while (look) {
                const int i = __ffs(look) - 1;
                look &= look - 1;
                const float s = scale_up(__shfl_sync(0xffffffffu, scale, i));
                const uint8_t* row = i < 16 ? kc + i * P.k_token : vc + (i - 16) * P.v_token;
                for (int x = 4 * lane; x < P.D; x += 128) {
                    uint32_t a, b;
                    half_codes(*reinterpret_cast<const uint32_t*>(row + x), a, b);
                    const float2 f = __half22float2(u32_as_h2(a)), g = __half22float2(u32_as_h2(b));
                    if (fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(g.x), fabsf(g.y))) * s > 65536.f) set_err(P.err, ERR_FP16_RANGE);
                }
            }
        }
        int t0 = t_lane, c0 = c_lane;                       // token and piece of the lane's first load of a round
        for (int n0 = 0; n0 < pieces; n0 += 32 * DEPTH) {
            uint2 k[DEPTH], x[DEPTH];
            int t = t0, c = c0;
            const auto step = [&]() {
                t += t_step;
                c += c_step;
                if (c >= lpr) {
                    c -= lpr;
                    ++t;
                }
            };
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                k[i] = x[i] = make_uint2(0, 0);
                if (t < 16 && tok >= 0 && taken(tok + t)) {
                    k[i] = __ldcs(reinterpret_cast<const uint2*>(kc + t * P.k_token + 8 * c));
                    x[i] = __ldcs(reinterpret_cast<const uint2*>(vc + t * P.v_token + 8 * c));
                }
                step();
            }
            t = t0;
            c = c0;
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                const float sk = scale_up(__shfl_sync(0xffffffffu, scale, t & 15)), sv = scale_up(__shfl_sync(0xffffffffu, scale, 16 + (t & 15)));
                if (t < 16 && taken(tok + t)) {             // (rows in front of the cache too, as zeros)
                    put8(ko + t * ors + 8 * c, k[i], sk);
                    put8(vo + t * vrs + 8 * c, x[i], sv);
                }
                step();
            }
            t0 = t;
            c0 = c;
        }
    }
}

template <typename TO, int DEPTH>
cudaError_t launch_read_d(const ReadParams& p, int sms, cudaStream_t st) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms * rd_blocks(DEPTH));
    cfg.blockDim = dim3(RD_THREADS);
    cfg.dynamicSmemBytes = 4 * (p.B + 1);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_read_kernel<TO, DEPTH>, p);
}
template <typename TO>
cudaError_t launch_read_t(const ReadParams& p, int sms, cudaStream_t st) {
    return p.D <= 64 ? launch_read_d<TO, 4>(p, sms, st) : launch_read_d<TO, 8>(p, sms, st);
}

}  // namespace

cudaError_t launch_paged_read(const ReadParams& p, int out_dtype, int sms, cudaStream_t st) {
    if (out_dtype == PCK_DT_F16) return launch_read_t<__half>(p, sms, st);
    if (out_dtype == PCK_DT_BF16) return launch_read_t<__nv_bfloat16>(p, sms, st);
    return launch_read_t<float>(p, sms, st);
}

cudaError_t launch_append_e4m3(const RopeParams& p, int in_dtype, int sms, cudaStream_t st) {
    if (in_dtype == PCK_DT_F16) return launch_append_t<__half>(p, sms, st);
    if (in_dtype == PCK_DT_BF16) return launch_append_t<__nv_bfloat16>(p, sms, st);
    return launch_append_t<float>(p, sms, st);
}

}  // namespace pck
