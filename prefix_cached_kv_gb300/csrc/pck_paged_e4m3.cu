// pck_paged_e4m3.cu -- the append to a quantised paged cache, and rows of that cache read back.
//
// Reading back: out = code * 2^e, rounded once to the output's type (fp32 and bf16 hold it exactly; in fp16 what is beyond
// 65,504 becomes 65,504). D + 1 bytes in and 2 D or 4 D out per row, so HBM bounds it. A warp takes tiles of 16 tokens of one kv
// head, K and V: 8 codes a lane, so that its 16-byte stores lie side by side, with DEPTH loads of K and of V in flight before the
// first is used: 6.1 TB/s read and written on the long sessions (0.90 of a copy).
// The tiles of all sequences laid end to end are dealt to the warps from the lengths on the device (one block scan), so
// one long session and many short ones fill the GPU alike.
#include "pck_paged_rope_impl.cuh"

namespace pck {
namespace {

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
    const int64_t total = (int64_t)pre[P.B] * P.H, stride = (int64_t)gridDim.x * (RD_THREADS / 32);
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
        const int64_t sc = (pg * P.H + h) * P.page + slot;
        const uint32_t scale = tok >= 0 ? (lane < 16 ? P.k_scale : P.v_scale)[sc + (lane & 15)] : 0;    // of token lane % 16
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
    if (in_dtype == PCK_DT_F16) return launch_t<__half, E4m3>(p, sms, st);
    if (in_dtype == PCK_DT_BF16) return launch_t<__nv_bfloat16, E4m3>(p, sms, st);
    return launch_t<float, E4m3>(p, sms, st);
}

}  // namespace pck
