// pck_paged_e4m3.cu -- the append to a quantised paged cache, and rows of that cache read back.
//
// Reading back: out = code * 2^e, rounded once to the output's type (fp32 and bf16 hold it exactly; in fp16 what is beyond
// 65,504 becomes 65,504). D + 1 bytes in and 2 D or 4 D out per row, so HBM bounds it. A warp takes tiles of 16 tokens of one kv
// head, K and V: D/16 lanes a row, 16 codes a lane, RD_DEPTH rows of loads in flight per lane before the first is used.
// The tiles of all sequences laid end to end are dealt to the warps from the lengths on the device (one block scan), so
// one long session and many short ones fill the GPU alike.
#include "pck_paged_rope_impl.cuh"

namespace pck {
namespace {

constexpr int RD_THREADS = 256;
constexpr int RD_BLOCKS = 3;         // blocks per SM
constexpr int RD_DEPTH = 4;          // chunks of 16 codes of K, and of V, that a lane has in flight

template <typename TO>
struct Out16;   // 16 values stored
template <>
struct Out16<float> {
    static __device__ __forceinline__ void store(float* p, const float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
};
template <>
struct Out16<__half> {
    static __device__ __forceinline__ float held(float x) { return x > 65504.f ? 65504.f : x < -65504.f ? -65504.f : x; }   // (NaN stays)
    static __device__ __forceinline__ void store(__half* p, const float (&x)[16]) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = h2_as_u32(__floats2half2_rn(held(x[2 * i]), held(x[2 * i + 1])));
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
};
template <>
struct Out16<__nv_bfloat16> {
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[16]) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
};

template <typename TO>
__device__ __forceinline__ void put16(TO* p, const uint4& c, float s) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    float x[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a, b;
        half_codes(w[i], a, b);
        const float2 f = __half22float2(u32_as_h2(a)), g = __half22float2(u32_as_h2(b));
        x[4 * i] = f.x * s;
        x[4 * i + 1] = f.y * s;
        x[4 * i + 2] = g.x * s;
        x[4 * i + 3] = g.y * s;
    }
    Out16<TO>::store(p, x);
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

template <typename TO>
__global__ void __launch_bounds__(RD_THREADS, RD_BLOCKS) paged_read_kernel(const __grid_constant__ ReadParams P) {
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
    const int64_t total = (int64_t)pre[P.B] * P.H;
    const int lpr = P.D / 16, chunks = 16 * lpr;      // lanes of a row, 16-code chunks of a tile
    for (int64_t it = (int64_t)blockIdx.x * (RD_THREADS / 32) + warp; it < total; it += (int64_t)gridDim.x * (RD_THREADS / 32)) {
        const int v = static_cast<int>(it / P.H);
        const int h = static_cast<int>(it - (int64_t)v * P.H);
        int b = 0, hi = P.B - 1;
        while (b < hi) {
            const int mid = (b + hi + 1) >> 1;
            if (pre[mid] <= v) b = mid;
            else hi = mid - 1;
        }
        const ReadSpan s = read_span(P, b, false);
        const int j = v - pre[b];
        if (j < 0 || j >= s.n) continue;                    // (only where cu_rows made no sense)
        const int tok = (j < s.ns ? j : j - s.ns + s.w0) * 16;
        const auto taken = [&](int p) { return p < s.len && (p >= s.lo || static_cast<uint32_t>(p) < static_cast<uint32_t>(s.sinks)); };
        // the tile's page; a tile in front of the cache (padded rows) has none
        int64_t pg = 0;
        int pi = 0;
        if (tok >= 0) {
            pi = tok / P.page;
            pg = P.table[(int64_t)b * P.max_pages + pi];
            if (pg < 0 || pg >= P.n_pages) {
                if (lane == 0) set_err(P.err, ERR_PAGE_ID);
                pg = 0;                                     // read instead: the call's results are invalid
            }
        }
        const int slot = tok - pi * P.page;
        TO *ko = static_cast<TO*>(P.Ko), *vo = static_cast<TO*>(P.Vo);
        if (P.pages) {
            const int sp = (s.sinks + P.page - 1) / P.page, wp = s.lo / P.page;
            const int os = wp > sp && pi >= wp ? pi - wp + sp : pi;
            if (os >= P.slots) continue;                    // (only where kv_len or cu_rows made no sense)
            const int64_t out_page = (int64_t)b * P.slots + os;
            if (lane == 0 && h == 0) P.page_map[(int64_t)b * P.max_pages + pi] = static_cast<int32_t>(out_page);
            const int64_t off = ((out_page * P.H + h) * P.page + slot) * P.D;
            ko += off;
            vo += off;
        } else {
            const int64_t row = s.r0 + ((int64_t)tok - s.lo);
            ko += row * P.ko_row + h * P.ko_head;
            vo += row * P.vo_row + h * P.vo_head;
        }
        const int64_t ors = P.pages ? P.D : P.ko_row, vrs = P.pages ? P.D : P.vo_row;
        const uint8_t* kc = P.K + pg * P.k_page + h * P.k_head + slot * P.k_token;
        const uint8_t* vc = P.V + pg * P.v_page + h * P.v_head + slot * P.v_token;
        const int64_t sc = (pg * P.H + h) * P.page + slot;
        for (int c0 = 0; c0 < chunks; c0 += 32 * RD_DEPTH) {
            uint4 k[RD_DEPTH], x[RD_DEPTH];
            float sk[RD_DEPTH], sv[RD_DEPTH];
#pragma unroll
            for (int i = 0; i < RD_DEPTH; ++i) {
                const int c = c0 + 32 * i + lane, t = c / lpr, d = (c - t * lpr) * 16, p = tok + t;
                k[i] = x[i] = make_uint4(0, 0, 0, 0);
                sk[i] = sv[i] = 0.f;
                if (c < chunks && p >= 0 && taken(p)) {
                    k[i] = __ldcs(reinterpret_cast<const uint4*>(kc + t * P.k_token + d));
                    x[i] = __ldcs(reinterpret_cast<const uint4*>(vc + t * P.v_token + d));
                    sk[i] = scale_up(P.k_scale[sc + t]);
                    sv[i] = scale_up(P.v_scale[sc + t]);
                }
            }
#pragma unroll
            for (int i = 0; i < RD_DEPTH; ++i) {
                const int c = c0 + 32 * i + lane, t = c / lpr, d = (c - t * lpr) * 16, p = tok + t;
                if (c < chunks && taken(p)) {               // (rows in front of the cache too, as zeros)
                    put16(ko + t * ors + d, k[i], sk[i]);
                    put16(vo + t * vrs + d, x[i], sv[i]);
                }
            }
        }
    }
}

template <typename TO>
cudaError_t launch_read_t(const ReadParams& p, int sms, cudaStream_t st) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms * RD_BLOCKS);
    cfg.blockDim = dim3(RD_THREADS);
    cfg.dynamicSmemBytes = 4 * (p.B + 1);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_read_kernel<TO>, p);
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
