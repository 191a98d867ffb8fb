// pck_paged_rope_impl.cuh -- head norms with the rotary rotation, and the append of new keys and values to a
// paged cache (the quantising append shares what places a row and its angles).
//
// Per row x (one token, one head, D elements) and position t:
//   y = x * rsqrt(mean(x^2) + eps) * w                       (q and k heads with a norm)
//   (a, b) -> (a cos - b sin, b cos + a sin)                 for the R/2 pairs of the first R elements
// with cos and sin read from the caller's fp32 table row t. Norm, weight and rotation stay in fp32
// and are rounded once, to the output's type. V rows are copied (converted where the types differ).
//
// Every byte is read and written once, so HBM bounds it. A row is held by L = D/16 lanes (a power
// of two at least), each with two vectors of 8 elements: vector p and vector p + R/16 of the
// rotated part, which are the two halves of its pairs when the halves are split (and hold whole
// pairs when they are adjacent), so a rotation needs no exchange between lanes; the norm's sum takes
// log2 L shuffles. `spt` subwarps share a token and step over its heads, so the token's table row
// is read into registers once for H / spt heads: few subwarps per token while there are tokens
// enough to fill the SMs, many when there are few. 16,384 tokens of 64 + 8 heads of 128: 105-107 us, 5.8 TB/s read and
// written (0.85 of a copy); an append of 8 ragged prompts, 32 + 8 + 8 heads: 59 us, 5.5 TB/s.
#pragma once

#include "pck_paged.cuh"

namespace pck {
namespace {

constexpr int NR_THREADS = 256;
// Heads whose loads a lane has in flight, and blocks per SM (64 registers, 16 bytes a thread spilt): 16,384 tokens of 72
// heads in 106.7 us; one head 111, four heads 115 (3 blocks); five blocks spill many more (138).
constexpr int NR_HEADS = 2;
template <typename TI> __host__ __device__ constexpr int nr_blocks() { return sizeof(TI) == 4 ? 3 : 4; }   // fp32 rows take 80 registers, 16 bytes spilt

template <typename T>
struct Vec8;   // 8 elements: as they lie in memory (Raw), and as fp32
template <>
struct Vec8<__half> {
    typedef uint4 Raw;
    static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ void store(__half* p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec8<__nv_bfloat16> {
    typedef uint4 Raw;
    static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec8<float> {
    struct Raw {
        float4 a, b;
    };
    static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[8]) {
        const float4 a = r.a, b = r.b;
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// Where an append puts a row: offsets into the cache (of head 0), and its cache position. False: the row is not to be stored.
struct RowPlace {
    int64_t k, v, s;                 // s: of the scale bytes, [page][head][slot]
    int pos;
};
template <typename TI, int L>
__device__ __forceinline__ bool place_row(const RopeParams& P, int t, int lane, uint32_t mask, int h0, RowPlace& at) {
    int b = t, n_b_left = 1;
    if (P.cu_rows) {
        int cnt = 0;   // sequences whose rows start at or before t
        bool bad = false;
        for (int i = lane; i <= P.B; i += L) {
            const int r0 = P.cu_rows[i];
            cnt += r0 <= t;
            if (blockIdx.x == 0 && i < P.B) bad |= !rows_sound(r0, P.cu_rows[i + 1], P.T);
        }
        if (bad) set_err(P.err, ERR_KV_LEN);
#pragma unroll
        for (int o = L / 2; o; o >>= 1) cnt += __shfl_xor_sync(mask, cnt, o, L);
        b = cnt - 1;
        if (b < 0 || b >= P.B) return false;   // a row of no sequence
        const int r1 = P.cu_rows[b + 1];
        if (P.cu_rows[b] > t || r1 <= t) return false;   // (nor here: cu_rows does not ascend)
        n_b_left = r1 - t;
    }
    const int64_t p = (int64_t)P.kv_len[b] - n_b_left;
    if (p < 0) {                                // no such token: a padded sequence stores nothing, and its q is 0
        const float zero[8] = {};
        if (lane < P.D / 16)
            for (int h = h0; h < P.q.H; h += P.spt) {
                TI* dst = static_cast<TI*>(P.q.out) + (int64_t)t * P.q.out_row + (int64_t)h * P.q.out_head + 16 * lane;
                Vec8<TI>::store(dst, zero);
                Vec8<TI>::store(dst + 8, zero);
            }
        return false;
    }
    if (p >= (int64_t)P.max_pages * P.page) {
        if (lane == 0) set_err(P.err, ERR_KV_LEN);
        return false;
    }
    const int pi = static_cast<int>(p) / P.page, slot = static_cast<int>(p) - pi * P.page;
    const int pg = P.table[(int64_t)b * P.max_pages + pi];
    if (pg < 0 || pg >= P.n_pages) {
        if (lane == 0) set_err(P.err, ERR_PAGE_ID);
        return false;
    }
    at.k = pg * P.k_page + slot * P.k.out_row;
    at.v = pg * P.v_page + slot * P.v.out_row;
    at.s = (int64_t)pg * P.k.H * P.page + slot;
    at.pos = static_cast<int>(p);
    return true;
}

// The lane's cosines and sines: false where the position has no row of the table.
__device__ __forceinline__ bool load_angles(const RopeParams& P, int t, int lane, int pos, bool rot, int s0, int s1, float (&co)[8],
                                            float (&si)[8]) {
    if (P.positions) pos = P.positions[t];
    if (pos < 0 || pos >= P.n_pos) {
        if (lane == 0) set_err(P.err, ERR_ROPE_POS);
        return false;
    }
    if (rot) {
        const float* row = P.cos_sin + (int64_t)pos * P.R;
        // pairs 8 lane .. +7 of split halves; pairs 4 s0 .. and 4 s1 .. of adjacent ones
        const int i0 = P.interleaved ? 4 * s0 : 8 * lane, i1 = P.interleaved ? 4 * s1 : 8 * lane + 4;
        *reinterpret_cast<float4*>(co) = *reinterpret_cast<const float4*>(row + i0);
        *reinterpret_cast<float4*>(co + 4) = *reinterpret_cast<const float4*>(row + i1);
        *reinterpret_cast<float4*>(si) = *reinterpret_cast<const float4*>(row + P.R / 2 + i0);
        *reinterpret_cast<float4*>(si + 4) = *reinterpret_cast<const float4*>(row + P.R / 2 + i1);
    }
    return true;
}

// L: lanes per row. TI: type of the rows read (and of q written); TC: type of the cache (append).
template <typename TI, typename TC, int L>
__global__ void __launch_bounds__(NR_THREADS, nr_blocks<TI>()) norm_rope_kernel(const __grid_constant__ RopeParams P) {
    constexpr int SUBS = NR_THREADS / L;
    pdl_wait();      // inputs may come from the previous kernel of the stream
    pdl_release();
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    const int tok_per_block = SUBS / P.spt;
    const int64_t t64 = (int64_t)blockIdx.x * tok_per_block + sub / P.spt;
    const uint32_t mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31) / L * L);
    if (t64 >= P.T) return;
    const int t = static_cast<int>(t64);
    const int h0 = sub % P.spt;
    const int Ht = P.q.H + P.k.H + P.v.H;
    if (h0 >= Ht) return;

    RowPlace at = {};
    if (P.append && !place_row<TI, L>(P, t, lane, mask, h0, at)) return;
    const int64_t kbase = at.k, vbase = at.v;
    int pos = at.pos;
    const bool active = lane < P.D / 16;
    const int rv = P.R / 16;
    const bool rot = lane < rv;
    // the lane's two vectors (in units of 8 elements)
    const int s0 = rot ? lane : P.R / 8 + (lane - rv);
    const int s1 = rot ? lane + rv : s0 + (P.D - P.R) / 16;
    float co[8], si[8];
    if (P.R > 0) {
        if (!load_angles(P, t, lane, pos, rot, s0, s1, co, si)) return;
    }

    typedef typename Vec8<TI>::Raw Raw;
    auto elem = [&](const void* p, int64_t off) { return static_cast<const TI*>(p) + off; };
    // NR_HEADS heads at a time, all of their loads in flight before the first is used
    for (int hb = h0; hb < Ht; hb += NR_HEADS * P.spt) {
        Raw r0[NR_HEADS], r1[NR_HEADS];
#pragma unroll
        for (int k = 0; k < NR_HEADS; ++k) {
            const int hh = hb + k * P.spt;
            r0[k] = r1[k] = Raw{};
            if (hh < Ht && active) {
                const int cls = hh < P.q.H ? 0 : hh < P.q.H + P.k.H ? 1 : 2;
                const RowsArg& A = cls == 0 ? P.q : cls == 1 ? P.k : P.v;
                const int h = hh - (cls == 0 ? 0 : cls == 1 ? P.q.H : P.q.H + P.k.H);
                const TI* src = elem(A.in, (int64_t)t * A.in_row + (int64_t)h * A.in_head);
                r0[k] = *reinterpret_cast<const Raw*>(src + 8 * s0);
                r1[k] = *reinterpret_cast<const Raw*>(src + 8 * s1);
            }
        }
#pragma unroll
        for (int k = 0; k < NR_HEADS; ++k) {
            const int hh = hb + k * P.spt;
            if (hh >= Ht) break;
            const int cls = hh < P.q.H ? 0 : hh < P.q.H + P.k.H ? 1 : 2;
            const RowsArg& A = cls == 0 ? P.q : cls == 1 ? P.k : P.v;
            const int h = hh - (cls == 0 ? 0 : cls == 1 ? P.q.H : P.q.H + P.k.H);
            float x[8], y[8];
            Vec8<TI>::unpack(r0[k], x);
            Vec8<TI>::unpack(r1[k], y);
            if (A.norm) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
                for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o, L);
                const float r = rsqrtf(ss * P.inv_d + P.eps);
                if (A.w && active) {
                    float w0[8], w1[8];
                    Vec8<TI>::unpack(*reinterpret_cast<const Raw*>(elem(A.w, 8 * s0)), w0);
                    Vec8<TI>::unpack(*reinterpret_cast<const Raw*>(elem(A.w, 8 * s1)), w1);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = x[i] * r * w0[i];
                        y[i] = y[i] * r * w1[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] *= r;
                        y[i] *= r;
                    }
                }
            }
            if (rot && cls != 2) {
                if (P.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = x[2 * i], b = x[2 * i + 1], c = y[2 * i], d = y[2 * i + 1];
                        x[2 * i] = a * co[i] - b * si[i];
                        x[2 * i + 1] = b * co[i] + a * si[i];
                        y[2 * i] = c * co[4 + i] - d * si[4 + i];
                        y[2 * i + 1] = d * co[4 + i] + c * si[4 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a = x[i], b = y[i];
                        x[i] = a * co[i] - b * si[i];
                        y[i] = b * co[i] + a * si[i];
                    }
                }
            }
            if (!active) continue;
            if (P.append && cls != 0) {
                TC* dst = static_cast<TC*>(A.out) + (cls == 1 ? kbase : vbase) + (int64_t)h * A.out_head;
                Vec8<TC>::store(dst + 8 * s0, x);
                Vec8<TC>::store(dst + 8 * s1, y);
            } else {
                TI* dst = static_cast<TI*>(A.out) + (int64_t)t * A.out_row + (int64_t)h * A.out_head;
                Vec8<TI>::store(dst + 8 * s0, x);
                Vec8<TI>::store(dst + 8 * s1, y);
            }
        }
    }
}

template <typename TI, typename TC, int L>
cudaError_t launch_l(RopeParams p, int sms, cudaStream_t st) {
    constexpr int SUBS = NR_THREADS / L;
    // Subwarps per token: as few as still give every SM 2048 threads, at least one warp's worth (neighbouring heads
    // of a token share a warp's wide accesses). At 16,384 tokens of 72 heads: 106.7 us, with twice as many 108.7, with
    // four times 135.
    const int Ht = p.q.H + p.k.H + p.v.H;
    int spt = 32 / L;
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
    return cudaLaunchKernelEx(&cfg, norm_rope_kernel<TI, TC, L>, p);
}

template <typename TI, typename TC>
cudaError_t launch_t(const RopeParams& p, int sms, cudaStream_t st) {
    const int l = p.D / 16;
    if (l <= 2) return launch_l<TI, TC, 2>(p, sms, st);
    if (l <= 4) return launch_l<TI, TC, 4>(p, sms, st);
    if (l <= 8) return launch_l<TI, TC, 8>(p, sms, st);
    if (l <= 16) return launch_l<TI, TC, 16>(p, sms, st);
    return launch_l<TI, TC, 32>(p, sms, st);
}

}  // namespace
}  // namespace pck
