// pck_paged_rows.cu -- attention of ragged rows (prompts, prompt chunks) over a paged KV cache, causal,
// with an optional sliding window and first tokens that stay visible, on the 5th-generation tensor cores.
//
// Row i of the n rows of a sequence with len cached tokens stands at p = len - n + i and sees the keys
// j <= p, with a window W > 0 only those with j > p - W or j < sinks:
//   S = tau q K^T,  O = sum_j 2^(s_j' - m) v_j / l,  LSE = (m + log2 l) ln 2       (s' = s log2 e)
//
// 4 D flop per visible (row, head, key) against K and V read through L2 once per CTA: the tensor
// cores bound it, so the kernel's business is to feed them without a pause.
//  * A CTA owns two tiles of 128 query rows of one kv head (row = token * G + q head, so grouped heads
//    share every K and V tile) and walks its keys in blocks of 128. While one tile's softmax runs, the
//    other tile's MMAs do. TMEM: two S (128 columns each; P of a block overwrites its S as packed 16-bit
//    values) and two O (D columns each).
//  * One warp loads Q and rings of K and of V blocks by TMA with 128-byte swizzle, one box per page run (a box
//    is the largest power-of-two run of tokens that divides both the page and the block). K is the
//    K-major B operand of S = Q K^T as it lies; V, stored token by token, is the MN-major B operand of
//    O += P V, so nothing is transposed.
//  * One warp issues tcgen05.mma: S0(j+1) right behind O0 += P0(j) V(j), then the same for tile 1.
//  * Warps 0-3 and 4-7 are the tiles' softmax, a thread per row. p = 2^(s - m), m a little below the running maximum;
//    it is checked by the weights' sum and moved only when that passes its CAP: no pass over the scores looks for
//    a maximum, and O is rarely rescaled. p is rounded once to the cache's type for the second MMA (a
//    rounding like that of the 16-bit output); its fp32 sum takes the unrounded p.
//  * Keys: with a window, the sinks' boxes and then the window's are laid end to end, so no block is spent
//    on hidden keys and the pages between are never touched. Only blocks that some row does not see
//    whole are masked, by a bit mask per row and 32 keys.
//  * V rows that no row of the CTA sees (behind the last token, in front of the window) are zeroed in
//    shared memory, since 0 * NaN would keep what they hold. V rows of partly hidden blocks that are not
//    finite are cleared too, and added at the end by the rows that see them.
//  * Few rows over a long cache: the keys are split over n_split CTAs and a second kernel joins them.
// Measured: a prompt of 8192 rows, 32 / 8 heads of 128, bf16 355-369 us (1,490-1,550 TFLOP/s, 0.77-0.80 of cuBLAS bf16),
// fp16 360-379 us; heads of 64 260-267 us; 4096 rows on 16k tokens 640-675 us (3.4 waves of nearly equal CTAs: 0.87 of
// what an even load would take); ragged prompts with a window of 1024, 24 / 8 heads, 164 us. A block of both tiles takes
// ~3,000 cycles where its MMAs take 2,048: the chain softmax - hand-off - P V - S bounds it.
#include <algorithm>
#include <type_traits>

#include "pck_paged.cuh"

namespace pck {
namespace {

constexpr int RW_M = 128;              // rows of a tile
constexpr int RW_BLOCK = 128;          // keys of a block
constexpr int RW_THREADS = 384;        // two softmax warpgroups; MMA warp, load warp, two warps that look V over
constexpr int RW_MMA_WARP = 8, RW_LOAD_WARP = 9, RW_EDGE_WARP = 10;
// registers a thread: 168 at launch (384 x 168 <= 65,536); 216 x 256 + 72 x 128 = 384 x 168 after the split. (The compiler
// keeps to 168 for all and spills 80 bytes a thread at D = 128, 68 at 64.)
constexpr int RW_REGS_SOFTMAX = 216, RW_REGS_OTHER = 72;

template <int D>
struct RCfg {
    static constexpr int CH = D / 64;                          // 128-byte chunks of a row
    static constexpr int CHUNK = 128 * 128;                    // bytes of a chunk of 128 rows
    static constexpr int TILE = CH * CHUNK;                    // Q tile, K block or V block
    static constexpr int NK = D == 128 ? 2 : 4, NV = D == 128 ? 3 : 4;   // stages of the K ring and of the V ring
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_V = OFF_RING + NK * TILE;
    static constexpr int OFF_BAR = OFF_V + NV * TILE;
    static constexpr int BAR_BYTES = 768;                      // barriers, TMEM address, this CTA's rows, spoilt keys
    static constexpr int SMEM = OFF_BAR + BAR_BYTES + 1024;    // + alignment slack
    // TMEM: S of tile t at column 128 t, O at 256 + D t. P of a block overwrites its S, so the next S has to wait for
    // P V; at D = 64 there is room for P on its own (64 columns a tile), and the next S only waits for this one to be
    // read (8k prompt, 32 / 8 heads: 305 -> 267 us).
    static constexpr bool APART = D == 64;
    static constexpr int S_COL = 0, O_COL = 256, P_COL = APART ? 384 : 0, P_STEP = APART ? 64 : 128;
    static constexpr int TMEM_COLS = 512;
};

// ---------------------------------------------------------------- tcgen05 and TMA wrappers

// 128-byte swizzled operand descriptors: K-major (rows of 128 bytes, 8-row groups 1024 bytes apart) and
// MN-major (runs of 64 elements per token, 8-token groups 1024 bytes apart, runs `lbo` bytes apart).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
// fp32 accumulator; A and B both fp16 (fmt 0) or bf16 (fmt 1); b_mn: B is MN-major
__host__ __device__ constexpr uint32_t idesc_16(int fmt, int N, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(fmt) << 7) | (static_cast<uint32_t>(fmt) << 10) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(RW_M >> 4) << 24);
}
// The MMAs of one block and tile, issued by one elected lane of a converged warp: one election for all of
// them, the operands' descriptors advanced by constants. The whole warp walks the issuing loop with values
// that are warp-uniform; elected one by one, or issued from a lane's own branch, an MMA cost about 100
// cycles to issue where its 16 k run 64.
// D += A B^T over 64 elements of k (4 MMAs), A and B from shared memory; acc 0: the first one overwrites D
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p, e, t; .reg .b32 rx; .reg .b64 a1, a2, a3, b1, b2, b3;\n"
        "setp.ne.u32 p, %4, 0; setp.eq.u32 t, 0, 0;\n"
        "add.u64 a1, %1, 2; add.u64 a2, %1, 4; add.u64 a3, %1, 6;\n"
        "add.u64 b1, %2, 2; add.u64 b2, %2, 4; add.u64 b3, %2, 6;\n"
        "elect.sync rx|e, 0xffffffff;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t; }"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// D += A B over 128 k (8 MMAs), A from TMEM (8 columns an MMA), B MN-major (2048 bytes an MMA)
__device__ __forceinline__ void mma_ts8(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p, e, t; .reg .b32 rx, a1, a2, a3, a4, a5, a6, a7; .reg .b64 b1, b2, b3, b4, b5, b6, b7;\n"
        "setp.ne.u32 p, %4, 0; setp.eq.u32 t, 0, 0;\n"
        "add.u32 a1, %1, 8; add.u32 a2, %1, 16; add.u32 a3, %1, 24; add.u32 a4, %1, 32;\n"
        "add.u32 a5, %1, 40; add.u32 a6, %1, 48; add.u32 a7, %1, 56;\n"
        "add.u64 b1, %2, 128; add.u64 b2, %2, 256; add.u64 b3, %2, 384; add.u64 b4, %2, 512;\n"
        "add.u64 b5, %2, 640; add.u64 b6, %2, 768; add.u64 b7, %2, 896;\n"
        "elect.sync rx|e, 0xffffffff;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], b4, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b5, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b6, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b7, %3, t; }"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p, e; .reg .b32 rx; elect.sync rx|e, 0xffffffff; setp.ne.u32 p, %4, 0; "
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{ .reg .pred e; .reg .b32 rx; elect.sync rx|e, 0xffffffff; "
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }"
        ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void ld32(uint32_t taddr, float* f) {   // 32 columns of the thread's lane; not waited for
    uint32_t* r = reinterpret_cast<uint32_t*>(f);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tma5(uint32_t dst, const CUtensorMap* tm, int x, int c1, int c2, int c3, int c4, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(dst), "l"(tm), "r"(x), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar) : "memory");
}

__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    return x;
}
__device__ __forceinline__ void f2_unpack(uint64_t x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <typename T> struct IsBf16 { static constexpr bool value = false; };
template <> struct IsBf16<__nv_bfloat16> { static constexpr bool value = true; };

// Where the maximum stands when it moves (log2), and the sum of a block's weights up to which it stays. fp16 has no step
// below 2^-24: with the maximum at 2^0 a weight under 2^-25 of it vanished, however many keys had one (131,070 keys 25
// (log2) below one: O off by 3.9e-3 of the largest |v|, as much as it is). At 2^6 a weight is within 2^-31 of the largest
// one, and a block of weights of 1 still sums to 2^13. Ragged prompts with a window of 1024: 163.7 us at 2^0,
// 163.8 at 2^6, 167.6 at 2^7 (rows whose first block is mostly hidden pass the sum again); 8k prompts as before.
template <typename T> struct Weights {
    static constexpr float TOP = 6.f, CAP = 61440.f;      // (a weight is at most the sum, and fp16 ends at 65,504)
};
template <> struct Weights<__nv_bfloat16> {
    static constexpr float TOP = 0.f, CAP = 32768.f;
};
template <typename T> __device__ __forceinline__ uint32_t pack16(float a, float b);
template <> __device__ __forceinline__ uint32_t pack16<__half>(float a, float b) { return h2_as_u32(__floats2half2_rn(a, b)); }
template <> __device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T> __device__ __forceinline__ float2 unpack16(uint32_t u);
template <> __device__ __forceinline__ float2 unpack16<__half>(uint32_t u) { return __half22float2(u32_as_h2(u)); }
template <> __device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Bounded wait on an mbarrier phase that lets the warp sleep in the barrier: with a time hint (20 us) try_wait
// suspends it, without one it comes back soon and the polls take issue slots from the other tile's softmax.
// Gives up after 2^17 hints (over two seconds).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
    for (uint32_t it = 0; it < (1u << 17); ++it) {
        uint32_t ok;
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(20000u) : "memory");
        if (ok) return true;
    }
    return false;
}

// ---------------------------------------------------------------- which rows, which keys

struct RowTile {
    int b;          // sequence, or -1: no rows for this tile index
    int tok0;       // first row of the sequence in this CTA
    int n;          // rows of the sequence
    int row0;       // first row of the sequence among the call's T
    int len;        // its cached tokens, as given
};

// Tiles of tt rows that n rows take.
__device__ __forceinline__ uint32_t tiles_of(int n, int tt) { return (static_cast<uint32_t>(max(0, n)) + tt - 1u) / static_cast<uint32_t>(tt); }

// The sequence and rows of CTA tile `idx` (tiles of tt rows, the sequences' tiles end to end). One warp; PER sequences a
// lane at a time. (Row counts that make no sense, from a cu_rows that does not ascend, give some tile or none: the
// caller checks every index that follows from it.)
template <int PER>
__device__ __forceinline__ RowTile find_tile_by(const PagedAttn& P, int idx, int tt, int lane) {
    int64_t before = 0;
    for (int b0 = 0; b0 < P.B; b0 += 32 * PER) {
        const int bl = b0 + lane * PER;
        int cu[PER + 1], len[PER];
#pragma unroll
        for (int i = 0; i <= PER; ++i) cu[i] = P.cu_rows[min(bl + i, P.B)];
#pragma unroll
        for (int i = 0; i < PER; ++i) len[i] = PER == 1 && bl + i < P.B ? P.kv_len[bl + i] : 0;   // many: loaded once found
        int64_t sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += tiles_of(cu[i + 1] - cu[i], tt);
        int64_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, idx < before + inc);
        if (hit) {
            const int w = __ffs(hit) - 1;
            RowTile t = {-1, 0, 0, 0, 0};
            if (lane == w) {
                int64_t at = idx - before - (inc - sum);     // tile of the lane's sequences
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int n = max(0, cu[i + 1] - cu[i]);
                    const int64_t nt = tiles_of(n, tt);
                    if (t.b < 0 && at < nt) t = RowTile{bl + i, static_cast<int>(at * tt), n, cu[i], PER == 1 ? len[i] : P.kv_len[bl + i]};
                    at -= nt;
                }
            }
            t.b = __shfl_sync(0xffffffffu, t.b, w);
            t.tok0 = __shfl_sync(0xffffffffu, t.tok0, w);
            t.n = __shfl_sync(0xffffffffu, t.n, w);
            t.row0 = __shfl_sync(0xffffffffu, t.row0, w);
            t.len = __shfl_sync(0xffffffffu, t.len, w);
            return t;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    return RowTile{-1, 0, 0, 0, 0};
}
__device__ __forceinline__ RowTile find_tile(const PagedAttn& P, int idx, int tt, int lane) {
    return P.B <= 32 ? find_tile_by<1>(P, idx, tt, lane) : find_tile_by<8>(P, idx, tt, lane);
}

// Whether a sequence has more rows than max_rows (their tiles may be more than the grid was made for), or cu_rows makes
// no sense.
__device__ __forceinline__ bool bad_rows(const PagedAttn& P, int lane) {
    bool bad = false;
    for (int b = lane; b < P.B; b += 32) {
        const int r0 = P.cu_rows[b], r1 = P.cu_rows[b + 1];
        bad |= !rows_sound(r0, r1, P.T) || r1 - r0 > P.max_rows;
    }
    return __any_sync(0xffffffffu, bad);
}

// The keys of a CTA: boxes of the sinks, [0, se), then [ws, end), laid end to end: total keys, a multiple
// of the box. p0 and p1: first and last position of its rows.
struct Keys {
    int se, ws, total;
    __device__ __forceinline__ int key(int v) const { return v < se ? v : v - se + ws; }
};
__device__ __forceinline__ Keys keys_of(int p0, int p1, int window, int sinks, int box) {
    Keys k;
    k.se = 0;
    k.ws = 0;
    const int end = (p1 + box) & -box;           // p1 + 1 rounded up (box is a power of two)
    if (window > 0) {
        const int first = max(0, p0 - window + 1);
        k.ws = first & -box;
        const int s = min(sinks, p1 + 1);
        k.se = max(0, min((s + box - 1) & -box, k.ws));
    }
    k.total = p1 < 0 ? 0 : k.se + end - k.ws;
    return k;
}

// What a row at position p sees of the keys laid end to end: [0, a) and [b, c). (Where the sinks reach past
// their own boxes, se = ws and the layout is the keys' own order.)
struct Seen {
    int a, b, c;
};
__device__ __forceinline__ Seen seen_of(const Keys& k, int p, int window, int sinks) {
    Seen s;
    s.c = p + 1 - k.ws + k.se;
    s.b = window > 0 ? max(0, p - window + 1 - k.ws + k.se) : 0;
    s.a = window > 0 ? min(sinks, p + 1) : 0;
    return s;
}
__device__ __forceinline__ uint32_t low_mask(int n) { return n >= 32 ? ~0u : (1u << max(n, 0)) - 1u; }
// which of 32 keys from v on
__device__ __forceinline__ uint32_t seen32(const Seen& s, int v) { return low_mask(s.a - v) | (low_mask(s.c - v) & ~low_mask(s.b - v)); }

__device__ __forceinline__ int page_of(const PagedAttn& P, int b, int key) {
    const int pg = P.table[(int64_t)b * P.max_pages + key / P.page];
    if (pg < 0 || pg >= P.n_pages) {
        set_err(P.err, ERR_PAGE_ID);     // and page 0 is read instead
        return 0;
    }
    return pg;
}

// Keys of partly hidden blocks whose V is not finite: the MMAs ran with those V rows cleared (0 * NaN is NaN, and a row
// that does not see the key must not get it), and the rows that do see them add p V here, at the end. One record per
// partly hidden block: its number and a bit per key.
constexpr int RW_MAX_EDGE = 12;        // blocks that some row of a CTA sees and another does not: 8 at most
struct Spoilt {
    int any, n;
    struct {
        int block;
        uint32_t keys[4];
    } e[RW_MAX_EDGE];
};

template <typename T, int D>
__device__ __noinline__ void add_spoilt(const PagedAttn& P, const Spoilt* sp, int b, int g, int64_t qoff, int p, Keys K, float m, uint32_t o_tm) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(P.Q) + qoff);
    const Seen seen = seen_of(K, p, P.window, P.sinks);
    for (int c = 0; c < D; c += 32) {
        float o[32];
        ld32(o_tm + c, o);
        wait_ld();
        for (int e = 0; e < sp->n; ++e)
            for (int i = 0; i < RW_BLOCK; ++i) {
                if (!(sp->e[e].keys[i >> 5] >> (i & 31) & 1)) continue;
                const int v0 = sp->e[e].block * RW_BLOCK + i, key = K.key(v0);
                if (p < 0 || !(v0 < seen.a || (v0 >= seen.b && v0 < seen.c))) continue;
                const int64_t pg = page_of(P, b, key);
                const int slot = key % P.page;
                const int64_t* st = P.kv_stride;
                const uint4* k = reinterpret_cast<const uint4*>(static_cast<const T*>(P.k_base) + pg * st[0] + g * st[1] + slot * st[2]);
                const uint4* v = reinterpret_cast<const uint4*>(static_cast<const T*>(P.v_base) + pg * st[3] + g * st[4] + slot * st[5]) + c / 8;
                float s = 0.f;
                for (int d = 0; d < D / 8; ++d) {
                    const uint4 x = q[d], y = k[d];
                    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const float2 f = unpack16<T>(xw[h]), w = unpack16<T>(yw[h]);
                        s = fmaf(f.x, w.x, fmaf(f.y, w.y, s));
                    }
                }
                const float w = ex2_approx(fmaf(s, P.scale_log2, -m));
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint4 x = v[d];
                    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const float2 f = unpack16<T>(xw[h]);
                        o[8 * d + 2 * h] = fmaf(w, f.x, o[8 * d + 2 * h]);
                        o[8 * d + 2 * h + 1] = fmaf(w, f.y, o[8 * d + 2 * h + 1]);
                    }
                }
            }
        __syncwarp();
        st32(o_tm + c, reinterpret_cast<const uint32_t*>(o));
        wait_st();
    }
}

// Whether one of 8 packed values is infinite or NaN: then its product with 0 is NaN, and so is the sum.
template <typename T> __device__ __forceinline__ bool not_finite8(uint4 x);
template <> __device__ __forceinline__ bool not_finite8<__half>(uint4 x) {
    const __half2 z = __float2half2_rn(0.f);
    const __half2 a = __hfma2(u32_as_h2(x.x), z, __hmul2(u32_as_h2(x.y), z)), b = __hfma2(u32_as_h2(x.z), z, __hmul2(u32_as_h2(x.w), z));
    return (h2_as_u32(__hadd2(a, b)) & 0x7fff7fffu) != 0;
}
template <> __device__ __forceinline__ bool not_finite8<__nv_bfloat16>(uint4 x) {
    const __nv_bfloat162 z = __float2bfloat162_rn(0.f);
    auto v = [](const uint32_t& u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
    const __nv_bfloat162 s = __hadd2(__hfma2(v(x.x), z, __hmul2(v(x.y), z)), __hfma2(v(x.z), z, __hmul2(v(x.w), z)));
    return (*reinterpret_cast<const uint32_t*>(&s) & 0x7fff7fffu) != 0;
}

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

// Partial of a CTA: m [2][128], l [2][128], O [2][D/4][128] float4 (a warp's rows side by side).
__host__ __device__ constexpr size_t rows_partial_floats(int D) { return (size_t)2 * RW_M * (D + 2); }

template <typename T, int D>
__global__ void __launch_bounds__(RW_THREADS, 1) paged_rows_kernel(const __grid_constant__ PagedAttn P) {
    using C = RCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_base = smem_u32(smem);
    // barriers: Q of each tile; K ring full, empty; V ring full, empty, looked over; of each tile: S ready, P ready and S read (4 warps), O += P V done
    constexpr int B_Q = 0, B_KF = 16, B_KE = B_KF + 8 * C::NK, B_VF = B_KE + 8 * C::NK, B_VE = B_VF + 8 * C::NV,
                  B_X = B_VE + 8 * C::NV, B_S = B_X + 8 * C::NV, B_P = B_S + 16, B_R = B_P + 16, B_O = B_R + 16, B_DR = B_O + 16, N_BAR = B_DR / 8 + 1;
    const uint32_t bar = s_base + C::OFF_BAR;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8 * N_BAR);
    RowTile* s_tile = reinterpret_cast<RowTile*>(smem + C::OFF_BAR + 8 * N_BAR + 16);
    Spoilt* s_spoilt = reinterpret_cast<Spoilt*>(s_tile + 1);
    static_assert(8 * N_BAR + 16 + sizeof(RowTile) + sizeof(Spoilt) <= C::BAR_BYTES, "barrier area");
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int G = P.G, tpt = RW_M / G, tt = 2 * tpt;
    // later tiles first (they see the most keys); kv heads next to one another, then key splits
    const int per_tile = P.H_kv * P.n_split;
    const int tile_idx = P.row_tiles - 1 - blockIdx.x / per_tile;
    const int sub = blockIdx.x % per_tile;
    const int g = sub % P.H_kv, split = sub / P.H_kv;

    if (warp == RW_LOAD_WARP && lane == 0) {
        for (int i = 0; i < N_BAR; ++i) mbar_init(bar + 8 * i, (8 * i >= B_P && 8 * i < B_O) ? 4 : (8 * i >= B_X && 8 * i < B_S) ? 2 : 1);
        fence_mbar_init();
        s_spoilt->any = s_spoilt->n = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.tm_q) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.tm_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.tm_v) : "memory");
    }
    if (warp == RW_MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(C::TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    pdl_release();
    fence_proxy_async_all();     // the pages may have been written by the kernel before, and are read by TMA
    if (warp == RW_LOAD_WARP) {
        const RowTile t = find_tile(P, tile_idx, tt, lane);
        if (lane == 0) *s_tile = t;
        // Q at once: rows token * G + head; rows behind the sequence's hold others' or nothing
        if (t.b >= 0 && lane < (min(t.n - t.tok0, tt) > tpt ? 2 : 1)) {
            mbar_arrive_expect_tx(bar + B_Q + 8 * lane, C::CH * G * tpt * 128);
            for (int c = 0; c < C::CH; ++c)
                tma5(s_base + lane * C::TILE + c * C::CHUNK, &P.tm_q, 0, 0, t.row0 + t.tok0 + lane * tpt, c, g, bar + B_Q + 8 * lane);
        }
        __syncwarp();
        if (blockIdx.x == 0 && bad_rows(P, lane) && lane == 0) set_err(P.err, ERR_KV_LEN);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    const RowTile rt = *s_tile;

    if (rt.b >= 0) {
        const int b = rt.b;
        int len = rt.len;
        if (len > (int64_t)P.max_pages * P.page) {
            if (tid == 0) set_err(P.err, ERR_KV_LEN);
            len = P.max_pages * P.page;
        }
        len = max(len, 0);
        const int rows_here = min(rt.n - rt.tok0, tt);          // rows (tokens) of this CTA
        const int ntile = rows_here > tpt ? 2 : 1;
        const int p0 = len - rt.n + rt.tok0, p1 = p0 + rows_here - 1;
        const int box = P.box;
        const Keys K = keys_of(p0, p1, P.window, P.sinks, box);
        const int nblk_all = (K.total + RW_BLOCK - 1) / RW_BLOCK;
        // (at most 2^23 blocks and 152 splits: within 32 bits)
        const int j0 = P.n_split == 1 ? 0 : static_cast<int>(static_cast<uint32_t>(nblk_all) * split / static_cast<uint32_t>(P.n_split));
        const int j1 = P.n_split == 1 ? nblk_all : static_cast<int>(static_cast<uint32_t>(nblk_all) * (split + 1) / static_cast<uint32_t>(P.n_split));
        const int nb = j1 - j0;
        auto keys_in = [&](int j) { return min(RW_BLOCK, K.total - (j0 + j) * RW_BLOCK); };   // of block j of this CTA
        bool failed = false;

        if (warp >= RW_MMA_WARP) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(RW_REGS_OTHER));
            if (warp == RW_LOAD_WARP) {
                // ------------------------------------------------------------ loads
                if (nb > 0) {
                    const int bpb = RW_BLOCK / box;     // boxes of a whole block
                    int pg = 0, tok = 0;
                    auto locate = [&](int j) {          // lane i: page and token of box i of block j
                        const int v = (j0 + j) * RW_BLOCK + lane * box;
                        if (lane < bpb && v < K.total) {
                            const int key = K.key(v);
                            pg = page_of(P, b, key);
                            tok = key % P.page;
                        }
                    };
                    locate(0);
                    auto load = [&](int j, const CUtensorMap* tm, int full, int empty, int off, int n) -> bool {
                        const int st = j % n, nk = keys_in(j);
                        if (j >= n && !__all_sync(0xffffffffu, wait_bar(bar + empty + 8 * st, (j / n - 1) & 1))) return false;
                        if (lane == 0) mbar_arrive_expect_tx(bar + full + 8 * st, nk * D * 2);
                        __syncwarp();
                        if (lane * box < nk) {
                            const uint32_t dst = s_base + off + st * C::TILE + lane * box * 128;
                            for (int c = 0; c < C::CH; ++c) tma5(dst + c * C::CHUNK, tm, 0, tok, c, g, pg, bar + full + 8 * st);
                        }
                        return true;
                    };
                    int jk = 0, jv = 0;      // blocks whose K, V were issued
                    for (; jv < nb; ++jv) {
                        if (!load(jk, &P.tm_k, B_KF, B_KE, C::OFF_RING, C::NK)) break;
                        ++jk;
                        if (!load(jv, &P.tm_v, B_VF, B_VE, C::OFF_V, C::NV)) break;
                        if (jv + 1 < nb) locate(jv + 1);
                    }
                    if (jv < nb && lane == 0) set_err(P.err, ERR_ROWS_LOAD);
                    // the copies in flight land before the CTA can end, whatever the other warps do (Q's below)
                    for (int j = max(0, jk - C::NK); j < jk; ++j)
                        if (!__all_sync(0xffffffffu, wait_bar(bar + B_KF + 8 * (j % C::NK), (j / C::NK) & 1))) break;
                    for (int j = max(0, jv - C::NV); j < jv; ++j)
                        if (!__all_sync(0xffffffffu, wait_bar(bar + B_VF + 8 * (j % C::NV), (j / C::NV) & 1))) break;
                }
                for (int t = 0; t < ntile; ++t)
                    if (!__all_sync(0xffffffffu, wait_bar(bar + B_Q + 8 * t, 0))) break;
            } else if (warp == RW_MMA_WARP) {
                // ------------------------------------------------------------ MMAs
                // broadcasts, so that the compiler sees them as uniform
                const int nbu = __shfl_sync(0xffffffffu, nb, 0), ntu = __shfl_sync(0xffffffffu, ntile, 0);
                const int nk_last = __shfl_sync(0xffffffffu, nb > 0 ? keys_in(nb - 1) : 0, 0);
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                constexpr int FMT = IsBf16<T>::value ? 1 : 0;
                constexpr uint32_t ID_PV = idesc_16(FMT, D, 1), ID_S = idesc_16(FMT, RW_BLOCK, 0);
                const uint64_t q_desc = desc_sw128(s_base, 16);
                const uint64_t k_desc = desc_sw128(s_base + C::OFF_RING, 16);
                const uint64_t v_desc = desc_sw128(s_base + C::OFF_V, C::CHUNK);
                auto wait = [&](int off, int phase) {
                    if (!failed && !__all_sync(0xffffffffu, wait_bar(bar + off, phase & 1))) failed = true;
                    return !failed;
                };
                auto issue_S = [&](int t, int j) {   // S_t = Q_t K(j)^T
                    const int st = j % C::NK;
                    const uint32_t id = j + 1 < nbu ? ID_S : idesc_16(FMT, nk_last, 0);
                    const uint64_t qd = q_desc + static_cast<uint64_t>((t * C::TILE) >> 4), kd = k_desc + static_cast<uint64_t>((st * C::TILE) >> 4);
#pragma unroll
                    for (int c = 0; c < C::CH; ++c)
                        mma_ss4(tm + C::S_COL + 128 * t, qd + c * (C::CHUNK >> 4), kd + c * (C::CHUNK >> 4), id, c > 0);
                    commit(bar + B_S + 8 * t);
                    if (t == ntu - 1) commit(bar + B_KE + 8 * st);
                };
                auto issue_PV = [&](int t, int j) {  // O_t += P_t V(j)
                    const int st = j % C::NV;
                    const uint64_t vd = v_desc + static_cast<uint64_t>((st * C::TILE) >> 4);
                    const uint32_t d = tm + C::O_COL + D * t, a = tm + C::P_COL + C::P_STEP * t;
                    if (j + 1 < nbu || nk_last == RW_BLOCK) {
                        mma_ts8(d, a, vd, ID_PV, j > 0);
                    } else {
                        for (int u = 0; 16 * u < nk_last; ++u)
                            mma_ts(d, a + 8 * u, vd + static_cast<uint64_t>(u * (2048 >> 4)), ID_PV, j > 0 || u > 0);
                    }
                    commit(bar + B_O + 8 * t);
                    if (t == ntu - 1) commit(bar + B_VE + 8 * st);
                };
                if (nbu > 0 && wait(B_KF, 0)) {
                    for (int t = 0; t < ntu; ++t)
                        if (wait(B_Q + 8 * t, 0)) issue_S(t, 0);
                    for (int j = 0; j < nbu && !failed; ++j) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (t >= ntu) break;
                            if (t == 0 && !(wait(B_VF + 8 * (j % C::NV), j / C::NV) && wait(B_X + 8 * (j % C::NV), j / C::NV) &&
                                            (j + 1 == nbu || wait(B_KF + 8 * ((j + 1) % C::NK), (j + 1) / C::NK)))) break;
                            if (C::APART && j + 1 < nbu) {
                                if (!wait(B_R + 8 * t, j)) break;
                                fence_after();
                                issue_S(t, j + 1);
                            }
                            if (!wait(B_P + 8 * t, j)) break;
                            fence_after();
                            issue_PV(t, j);
                            if (!C::APART && j + 1 < nbu) issue_S(t, j + 1);
                        }
                    }
                }
                if (failed && lane == 0) set_err(P.err, ERR_ROWS_MMA);
                commit(bar + B_DR);      // no MMA writes TMEM any more when the CTA gives it back
                __all_sync(0xffffffffu, wait_bar(bar + B_DR, 0));
            } else {
                // -------------------------------------------------------- V blocks looked over (the two warps left)
                // Where a block is partly hidden from the CTA's rows, V rows that none of them sees are cleared (they
                // may hold anything), and so are those that are not finite, which are put on record. A warp takes 64 V
                // rows, 8 lanes of 16 bytes a row and chunk. Other blocks are passed on as they are.
                const int w = warp - RW_EDGE_WARP;
                int n_edge = 0;
                for (int j = 0; j < nb && !failed; ++j) {
                    const int st = j % C::NV, v0 = (j0 + j) * RW_BLOCK, nk = keys_in(j);
                    const int ka = K.key(v0), kz = K.key(v0 + nk - 1);
                    if (!__all_sync(0xffffffffu, wait_bar(bar + B_VF + 8 * st, (j / C::NV) & 1))) {
                        failed = true;
                        break;
                    }
                    if (kz > p0 || kz - ka != nk - 1 || (P.window > 0 && ka <= p1 - P.window && kz >= P.sinks)) {
                        bool cleared = false;
                        for (int h = 0; h < 2; ++h) {
                            const int r = 64 * w + 32 * h + lane, key = K.key(v0 + r);
                            const uint32_t clear = __ballot_sync(0xffffffffu, r < nk && (key > p1 || (P.window > 0 && key <= p0 - P.window && key >= P.sinks)));
                            const uint32_t live = __ballot_sync(0xffffffffu, r < nk) & ~clear;
                            uint8_t* rows = smem + C::OFF_V + st * C::TILE + (64 * w + 32 * h) * 128 + lane * 16;
                            uint32_t spoilt = 0;
                            if (live && n_edge < RW_MAX_EDGE) {
                                uint32_t bad = 0;          // bit i: this lane's piece of row 4 i + lane / 8
#pragma unroll
                                for (int i = 0; i < 8; ++i)
#pragma unroll
                                    for (int c = 0; c < C::CH; ++c)
                                        bad |= static_cast<uint32_t>(not_finite8<T>(*reinterpret_cast<const uint4*>(rows + c * C::CHUNK + i * 512))) << i;
                                if (__any_sync(0xffffffffu, bad)) {
                                    for (int i = 0; i < 8; ++i) {
                                        const uint32_t f = __ballot_sync(0xffffffffu, bad >> i & 1);
                                        for (int q = 0; q < 4; ++q) spoilt |= (f >> (8 * q) & 0xffu ? 1u : 0u) << (4 * i + q);
                                    }
                                    spoilt &= live;
                                }
                            }
                            if (n_edge < RW_MAX_EDGE && lane == 0) {
                                s_spoilt->e[n_edge].block = j0 + j;
                                s_spoilt->e[n_edge].keys[2 * w + h] = spoilt;
                                s_spoilt->n = n_edge + 1;
                                if (spoilt) s_spoilt->any = 1;
                            }
                            if (clear | spoilt) {
                                for (int i = 0; i < 8; ++i)
                                    if ((clear | spoilt) >> (4 * i + (lane >> 3)) & 1)
                                        for (int c = 0; c < C::CH; ++c) *reinterpret_cast<uint4*>(rows + c * C::CHUNK + i * 512) = make_uint4(0, 0, 0, 0);
                                cleared = true;
                            }
                        }
                        if (n_edge < RW_MAX_EDGE) ++n_edge;
                        if (cleared) fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(bar + B_X + 8 * st);
                }
                if (failed && lane == 0) set_err(P.err, ERR_ROWS_LOAD);
                // the record is complete, for either tile
                asm volatile("barrier.cta.arrive 1, 192;" ::: "memory");
                if (ntile == 2) asm volatile("barrier.cta.arrive 2, 192;" ::: "memory");
            }
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(RW_REGS_SOFTMAX));
            if (warp < 4 * ntile) {
                // -------------------------------------------------------- softmax: row r of tile t
                const int t = warp >> 2, r = (warp & 3) * 32 + lane;
                const int rtok = t * tpt + r / G;                     // token of the CTA
                const int64_t trow = (int64_t)rt.row0 + rt.tok0 + rtok;
                const bool row_ok = r < tpt * G && rtok < rows_here && trow >= 0 && trow < P.T;
                const int p = row_ok ? p0 + rtok : -1;
                const int hq = g * G + r % G;
                // positions of the tile's first and last rows
                const int pa = p0 + t * tpt, pz = min(p1, pa + tpt - 1);
                const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
                const uint32_t s_tm = tmem + C::S_COL + 128 * t + lane_base, p_tm = tmem + C::P_COL + C::P_STEP * t + lane_base, o_tm = tmem + C::O_COL + D * t + lane_base;
                const float sc = P.scale_log2;
                const Seen seen = seen_of(K, p, P.window, P.sinks);
                float m = -INFINITY, l = 0.f;
                // A wait that runs out only marks the warp: it goes on, without work, to the barrier at the end.
                for (int j = 0; j < nb; ++j) {
                    const int v0 = (j0 + j) * RW_BLOCK, nk = keys_in(j);
                    const int ka = K.key(v0), kz = K.key(v0 + nk - 1);
                    if (!__all_sync(0xffffffffu, !failed && wait_bar(bar + B_S + 8 * t, j & 1))) failed = true;
                    fence_after();
                    // every row of the tile sees the whole block, or masks: 16 keys at a time
                    const bool full = nk == RW_BLOCK && kz - ka == RW_BLOCK - 1 && kz <= pa &&
                                      (P.window <= 0 || ka > pz - P.window || kz < P.sinks);
                    // per 32 keys: bits of those the row sees; and whether the warp's rows see all of them, or none
                    uint32_t see[RW_BLOCK / 32];
                    uint32_t part = 0, none = 0;
                    if (!full) {
#pragma unroll
                        for (int c = 0; c < RW_BLOCK / 32; ++c) {
                            see[c] = seen32(seen, v0 + 32 * c);
                            if (__all_sync(0xffffffffu, see[c] == 0)) none |= 1u << c;
                            else if (!__all_sync(0xffffffffu, see[c] == ~0u || !row_ok)) part |= 1u << c;
                        }
                    }
                    auto mask = [&](int c, float* x) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = see[c] & (1u << i) ? x[i] : -INFINITY;
                    };
                    // p = 2^(s - m) at the running maximum, packed, and their sum
                    uint32_t pk[RW_BLOCK / 2];
                    float bs = 0.f;
                    auto weights = [&](auto masked) {
                        const float ms = m > -INFINITY ? m : 0.f;
                        const uint64_t sc2 = f2_pack(sc, sc), nm2 = f2_pack(-ms, -ms);
                        uint64_t acc[2] = {0, 0};
                        float x[2][32];
                        ld32(s_tm, x[0]);
                        wait_ld();
#pragma unroll
                        for (int c = 0; c < RW_BLOCK / 32; ++c) {   // the next chunk's load runs under this one's arithmetic
                            if (c + 1 < RW_BLOCK / 32) ld32(s_tm + 32 * (c + 1), x[(c + 1) & 1]);
                            float* y = x[c & 1];
                            if (masked && (none >> c & 1)) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) pk[16 * c + i] = 0;
                            } else {
                                if (masked && (part >> c & 1)) mask(c, y);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    float x0, x1;
                                    f2_unpack(f2_fma(f2_pack(y[2 * i], y[2 * i + 1]), sc2, nm2), x0, x1);
                                    x0 = ex2_approx(x0);
                                    x1 = ex2_approx(x1);
                                    acc[i & 1] = f2_add(acc[i & 1], f2_pack(x0, x1));
                                    pk[16 * c + i] = pack16<T>(x0, x1);
                                }
                            }
                            if (c + 1 < RW_BLOCK / 32) wait_ld();
                        }
                        float a0, a1, b0, b1;
                        f2_unpack(acc[0], a0, a1);
                        f2_unpack(acc[1], b0, b1);
                        bs = (a0 + a1) + (b0 + b1);
                    };
                    // The maximum moves only when it has to: a sum up to CAP bounds every p by it, which fp16 and
                    // bf16 hold as exactly as smaller ones. Otherwise (and where a row has no maximum yet) the block's
                    // maximum is found, O and l are rescaled, and the weights taken again.
                    bool again = true;
                    if (j > 0) {
                        if (!failed) {
                            if (full) weights(std::false_type());
                            else weights(std::true_type());
                        }
                        again = __any_sync(0xffffffffu, row_ok && (!(bs <= Weights<T>::CAP) || m == -INFINITY));
                    }
                    if (again) {
                        float bm = -INFINITY;
                        if (!failed) {
#pragma unroll
                            for (int c = 0; c < RW_BLOCK / 32; ++c) {
                                if (none >> c & 1) continue;
                                float x[32];
                                ld32(s_tm + 32 * c, x);
                                wait_ld();
                                if (part >> c & 1) mask(c, x);
                                float b0 = fmaxf(x[0], x[1]), b1 = fmaxf(x[2], x[3]);
#pragma unroll
                                for (int i = 4; i < 32; i += 4) {
                                    b0 = fmaxf(b0, fmaxf(x[i], x[i + 1]));
                                    b1 = fmaxf(b1, fmaxf(x[i + 2], x[i + 3]));
                                }
                                bm = fmaxf(bm, fmaxf(b0, b1));
                            }
                        }
                        const float mn = fmaxf(m, bm * sc - Weights<T>::TOP);
                        const float al = mn > m ? ex2_approx(m - mn) : 1.0f;     // 0 from m = -inf
                        if (j > 0) {   // O is quiet once P V of the previous block is done
                            if (!__all_sync(0xffffffffu, !failed && wait_bar(bar + B_O + 8 * t, (j - 1) & 1))) failed = true;
                            fence_after();
                            if (!failed) {
#pragma unroll 1
                                for (int c = 0; c < D; c += 32) {
                                    float o[32];
                                    ld32(o_tm + c, o);
                                    wait_ld();
#pragma unroll
                                    for (int i = 0; i < 32; ++i) o[i] *= al;
                                    st32(o_tm + c, reinterpret_cast<const uint32_t*>(o));
                                }
                            }
                        }
                        l *= al;
                        m = mn;
                        if (!failed) {
                            if (full) weights(std::false_type());
                            else weights(std::true_type());
                        }
                    }
                    if (!failed) {
                        if (C::APART) {
                            fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar + B_R + 8 * t);
                            // P's columns are free once P V of the previous block is done
                            if (j > 0) {
                                if (!__all_sync(0xffffffffu, wait_bar(bar + B_O + 8 * t, (j - 1) & 1))) failed = true;
                                fence_after();
                            }
                        }
                        st32(p_tm, pk);
                        st32(p_tm + 32, pk + 32);
                        l += bs;
                        wait_st();
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar + B_P + 8 * t);
                    }
                }
                if (nb > 0 && !failed && !__all_sync(0xffffffffu, wait_bar(bar + B_O + 8 * t, (nb - 1) & 1))) {
                    set_err(P.err, ERR_ROWS_O);
                    failed = true;
                } else if (failed) {
                    set_err(P.err, ERR_ROWS_SOFTMAX);
                }
                fence_after();
                // without keys nothing else has waited for Q, over which the result is staged
                if (nb == 0 && !__all_sync(0xffffffffu, wait_bar(bar + B_Q + 8 * t, 0))) failed = true;
                // the record of spoilt keys is complete
                asm volatile("barrier.cta.sync %0, 192;" ::"r"(1 + t) : "memory");
                if (!failed) {
                    const int row = static_cast<int>(trow * P.row_heads + hq);      // (T row_heads < 2^31)
                    const bool direct = P.n_split == 1;
                    RowEnd e = {1.f, 0.f, 0.f, false};
                    if (direct && row_ok) e = row_end(P, row, m, l);
                    float* part = P.ws + ((size_t)tile_idx * per_tile + sub) * rows_partial_floats(D);
                    // the warp's 32 result rows, staged over the tile's Q (which no MMA reads any more)
                    uint8_t* stage = smem + t * C::TILE + (warp & 3) * 32 * (D * 2);
                    if (nb > 0 && s_spoilt->any)
                        add_spoilt<T, D>(P, s_spoilt, b, g, trow * P.q_row + (int64_t)hq * P.q_head, p, K, m, o_tm);
                    const bool nothing = __any_sync(0xffffffffu, l == 0.f);
#pragma unroll 2
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        if (nb > 0) {
                            ld32(o_tm + c, o);
                            wait_ld();
                        }
                        if (nothing && l == 0.f) {     // nothing seen (and O unwritten where the CTA has no keys)
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = 0.f;
                        }
                        if (direct) {
                            const float4* pr = reinterpret_cast<const float4*>(P.O_prior + (int64_t)row * D + c);
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                float x[8];
#pragma unroll
                                for (int q = 0; q < 8; ++q) x[q] = o[i + q] * e.wo;
                                if (e.prior) {
                                    const float4 a = pr[i / 4], c4 = pr[i / 4 + 1];
                                    x[0] = fmaf(a.x, e.wp, x[0]); x[1] = fmaf(a.y, e.wp, x[1]);
                                    x[2] = fmaf(a.z, e.wp, x[2]); x[3] = fmaf(a.w, e.wp, x[3]);
                                    x[4] = fmaf(c4.x, e.wp, x[4]); x[5] = fmaf(c4.y, e.wp, x[5]);
                                    x[6] = fmaf(c4.z, e.wp, x[6]); x[7] = fmaf(c4.w, e.wp, x[7]);
                                }
                                *reinterpret_cast<uint4*>(stage + lane * (D * 2) + (((c + i) / 8 ^ lane) & (D / 8 - 1)) * 16) =
                                    make_uint4(pack16<T>(x[0], x[1]), pack16<T>(x[2], x[3]), pack16<T>(x[4], x[5]), pack16<T>(x[6], x[7]));
                            }
                        } else {   // [D/4][128 rows] float4
                            float4* po = reinterpret_cast<float4*>(part + 4 * RW_M) + ((size_t)t * (D / 4) + c / 4) * RW_M + r;
#pragma unroll
                            for (int i = 0; i < 32; i += 4) po[(i / 4) * RW_M] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                    if (direct) {
                        // whole rows out, 512 contiguous bytes of neighbouring heads an instruction
                        __syncwarp();
                        constexpr int CR = D / 8, RPI = 32 / CR;      // 16-byte pieces a row, rows an instruction
                        const uint32_t ok = __ballot_sync(0xffffffffu, row_ok);
                        const int piece = lane & (CR - 1);
#pragma unroll
                        for (int i = 0; i < 32; i += RPI) {
                            const int rr = i + lane / CR;
                            const int64_t dst = __shfl_sync(0xffffffffu, row, rr);   // (widened)
                            if (ok >> rr & 1)
                                *reinterpret_cast<uint4*>(static_cast<T*>(P.O) + dst * D + piece * 8) =
                                    *reinterpret_cast<const uint4*>(stage + rr * (D * 2) + ((piece ^ rr) & (CR - 1)) * 16);
                        }
                        if (row_ok && P.LSE) P.LSE[row] = e.lse;
                    } else {
                        part[t * RW_M + r] = m;
                        part[2 * RW_M + t * RW_M + r] = l;
                    }
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == RW_MMA_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
}

// Joins the n_split partials: a CTA per tile of 128 rows and 32 columns, a thread per row.
template <typename T, int D>
__global__ void __launch_bounds__(RW_M) paged_rows_join_kernel(const __grid_constant__ PagedAttn P) {
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31, r = threadIdx.x;
    const int tpt = RW_M / P.G, tt = 2 * tpt;
    const int tile_idx = blockIdx.x / P.H_kv, g = blockIdx.x % P.H_kv;
    const int t = blockIdx.y & 1, c0 = (blockIdx.y >> 1) * 32;
    const RowTile rt = find_tile(P, tile_idx, tt, lane);
    if (rt.b < 0) return;
    const int rtok = t * tpt + r / P.G;
    const int64_t trow = (int64_t)rt.row0 + rt.tok0 + rtok;
    if (r >= tpt * P.G || rtok >= min(rt.n - rt.tok0, tt) || trow < 0 || trow >= P.T) return;
    const int64_t row = trow * P.row_heads + g * P.G + r % P.G;
    auto part = [&](int s) { return P.ws + ((size_t)tile_idx * P.H_kv * P.n_split + (size_t)s * P.H_kv + g) * rows_partial_floats(D); };
    float M = -INFINITY, L = 0.f;
#pragma unroll 4
    for (int s = 0; s < P.n_split; ++s) M = fmaxf(M, part(s)[t * RW_M + r]);
    float4 acc[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int s = 0; s < P.n_split; ++s) {
        const float* p = part(s);
        const float m = p[t * RW_M + r];
        const float w = m > -INFINITY ? ex2_approx(m - M) : 1.f;   // (a part without keys holds zeros)
        L = fmaf(w, p[2 * RW_M + t * RW_M + r], L);
        const float4* po = reinterpret_cast<const float4*>(p + 4 * RW_M) + ((size_t)t * (D / 4) + c0 / 4) * RW_M + r;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float4 v = po[c * RW_M];
            acc[c].x = fmaf(w, v.x, acc[c].x);
            acc[c].y = fmaf(w, v.y, acc[c].y);
            acc[c].z = fmaf(w, v.z, acc[c].z);
            acc[c].w = fmaf(w, v.w, acc[c].w);
        }
    }
    const RowEnd e = row_end(P, row, M, L);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(P.O) + row * D + c0);
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
        float4 x = acc[c], y = acc[c + 1];
        x = make_float4(x.x * e.wo, x.y * e.wo, x.z * e.wo, x.w * e.wo);
        y = make_float4(y.x * e.wo, y.y * e.wo, y.z * e.wo, y.w * e.wo);
        if (e.prior) {
            const float4* pr = reinterpret_cast<const float4*>(P.O_prior + row * D + c0 + 4 * c);
            const float4 a = pr[0], b = pr[1];
            x.x = fmaf(a.x, e.wp, x.x); x.y = fmaf(a.y, e.wp, x.y); x.z = fmaf(a.z, e.wp, x.z); x.w = fmaf(a.w, e.wp, x.w);
            y.x = fmaf(b.x, e.wp, y.x); y.y = fmaf(b.y, e.wp, y.y); y.z = fmaf(b.z, e.wp, y.z); y.w = fmaf(b.w, e.wp, y.w);
        }
        dst[c / 2] = make_uint4(pack16<T>(x.x, x.y), pack16<T>(x.z, x.w), pack16<T>(y.x, y.y), pack16<T>(y.z, y.w));
    }
    if (c0 == 0 && P.LSE) P.LSE[row] = e.lse;
}

template <typename T, int D>
cudaError_t launch_t(PagedAttn& p, cudaStream_t st) {
    using C = RCfg<D>;
    static_assert(C::SMEM <= 232448, "one CTA's shared memory");
    cudaError_t e = allow_smem<paged_rows_kernel<T, D>>(C::SMEM, p.device);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.row_tiles * p.H_kv * p.n_split);
    cfg.blockDim = dim3(RW_THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_rows_kernel<T, D>, p);
    if (e != cudaSuccess || p.n_split == 1) return e;
    cfg.gridDim = dim3(p.row_tiles * p.H_kv, 2 * (D / 32));
    cfg.blockDim = dim3(RW_M);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, paged_rows_join_kernel<T, D>, p);
}

}  // namespace

bool paged_rows_dim_ok(int D) { return D == 64 || D == 128; }
int paged_rows_box(int page) {
    int box = 16;
    while (box < RW_BLOCK && page % (2 * box) == 0) box *= 2;
    return box;
}
int paged_rows_tok_per_tile(int G) { return RW_M / G; }

size_t paged_rows_plan(PagedAttn& p, int D, int sms) {
    const int tt = 2 * (RW_M / p.G);
    // at most, whatever the sequences' shares
    p.row_tiles = static_cast<int>(std::min<int64_t>(p.T / tt + std::min(p.B, p.T), (int64_t)p.B * ((p.max_rows + tt - 1) / tt)));
    p.box = paged_rows_box(p.page);
    // Keys are split when the row tiles leave SMs idle: as many splits as fill them once, each of at least 4 blocks
    // of the longest cache the table can hold. The tiles are taken as those of full ones, or one per sequence.
    const int64_t tiles = std::max<int64_t>((p.T + tt - 1) / tt, std::min(p.B, p.T));
    const int64_t ctas = std::min<int64_t>(tiles, p.row_tiles) * p.H_kv;
    int64_t bound = (int64_t)p.max_pages * p.page;
    if (p.window > 0) {
        const int64_t w = (int64_t)p.window + tt + p.sinks + 2 * p.box;
        if (w < bound) bound = w;
    }
    int64_t ns = ctas >= sms ? 1 : sms / ctas;
    const int64_t most = bound / (4 * RW_BLOCK);
    if (ns > most) ns = most;
    p.n_split = ns < 1 ? 1 : static_cast<int>(ns);
    return p.n_split == 1 ? 0 : (size_t)p.row_tiles * p.H_kv * p.n_split * rows_partial_floats(D) * sizeof(float);
}

cudaError_t launch_paged_rows(PagedAttn& p, int D, cudaStream_t st) {
    if (p.dtype == PCK_DT_F16) return D == 64 ? launch_t<__half, 64>(p, st) : launch_t<__half, 128>(p, st);
    return D == 64 ? launch_t<__nv_bfloat16, 64>(p, st) : launch_t<__nv_bfloat16, 128>(p, st);
}

}  // namespace pck
