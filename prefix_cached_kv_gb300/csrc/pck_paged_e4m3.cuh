// pck_paged_e4m3.cuh -- the quantised paged cache (internal to libpck): its element format, and the parameter blocks
// and launchers of the operators that only it has.
//
// A head row of a token is D codes in e4m3 (1-4-3 bits, largest value 448, NaN = 0x7f, no infinities) and one scale, a power
// of two 2^e held as its biased exponent e + 127 in a byte (E8M0: 0 .. 254, and 255 is NaN; the append writes 1 .. 247). A
// value is code * 2^e: exact in fp32 (below 2^128) and, for e of -124 .. 119, in bf16. A floating code has the same relative step
// whatever the scale, so the scale only keeps the row in range, and a power of two keeps every other rounding out of the format.
#pragma once

#include "pck_paged.cuh"

namespace pck {

// Two codes, the first in the low byte (NaN stays NaN; what is beyond 448 becomes 448).
__device__ __forceinline__ uint32_t codes2(float x0, float x1) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(x0), "f"(x1));
    return r;
}
// The four codes of a word as two pairs of fp16 values (exact), the first two in `a`.
__device__ __forceinline__ void half_codes(uint32_t w, uint32_t& a, uint32_t& b) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }" : "=r"(a), "=r"(b) : "r"(w));
}

// The scale's byte for a row whose largest finite magnitude is a (finite): 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_byte(float a) {
    const uint32_t u = __float_as_uint(a);
    return max(1, static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u));
}
__device__ __forceinline__ float scale_down(int byte) { return __uint_as_float(static_cast<uint32_t>(254 - byte) << 23); }   // 2^-e
__device__ __forceinline__ float scale_up(uint32_t byte) {                                                                    // 2^e
    return __uint_as_float(byte == 255 ? 0x7fffffffu : max(byte << 23, 0x00400000u));    // (2^-127 is a subnormal fp32)
}

// Rows of the cache read back into the caller's rows, or into 16-bit pages of a workspace (one read of the codes either way).
struct ReadParams {
    const uint8_t *K, *V;            // codes
    const uint8_t *k_scale, *v_scale;
    int64_t k_page, k_head, k_token, v_page, v_head, v_token;
    int H, D, page, max_pages, B, T;
    int scale_heads;                 // heads of a page's scales (H, or more where a call takes some kv heads at a time)
    int64_t n_pages;
    const int32_t* cu_rows;
    const int32_t* kv_len;
    const int32_t* table;
    int max_rows;                    // rows read of a sequence at most
    int* err;
    void *Ko, *Vo;
    int64_t ko_row, ko_head, vo_row, vo_head;   // rows: strides of the outputs in elements
    // pages: the tokens that the rows see, sequence b's page i at slot i (behind the sinks' pages: counted from the window's
    // first) of its `slots` output pages [slot][head][token][D], whose numbers go to page_map [B, max_pages]; or (by_page) a page of
    // the cache at its own number, which sequences that share it write alike
    int pages, by_page, slots, window, sinks;
    int32_t* page_map;
};
cudaError_t launch_paged_read(const ReadParams& p, int out_dtype, int sms, cudaStream_t st);

// One-token attention over codes.
int paged_token_e4m3_box(const PagedAttn& p, int D);         // tokens of a TMA tile load, of a planned call
size_t paged_token_e4m3_plan(PagedAttn& p, int D, int sms);  // how the call is cut; its workspace in bytes
cudaError_t launch_paged_token_e4m3(PagedAttn& p, int D, cudaStream_t st);
cudaError_t launch_paged_token_e4m3_128(PagedAttn& p, cudaStream_t st);
cudaError_t launch_paged_token_e4m3_wide(PagedAttn& p, int D, cudaStream_t st);

cudaError_t launch_append_e4m3(const RopeParams& p, int in_dtype, int sms, cudaStream_t st);

}  // namespace pck
