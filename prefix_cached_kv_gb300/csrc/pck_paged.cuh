// pck_paged.cuh -- parameter blocks, launchers and element helpers of the paged-tail operators
// (internal to libpck): head norms with the rotary rotation, the append to a paged cache, and
// attention over that cache.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/pck.h"
#include "pck_common.cuh"

namespace pck {

// Device error codes of these operators (pck_sync reports them).
constexpr int ERR_PAGE_ID = 8;       // a page number of the table outside [0, n_pages)
constexpr int ERR_ROPE_POS = 9;      // a position outside the rotary table
constexpr int ERR_KV_LEN = 10;       // a cache length beyond the table, more rows than max_rows, or cu_rows that makes no sense
constexpr int ERR_PAGED_TOKEN = 11;  // one-token attention: a page tile never landed
constexpr int ERR_ROWS_LOAD = 12;    // row attention: producer, MMA warp, softmax, final O
constexpr int ERR_ROWS_MMA = 13;
constexpr int ERR_ROWS_SOFTMAX = 14;
constexpr int ERR_ROWS_O = 15;
constexpr int ERR_FP16_RANGE = 16;   // row attention over a quantised cache with an fp16 q: a value that fp16 cannot hold

constexpr float PG_LN2 = 0.69314718055994530942f;
constexpr float PG_LOG2E = 1.4426950408889634074f;
constexpr int PG_SUB = 16;           // tokens per cache tile of the one-token kernel (and the page granule)

// A strided set of rows [T, H, D], innermost contiguous; strides in elements.
struct RowsArg {
    const void* in;
    void* out;
    int64_t in_row, in_head, out_row, out_head;
    const void* w;       // norm weight [D] or nullptr (no weight)
    int H;
    int norm;            // 1: RMS norm of each head
};

struct RopeParams {
    RowsArg q, k, v;                 // v: append only (copied), H = 0 otherwise
    int T, D, R, interleaved;
    float eps, inv_d;
    const float* cos_sin;            // [n_pos, R]: R/2 cosines, R/2 sines
    int n_pos;
    const int32_t* positions;        // [T] or nullptr (append: the row's cache position)
    // append: destination pages of k and v (out strides: page, head, token)
    int append;
    uint8_t *k_scale, *v_scale;      // a quantised cache's scales [n_pages, H_kv, page]
    int B, page, max_pages;
    int64_t n_pages, k_page, v_page;
    const int32_t* cu_rows;
    const int32_t* kv_len;
    const int32_t* table;
    int* err;
    int spt;                         // subwarps that share a token
};

cudaError_t launch_norm_rope(const RopeParams& p, int in_dtype, int cache_dtype, int sms, cudaStream_t st);

// Attention over the pages.
struct PagedAttn {
    CUtensorMap tm_k, tm_v, tm_q;    // tm_q: row attention only
    const void* Q;
    void* O;
    float* LSE;
    const float* O_prior;            // [T, H_q, D], or nullptr
    const float* LSE_prior;          // [T, H_q]
    int64_t q_row, q_head;           // strides of Q in elements; O, LSE and the priors are contiguous
    const int32_t* cu_rows;
    const int32_t* kv_len;
    const int32_t* table;
    int B, T, H_q, H_kv, G;          // G = H_q / H_kv
    int page, max_pages;
    int n_pages;
    int window, sinks;
    int max_rows;                    // bound on a sequence's rows
    float scale_log2;                // tau * log2(e)
    int dtype, device;
    float* ws;                       // partials, then the join descriptors
    int* err;
    // one-token kernel
    int heads_per_group, n_groups;   // q heads of a kv head that share a work item, and items per kv head
    int cols;                        // columns of a work item: rows x heads
    int mode;                        // how the call is cut
    int n_ctas;
    const uint8_t *k_scale, *v_scale;   // a quantised cache's scales [n_pages, H_kv, page]
    int pieces;                      // its pages are no multiples of a unit: loaded 16 tokens at a time, by the lanes
    // row kernel
    int n_split, row_tiles, box;     // key splits, row tiles of the grid, tokens of a TMA box
    int row_heads;                   // heads of a row of O, LSE and the priors: H_q, or more where a call takes some kv heads at a time
    const void *k_base, *v_base;
    int64_t kv_stride[6];            // k page, head, token; v page, head, token (elements)
};

bool paged_token_dim_ok(int D);
int paged_token_cols(int D);                              // columns (rows x q heads of a kv head) that a work item can have
bool paged_token_rows_ok(int G, int max_rows, int D);     // ragged rows few enough for the one-token kernel
constexpr int paged_token_box_rows() { return PG_SUB; }   // tokens of a TMA tile load
size_t paged_token_plan(PagedAttn& p, int D, int sms);    // how the call is cut; its workspace in bytes
cudaError_t launch_paged_token(PagedAttn& p, int D, cudaStream_t st);
cudaError_t launch_paged_token_bf16(PagedAttn& p, int D, cudaStream_t st);
bool paged_rows_dim_ok(int D);
int paged_rows_box(int page);             // tokens of a TMA box
int paged_rows_tok_per_tile(int G);
size_t paged_rows_plan(PagedAttn& p, int D, int sms);
cudaError_t launch_paged_rows(PagedAttn& p, int D, cudaStream_t st);

// The context behind a handle (pck_api.cu).
struct CtxView {
    int device, sms;
    int* dev_err;
};
CtxView ctx_view(pck_ctx* c);
int ctx_fail(pck_ctx* c, int code, const char* fmt, ...);
void ctx_count_query(pck_ctx* c);

// Lets a kernel have `bytes` of dynamic shared memory, once per kernel and device. (Two threads may both do it: it is
// the same setting.)
template <auto KERNEL>
inline cudaError_t allow_smem(int bytes, int device) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Whether [r0, r1) can be a sequence's rows among T.
__device__ __forceinline__ bool rows_sound(int r0, int r1, int T) { return r0 >= 0 && r1 >= r0 && r1 <= T; }

// Orders this thread's earlier view of memory (ordinary loads and stores) before its later TMA accesses.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace pck
