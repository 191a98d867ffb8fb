// pck_paged_api.cu -- C entries of the paged-tail operators: argument checks on the host, tensor
// maps, launches. Nothing is launched for a call that is refused.
#include <cuda.h>
#include <cuda_runtime.h>

#include "pck_paged.cuh"
#include "pck_paged_e4m3.cuh"

using namespace pck;

namespace {

// Sets the context's device for the length of a call and puts the caller's back.
struct DeviceScope {
    int before = -1;
    bool ok = false;
    explicit DeviceScope(int device) {
        int cur = 0;
        if (cudaGetDevice(&cur) != cudaSuccess) return;
        if (cur != device) {
            if (cudaSetDevice(device) != cudaSuccess) return;
            before = cur;
        }
        ok = true;
    }
    ~DeviceScope() {
        if (before >= 0) cudaSetDevice(before);
    }
};

constexpr int DT_E4M3 = -1;             // run_rope: the append to a quantised cache
constexpr int MAX_TOKENS = 1 << 30;     // of one sequence, by the table's width; windows and sinks are cut to it

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool stride_ok(int64_t s, int64_t extent, int elems) { return extent <= 1 || (s > 0 && s % elems == 0 && s < (int64_t(1) << 36)); }

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = []() -> EncodeFn {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// Pages as {64 elements, token, D/64, head, page} with a box of `rows` tokens and `chunks` runs of 64
// elements, 128-byte swizzle: shared memory then holds [chunk][token][128 B] tiles.
bool encode_pages(CUtensorMap* tm, int dtype, void* base, int page_size, int D, int H, int64_t n_pages, int64_t s_tok,
                  int64_t s_head, int64_t s_page, int rows, int chunks) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    // a dimension of one element is never stepped over: any legal stride will do
    const int64_t st = page_size > 1 ? s_tok : D, sh = H > 1 ? s_head : D, sp = n_pages > 1 ? s_page : D;
    const cuuint64_t dims[5] = {64, (cuuint64_t)page_size, (cuuint64_t)(D / 64), (cuuint64_t)H, (cuuint64_t)n_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)st * 2, 128, (cuuint64_t)sh * 2, (cuuint64_t)sp * 2};
    const cuuint32_t box[5] = {64, (cuuint32_t)rows, (cuuint32_t)chunks, 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType dt = dtype == PCK_DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return fn(tm, dt, 5, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What both kinds of cache have in common; strides in multiples of `elems` elements (16 bytes).
template <typename Cache>
int check_pages(pck_ctx* c, const Cache* k, int elems) {
    if (k->H_kv < 1 || k->H_kv > PCK_MAX_HEADS) return ctx_fail(c, PCK_EINVAL, "H_kv=%d out of range [1, %d]", k->H_kv, PCK_MAX_HEADS);
    if (k->D < 16 || k->D > 512 || k->D % 16) return ctx_fail(c, PCK_EUNSUPPORTED, "D=%d is not a multiple of 16 up to 512", k->D);
    if (k->page_size < 16 || k->page_size % 16 || k->page_size > (1 << 20))
        return ctx_fail(c, PCK_EUNSUPPORTED, "page_size=%d is not a multiple of 16 (at most 2^20)", k->page_size);
    if (k->n_pages < 1 || k->n_pages >= (int64_t(1) << 31)) return ctx_fail(c, PCK_EINVAL, "n_pages=%lld out of range", (long long)k->n_pages);
    if (!aligned16(k->K) || !aligned16(k->V)) return ctx_fail(c, PCK_EINVAL, "K and V must be 16-byte aligned");
    if (!stride_ok(k->k_page, k->n_pages, elems) || !stride_ok(k->k_head, k->H_kv, elems) || !stride_ok(k->k_token, k->page_size, elems) ||
        !stride_ok(k->v_page, k->n_pages, elems) || !stride_ok(k->v_head, k->H_kv, elems) || !stride_ok(k->v_token, k->page_size, elems))
        return ctx_fail(c, PCK_EINVAL, "cache strides must be positive multiples of %d elements", elems);
    return PCK_OK;
}

int check_cache(pck_ctx* c, const pck_paged_cache* k) {
    if (!k || !k->K || !k->V) return ctx_fail(c, PCK_EINVAL, "NULL cache");
    if (k->dtype != PCK_DT_F16 && k->dtype != PCK_DT_BF16) return ctx_fail(c, PCK_EINVAL, "cache dtype %d is not fp16 or bf16", k->dtype);
    return check_pages(c, k, 8);
}

int check_cache(pck_ctx* c, const pck_paged_cache_e4m3* k) {
    if (!k || !k->K || !k->V || !k->K_scale || !k->V_scale) return ctx_fail(c, PCK_EINVAL, "NULL cache or scales");
    if (!aligned16(k->K_scale) || !aligned16(k->V_scale)) return ctx_fail(c, PCK_EINVAL, "K_scale and V_scale must be 16-byte aligned");
    return check_pages(c, k, 16);
}

int check_batch(pck_ctx* c, const pck_paged_batch* b, int page_size) {
    if (!b) return ctx_fail(c, PCK_EINVAL, "NULL batch");
    if (b->B < 0 || b->T < 0) return ctx_fail(c, PCK_EINVAL, "B=%d T=%d", b->B, b->T);
    if (b->B > PCK_PAGED_MAX_BATCH) return ctx_fail(c, PCK_EUNSUPPORTED, "B=%d above %d", b->B, PCK_PAGED_MAX_BATCH);
    if (b->B == 0 || b->T == 0) return PCK_OK;
    if (!b->kv_len || !b->table) return ctx_fail(c, PCK_EINVAL, "NULL kv_len or table");
    if (b->max_pages < 1 || (int64_t)b->max_pages * page_size > MAX_TOKENS)
        return ctx_fail(c, PCK_EINVAL, "max_pages=%d out of range", b->max_pages);
    if (b->max_rows < 1) return ctx_fail(c, PCK_EINVAL, "max_rows=%d", b->max_rows);
    if (!b->cu_rows && b->T != b->B)
        return ctx_fail(c, PCK_EINVAL, "without cu_rows there is one row per sequence (T=%d, B=%d)", b->T, b->B);
    return PCK_OK;
}

int elems16(int dtype) { return dtype == PCK_DT_F32 ? 4 : 8; }

int check_rows(pck_ctx* c, const pck_rows* r, const char* name, int T, int D, int dtype, bool out) {
    if (r->H < 1 || r->H > 1024) return ctx_fail(c, PCK_EINVAL, "%s: H=%d out of range [1, 1024]", name, r->H);
    const int e = elems16(dtype);
    if (!aligned16(r->in) || !aligned16(r->weight) || (out && (!r->out || !aligned16(r->out))))
        return ctx_fail(c, PCK_EINVAL, "%s: pointers must be set and 16-byte aligned", name);
    if (!stride_ok(r->in_row, T, e) || !stride_ok(r->in_head, r->H, e) ||
        (out && (!stride_ok(r->out_row, T, e) || !stride_ok(r->out_head, r->H, e))))
        return ctx_fail(c, PCK_EINVAL, "%s: strides must be positive multiples of %d elements", name, e);
    (void)D;
    return PCK_OK;
}

int check_rope(pck_ctx* c, const pck_rotary* r, int D, bool need_positions) {
    if (!r) return PCK_OK;
    if (r->R < 16 || r->R > D || r->R % 16) return ctx_fail(c, PCK_EUNSUPPORTED, "R=%d is not a multiple of 16 up to D=%d", r->R, D);
    if (!r->cos_sin || !aligned16(r->cos_sin)) return ctx_fail(c, PCK_EINVAL, "cos_sin must be set and 16-byte aligned");
    if (r->n_pos < 1) return ctx_fail(c, PCK_EINVAL, "n_pos=%d", r->n_pos);
    if (need_positions && !r->positions) return ctx_fail(c, PCK_EINVAL, "positions must be given");
    return PCK_OK;
}

RowsArg rows_arg(const pck_rows* r, bool norm) {
    RowsArg a = {};
    if (!r || !r->in) return a;
    a.in = r->in;
    a.out = r->out;
    a.in_row = r->in_row;
    a.in_head = r->in_head;
    a.out_row = r->out_row;
    a.out_head = r->out_head;
    a.w = r->weight;
    a.H = r->H;
    a.norm = norm;
    return a;
}

void set_rope(RopeParams& p, const pck_rotary* r) {
    if (!r) return;
    p.R = r->R;
    p.interleaved = r->interleaved != 0;
    p.cos_sin = r->cos_sin;
    p.n_pos = r->n_pos;
    p.positions = r->positions;
}

int run_rope(pck_ctx* c, const RopeParams& p, int in_dtype, int cache_dtype, void* stream) {
    const CtxView v = ctx_view(c);
    DeviceScope dev(v.device);
    if (!dev.ok) return ctx_fail(c, PCK_ECUDA, "cannot select device %d", v.device);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache_dtype == DT_E4M3 ? launch_append_e4m3(p, in_dtype, v.sms, st) : launch_norm_rope(p, in_dtype, cache_dtype, v.sms, st);
    return e == cudaSuccess ? PCK_OK : ctx_fail(c, PCK_ECUDA, "launch: %s", cudaGetErrorString(e));
}

bool dtype_any(int d) { return d == PCK_DT_F32 || d == PCK_DT_F16 || d == PCK_DT_BF16; }

// Shapes of an attention call, checked; fills the parts of p that its plan needs.
int attend_shape(pck_ctx* c, const pck_paged_cache* k, const pck_paged_batch* b, int H_q, int window, int sinks, PagedAttn& p) {
    int rc = check_cache(c, k);
    if (rc != PCK_OK) return rc;
    rc = check_batch(c, b, k->page_size);
    if (rc != PCK_OK) return rc;
    if (H_q < 1 || H_q > 1024 || H_q % k->H_kv) return ctx_fail(c, PCK_EINVAL, "H_q=%d is not a multiple of H_kv=%d (at most 1024)", H_q, k->H_kv);
    if (window < 0 || sinks < 0) return ctx_fail(c, PCK_EINVAL, "window=%d sinks=%d", window, sinks);
    p.max_rows = b->max_rows < b->T ? b->max_rows : b->T;     // no sequence has more rows than there are
    if (b->cu_rows) {
        if (!paged_token_rows_ok(H_q / k->H_kv, p.max_rows, k->D)) {
            if (!paged_rows_dim_ok(k->D)) return ctx_fail(c, PCK_EUNSUPPORTED, "D=%d with %d rows of a sequence: 64 or 128", k->D, p.max_rows);
            if (H_q / k->H_kv > 128) return ctx_fail(c, PCK_EUNSUPPORTED, "%d q heads per kv head: at most 128 with cu_rows", H_q / k->H_kv);
        }
    } else if (!paged_token_dim_ok(k->D)) {
        return ctx_fail(c, PCK_EUNSUPPORTED, "D=%d: 64, 128, 192 or 256", k->D);
    }
    p.B = b->B;
    p.T = b->T;
    p.H_q = H_q;
    p.H_kv = k->H_kv;
    p.G = H_q / k->H_kv;
    p.page = k->page_size;
    p.max_pages = b->max_pages;
    p.n_pages = static_cast<int>(k->n_pages);
    p.window = window < MAX_TOKENS ? window : MAX_TOKENS;
    p.sinks = sinks < MAX_TOKENS ? sinks : MAX_TOKENS;
    p.cu_rows = b->cu_rows;
    p.dtype = k->dtype;
    if ((int64_t)b->B * (((int64_t)b->max_pages * k->page_size + PG_SUB - 1) / PG_SUB + 64) >= (int64_t(1) << 31))
        return ctx_fail(c, PCK_EUNSUPPORTED, "B=%d sequences of up to %lld tokens", b->B, (long long)b->max_pages * k->page_size);
    if ((int64_t)b->T * H_q >= (int64_t(1) << 31)) return ctx_fail(c, PCK_EUNSUPPORTED, "T=%d, H_q=%d", b->T, H_q);
    return PCK_OK;
}

// Ragged rows go to the tensor-core kernel, which works on 128-row tiles, unless a sequence's rows fit the columns of
// the one-token kernel, which reads the cache at HBM's rate: 4 sequences of 20-32k tokens, 32 / 8 heads of 128, 4 rows
// each, 84 us against 136.
bool tiled_rows(const PagedAttn& p, int D) { return p.cu_rows && !paged_token_rows_ok(p.G, p.max_rows, D); }
size_t attend_plan(PagedAttn& p, int D, int sms) { return tiled_rows(p, D) ? paged_rows_plan(p, D, sms) : paged_token_plan(p, D, sms); }

// Q [T, H_q, D] as {64 elements, q head of the group, token, D/64, kv head} with a box of all G heads of `tokens`
// tokens: row token * G + head of a tile.
bool encode_q(CUtensorMap* tm, const PagedAttn& p, int D, int tokens) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const int64_t sh = p.H_q > 1 ? p.q_head : D, st = p.T > 1 ? p.q_row : D;
    const cuuint64_t dims[5] = {64, (cuuint64_t)p.G, (cuuint64_t)p.T, (cuuint64_t)(D / 64), (cuuint64_t)p.H_kv};
    const cuuint64_t strides[4] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2, 128, (cuuint64_t)(sh * p.G) * 2};
    const cuuint32_t box[5] = {64, (cuuint32_t)p.G, (cuuint32_t)tokens, 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType dt = p.dtype == PCK_DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return fn(tm, dt, 5, const_cast<void*>(p.Q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The append to either kind of cache; dtype_ok: whether the rows' type suits it.
template <typename Cache>
int append_rows(pck_ctx* c, const Cache* cache, const pck_paged_batch* batch, int dtype, bool dtype_ok, const pck_rows* Q,
                const pck_rows* K, const pck_rows* V, int norm, float eps, const pck_rotary* rope, RopeParams& p) {
    int rc = check_cache(c, cache);
    if (rc != PCK_OK) return rc;
    if ((rc = check_batch(c, batch, cache->page_size)) != PCK_OK) return rc;
    if (!dtype_ok) return ctx_fail(c, PCK_EINVAL, "dtype=%d does not suit the cache (its own type or fp32)", dtype);
    if (batch->T == 0 || batch->B == 0) return PCK_OK;
    if (!K || !K->in || !V || !V->in) return ctx_fail(c, PCK_EINVAL, "NULL K or V");
    if (K->H != cache->H_kv || V->H != cache->H_kv) return ctx_fail(c, PCK_EINVAL, "K and V have %d and %d heads, the cache %d", K->H, V->H, cache->H_kv);
    if (norm && !(eps >= 0.f)) return ctx_fail(c, PCK_EINVAL, "eps=%g", eps);
    const int T = batch->T, D = cache->D;
    if (Q && Q->in && (rc = check_rows(c, Q, "Q", T, D, dtype, true)) != PCK_OK) return rc;
    if ((rc = check_rows(c, K, "K", T, D, dtype, false)) != PCK_OK) return rc;
    if ((rc = check_rows(c, V, "V", T, D, dtype, false)) != PCK_OK) return rc;
    if ((rc = check_rope(c, rope, D, false)) != PCK_OK) return rc;
    p.q = rows_arg(Q, norm != 0);
    p.k = rows_arg(K, norm != 0);
    p.v = rows_arg(V, false);
    p.k.out = cache->K;
    p.k.out_row = cache->k_token;
    p.k.out_head = cache->k_head;
    p.v.out = cache->V;
    p.v.out_row = cache->v_token;
    p.v.out_head = cache->v_head;
    p.T = T;
    p.D = D;
    p.eps = eps;
    set_rope(p, rope);
    p.append = 1;
    p.B = batch->B;
    p.page = cache->page_size;
    p.max_pages = batch->max_pages;
    p.n_pages = cache->n_pages;
    p.k_page = cache->k_page;
    p.v_page = cache->v_page;
    p.cu_rows = batch->cu_rows;
    p.kv_len = batch->kv_len;
    p.table = batch->table;
    p.err = ctx_view(c).dev_err;
    return PCK_OK;
}

// Pages of codes as {CHB codes, token, D / CHB, head, page} with a box of `rows` tokens and all of a row's D / CHB runs, swizzled
// by their width: runs of 128 codes where D has them, of 64 otherwise.
bool encode_codes(CUtensorMap* tm, void* base, int page_size, int D, int H, int64_t n_pages, int64_t s_tok, int64_t s_head,
                  int64_t s_page, int rows) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const int run = D % 128 == 0 ? 128 : 64;
    const int64_t st = page_size > 1 ? s_tok : D, sh = H > 1 ? s_head : D, sp = n_pages > 1 ? s_page : D;
    const cuuint64_t dims[5] = {(cuuint64_t)run, (cuuint64_t)page_size, (cuuint64_t)(D / run), (cuuint64_t)H, (cuuint64_t)n_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)st, (cuuint64_t)run, (cuuint64_t)sh, (cuuint64_t)sp};
    const cuuint32_t box[5] = {(cuuint32_t)run, (cuuint32_t)rows, (cuuint32_t)(D / run), 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              run == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The parts of an attention call that its kernels read beside its shape.
void attend_args(PagedAttn& p, const CtxView& v, const pck_paged_batch* batch, int D, const void* Q, int64_t q_row, int64_t q_head,
                 const float* O_prior, const float* LSE_prior, void* O, float* LSE, void* workspace) {
    p.Q = Q;
    p.O = O;
    p.LSE = LSE;
    p.O_prior = O_prior;
    p.LSE_prior = LSE_prior;
    p.q_row = q_row;
    p.q_head = q_head;
    p.kv_len = batch->kv_len;
    p.table = batch->table;
    p.scale_log2 = PG_LOG2E / sqrtf(static_cast<float>(D));
    p.ws = static_cast<float*>(workspace);
    p.err = v.dev_err;
    p.device = v.device;
}

int check_attend_rows(pck_ctx* c, int T, int H_q, const void* Q, int64_t q_row, int64_t q_head, const float* O_prior,
                      const float* LSE_prior, const void* O, const void* workspace) {
    if (!Q || !O) return ctx_fail(c, PCK_EINVAL, "NULL Q or O");
    if (!aligned16(Q) || !aligned16(O) || !aligned16(O_prior) || !aligned16(workspace))
        return ctx_fail(c, PCK_EINVAL, "Q, O, O_prior and the workspace must be 16-byte aligned");
    if (!stride_ok(q_row, T, 8) || !stride_ok(q_head, H_q, 8)) return ctx_fail(c, PCK_EINVAL, "Q strides must be positive multiples of 8");
    if ((O_prior != nullptr) != (LSE_prior != nullptr)) return ctx_fail(c, PCK_EINVAL, "O_prior and LSE_prior go together");
    return PCK_OK;
}

// row_heads: heads of a row of O, LSE and the priors, of which the call's H_q are neighbours (tiled rows only: else H_q).
int attend_run(pck_ctx* c, const pck_paged_cache* cache, const pck_paged_batch* batch, int H_q, int row_heads, const void* Q, int64_t q_row,
               int64_t q_head, int window, int sinks, const float* O_prior, const float* LSE_prior, void* O, float* LSE,
               void* workspace, size_t workspace_bytes, void* stream) {
    PagedAttn p = {};
    const int rc = attend_shape(c, cache, batch, H_q, window, sinks, p);
    if (rc != PCK_OK) return rc;
    if (p.B == 0 || p.T == 0) return PCK_OK;
    const int rc2 = check_attend_rows(c, p.T, H_q, Q, q_row, q_head, O_prior, LSE_prior, O, workspace);
    if (rc2 != PCK_OK) return rc2;
    const CtxView v = ctx_view(c);
    const int D = cache->D;
    const size_t need = attend_plan(p, D, v.sms);
    if (workspace_bytes < need || (need && !workspace))
        return ctx_fail(c, PCK_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    attend_args(p, v, batch, D, Q, q_row, q_head, O_prior, LSE_prior, O, LSE, workspace);
    p.row_heads = row_heads;
    p.k_base = cache->K;
    p.v_base = cache->V;
    const int64_t strides[6] = {cache->k_page, cache->k_head, cache->k_token, cache->v_page, cache->v_head, cache->v_token};
    for (int i = 0; i < 6; ++i) p.kv_stride[i] = strides[i];
    const bool ragged = tiled_rows(p, D);
    const int rows = ragged ? p.box : paged_token_box_rows(), chunks = ragged ? 1 : D / 64;
    DeviceScope dev(v.device);
    if (!dev.ok) return ctx_fail(c, PCK_ECUDA, "cannot select device %d", v.device);
    if (!encode_pages(&p.tm_k, p.dtype, cache->K, p.page, D, p.H_kv, cache->n_pages, cache->k_token, cache->k_head, cache->k_page, rows, chunks) ||
        !encode_pages(&p.tm_v, p.dtype, cache->V, p.page, D, p.H_kv, cache->n_pages, cache->v_token, cache->v_head, cache->v_page, rows, chunks))
        return ctx_fail(c, PCK_ECUDA, "the driver refused the cache's tensor map");
    if (ragged && !encode_q(&p.tm_q, p, D, paged_rows_tok_per_tile(p.G))) return ctx_fail(c, PCK_ECUDA, "the driver refused Q's tensor map");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = ragged ? launch_paged_rows(p, D, st) : launch_paged_token(p, D, st);
    if (e != cudaSuccess) return ctx_fail(c, PCK_ECUDA, "launch: %s", cudaGetErrorString(e));
    return PCK_OK;
}

// Attention over a quantised cache. One row of a sequence, or a few: over the codes. More: through 16-bit pages: what the rows see is read back
// into pages of the workspace (of Q's type, in the order of the sequences or, where the tables are wide, at their own numbers), and those
// are attended to.
// The tables' width, which is all that the host knows, may name far more pages than the rows see. So a call whose pages could take more
// than EXPAND_BYTES, or half of the cache's codes where that is more, goes through its kv heads some at a time, and through its sequences
// where one head's pages are still too many: a large cache and the workspace together stay below the bytes of a 16-bit cache. A part costs its
// launches and a wave that it may not fill: 24 prompts of 300 tokens (32 / 8 heads of 128) in tables of 131k tokens over 6.1 GiB of codes
// take 126 us in 4 parts with 3 GiB, 86 in one with 12 GiB, 179 in 8 with 1.5 GiB (a quarter of the codes).
constexpr int64_t EXPAND_BYTES = int64_t(4) << 30;

struct Expanded {
    PagedAttn p;                     // over the codes: its shape
    bool direct;
    int heads, seqs;                 // kv heads and sequences of a part: all of them, or fewer
    pck_paged_cache cache;           // a part's pages in the workspace (of `heads` kv heads); K and V are set by the call
    int slots;                       // pages of a sequence
    bool by_page;                    // as many pages as the cache has: fewer than a part's tables could name
    size_t off_v, off_map, off_inner, total;    // workspace: K, V, page map, the attention's own
};

// A part of a call: sequences from b0 on.
pck_paged_batch part_of(const pck_paged_batch* b, int b0, int seqs) {
    pck_paged_batch x = *b;
    x.B = seqs;
    x.cu_rows += b0;                 // (tiled rows have them)
    x.kv_len += b0;
    x.table += (int64_t)b0 * b->max_pages;
    return x;
}

int expand_shape(pck_ctx* c, const pck_paged_cache_e4m3* k, const pck_paged_batch* b, int q_dtype, int H_q, int window, int sinks, Expanded& x) {
    x = Expanded{};
    int rc = check_cache(c, k);
    if (rc != PCK_OK) return rc;
    if ((rc = check_batch(c, b, k->page_size)) != PCK_OK) return rc;
    if (q_dtype != PCK_DT_F16 && q_dtype != PCK_DT_BF16) return ctx_fail(c, PCK_EINVAL, "q_dtype=%d is not fp16 or bf16", q_dtype);
    if (window < 0 || sinks < 0) return ctx_fail(c, PCK_EINVAL, "window=%d sinks=%d", window, sinks);
    // the shape's checks are those of a 16-bit cache of this geometry (contiguous: its strides are not looked at)
    const int64_t page = k->page_size;
    void* const some = reinterpret_cast<void*>(256);                     // stands for the workspace
    x.cache = pck_paged_cache{some, some, q_dtype, k->H_kv, k->D, k->page_size, k->n_pages,
                              k->H_kv * page * k->D, page * k->D, k->D, k->H_kv * page * k->D, page * k->D, k->D};
    if ((rc = attend_shape(c, &x.cache, b, H_q, window, sinks, x.p)) != PCK_OK) return rc;
    if (x.p.B == 0 || x.p.T == 0) return PCK_OK;
    x.direct = !tiled_rows(x.p, k->D);
    const int sms = ctx_view(c).sms;
    if (x.direct) {
        x.total = paged_token_e4m3_plan(x.p, k->D, sms);
        return PCK_OK;
    }
    int64_t slots = b->max_pages;
    if (window > 0) {
        const int64_t rows = b->max_rows < b->T ? b->max_rows : b->T;
        const int64_t some = (sinks + page - 1) / page + (window + rows) / page + 2;
        if (some < slots) slots = some;
    }
    const int64_t one = page * k->D * 4;                                 // bytes of a page of one kv head, K and V
    const auto pages_of = [&](int64_t seqs) { return k->n_pages < seqs * slots ? k->n_pages : seqs * slots; };
    const int64_t half = k->n_pages * k->H_kv * page * k->D, budget = half > EXPAND_BYTES ? half : EXPAND_BYTES;
    // as many as the budget holds, at least one, and the parts as even as they come
    const auto even = [](int n, int64_t most) {
        const int64_t m = most < 1 ? 1 : most > n ? n : most, parts = (n + m - 1) / m;
        return static_cast<int>((n + parts - 1) / parts);
    };
    x.heads = even(k->H_kv, budget / (pages_of(b->B) * one));
    x.seqs = pages_of(b->B) * one <= budget ? b->B : even(b->B, budget / (slots * one));
    x.by_page = k->n_pages < x.seqs * slots;
    x.slots = static_cast<int>(slots);
    const int64_t pages = pages_of(x.seqs), H = x.heads;
    x.cache = pck_paged_cache{some, some, q_dtype, x.heads, k->D, k->page_size, pages,
                              H * page * k->D, page * k->D, k->D, H * page * k->D, page * k->D, k->D};
    const size_t side = (size_t)pages * H * page * k->D * 2;             // a multiple of 512 bytes
    x.off_v = side;
    x.off_map = 2 * side;
    x.off_inner = x.off_map + (((size_t)x.seqs * b->max_pages * 4 + 255) & ~size_t(255));
    // the attention's own: the most that a part takes (the last ones may be smaller, and are then split further)
    size_t inner = 0;
    const int G = H_q / k->H_kv, last_h = k->H_kv - (k->H_kv - 1) / x.heads * x.heads, last_b = b->B - (b->B - 1) / x.seqs * x.seqs;
    for (const int nh : {x.heads, last_h})
        for (const int nb : {x.seqs, last_b}) {
            PagedAttn p = {};
            pck_paged_cache part = x.cache;
            part.H_kv = nh;
            const pck_paged_batch pb = part_of(b, 0, nb);
            if ((rc = attend_shape(c, &part, &pb, nh * G, window, sinks, p)) != PCK_OK) return rc;
            const size_t need = paged_rows_plan(p, k->D, sms);
            if (need > inner) inner = need;
        }
    x.total = x.off_inner + inner;
    return PCK_OK;
}

void read_params(pck_ctx* c, const pck_paged_cache_e4m3* k, const pck_paged_batch* b, ReadParams& p) {
    p.K = static_cast<const uint8_t*>(k->K);
    p.V = static_cast<const uint8_t*>(k->V);
    p.k_scale = k->K_scale;
    p.v_scale = k->V_scale;
    p.k_page = k->k_page;
    p.k_head = k->k_head;
    p.k_token = k->k_token;
    p.v_page = k->v_page;
    p.v_head = k->v_head;
    p.v_token = k->v_token;
    p.H = p.scale_heads = k->H_kv;
    p.D = k->D;
    p.page = k->page_size;
    p.n_pages = k->n_pages;
    p.B = b->B;
    p.T = b->T;
    p.max_pages = b->max_pages;
    p.cu_rows = b->cu_rows;
    p.kv_len = b->kv_len;
    p.table = b->table;
    p.err = ctx_view(c).dev_err;
}

int run_read(pck_ctx* c, const ReadParams& p, int out_dtype, void* stream) {
    const CtxView v = ctx_view(c);
    DeviceScope dev(v.device);
    if (!dev.ok) return ctx_fail(c, PCK_ECUDA, "cannot select device %d", v.device);
    const cudaError_t e = launch_paged_read(p, out_dtype, v.sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PCK_OK : ctx_fail(c, PCK_ECUDA, "launch: %s", cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int pck_qk_norm_rope(pck_ctx* c, int dtype, int T, int D, const pck_rows* Q, const pck_rows* K, int norm, float eps,
                     const pck_rotary* rope, void* stream) {
    if (!c) return PCK_EINVAL;
    if (!dtype_any(dtype)) return ctx_fail(c, PCK_EINVAL, "dtype=%d", dtype);
    if (T < 0) return ctx_fail(c, PCK_EINVAL, "T=%d", T);
    if (D < 16 || D > 512 || D % 16) return ctx_fail(c, PCK_EUNSUPPORTED, "D=%d is not a multiple of 16 up to 512", D);
    if (!norm && !rope) return ctx_fail(c, PCK_EINVAL, "neither a norm nor a rotation");
    if (T == 0) return PCK_OK;
    if ((!Q || !Q->in) && (!K || !K->in)) return ctx_fail(c, PCK_EINVAL, "neither Q nor K");
    if (norm && !(eps >= 0.f)) return ctx_fail(c, PCK_EINVAL, "eps=%g", eps);
    int rc = PCK_OK;
    if (Q && Q->in && (rc = check_rows(c, Q, "Q", T, D, dtype, true)) != PCK_OK) return rc;
    if (K && K->in && (rc = check_rows(c, K, "K", T, D, dtype, true)) != PCK_OK) return rc;
    if ((rc = check_rope(c, rope, D, true)) != PCK_OK) return rc;
    RopeParams p = {};
    p.q = rows_arg(Q, norm != 0);
    p.k = rows_arg(K, norm != 0);
    p.T = T;
    p.D = D;
    p.eps = eps;
    set_rope(p, rope);
    p.err = ctx_view(c).dev_err;
    return run_rope(c, p, dtype, PCK_DT_F16, stream);
}

int pck_paged_append(pck_ctx* c, const pck_paged_cache* cache, const pck_paged_batch* batch, int dtype, const pck_rows* Q,
                     const pck_rows* K, const pck_rows* V, int norm, float eps, const pck_rotary* rope, void* stream) {
    if (!c) return PCK_EINVAL;
    RopeParams p = {};
    const int rc = append_rows(c, cache, batch, dtype, cache && (dtype == cache->dtype || dtype == PCK_DT_F32), Q, K, V, norm, eps, rope, p);
    if (rc != PCK_OK || p.T == 0) return rc;
    return run_rope(c, p, dtype, cache->dtype, stream);
}

int pck_paged_append_e4m3(pck_ctx* c, const pck_paged_cache_e4m3* cache, const pck_paged_batch* batch, int dtype, const pck_rows* Q,
                          const pck_rows* K, const pck_rows* V, int norm, float eps, const pck_rotary* rope, void* stream) {
    if (!c) return PCK_EINVAL;
    RopeParams p = {};
    const int rc = append_rows(c, cache, batch, dtype, dtype_any(dtype), Q, K, V, norm, eps, rope, p);
    if (rc != PCK_OK || p.T == 0) return rc;
    p.k_scale = cache->K_scale;
    p.v_scale = cache->V_scale;
    return run_rope(c, p, dtype, DT_E4M3, stream);
}

int pck_paged_workspace(pck_ctx* c, const pck_paged_cache* cache, const pck_paged_batch* batch, int H_q, int window, int sinks,
                        size_t* bytes) {
    if (!c) return PCK_EINVAL;
    if (!bytes) return ctx_fail(c, PCK_EINVAL, "NULL bytes");
    PagedAttn p = {};
    const int rc = attend_shape(c, cache, batch, H_q, window, sinks, p);
    if (rc != PCK_OK) return rc;
    *bytes = p.B == 0 || p.T == 0 ? 0 : attend_plan(p, cache->D, ctx_view(c).sms);
    return PCK_OK;
}

int pck_paged_attend(pck_ctx* c, const pck_paged_cache* cache, const pck_paged_batch* batch, int H_q, const void* Q, int64_t q_row,
                     int64_t q_head, int window, int sinks, const float* O_prior, const float* LSE_prior, void* O, float* LSE,
                     void* workspace, size_t workspace_bytes, void* stream) {
    if (!c) return PCK_EINVAL;
    const int rc = attend_run(c, cache, batch, H_q, H_q, Q, q_row, q_head, window, sinks, O_prior, LSE_prior, O, LSE, workspace, workspace_bytes, stream);
    if (rc == PCK_OK && batch->B > 0 && batch->T > 0) ctx_count_query(c);
    return rc;
}

int pck_paged_workspace_e4m3(pck_ctx* c, const pck_paged_cache_e4m3* cache, const pck_paged_batch* batch, int q_dtype, int H_q, int window,
                             int sinks, size_t* bytes) {
    if (!c) return PCK_EINVAL;
    if (!bytes) return ctx_fail(c, PCK_EINVAL, "NULL bytes");
    Expanded x;
    const int rc = expand_shape(c, cache, batch, q_dtype, H_q, window, sinks, x);
    if (rc != PCK_OK) return rc;
    *bytes = x.total;
    return PCK_OK;
}

int pck_paged_attend_e4m3(pck_ctx* c, const pck_paged_cache_e4m3* cache, const pck_paged_batch* batch, int q_dtype, int H_q, const void* Q,
                          int64_t q_row, int64_t q_head, int window, int sinks, const float* O_prior, const float* LSE_prior, void* O,
                          float* LSE, void* workspace, size_t workspace_bytes, void* stream) {
    if (!c) return PCK_EINVAL;
    Expanded x;
    int rc = expand_shape(c, cache, batch, q_dtype, H_q, window, sinks, x);
    if (rc != PCK_OK || x.p.B == 0 || x.p.T == 0) return rc;
    if ((rc = check_attend_rows(c, batch->T, H_q, Q, q_row, q_head, O_prior, LSE_prior, O, workspace)) != PCK_OK) return rc;
    if (workspace_bytes < x.total || (x.total && !workspace))
        return ctx_fail(c, PCK_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, x.total);
    if (x.direct) {
        const CtxView v = ctx_view(c);
        PagedAttn& p = x.p;
        attend_args(p, v, batch, cache->D, Q, q_row, q_head, O_prior, LSE_prior, O, LSE, workspace);
        p.k_scale = cache->K_scale;
        p.v_scale = cache->V_scale;
        p.k_base = cache->K;
        p.v_base = cache->V;
        const int64_t strides[6] = {cache->k_page, cache->k_head, cache->k_token, cache->v_page, cache->v_head, cache->v_token};
        for (int i = 0; i < 6; ++i) p.kv_stride[i] = strides[i];
        DeviceScope dev(v.device);
        if (!dev.ok) return ctx_fail(c, PCK_ECUDA, "cannot select device %d", v.device);
        const int rows = paged_token_e4m3_box(p, cache->D);     // (pages in pieces are not loaded by tiles)
        if (!p.pieces && (!encode_codes(&p.tm_k, cache->K, p.page, cache->D, p.H_kv, cache->n_pages, cache->k_token, cache->k_head, cache->k_page, rows) ||
            !encode_codes(&p.tm_v, cache->V, p.page, cache->D, p.H_kv, cache->n_pages, cache->v_token, cache->v_head, cache->v_page, rows)))
            return ctx_fail(c, PCK_ECUDA, "the driver refused the cache's tensor map");
        const cudaError_t e = launch_paged_token_e4m3(p, cache->D, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return ctx_fail(c, PCK_ECUDA, "launch: %s", cudaGetErrorString(e));
        ctx_count_query(c);
        return PCK_OK;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    x.cache.K = ws;
    x.cache.V = ws + x.off_v;
    int32_t* const map = reinterpret_cast<int32_t*>(ws + x.off_map);
    const int64_t D = cache->D, G = H_q / cache->H_kv;
    for (int b0 = 0; b0 < batch->B; b0 += x.seqs) {
        pck_paged_batch part = part_of(batch, b0, batch->B - b0 < x.seqs ? batch->B - b0 : x.seqs);
        for (int h0 = 0; h0 < cache->H_kv; h0 += x.heads) {
            const int nh = cache->H_kv - h0 < x.heads ? cache->H_kv - h0 : x.heads;
            ReadParams p = {};
            read_params(c, cache, &part, p);
            p.K += h0 * cache->k_head;
            p.V += h0 * cache->v_head;
            p.k_scale += (int64_t)h0 * p.page;
            p.v_scale += (int64_t)h0 * p.page;
            p.H = nh;
            p.max_rows = batch->max_rows < batch->T ? batch->max_rows : batch->T;
            p.Ko = x.cache.K;
            p.Vo = x.cache.V;
            p.pages = 1;
            p.slots = x.slots;
            p.by_page = x.by_page;
            p.window = window < MAX_TOKENS ? window : MAX_TOKENS;
            p.sinks = sinks < MAX_TOKENS ? sinks : MAX_TOKENS;
            p.page_map = map;
            if ((rc = run_read(c, p, q_dtype, stream)) != PCK_OK) return rc;
            pck_paged_cache pages = x.cache;
            pages.H_kv = nh;
            pages.k_page = pages.v_page = nh * pages.k_head;
            pck_paged_batch mapped = part;
            mapped.table = map;
            const int64_t head = h0 * G;                 // the part's first q head
            if ((rc = attend_run(c, &pages, &mapped, static_cast<int>(nh * G), H_q, static_cast<const uint8_t*>(Q) + head * q_head * 2, q_row, q_head,
                                 window, sinks, O_prior ? O_prior + head * D : nullptr, LSE_prior ? LSE_prior + head : nullptr,
                                 static_cast<uint8_t*>(O) + head * D * 2, LSE ? LSE + head : nullptr, ws + x.off_inner,
                                 workspace_bytes - x.off_inner, stream)) != PCK_OK) return rc;
        }
    }
    ctx_count_query(c);
    return PCK_OK;
}

int pck_paged_read_e4m3(pck_ctx* c, const pck_paged_cache_e4m3* cache, const pck_paged_batch* batch, int dtype, const pck_rows* K,
                        const pck_rows* V, void* stream) {
    if (!c) return PCK_EINVAL;
    int rc = check_cache(c, cache);
    if (rc != PCK_OK) return rc;
    if ((rc = check_batch(c, batch, cache->page_size)) != PCK_OK) return rc;
    if (!dtype_any(dtype)) return ctx_fail(c, PCK_EINVAL, "dtype=%d", dtype);
    if (batch->T == 0 || batch->B == 0) return PCK_OK;
    if (!K || !V) return ctx_fail(c, PCK_EINVAL, "NULL K or V");
    const int e = elems16(dtype);
    for (const pck_rows* r : {K, V}) {
        if (!r->out || !aligned16(r->out)) return ctx_fail(c, PCK_EINVAL, "K and V: outputs must be set and 16-byte aligned");
        if (r->H != cache->H_kv) return ctx_fail(c, PCK_EINVAL, "%d heads, the cache has %d", r->H, cache->H_kv);
        if (!stride_ok(r->out_row, batch->T, e) || !stride_ok(r->out_head, r->H, e))
            return ctx_fail(c, PCK_EINVAL, "K and V: strides must be positive multiples of %d elements", e);
    }
    ReadParams p = {};
    read_params(c, cache, batch, p);
    p.max_rows = batch->T;
    p.Ko = K->out;
    p.Vo = V->out;
    p.ko_row = K->out_row;
    p.ko_head = K->out_head;
    p.vo_row = V->out_row;
    p.vo_head = V->out_head;
    return run_read(c, p, dtype, stream);
}

}  // extern "C"
