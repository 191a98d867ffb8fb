// pck_paged_api.cu -- C entries of the paged-tail operators: argument checks on the host, tensor
// maps, launches. Nothing is launched for a call that is refused.
#include <cuda.h>
#include <cuda_runtime.h>

#include "pck_paged.cuh"

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

int check_cache(pck_ctx* c, const pck_paged_cache* k) {
    if (!k || !k->K || !k->V) return ctx_fail(c, PCK_EINVAL, "NULL cache");
    if (k->dtype != PCK_DT_F16 && k->dtype != PCK_DT_BF16) return ctx_fail(c, PCK_EINVAL, "cache dtype %d is not fp16 or bf16", k->dtype);
    if (k->H_kv < 1 || k->H_kv > PCK_MAX_HEADS) return ctx_fail(c, PCK_EINVAL, "H_kv=%d out of range [1, %d]", k->H_kv, PCK_MAX_HEADS);
    if (k->D < 16 || k->D > 512 || k->D % 16) return ctx_fail(c, PCK_EUNSUPPORTED, "D=%d is not a multiple of 16 up to 512", k->D);
    if (k->page_size < 16 || k->page_size % 16 || k->page_size > (1 << 20))
        return ctx_fail(c, PCK_EUNSUPPORTED, "page_size=%d is not a multiple of 16 (at most 2^20)", k->page_size);
    if (k->n_pages < 1 || k->n_pages >= (int64_t(1) << 31)) return ctx_fail(c, PCK_EINVAL, "n_pages=%lld out of range", (long long)k->n_pages);
    if (!aligned16(k->K) || !aligned16(k->V)) return ctx_fail(c, PCK_EINVAL, "K and V must be 16-byte aligned");
    if (!stride_ok(k->k_page, k->n_pages, 8) || !stride_ok(k->k_head, k->H_kv, 8) || !stride_ok(k->k_token, k->page_size, 8) ||
        !stride_ok(k->v_page, k->n_pages, 8) || !stride_ok(k->v_head, k->H_kv, 8) || !stride_ok(k->v_token, k->page_size, 8))
        return ctx_fail(c, PCK_EINVAL, "cache strides must be positive multiples of 8 elements");
    return PCK_OK;
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
    const cudaError_t e = launch_norm_rope(p, in_dtype, cache_dtype, v.sms, static_cast<cudaStream_t>(stream));
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
    int rc = check_cache(c, cache);
    if (rc != PCK_OK) return rc;
    if ((rc = check_batch(c, batch, cache->page_size)) != PCK_OK) return rc;
    if (dtype != cache->dtype && dtype != PCK_DT_F32) return ctx_fail(c, PCK_EINVAL, "dtype=%d is neither the cache's nor fp32", dtype);
    if (batch->T == 0 || batch->B == 0) return PCK_OK;
    if (!K || !K->in || !V || !V->in) return ctx_fail(c, PCK_EINVAL, "NULL K or V");
    if (K->H != cache->H_kv || V->H != cache->H_kv) return ctx_fail(c, PCK_EINVAL, "K and V have %d and %d heads, the cache %d", K->H, V->H, cache->H_kv);
    if (norm && !(eps >= 0.f)) return ctx_fail(c, PCK_EINVAL, "eps=%g", eps);
    const int T = batch->T, D = cache->D;
    if (Q && Q->in && (rc = check_rows(c, Q, "Q", T, D, dtype, true)) != PCK_OK) return rc;
    if ((rc = check_rows(c, K, "K", T, D, dtype, false)) != PCK_OK) return rc;
    if ((rc = check_rows(c, V, "V", T, D, dtype, false)) != PCK_OK) return rc;
    if ((rc = check_rope(c, rope, D, false)) != PCK_OK) return rc;
    RopeParams p = {};
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
    return run_rope(c, p, dtype, cache->dtype, stream);
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
    PagedAttn p = {};
    const int rc = attend_shape(c, cache, batch, H_q, window, sinks, p);
    if (rc != PCK_OK) return rc;
    if (p.B == 0 || p.T == 0) return PCK_OK;
    if (!Q || !O) return ctx_fail(c, PCK_EINVAL, "NULL Q or O");
    if (!aligned16(Q) || !aligned16(O) || !aligned16(O_prior) || !aligned16(workspace))
        return ctx_fail(c, PCK_EINVAL, "Q, O, O_prior and the workspace must be 16-byte aligned");
    if (!stride_ok(q_row, p.T, 8) || !stride_ok(q_head, H_q, 8)) return ctx_fail(c, PCK_EINVAL, "Q strides must be positive multiples of 8");
    if ((O_prior != nullptr) != (LSE_prior != nullptr)) return ctx_fail(c, PCK_EINVAL, "O_prior and LSE_prior go together");
    const CtxView v = ctx_view(c);
    const int D = cache->D;
    const size_t need = attend_plan(p, D, v.sms);
    if (workspace_bytes < need || (need && !workspace))
        return ctx_fail(c, PCK_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
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
    ctx_count_query(c);
    return PCK_OK;
}

}  // extern "C"
