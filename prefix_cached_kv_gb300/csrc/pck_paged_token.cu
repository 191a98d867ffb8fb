// pck_paged_token.cu -- one-token attention over a paged cache: how a call is cut, and the fp16 kernels.
#include "pck_paged_token_impl.cuh"

namespace pck {

bool paged_token_dim_ok(int D) { return D == 64 || D == 128 || D == 192 || D == 256; }

int paged_token_cols(int D) { return D <= 128 ? 16 : 8; }
bool paged_token_rows_ok(int G, int max_rows, int D) { return paged_token_dim_ok(D) && (int64_t)G * max_rows <= paged_token_cols(D); }

// How a call is cut; fills heads_per_group, n_groups, cols, mode and n_ctas, and returns the workspace
// bytes. Up to 8 q heads (16 at D <= 128) share a work item and one read of the kv head; more are
// split evenly into several items. A few rows of a sequence share it as well.
size_t paged_token_plan(PagedAttn& p, int D, int sms) {
    const int most = paged_token_cols(D);
    const int rows = p.cu_rows ? p.max_rows : 1;
    p.n_groups = (p.G * rows + most - 1) / most;       // 1 with more than one row
    p.heads_per_group = (p.G + p.n_groups - 1) / p.n_groups;
    p.cols = p.heads_per_group * rows;
    int64_t bound = ((int64_t)p.max_pages * p.page + PG_SUB - 1) / PG_SUB;   // units of one item
    int64_t direct = TK_DIRECT_UNITS;
    if (p.window > 0) {
        const int64_t edges = 1 + ((int64_t)p.sinks + PG_SUB - 1) / PG_SUB;    // units beside the window's own
        const int64_t w = ((int64_t)p.window + rows + PG_SUB - 1) / PG_SUB + edges;
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
    const size_t ranges = is_split(p.mode) ? (size_t)p.n_ctas * (p.mode == TK_WARP ? warps_sm(D, TK_WARP) : 1) : 0;
    return ranges * (2 * slot_floats(D, p.cols) * sizeof(float) + sizeof(JoinDesc));
}

cudaError_t launch_paged_token(PagedAttn& p, int D, cudaStream_t st) {
    return p.dtype == PCK_DT_F16 ? launch_d<__half>(p, D, st) : launch_paged_token_bf16(p, D, st);
}

}  // namespace pck
