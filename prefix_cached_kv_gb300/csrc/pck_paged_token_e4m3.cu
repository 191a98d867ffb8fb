// pck_paged_token_e4m3.cu -- one-token attention over a quantised paged cache: how a call is cut, and the kernels of D = 64.
#include "pck_paged_token_e4m3_impl.cuh"

namespace pck {

int paged_token_e4m3_box(const PagedAttn& p, int D) { return sub8(D, p.mode); }

// Items per SM above which a range is a warp's: where an item could have a CTA of its own (64 x 500 tokens, 3.4 per SM: 23.2 us with
// one, 25.2 with a range per warp), and where it could not (64 ragged sequences of 100-16k tokens at D = 64: 57 us with a range per
// warp, 59 per half CTA; at D = 128 with pages of 16 tokens 84 against 86, of 64 78.5 against 77.8).
constexpr int T8_FEW_SHORT = 6, T8_FEW = 2;
// Tokens up to which an item gets a CTA: by the table's width (one sequence of 1000 tokens 12.3 us, of 2000, cut, 12.6), and where a window
// bounds them, so that most items have that length, and they fill the CTAs (32 windows of 2048 tokens, 8 kv heads: 29.6 us against 34.1
// cut, of 4000 51 against 54).
constexpr int T8_ITEM = 1024, T8_ITEM_WINDOW = 4096;

// How a call is cut; fills heads_per_group, n_groups, cols, mode, pieces and n_ctas, and returns the workspace bytes.
size_t paged_token_e4m3_plan(PagedAttn& p, int D, int sms) {
    const int most = paged_token_cols(D);
    const int rows = p.cu_rows ? p.max_rows : 1;
    p.n_groups = (p.G * rows + most - 1) / most;       // 1 with more than one row
    p.heads_per_group = (p.G + p.n_groups - 1) / p.n_groups;
    p.cols = p.heads_per_group * rows;
    const int64_t items = (int64_t)p.B * p.H_kv * p.n_groups;
    const bool spread = items > sms;                    // more than one item per SM
    int64_t bound = (int64_t)p.max_pages * p.page, direct = T8_ITEM;          // tokens of one item
    if (p.window > 0 && (int64_t)p.window + p.sinks < bound) {
        bound = (int64_t)p.window + (p.sinks > 256 ? p.sinks - 256 : 0);
        const int64_t slots = sms * (spread ? 2 : 1), left = items % slots;
        if (items >= slots ? left == 0 || left * 2 >= slots : items * 4 >= slots * 3) direct = T8_ITEM_WINDOW;
    }
    p.mode = items > (int64_t)T8_FEW_SHORT * sms ? TK_WARP
             : bound <= direct           ? (spread ? TK_ITEM_HALF : TK_ITEM)
             : items > (int64_t)T8_FEW * sms ? TK_WARP
                                           : (spread ? TK_CTA_HALF : TK_CTA);
    p.pieces = p.page % sub8(D, p.mode) != 0;
    p.n_ctas = is_split(p.mode) ? sms * per_sm(p.mode) : static_cast<int>(items);
    const size_t ranges = is_split(p.mode) ? (size_t)p.n_ctas * (p.mode == TK_WARP ? warps_sm8(D, TK_WARP) : 1) : 0;
    return ranges * (2 * slot_floats(D, p.cols) * sizeof(float) + sizeof(JoinDesc));
}

cudaError_t launch_paged_token_e4m3(PagedAttn& p, int D, cudaStream_t st) {
    return D == 64 ? launch8_d<64>(p, st) : D == 128 ? launch_paged_token_e4m3_128(p, st) : launch_paged_token_e4m3_wide(p, D, st);
}

}  // namespace pck
