// kvo_paged_chunk_attn of a few new tokens of each request: at most 16 rows (tokens x query heads of a group), the kernels
// of the decode attention with a number of visible keys for each row.  Up to 8 rows cost what one does; 16 are two tiles of the
// products' 8 columns, with twice the exponentials, and bound by issue slots where 8 are by HBM.  Measured (32 query and 8 KV
// heads of 128, 4 tokens each): 48 requests of 8K to 32K tokens in e4m3 350 us, 5.6 TB/s (one token each 297), 16 of 32K in
// bf16 323 us, 6.6 TB/s, one of 500 7.9 us.  Both ways at 16 rows, here and as tiles of 128 rows on tcgen05: 48 behind 16K in
// e4m3 293 and 365 us (12 rows 291, 366; 8 rows 249, 365), in bf16 485 and 468; one behind 4096 in e4m3 13 and 27, in bf16 12 and
// 24, behind 32K 33 and 45, 49 and 48.  20 rows, which only the tiles hold: 367, 471, one behind 32K 45 and 54.
#include "paged_few.cuh"

#include "paged_attn.cuh"

namespace kvo {

namespace {

// Rows that a call's kernels hold, for at most max_new tokens of r heads.
int few_rows(int r, int64_t max_new) { return max_new * r <= 8 ? 8 : 16; }
int64_t few_tokens(const kvo_paged_cache* c, int64_t max_len) {
    const int64_t cap = (int64_t)c->max_pages * c->page_size;
    return max_len > 0 && max_len < cap ? max_len : cap;
}

}  // namespace

size_t paged_few_workspace(const kvo_paged_cache* c, int r, int64_t max_new, int64_t max_len) {
    const int G = c->batch * c->n_kv_heads, rows = few_rows(r, max_new);
    return paged_attn_workspace(paged_attn_plan(std::max(G, 1), rows, few_tokens(c, max_len)), G, rows, c->head_dim);
}

cudaError_t launch_paged_few(const kvo_paged_cache* c, const CUtensorMap& mk, const CUtensorMap& mv, const void* q, int64_t q_stride,
                             int64_t total, int r, const int32_t* cu, const int32_t* lens, int64_t max_new, int64_t max_len, void* o,
                             float* lse, void* workspace, int32_t* status, cudaStream_t s) {
    const int G = c->batch * c->n_kv_heads, rows = few_rows(r, max_new), D = c->head_dim;
    const bool fp8 = c->format == KVO_PAGES_E4M3;
    const PaPlan plan = paged_attn_plan(G, rows, few_tokens(c, max_len));
    PagedAttnArgs A{};
    A.q = (const uint16_t*)q;
    A.q_stride = q_stride;
    A.total = total;
    A.cu = cu;
    A.most = rows;
    A.scale[0] = fp8 ? c->k_scale : nullptr;
    A.scale[1] = fp8 ? c->v_scale : nullptr;
    A.table = c->table;
    A.lens = lens;
    A.o = (uint16_t*)o;
    A.lse = lse;
    uint8_t* ws = (uint8_t*)workspace;
    A.info = (int2*)ws;
    A.part_ml = (float4*)(ws + round256((size_t)G * sizeof(int2)));
    A.part_o = (float*)((uint8_t*)A.part_ml + round256((size_t)2 * plan.ctas * PA_WARPS * rows * sizeof(float4)));
    A.status = status;
    A.hkv = c->n_kv_heads;
    A.r = r;
    A.page = c->page_size;
    A.shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
    A.n_pages = c->n_pages;
    A.max_pages = c->max_pages;
    A.G = G;
    A.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
    A.warps = plan.ctas * PA_WARPS;
    A.wait_ns = call_wait.limit_ns;
    A.skip = call_wait.skip;
#define KVO_FEW(D_, F_) (rows == 8 ? paged_attn_launch<D_, F_, 1, true>(mk, mv, A, plan, s) : paged_attn_launch<D_, F_, 2, true>(mk, mv, A, plan, s))
    if (D == 128) return fp8 ? KVO_FEW(128, true) : KVO_FEW(128, false);
    return fp8 ? KVO_FEW(64, true) : KVO_FEW(64, false);
#undef KVO_FEW
}

}  // namespace kvo
