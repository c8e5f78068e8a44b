// kvo_paged_attn: decode attention of one query token per request over a paged cache; the kernels are in paged_attn.cuh.
#include "paged_attn.cuh"

namespace kvo {

// How a call is cut.
// cluster > 0: that many CTAs per group in a cluster and no second launch.  Taken where the groups' clusters fit the
// device at once with at most 1536 tokens a CTA, i.e. where latency counts: e4m3, 8 KV heads of 128, one request of
// 4096 tokens 9.1 us against 13.5 as ranges, 4 of 8192 16.3 against 20.2, 16 of 4096 28.6 against 33.3; from 24576 on
// (1536 tokens a CTA) ranges are as fast or faster (20.7).
// cluster 0: ranges of equal cost over `ctas` CTAs, two to an SM (three are slower: 16 x 64K-128K 457 us against 430), with
// at least 8 subtiles each at the lengths the caller bounds.  The host does not know the lengths: where they differ a
// cluster per group waits for the longest (16 x 512-4096: 19.8 us against 20.0 as ranges).
// CTAs in clusters that start at once: three to an SM (448 in sevens do not), two with 16 heads' registers; clusters of
// 16 fill a GPC less well (384, or 256 of 16 heads, do not start at once: 3 x 4096 tokens 19.9 us, 15.2 as ranges).
int paged_attn_fit(int r, int cluster) { return cluster < 16 ? (r <= 8 ? 400 : 280) : (r <= 8 ? 300 : 200); }
PaPlan paged_attn_plan(int64_t groups, int r, int64_t max_tokens) {
    const int64_t want = std::max<int64_t>(1, (max_tokens + 127) / 128);
    int64_t s = 0;
    for (int c : {1, 2, 3, 4, 6, 8, 12, 16})
        if (c * groups <= paged_attn_fit(r, c) && (c <= want || c == 1)) s = c;
    if (s && max_tokens <= 1536 * s) return {(int)s, (int)(s * groups)};
    const int64_t subs = groups * ((max_tokens + PA_SUB - 1) / PA_SUB);
    return {0, (int)std::min<int64_t>(PA_SLOTS, std::max<int64_t>(1, (subs + 7) / 8))};
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

size_t paged_attn_workspace(const PaPlan& plan, int G, int r, int d) {
    if (plan.cluster) return 0;
    const int warps = plan.ctas * PA_WARPS;
    return round256((size_t)G * sizeof(int2)) + round256((size_t)2 * warps * r * sizeof(float4)) +
           (size_t)2 * warps * r * d * sizeof(float);
}

}  // namespace kvo

namespace {

int64_t paged_attn_bound(const kvo_paged_cache* c, int n_blocks, int64_t max_len) {
    const int64_t cap = (int64_t)c->max_pages * c->page_size;
    int64_t n = max_len > 0 && max_len < cap ? max_len : cap;
    if (n_blocks > 0) n = (int64_t)n_blocks * c->page_size;
    return n;
}

const char* paged_attn_error(const kvo_paged_cache* c, int n_q_heads, int n_blocks, int64_t max_len) {
    if (const char* m = kvo::paged_cache_error(c)) return m;
    if (n_q_heads < c->n_kv_heads || n_q_heads % c->n_kv_heads) return "n_q_heads must be a multiple of n_kv_heads";
    if (n_q_heads / c->n_kv_heads > 16) return "n_q_heads / n_kv_heads must be <= 16";
    if (max_len < 0) return "max_len must be >= 0";
    if (n_blocks < 0 || (int64_t)n_blocks * c->page_size >= (1 << 30)) return "n_blocks * page_size must fit in 30 bits";
    return nullptr;
}

}  // namespace

extern "C" kvo_status kvo_paged_attn_workspace(const kvo_paged_cache* cache, int n_q_heads, int n_blocks,
                                               int64_t max_len, size_t* bytes_out) {
    using namespace kvo;
    auto bad = [](const char* m) { set_last_error(m); return KVO_ERR_INVALID; };
    if (!bytes_out) return bad("null output pointer");
    *bytes_out = 0;
    if (const char* m = paged_attn_error(cache, n_q_heads, n_blocks, max_len)) return bad(m);
    const int G = cache->batch * cache->n_kv_heads;
    *bytes_out = paged_attn_workspace(paged_attn_plan(std::max(G, 1), n_q_heads / cache->n_kv_heads, paged_attn_bound(cache, n_blocks, max_len)), G,
                                      n_q_heads / cache->n_kv_heads, cache->head_dim);
    return KVO_OK;
}

extern "C" kvo_status kvo_paged_attn(const kvo_paged_cache* cache, const void* q, int n_q_heads, const int32_t* lens,
                                     int64_t max_len, const int32_t* blocks, const int32_t* counts, int n_blocks,
                                     void* o, float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                                     kvo_stream_t stream) {
    using namespace kvo;
    auto bad = [](const char* m) { set_last_error(m); return KVO_ERR_INVALID; };
    if (const char* m = paged_attn_error(cache, n_q_heads, blocks ? n_blocks : 0, max_len)) return bad(m);
    if (cache->batch == 0) return KVO_OK;
    if (!q || !lens || !o || !lse) return bad("null pointer argument");
    if (blocks && n_blocks < 1) return bad("blocks needs n_blocks >= 1");
    if (counts && !blocks) return bad("counts needs blocks");
    if ((uintptr_t)q % 16 || (uintptr_t)o % 16 || (uintptr_t)workspace % 256)
        return bad("q and o must be 16-byte aligned, the workspace 256-byte aligned");
    const int G = cache->batch * cache->n_kv_heads, r = n_q_heads / cache->n_kv_heads, D = cache->head_dim;
    const PaPlan plan = paged_attn_plan(G, r, paged_attn_bound(cache, blocks ? n_blocks : 0, max_len));
    const size_t need = paged_attn_workspace(plan, G, r, D);
    if (need && (!workspace || workspace_bytes < need)) return bad("the workspace is too small (kvo_paged_attn_workspace)");
    const int64_t bytes = 2ll * cache->batch * n_q_heads * D;
    if (ranges_meet(o, bytes, q, bytes)) return bad("o must not overlap q");
    const int64_t pool = page_bytes(cache), scales = scale_bytes(cache), b = cache->batch;
    const Bytes to_o{o, bytes}, to_lse{lse, 4 * b * n_q_heads}, to_ws{workspace, (int64_t)need};
    bool meet = meets_any(to_o, {to_lse, to_ws}) || meets_any(to_lse, {to_ws});
    for (const Bytes& x : {to_o, to_lse, to_ws})
        meet |= meets_any(x, {{q, bytes}, {cache->k_pages, pool}, {cache->v_pages, pool}, {cache->k_scale, scales}, {cache->v_scale, scales},
                              {cache->table, 4 * b * cache->max_pages}, {lens, 4 * b}, {blocks, 4ll * G * n_blocks}, {counts, 4ll * G}});
    if (meet) return bad("o, lse and the workspace must be apart from each other and from all that the call reads");
    const bool fp8 = cache->format == KVO_PAGES_E4M3;
    const int rb = fp8 ? D : 2 * D;
    CUtensorMap mk, mv;
    const uint64_t rows = (uint64_t)cache->n_pages * cache->n_kv_heads * cache->page_size;
    if (!tensor_map_rows(&mk, cache->k_pages, fp8 ? 1 : 2, D, rows, rb > 128 ? 128 : rb, PA_SUB) ||
        !tensor_map_rows(&mv, cache->v_pages, fp8 ? 1 : 2, D, rows, rb > 128 ? 128 : rb, PA_SUB)) {
        set_last_error("cuTensorMapEncodeTiled failed for the pages");
        return KVO_ERR_CUDA;
    }
    PagedAttnArgs A{};
    A.q = (const uint16_t*)q;
    A.scale[0] = fp8 ? cache->k_scale : nullptr;
    A.scale[1] = fp8 ? cache->v_scale : nullptr;
    A.table = cache->table;
    A.lens = lens;
    A.blocks = blocks;
    A.counts = counts;
    A.o = (uint16_t*)o;
    A.lse = lse;
    uint8_t* ws = (uint8_t*)workspace;
    A.info = (int2*)ws;
    A.part_ml = (float4*)(ws + round256((size_t)G * sizeof(int2)));
    A.part_o = (float*)((uint8_t*)A.part_ml + round256((size_t)2 * plan.ctas * PA_WARPS * r * sizeof(float4)));
    A.status = status;
    A.hkv = cache->n_kv_heads;
    A.r = r;
    A.page = cache->page_size;
    A.shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : cache->page_size == 64 ? 6 : 7;
    A.n_pages = cache->n_pages;
    A.max_pages = cache->max_pages;
    A.n_blocks = n_blocks;
    A.G = G;
    A.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
    A.warps = plan.ctas * PA_WARPS;
    A.wait_ns = call_wait.limit_ns;
    A.skip = call_wait.skip;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
#define KVO_PAGED(D_, F_) (r <= 8 ? kvo::paged_attn_launch<D_, F_, 1, false>(mk, mv, A, plan, s) : kvo::paged_attn_launch<D_, F_, 2, false>(mk, mv, A, plan, s))
    if (D == 128) e = fp8 ? KVO_PAGED(128, true) : KVO_PAGED(128, false);
    else e = fp8 ? KVO_PAGED(64, true) : KVO_PAGED(64, false);
#undef KVO_PAGED
    if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
    return KVO_OK;
}
