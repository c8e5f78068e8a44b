// The pages of a paged cache through their life: kvo_paged_reserve, kvo_paged_fork, kvo_paged_compact keep the book of
// who holds which page, kvo_paged_copy moves what pages hold.
//
// The book is the table (page ids of each request), `held` (how many of them a request has) and refs[page], how often a
// page is named; 0 is free.  Free pages are always handed out lowest first, in the order of the requests, so results do
// not depend on timing: refs change by integer atomics, whose order does not matter, and ranks come from prefix sums.
//
// What bounds the book's calls is latency: a look at refs (1 MB for 262144 pages, 0.2 us of HBM) and two dependent passes
// over it with a sum over all pages between.  One cluster of 8 CTAs takes them in one launch, exchanging the CTAs' sums
// through distributed shared memory; rows of the table, which may be long, are moved by other CTAs.
//
// Measured (replayed graph): 256 requests of 2000 to 16384 tokens forked in a pool of 196608 pages of 16 9.3 us (1.2 for the rows'
// uses, 3 for the look at refs, 2 for the ranks, 2 for pages and lists), 32 beams 8.0 in one launch; room for 64 prompts in a pool of
// 262144 7.4 us; such a pool compacted 20 us (3 for the look, 2 for the ranks, 3 and 6 for the two lists, 4 for the rows), one of 2048
// pages 8.7.  Clusters of 16 CTAs: 11.4 us for the 256, 11.2 for the prompts, 19.3 for the compaction.  A run of pages to each
// warp instead of rounds (below): 14.4, 14 and 22, as few warps hold what is given out.
#include <algorithm>

#include "kvo_internal.cuh"
#include "launch.cuh"
#include "paged.cuh"
#include "tma_ptx.cuh"

namespace kvo {

constexpr int PG_THREADS = 1024;
constexpr int PG_CLUSTER = 8;
constexpr int PG_BATCH = 8192;                // requests of a call
constexpr int PG_ROW_THREADS = 256;
// A fork is one launch, of one cluster, up to so many requests (rows that its threads take at once) and entries of the table.
// Measured in us, one launch and two: 16 requests 7.4 and 7.6, 32 of 512 entries 8.3 and 7.7 (and a launch less on the host), 64
// 9.5 and 7.6, 256 18.8 and 8.1, 1024 of 64 entries 57 and 9.5; 32 of 8192 18.5 and 15.4.
constexpr int PG_ONE_BATCH = 32;
constexpr int64_t PG_ONE = 1 << 15;

struct Book {
    int32_t* table;
    int32_t* held;
    int32_t* refs;
    int32_t* status;
    int batch, max_pages, n_pages, page;
};

__device__ __forceinline__ void pg_report(const Book& B, int bits) {
    if (B.status) atomicOr(B.status, bits);
}

// The sum of `sums` over the warps before this one, and of all.
__device__ __forceinline__ int warps_before(const int* sums, int& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = sums[lane];                 // 32 warps
    int c = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += x;
    }
    all = __shfl_sync(0xffffffffu, c, 31);
    return __shfl_sync(0xffffffffu, c - t, warp);
}
// Exclusive sum over the CTA's threads; `all` gets the sum of all.  sums: 32 words that nothing else uses.
__device__ __forceinline__ int block_sum(int v, int* sums, int& all) {
    const int lane = threadIdx.x & 31;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
    }
    if (lane == 31) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    return s - v + warps_before(sums, all);
}

// The pages are dealt to the cluster's warps in rounds, at most 32 of them: a run of k groups of 32 pages to each warp, in the
// order of CTAs and warps, then the next round.  The lowest free pages, which are given out first, lie in every warp's hands.
struct Deal {
    int warps, mine, k, rounds;               // `mine`: this warp among them
};
// The first `idle` CTAs of a cluster of several take none.
__device__ __forceinline__ Deal pg_deal(const Book& B, int idle = 0) {
    const int ctas = (int)cluster_size(), skip = ctas > 1 ? idle : 0, groups = B.n_pages / 32 + (B.n_pages % 32 > 0);
    Deal d;
    d.warps = (ctas - skip) * (PG_THREADS / 32);
    d.mine = ((int)cluster_rank() - skip) * (PG_THREADS / 32) + (int)(threadIdx.x >> 5);
    d.k = (groups - 1) / (32 * d.warps) + 1;
    d.rounds = d.mine < 0 ? 0 : (groups - 1) / (d.warps * d.k) + 1;
    return d;
}
// The warp's groups number rounds * k.  The first page of its j-th; behind all pages where there is none.
__device__ __forceinline__ uint32_t pg_first(const Deal& d, int j) {
    const int round = j / d.k;
    return round < d.rounds ? ((uint32_t)(round * d.warps + d.mine) * d.k + (j - round * d.k)) * 32 : 1u << 31;
}
// Whole warp, its groups j0 .. j0 + 31: lane i gets the i-th one's free pages, a bit each.  Loops that stay loops: these
// kernels run for some microseconds, and every line of code that they pass has to be fetched.
__device__ __forceinline__ unsigned pg_masks(const Book& B, uint32_t first) {
    constexpr int AT_ONCE = 16;
    const int lane = threadIdx.x & 31;
    unsigned mask = 0;
#pragma unroll 1
    for (int h = 0; h < 32; h += AT_ONCE) {
        int v[AT_ONCE];
        if (__shfl_sync(0xffffffffu, first, h) >= (uint32_t)B.n_pages) break;
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const uint32_t p = __shfl_sync(0xffffffffu, first, h + i) + lane;
            v[i] = p < (uint32_t)B.n_pages ? B.refs[p] : -1;
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const unsigned m = __ballot_sync(0xffffffffu, v[i] == 0);
            if (lane == h + i) mask = m;
        }
    }
    return mask;
}
// Of a group of 32 pages: how many are free before this lane's, and in all.
__device__ __forceinline__ int pg_free_before(int v, int& all) {
    const unsigned free = __ballot_sync(0xffffffffu, v == 0);
    all = __popc(free);
    return __popc(free & ((1u << (threadIdx.x & 31)) - 1));
}
struct Ranks {
    int count[32][33];                        // [round][warp]
    int total[32];                            // of the rounds, in this CTA
};
// The warp's free pages, counted by rounds; returns the masks of its first 32 groups.
__device__ __forceinline__ unsigned pg_count_free(const Book& B, const Deal& d, Ranks& R) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = d.rounds * d.k;
    unsigned mask0 = 0;
    R.count[lane][warp] = 0;
    __syncwarp();
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += 32) {
        const unsigned mask = pg_masks(B, pg_first(d, j0 + lane));
        if (j0 == 0) mask0 = mask;
        if (mask) atomicAdd(&R.count[(j0 + lane) / d.k][warp], __popc(mask));
    }
    return mask0;
}
// Whole warp: f(page, rank) for its free pages, a page to a lane, rank by rank from round to round, up to rank n.  rank: of
// round `lane`, from pg_rank; mask0: from pg_count_free.
template <typename F>
__device__ __forceinline__ void pg_give(const Book& B, const Deal& d, unsigned mask0, int rank, int n, F&& f) {
    const int lane = threadIdx.x & 31, groups = d.rounds * d.k;
    if (d.k == 1) {                           // a round is a group: half as much to do for each
        uint32_t p = (uint32_t)d.mine * 32 + lane;
#pragma unroll 2
        for (int i = 0; i < groups; ++i, p += (uint32_t)d.warps * 32) {
            const unsigned m = __shfl_sync(0xffffffffu, mask0, i);
            const int at = __shfl_sync(0xffffffffu, rank, i);
            if (at >= n) return;              // ranks ascend from round to round
            const int r = at + __popc(m & ((1u << lane) - 1));
            if ((m >> lane & 1) && r < n) f((int)p, r);
        }
        return;
    }
    int at = 0, in = 0, round = 0;
#pragma unroll 1
    for (int j0 = 0; j0 < groups; j0 += 32) {
        const uint32_t first = pg_first(d, j0 + lane);
        const unsigned mask = j0 == 0 ? mask0 : pg_masks(B, first);
#pragma unroll 1
        for (int i = 0; i < 32 && j0 + i < groups; ++i) {
            if (in == 0) {
                at = __shfl_sync(0xffffffffu, rank, round++);
                if (at >= n) return;
            }
            const unsigned m = __shfl_sync(0xffffffffu, mask, i);
            const uint32_t p = __shfl_sync(0xffffffffu, first, i) + lane;
            const int r = at + __popc(m & ((1u << lane) - 1));
            if ((m >> lane & 1) && r < n) f((int)p, r);
            at += __popc(m);
            if (++in == d.k) in = 0;
        }
    }
}
// Free pages before this warp's run of round `lane`, of `free` in all, from the counts.  Barriers of this CTA and of the
// cluster: what any thread of the cluster wrote before is seen by all after it.
__device__ __forceinline__ int pg_rank(Ranks& R, int& free) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = (int)cluster_rank(), ctas = (int)cluster_size();
    __syncthreads();
    const int mine = R.count[warp][lane];     // this warp sums round `warp` up
    int c = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += x;
    }
    R.count[warp][lane] = c - mine;
    if (lane == 31) R.total[warp] = c;
    cluster_barrier();
    int all = 0, before = 0;
    uint32_t t[PG_CLUSTER];
#pragma unroll
    for (int q = 0; q < PG_CLUSTER; ++q) t[q] = q < ctas ? ld_cluster_u32(&R.total[lane], q) : 0;
#pragma unroll
    for (int q = 0; q < PG_CLUSTER; ++q) {
        all += (int)t[q];
        if (q < me) before += (int)t[q];
    }
    c = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += x;
    }
    free = __shfl_sync(0xffffffffu, c, 31);
    return c - all + before + R.count[lane][warp];
}

// ------------------------------------------------------------------ reserve
__global__ void __launch_bounds__(PG_THREADS, 1) pages_reserve_kernel(const Book B, const int32_t* want) {
    extern __shared__ int32_t smem[];
    int32_t* end = smem;                      // [batch]: pages asked for by the requests up to this one
    int32_t* had = smem + B.batch;            // [batch]: pages held before
    __shared__ int sums[32], given;
    __shared__ Ranks ranks;
    grid_wait();
    const int tid = threadIdx.x;
    if (tid == 0) given = 0;
    const int per = (B.batch + PG_THREADS - 1) / PG_THREADS, b0 = min(tid * per, B.batch), b1 = min(b0 + per, B.batch);
    int need = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const int w = want[b], h = B.held[b];
        const int pages = (int)(((unsigned)max(w, 0) + B.page - 1) / B.page);
        const bool bad = w < 0 || pages > B.max_pages || h < 0 || h > B.max_pages;
        if (bad && cluster_rank() == 0) pg_report(B, KVO_DEV_BAD_COUNT);
        if (!bad) need += max(pages - h, 0);
        end[b] = need;
        had[b] = h;
    }
    const Deal deal = pg_deal(B);
    const unsigned mask0 = pg_count_free(B, deal, ranks);
    int all, free;
    const int asked_before = block_sum(need, sums, all);
#pragma unroll 1
    for (int b = b0; b < b1; ++b) end[b] += asked_before;
    const int rank = pg_rank(ranks, free);         // (also a barrier of this CTA, for `end`)
    int last = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b)
        if (end[b] <= free) last = end[b];
    if (last) atomicMax(&given, last);
    __syncthreads();
    const int n = given;
    if (cluster_rank() == 0)
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int mine = end[b] - (b ? end[b - 1] : 0);
            if (mine && end[b] <= n) B.held[b] = had[b] + mine;
            if (mine && end[b] > n) pg_report(B, KVO_DEV_NO_PAGES);
        }
    pg_give(B, deal, mask0, rank, n, [&](int p, int r) {
        int b = 0;                            // the first request that asked for more than r pages with those before it
        for (int len = B.batch; len > 1;) {
            const int half = len / 2;
            if (end[b + half - 1] <= r) b += half;
            len -= half;
        }
        while (end[b] <= r) ++b;
        B.table[(int64_t)b * B.max_pages + had[b] + r - (b ? end[b - 1] : 0)] = p;
        B.refs[p] = 1;
    });
    cluster_barrier();                        // nobody leaves while its sum is read
}

// ------------------------------------------------------------------ fork
struct ForkArgs {
    Book book;
    const int32_t* parent;
    const int32_t* keep;
    int32_t* src;
    int32_t* dst;
    int32_t* count;
    int32_t* rows;                            // [batch][max_pages]: the new rows of requests that change parents
    int4* meta;                               // [batch]: pages before, pages after, the part-filled last one or -1, parent
    int32_t* list;                            // [batch]: the requests that get a copy, then their number
    int slots;                                // of the hash table, a power of two >= 2 batch
};

// The new row of request b, read from the table as it was, and every page's new number of uses; by PG_ROW_THREADS threads,
// of which this is the t-th.
__device__ __forceinline__ void fork_gather(const ForkArgs& A, int b, int t) {
    constexpr int AT_ONCE = 4;
    const Book& B = A.book;
    auto clamped = [&](int held) { return min(max(held, 0), B.max_pages); };
    const int held = B.held[b], before = clamped(held), keep = A.keep[b];
    int p = A.parent[b], after = before, part = 0;
    bool bad = false;
    if (p < -1 || p >= B.batch) bad = true;
    else if (p < 0) after = 0;
    else {
        const int pages = (int)(((unsigned)max(keep, 0) + B.page - 1) / B.page), most = p == b ? before : clamped(B.held[p]);
        if (keep < 0 || pages > most) bad = true;
        else { after = pages; part = keep % B.page; }
    }
    if (bad) { p = b; after = before; part = 0; }             // stays as it is
    if ((bad || held != before) && t == 0) pg_report(B, KVO_DEV_BAD_COUNT);
    const int32_t* old = B.table + (int64_t)b * B.max_pages;
    const int32_t* from = B.table + (int64_t)max(p, 0) * B.max_pages;
    int32_t* to = A.rows + (int64_t)b * B.max_pages;
    bool wrong = false;
    auto use = [&](int page, int n) {
        if (page < 0 || page >= B.n_pages) wrong = true;
        else atomicAdd(B.refs + page, n);
    };
    const int end = max(after, before);
    for (int j0 = (p == b ? after : 0) + t; j0 < end; j0 += PG_ROW_THREADS * AT_ONCE) {
        int o[AT_ONCE], e[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int j = j0 + i * PG_ROW_THREADS;
            o[i] = j < before ? old[j] : -1;
            e[i] = j < after ? from[j] : -1;
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int j = j0 + i * PG_ROW_THREADS;
            if (j < after) to[j] = e[i];
            if (j < after && j < before && e[i] == o[i]) continue;
            if (j < after) use(e[i], 1);
            if (j < before) use(o[i], -1);
        }
    }
    if (t == 0) {
        int last = -1;
        if (part && after) {
            last = from[after - 1];
            if (last < 0 || last >= B.n_pages) { wrong = true; last = -1; }
        }
        A.meta[b] = make_int4(before, after, last, p);
    }
    if (wrong) pg_report(B, KVO_DEV_BAD_BLOCK_ID);
}
// Writes the new row of request b, but for the entry of a part-filled last page.
__device__ __forceinline__ void fork_write(const ForkArgs& A, int b, int t) {
    constexpr int AT_ONCE = 4;
    const Book& B = A.book;
    const int4 m = A.meta[b];
    const int before = m.x, after = m.y, end = max(after, before);
    int32_t* to = B.table + (int64_t)b * B.max_pages;
    const int32_t* from = A.rows + (int64_t)b * B.max_pages;
    for (int j0 = (m.w == b ? after : 0) + t; j0 < end; j0 += PG_ROW_THREADS * AT_ONCE) {
        int e[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int j = j0 + i * PG_ROW_THREADS;
            e[i] = j < after ? from[j] : -1;
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int j = j0 + i * PG_ROW_THREADS;
            if (j < end && (m.z < 0 || j != after - 1)) to[j] = e[i];
        }
    }
}

// The first of two launches, a CTA per request.
__global__ void __launch_bounds__(PG_ROW_THREADS) pages_fork_rows_kernel(const ForkArgs A) {
    grid_wait();
    grid_launch_next();
    fork_gather(A, blockIdx.x, threadIdx.x);
}

// The second.  The first cluster settles the part-filled pages: a request that will write into one must be alone with it.
// The other CTAs write the rows.  ONE: one launch of one cluster does it all (PG_ONE).
template <bool ONE>
__global__ void __launch_bounds__(PG_THREADS, 1) pages_fork_kernel(const ForkArgs A) {
    constexpr int AT_ONCE = PG_THREADS / PG_ROW_THREADS;
    const Book& B = A.book;
    extern __shared__ int32_t smem[];
    __shared__ int sums[32];
    __shared__ Ranks ranks;
    const int tid = threadIdx.x;
    int32_t *key = smem, *first = smem + A.slots, *holders = smem + 2 * A.slots;
    if (cluster_rank() == 0)
        for (int i = tid; i < A.slots; i += PG_THREADS) { key[i] = -1; first[i] = INT32_MAX; holders[i] = 0; }
    grid_wait();
    const int ctas = ONE ? (int)gridDim.x : (int)(gridDim.x - cluster_size()), cta_row = (ONE ? (int)blockIdx.x : (int)(blockIdx.x - cluster_size())) * AT_ONCE + tid / PG_ROW_THREADS;
    if (ONE) {
        for (int b = cta_row; b < B.batch; b += ctas * AT_ONCE) fork_gather(A, b, tid % PG_ROW_THREADS);
        cluster_barrier();
        for (int b = cta_row; b < B.batch; b += ctas * AT_ONCE) fork_write(A, b, tid % PG_ROW_THREADS);
    } else if (cta_row >= 0) {
        for (int b = cta_row; b < B.batch; b += ctas * AT_ONCE) fork_write(A, b, tid % PG_ROW_THREADS);
        return;
    } else {
        __syncthreads();                      // the table of part-filled pages is laid out (above, the cluster's barrier says so)
    }
    const Deal deal = pg_deal(B, 1);          // the first CTA has the part-filled pages to do
    const unsigned mask0 = pg_count_free(B, deal, ranks);
    int free, first_rank = 0;                 // (first CTA) copies of the requests before this thread's
    unsigned mine = 0;                        // which of its up to 8 get one
    static_assert(PG_BATCH / PG_THREADS <= 32, "a bit to a request");
    const int per = (B.batch + PG_THREADS - 1) / PG_THREADS, b0 = min(tid * per, B.batch), b1 = min(b0 + per, B.batch);
    int total = 0;
    if (cluster_rank() == 0) {
        auto find = [&](int page) {           // its slot; there are twice as many slots as pages
            uint32_t i = (uint32_t)page * 2654435761u >> 7 & (A.slots - 1);
            while (true) {
                const int k = atomicCAS(key + i, -1, page);
                if (k == -1 || k == page) return i;
                i = (i + 1) & (A.slots - 1);
            }
        };
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int page = A.meta[b].z;
            if (page < 0) continue;
            const uint32_t i = find(page);
            atomicMin(first + i, b);
            atomicAdd(holders + i, 1);
        }
        __syncthreads();
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int page = A.meta[b].z;
            if (page < 0) continue;
            const int uses = B.refs[page];
            const uint32_t i = find(page);
            if (first[i] != b || uses != holders[i]) mine |= 1u << (b - b0);
        }
        first_rank = block_sum(__popc(mine), sums, total);
        int at = first_rank;
#pragma unroll 1
        for (int b = b0; b < b1; ++b)
            if (mine >> (b - b0) & 1) A.list[at++] = b;
        if (tid == 0) A.list[B.batch] = total;
    }
    const int rank = pg_rank(ranks, free);
    const int n = min(__ldcg(A.list + B.batch), free);
    if (cluster_rank() == 0) {
        int at = first_rank;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int4 m = A.meta[b];
            const bool copied = mine >> (b - b0) & 1;
            const bool lost = copied && at >= n;
            if (copied) {
                ++at;
                atomicSub(B.refs + m.z, 1);   // others hold it, or hold on to it: it does not become free
            }
            if (lost) pg_report(B, KVO_DEV_NO_PAGES);
            if (m.z >= 0 && (!copied || lost)) B.table[(int64_t)b * B.max_pages + m.y - 1] = lost ? -1 : m.z;
            B.held[b] = m.y - lost;
        }
        for (int i = n + tid; i < B.batch; i += PG_THREADS) A.src[i] = A.dst[i] = -1;
        if (tid == 0) *A.count = n;
    }
    pg_give(B, deal, mask0, rank, n, [&](int p, int r) {
        const int b = __ldcg(A.list + r);
        const int4 m = A.meta[b];
        B.table[(int64_t)b * B.max_pages + m.y - 1] = p;
        B.refs[p] = 1;
        A.src[r] = m.z;
        A.dst[r] = p;
    });
    cluster_barrier();                        // nobody leaves while its sum is read
}

// ------------------------------------------------------------------ compact
struct CompactArgs {
    Book book;
    int32_t* table_out;
    int32_t* refs_out;
    int32_t* src;
    int32_t* dst;
    int32_t* count;
    int32_t* head;                            // [0]: the pages in use, L; [1]: the moves
    int32_t* to;                              // [n_pages]: where page p >= L goes
};

// First launch, one cluster: L pages are in use; the i-th of those at L and behind goes to the i-th free one before L.
__global__ void __launch_bounds__(PG_THREADS, 1) pages_compact_kernel(const CompactArgs A) {
    const Book& B = A.book;
    __shared__ Ranks ranks;
    __shared__ int below;                     // free pages before L among this CTA's
    if (threadIdx.x == 0) below = 0;
    grid_wait();
    grid_launch_next();
    const Deal deal = pg_deal(B);
    const int lane = threadIdx.x & 31, groups = deal.rounds * deal.k;
    const unsigned mask0 = pg_count_free(B, deal, ranks);
    int free, mine = 0;
    const int rank = pg_rank(ranks, free);
    const int live = B.n_pages - free;
    pg_give(B, deal, mask0, rank, free, [&](int p, int r) {
        if (p < live) { A.dst[r] = p; ++mine; }
    });
    mine = (int)__reduce_add_sync(0xffffffffu, (unsigned)mine);
    if (lane == 0 && mine) atomicAdd(&below, mine);
    cluster_barrier();
    int moves = lane < (int)cluster_size() ? (int)ld_cluster_u32(&below, lane) : 0;
    moves = (int)__reduce_add_sync(0xffffffffu, (unsigned)moves);
    if (cluster_rank() == 0 && threadIdx.x == 0) {
        A.head[0] = live;
        A.head[1] = moves;
    }
    constexpr int AT_ONCE = 8;                // groups whose places are fetched together: a store may not pass a load
    int before = moves;
#pragma unroll 1
    for (int j0 = 0; j0 < groups; j0 += AT_ONCE) {
        const int j = j0 + (lane & (AT_ONCE - 1)), round = j / deal.k;
        const uint32_t first = pg_first(deal, j);
        // Free pages before L may have been filled meanwhile: counted are those from L on.
        const int at_round = __shfl_sync(0xffffffffu, rank, round & 31), start = first >= (uint32_t)live ? at_round : moves;
        const unsigned begins = __ballot_sync(0xffffffffu, j == round * deal.k);
        if (__shfl_sync(0xffffffffu, first, AT_ONCE - 1) + 32 <= (uint32_t)live) continue;      // (all before L: `before` is `moves`)
        int p[AT_ONCE], v[AT_ONCE], at[AT_ONCE], to[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const uint32_t x = __shfl_sync(0xffffffffu, first, i) + lane;
            p[i] = (int)x;
            v[i] = x >= (uint32_t)live && x < (uint32_t)B.n_pages ? B.refs[x] : INT32_MIN;
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int s = __shfl_sync(0xffffffffu, start, i);
            if (begins >> i & 1) before = s;
            int here;
            at[i] = p[i] - (before + pg_free_before(v[i], here)) - (live - moves);
            before += here;
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) to[i] = v[i] != INT32_MIN && v[i] != 0 ? __ldcg(A.dst + at[i]) : p[i];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            if (v[i] != INT32_MIN && v[i] != 0) {
                A.src[at[i]] = p[i];
                A.refs_out[to[i]] = v[i];
                if (A.refs_out == B.refs) A.refs_out[p[i]] = 0;
            }
            if (v[i] != INT32_MIN) A.to[p[i]] = to[i];
        }
    }
    if (cluster_rank() == 0 && threadIdx.x == 0) *A.count = moves;
    cluster_barrier();                        // nobody leaves while its sum is read
}

// Second launch.  A CTA per request: the rows' entries follow their pages.  All CTAs: what the first leaves of the lists,
// and of refs that go elsewhere.
__global__ void __launch_bounds__(PG_ROW_THREADS) pages_compact_rows_kernel(const CompactArgs A) {
    constexpr int AT_ONCE = 4;
    const Book& B = A.book;
    grid_wait();
    const int b = blockIdx.x, live = A.head[0], moves = A.head[1], stripe = gridDim.x * PG_ROW_THREADS;
    for (int i = moves + b * PG_ROW_THREADS + threadIdx.x; i < B.n_pages / 2; i += stripe) A.src[i] = A.dst[i] = -1;
    if (A.refs_out != B.refs)
        for (int p = b * PG_ROW_THREADS + threadIdx.x; p < B.n_pages; p += stripe) {
            const int v = B.refs[p];
            if (p >= live || v != 0) A.refs_out[p] = p >= live ? 0 : v;
        }
    if (b >= B.batch) return;
    int held = B.held[b];
    if ((held < 0 || held > B.max_pages) && threadIdx.x == 0) pg_report(B, KVO_DEV_BAD_COUNT);
    held = min(max(held, 0), B.max_pages);
    const int32_t* from = B.table + (int64_t)b * B.max_pages;
    int32_t* to = A.table_out + (int64_t)b * B.max_pages;
    const int end = A.table_out == B.table ? held : B.max_pages;
    bool wrong = false;
    for (int j = threadIdx.x; j < end; j += PG_ROW_THREADS * AT_ONCE) {
        int e[AT_ONCE], t[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) e[i] = j + i * PG_ROW_THREADS < end ? from[j + i * PG_ROW_THREADS] : 0;
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const bool named = j + i * PG_ROW_THREADS < held, in = e[i] >= 0 && e[i] < B.n_pages;
            wrong |= named && !in;
            t[i] = named && in && e[i] >= live ? A.to[e[i]] : e[i];
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
            if (j + i * PG_ROW_THREADS < end) to[j + i * PG_ROW_THREADS] = t[i];
    }
    if (wrong) pg_report(B, KVO_DEV_BAD_BLOCK_ID);
}

// ------------------------------------------------------------------ copy
struct CopyArgs {
    uint8_t* pages[2];
    float* scale[2];
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;                     // or NULL: all `moves`
    int32_t* status;
    int64_t layer_bytes;                      // of one layer's K (or V)
    int page_bytes, n_pages, hkv, layers, moves, pieces;
};
constexpr int PC_CTAS = 152 * 24, PC_THREADS = 256, PC_LOADS = 8, PC_PIECE = PC_THREADS * PC_LOADS * 16;

// Bound by HBM: every byte is read once and written once.  A piece is 32 KB of a page (or a page, where that is smaller), eight
// 16-byte loads to a thread.  501 pages of 4 layers, 263 MB read and as many written, 82 us: 6.4 TB/s, 0.95 of a measured copy.
// Up to 24 CTAs to an SM are launched, 6 or so run at a time: as they end others take over, which balances better than long
// strides (6: 87 us, 12: 84.6, 54: 79.8), but a call whose count is 0 starts them all (4.4 us; 1.9 with 6, 8.7 with 54).
__global__ void __launch_bounds__(PC_THREADS) pages_copy_kernel(const CopyArgs A) {
    grid_wait();
    int n = A.moves;
    if (A.count) {
        const int c = *A.count;
        if ((c < 0 || c > n) && blockIdx.x == 0 && threadIdx.x == 0 && A.status) atomicOr(A.status, KVO_DEV_BAD_COUNT);
        n = min(max(c, 0), n);
    }
    const int64_t units = (int64_t)n * A.pieces * 2 * A.layers;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int piece = (int)(u % A.pieces), kv = (int)(u / A.pieces & 1);
        const int64_t m = u / A.pieces >> 1;
        const int layer = (int)(m / n), i = (int)(m - (int64_t)layer * n);
        const int s = A.src[i], d = A.dst[i];
        if (s < 0 || s >= A.n_pages || d < 0 || d >= A.n_pages) {
            if (threadIdx.x == 0 && A.status) atomicOr(A.status, KVO_DEV_BAD_BLOCK_ID);
            continue;
        }
        if (s == d) continue;
        uint8_t* base = A.pages[kv] + layer * A.layer_bytes;
        const int off = piece * PC_PIECE, bytes = min(PC_PIECE, A.page_bytes - off);
        const uint4* from = reinterpret_cast<const uint4*>(base + (int64_t)s * A.page_bytes + off);
        uint4* to = reinterpret_cast<uint4*>(base + (int64_t)d * A.page_bytes + off);
        uint4 v[PC_LOADS];
#pragma unroll
        for (int e = 0; e < PC_LOADS; ++e)
            if ((e * PC_THREADS + (int)threadIdx.x) * 16 < bytes) v[e] = __ldcs(from + e * PC_THREADS + threadIdx.x);
#pragma unroll
        for (int e = 0; e < PC_LOADS; ++e)
            if ((e * PC_THREADS + (int)threadIdx.x) * 16 < bytes) to[e * PC_THREADS + threadIdx.x] = v[e];
        if (A.scale[kv] && piece == 0) {
            float* sc = A.scale[kv] + (int64_t)layer * A.n_pages * A.hkv;
            for (int h = threadIdx.x; h < A.hkv; h += PC_THREADS) sc[(int64_t)d * A.hkv + h] = sc[(int64_t)s * A.hkv + h];
        }
    }
}

// ------------------------------------------------------------------ host
const char* book_error(const kvo_page_book* b) {
    if (!b) return "null book";
    if (b->batch < 0 || b->batch > PG_BATCH) return "batch must be in 0..8192";
    if (b->n_pages < 1 || b->max_pages < 1) return "need n_pages >= 1 and max_pages >= 1";
    if (b->page_size < 1 || (int64_t)b->max_pages * b->page_size > INT32_MAX) return "need page_size >= 1 and max_pages * page_size below 2^31";
    if (b->n_pages > 1 << 30 || b->max_pages > 1 << 30) return "n_pages and max_pages must be at most 2^30";      // (kernels step past them)
    if ((int64_t)b->batch * b->max_pages > INT32_MAX) return "batch * max_pages must fit in 31 bits";
    if (!b->refs || (b->batch > 0 && (!b->table || !b->held))) return "null table, held or refs";
    if ((uintptr_t)b->refs % 16) return "refs must be 16-byte aligned";
    return nullptr;
}
Book device_book(const kvo_page_book* b, int32_t* status) {
    return {b->table, b->held, b->refs, status, b->batch, b->max_pages, b->n_pages, b->page_size};
}
Bytes table_of(const kvo_page_book* b) { return {b->table, 4ll * b->batch * b->max_pages}; }
Bytes held_of(const kvo_page_book* b) { return {b->held, 4ll * b->batch}; }
Bytes refs_of(const kvo_page_book* b) { return {b->refs, 4ll * b->n_pages}; }
// Whether a range of `some` shares a byte with another of them, or with one of `others`.
bool any_meet(std::initializer_list<Bytes> some, std::initializer_list<Bytes> others) {
    for (const Bytes* x = some.begin(); x != some.end(); ++x) {
        if (meets_any(*x, others)) return true;
        for (const Bytes* y = x + 1; y != some.end(); ++y)
            if (meets_any(*x, {*y})) return true;
    }
    return false;
}
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
// CTAs of the cluster that looks at refs: one for pools of up to 4 groups of 32 pages to a warp, without barriers of clusters.
int pages_cluster(int n_pages) { return n_pages <= 4 * PG_THREADS ? 1 : PG_CLUSTER; }

size_t fork_workspace(const kvo_page_book* b) {
    return up256((size_t)b->batch * sizeof(int4)) + up256(((size_t)b->batch + 1) * 4) + up256((size_t)b->batch * b->max_pages * 4);
}
size_t compact_workspace(const kvo_page_book* b) { return 256 + up256((size_t)b->n_pages * 4); }

cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>& done, int bytes) {
    if (!first_on_device(done)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) mark_on_device(done);
    return e;
}

}  // namespace kvo

namespace {

kvo_status refuse(const char* m) {
    kvo::set_last_error(m);
    return KVO_ERR_INVALID;
}
kvo_status launched(cudaError_t e) {
    if (e == cudaSuccess) return KVO_OK;
    kvo::set_last_error(cudaGetErrorString(e));
    return KVO_ERR_CUDA;
}

}  // namespace

extern "C" kvo_status kvo_paged_reserve(const kvo_page_book* book, const int32_t* want, int32_t* status, kvo_stream_t stream) {
    using namespace kvo;
    if (const char* m = book_error(book)) return refuse(m);
    if (book->batch == 0) return KVO_OK;
    if (!want) return refuse("null pointer argument");
    if (any_meet({table_of(book), held_of(book), refs_of(book)}, {{want, 4ll * book->batch}}))
        return refuse("table, held and refs must be apart from each other and from want");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem((const void*)pages_reserve_kernel, done, PG_BATCH * 8);
    if (e == cudaSuccess) {
        const int cluster = pages_cluster(book->n_pages);
        e = launch_dependent(pages_reserve_kernel, dim3(cluster), PG_THREADS, (size_t)book->batch * 8, (cudaStream_t)stream, cluster,
                             device_book(book, status), want);
    }
    return launched(e);
}

extern "C" kvo_status kvo_paged_fork_workspace(const kvo_page_book* book, size_t* bytes_out) {
    if (!bytes_out) return refuse("null output pointer");
    *bytes_out = 0;
    if (const char* m = kvo::book_error(book)) return refuse(m);
    *bytes_out = kvo::fork_workspace(book);
    return KVO_OK;
}

extern "C" kvo_status kvo_paged_fork(const kvo_page_book* book, const int32_t* parent, const int32_t* keep, int32_t* src,
                                     int32_t* dst, int32_t* count, void* workspace, size_t workspace_bytes, int32_t* status,
                                     kvo_stream_t stream) {
    using namespace kvo;
    if (const char* m = book_error(book)) return refuse(m);
    if (!count) return refuse("null pointer argument");
    cudaStream_t s = (cudaStream_t)stream;
    if (book->batch == 0) return launched(cudaMemsetAsync(count, 0, 4, s));
    if (!parent || !keep || !src || !dst) return refuse("null pointer argument");
    const size_t need = fork_workspace(book);
    if (!workspace || workspace_bytes < need) return refuse("the workspace is too small (kvo_paged_fork_workspace)");
    if ((uintptr_t)workspace % 256) return refuse("the workspace must be 256-byte aligned");
    const int64_t b4 = 4ll * book->batch;
    if (any_meet({table_of(book), held_of(book), refs_of(book), {src, b4}, {dst, b4}, {count, 4}, {workspace, (int64_t)need}},
                 {{parent, b4}, {keep, b4}}))
        return refuse("what the call writes must be apart from each other and from parent and keep");
    ForkArgs A{};
    A.book = device_book(book, status);
    A.parent = parent;
    A.keep = keep;
    A.src = src;
    A.dst = dst;
    A.count = count;
    uint8_t* ws = (uint8_t*)workspace;
    A.meta = (int4*)ws;
    A.list = (int32_t*)(ws + up256((size_t)book->batch * sizeof(int4)));
    A.rows = (int32_t*)((uint8_t*)A.list + up256(((size_t)book->batch + 1) * 4));
    A.slots = 32;
    while (A.slots < 2 * book->batch) A.slots *= 2;
    static std::atomic<uint64_t> done_one{0}, done_two{0};
    const int cluster = pages_cluster(book->n_pages), rows = (book->batch + 3) / 4;
    if (book->batch <= PG_ONE_BATCH && (int64_t)book->batch * book->max_pages <= PG_ONE) {
        const cudaError_t e = allow_smem((const void*)pages_fork_kernel<true>, done_one, 2 * PG_BATCH * 12);
        if (e != cudaSuccess) return launched(e);
        const int ctas = std::max(cluster, rows > 1 ? PG_CLUSTER : 1);
        return launched(launch_dependent(pages_fork_kernel<true>, dim3(ctas), PG_THREADS, (size_t)A.slots * 12, s, ctas, A));
    }
    cudaError_t e = allow_smem((const void*)pages_fork_kernel<false>, done_two, 2 * PG_BATCH * 12);
    if (e != cudaSuccess) return launched(e);
    e = launch_dependent(pages_fork_rows_kernel, dim3(book->batch), PG_ROW_THREADS, 0, s, 0, A);
    if (e != cudaSuccess) return launched(e);
    const int ctas = cluster + (std::min(rows, 128) + cluster - 1) / cluster * cluster;
    return launched(launch_dependent(pages_fork_kernel<false>, dim3(ctas), PG_THREADS, (size_t)A.slots * 12, s, cluster, A));
}

extern "C" kvo_status kvo_paged_compact_workspace(const kvo_page_book* book, size_t* bytes_out) {
    if (!bytes_out) return refuse("null output pointer");
    *bytes_out = 0;
    if (const char* m = kvo::book_error(book)) return refuse(m);
    *bytes_out = kvo::compact_workspace(book);
    return KVO_OK;
}

extern "C" kvo_status kvo_paged_compact(const kvo_page_book* book, int32_t* table_out, int32_t* refs_out, int32_t* src,
                                        int32_t* dst, int32_t* count, void* workspace, size_t workspace_bytes,
                                        int32_t* status, kvo_stream_t stream) {
    using namespace kvo;
    if (const char* m = book_error(book)) return refuse(m);
    if (!table_out) table_out = book->table;
    if (!refs_out) refs_out = book->refs;
    if (!count || (book->n_pages > 1 && (!src || !dst))) return refuse("null pointer argument");
    const size_t need = compact_workspace(book);
    if (!workspace || workspace_bytes < need) return refuse("the workspace is too small (kvo_paged_compact_workspace)");
    if ((uintptr_t)workspace % 256) return refuse("the workspace must be 256-byte aligned");
    const int64_t half = 4ll * (book->n_pages / 2);
    const Bytes table = table_of(book), refs = refs_of(book);
    if (any_meet({{src, half}, {dst, half}, {count, 4}, {workspace, (int64_t)need}, {table_out, table.n}, {refs_out, refs.n}}, {held_of(book)}) ||
        any_meet({{src, half}, {dst, half}, {count, 4}, {workspace, (int64_t)need}}, {table, refs}) ||
        (table_out != book->table && meets_any({table_out, table.n}, {table, refs})) ||
        (refs_out != book->refs && meets_any({refs_out, refs.n}, {table, refs})))
        return refuse("what the call writes must be apart from each other and from what it reads (table_out and refs_out may be table and refs)");
    CompactArgs A{};
    A.book = device_book(book, status);
    A.table_out = table_out;
    A.refs_out = refs_out;
    A.src = src;
    A.dst = dst;
    A.count = count;
    A.head = (int32_t*)workspace;
    A.to = A.head + 64;
    cudaStream_t s = (cudaStream_t)stream;
    const int cluster = pages_cluster(book->n_pages);
    cudaError_t e = launch_dependent(pages_compact_kernel, dim3(cluster), PG_THREADS, 0, s, cluster, A);
    const int stripes = (int)std::min<int64_t>(304, (book->n_pages + 4ll * PG_ROW_THREADS - 1) / (4 * PG_ROW_THREADS));
    if (e == cudaSuccess)
        e = launch_dependent(pages_compact_rows_kernel, dim3(std::max(book->batch, stripes)), PG_ROW_THREADS, 0, s, 0, A);
    return launched(e);
}

extern "C" kvo_status kvo_paged_copy(const kvo_paged_cache* pools, int layers, const int32_t* src, const int32_t* dst, int moves,
                                     const int32_t* count, int32_t* status, kvo_stream_t stream) {
    using namespace kvo;
    if (!pools) return refuse("null cache");
    kvo_paged_cache c = *pools;               // a call without requests: table and batch are not looked at
    c.batch = 0;
    c.max_pages = 1;
    if (const char* m = paged_cache_error(&c)) return refuse(m);
    if (layers < 0 || moves < 0) return refuse("layers and moves must be >= 0");
    const int64_t layer = page_bytes(&c), scales = scale_bytes(&c);
    if (layer / c.n_pages > (1 << 30)) return refuse("a page must be at most 2^30 bytes");
    if (layers > 65536 || layer > INT64_MAX / 4 / std::max(layers, 1)) return refuse("layers must be <= 65536");
    if (layers == 0 || moves == 0) return KVO_OK;
    if (!src || !dst) return refuse("null pointer argument");
    const Bytes k{c.k_pages, layer * layers}, v{c.v_pages, layer * layers}, ks{c.k_scale, scales * layers}, vs{c.v_scale, scales * layers};
    if (any_meet({k, v, ks, vs}, {{src, 4ll * moves}, {dst, 4ll * moves}, {count, 4}}))
        return refuse("pools and scales must be apart from each other and from src, dst and count");
    CopyArgs A{};
    A.pages[0] = (uint8_t*)c.k_pages;
    A.pages[1] = (uint8_t*)c.v_pages;
    A.scale[0] = scales ? c.k_scale : nullptr;
    A.scale[1] = scales ? c.v_scale : nullptr;
    A.src = src;
    A.dst = dst;
    A.count = count;
    A.status = status;
    A.layer_bytes = layer;
    A.n_pages = c.n_pages;
    A.page_bytes = (int)(layer / c.n_pages);
    A.hkv = c.n_kv_heads;
    A.layers = layers;
    A.moves = moves;
    A.pieces = (A.page_bytes + PC_PIECE - 1) / PC_PIECE;
    const int64_t units = (int64_t)moves * A.pieces * 2 * layers;
    return launched(launch_dependent(pages_copy_kernel, dim3((unsigned)std::min<int64_t>(units, PC_CTAS)), PC_THREADS, 0, (cudaStream_t)stream, 0, A));
}
