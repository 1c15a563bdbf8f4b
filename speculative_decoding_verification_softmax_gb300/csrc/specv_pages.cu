// Pages of a key-value cache: reserve, commit, free, fork and compact.
//
// A page is free when its count of references is zero; there is no free list.
// Every call that takes pages finds the lowest free ones by a scan of the
// counts, so a result depends on the state alone (a stack of free pages would
// be in the order in which blocks happened to push) and the pool stays dense
// at its lower end.  The scan is 4 bytes a page: 1 MB for 262144 pages.
//
// Small calls are bound by their launches and chains of round trips: reserve and
// commit for 1024 requests over 250,000 pages take 20 us together, for 16 requests
// 11 us; a fork of 64 requests 20 us for the tables and 17 us for 122 MB of copied
// tokens (7.2 TB/s, partly from L2).  Large copies are bound by HBM: compact moves
// 0.6 GB of pages, 1.19 GB read and written, in 197 us, 6.0 TB/s.
#include <cooperative_groups.h>

#include <mutex>

#include "specv_cache.cuh"
#include "specv_trace.h"

namespace cg = cooperative_groups;

namespace specv {

constexpr int kPgThreads = 1024;
constexpr int kPgWarps = kPgThreads / 32;
constexpr int kPgCluster = 16;
constexpr int kPgPer = SPEC_MAX_BATCH / kPgThreads;  // requests of a thread
constexpr int kPgWords = 16;                         // words of 32 pages of a warp and pass
// Workspace words behind the status: number of moved pages.
constexpr int kPgMoved = 4;

// ----------------------------------------------------------- scan of the pool
// The cluster scans the counts in passes of (blocks * 16384) pages; in a pass
// a warp has 512 adjacent pages, read as 16 coalesced words whose ballots say
// which are free.  Blocks exchange their totals through distributed shared
// memory, one cluster barrier a pass.
struct PoolScan {
    int* s_warp;  // [kPgWarps + 1]
    int* s_cta;   // [2][kPgCluster]
    int ranks, rank, pages;
    int passes;
    int turn;
    bool started;

    // of the current pass
    int first;      // the warp's first page
    uint32_t word;  // lane j < 16: bit i set if page first + 32 j + i is free
    int before;     // free pages before the warp's first
    int total;      // free pages of all passes so far

    __device__ PoolScan(int* sw, int* sc, int n, int r, int p) : s_warp(sw), s_cta(sc), ranks(n), rank(r), pages(p) {
        // every block of the cluster runs before the first store to another one
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        started = false;
        passes = (int)(((long long)p + (long long)n * kPgWarps * kPgWords * 32 - 1) /
                       ((long long)n * kPgWarps * kPgWords * 32));
        turn = 0;
        total = 0;
    }

    // Reads pass `pass`; ref[j] keeps the counts if KEEP.
    template <bool KEEP>
    __device__ void read(const int32_t* ref_count, int pass, int32_t (&ref)[kPgWords]) {
        cg::cluster_group cluster = cg::this_cluster();
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const long long f = (((long long)pass * ranks + rank) * kPgWarps + warp) * (kPgWords * 32);
        first = f < pages ? (int)f : pages;
        int32_t v[kPgWords];
#pragma unroll
        for (int j = 0; j < kPgWords; ++j) {
            const long long p = f + 32 * j + lane;
            v[j] = p < pages ? __ldcg(ref_count + p) : 1;
        }
        int n = 0;
        word = 0;
#pragma unroll
        for (int j = 0; j < kPgWords; ++j) {
            const uint32_t w = __ballot_sync(0xffffffffu, v[j] == 0);
            if (lane == j) word = w;
            n += __popc(w);
            if (KEEP) ref[j] = v[j];
        }
        if (lane == 0) s_warp[warp] = n;
        if (!started) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        started = true;
        __syncthreads();
        if (warp == 0) {
            const int c = s_warp[lane];
            int x = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            s_warp[lane] = x - c;
            const int all = __shfl_sync(0xffffffffu, x, 31);
            if (lane < ranks) *cluster.map_shared_rank(&s_cta[turn * kPgCluster + rank], lane) = all;
        }
        cluster.sync();
        int base = total, sum = 0;
        for (int r = 0; r < ranks; ++r) {
            const int c = s_cta[turn * kPgCluster + r];
            if (r < rank) base += c;
            sum += c;
        }
        before = base + s_warp[warp];
        total += sum;
        turn ^= 1;
        __syncthreads();  // s_warp is free for the next pass
    }

    // The free pages before page first + 32 j + lane, for the word of j.
    __device__ __forceinline__ int rank_of(int j, uint32_t& w, int& upto) const {
        const int lane = threadIdx.x & 31;
        w = __shfl_sync(0xffffffffu, word, j);
        const int r = upto + __popc(w & ((1u << lane) - 1u));
        upto += __popc(w);
        return r;
    }
};

// Sums of needs stop at kMany, above any pool, so that they stay in 32 bits.
constexpr int kMany = 0x3fffffff;
__device__ __forceinline__ int add_needs(int a, int b) { return min(a + b, kMany); }

// Exclusive prefix over n <= 4096 values of at most kMany, four adjacent ones a
// thread, into out[0..n]; out[n] is the sum.
__device__ __forceinline__ void block_prefix(const int (&v)[kPgPer], int n, int* out, int* s_tmp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int x = 0;
#pragma unroll
    for (int i = 0; i < kPgPer; ++i) x = add_needs(x, v[i]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = add_needs(x, y);
    }
    if (lane == 31) s_tmp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = s_tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y = add_needs(y, z);
        }
        s_tmp[lane] = y;
    }
    __syncthreads();
    const int left = __shfl_up_sync(0xffffffffu, x, 1);
    int at = add_needs(warp ? s_tmp[warp - 1] : 0, lane ? left : 0);
#pragma unroll
    for (int i = 0; i < kPgPer; ++i) {
        const int b = tid * kPgPer + i;
        if (b < n) out[b] = at;
        at = add_needs(at, v[i]);
        if (b == n - 1) out[n] = at;
    }
    __syncthreads();
}

// The largest b with pref[b] <= r (pref[0] = 0, ascending, n + 1 entries, r < pref[n]).
__device__ __forceinline__ int owner_of(const int* pref, int n, int r) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pref[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Of the prefixes, the largest one that `free` pages cover.
__device__ __forceinline__ int covered(const int* pref, int n, int free) {
    return pref[n] <= free ? pref[n] : pref[owner_of(pref, n, free)];
}

// Gives one reference of a table entry back.
__device__ __forceinline__ void release(int32_t* ref_count, int pages, int page, int* status) {
    if (page < 0) return;
    if (page >= pages) {
        set_status(status, SPEC_ERR_PAGE);
        return;
    }
    if (atomicSub(ref_count + page, 1) <= 0) {
        atomicAdd(ref_count + page, 1);
        set_status(status, SPEC_ERR_PAGE);
    }
}

struct ReserveArgs {
    int32_t* table;
    int32_t* num;
    int32_t* ref;
    const int32_t* len;
    const int32_t* ell;
    int32_t* out_status;
    int* status;
    int pages, B, gamma, max_pages, page_size;
};

// Reserve: every block sums the requests' needs (4096 at most, four a thread),
// the cluster scans the pool, and the warp that sees the r-th free page gives
// it to the request whose range of needs holds r (a binary search in shared
// memory).  Latency bound: 1024 requests over a pool of 250,000 pages read 1 MB.
__global__ void __launch_bounds__(kPgThreads) k_reserve_pages(ReserveArgs a) {
    pdl_trigger();
    pdl_wait();
    __shared__ int s_pref[SPEC_MAX_BATCH + 1];
    __shared__ int s_num[SPEC_MAX_BATCH];
    __shared__ int s_warp[kPgWarps + 1], s_cta[2 * kPgCluster];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31;

    int grow[kPgPer], err[kPgPer];
#pragma unroll
    for (int i = 0; i < kPgPer; ++i) {
        const int b = tid * kPgPer + i;
        grow[i] = 0;
        err[i] = SPEC_OK;
        if (b < a.B) {
            const int ell = a.ell ? a.ell[b] : a.gamma, n = a.len[b], held = a.num[b];
            s_num[b] = held;
            if (ell < 0 || ell > a.gamma) err[i] = SPEC_ERR_VERIFY_LEN;
            else if (n < 0 || held < 0 || held > a.max_pages) err[i] = SPEC_ERR_CACHE_LEN;
            else {
                const long long need = ((long long)n + ell + a.page_size) / a.page_size;
                if (need > a.max_pages) err[i] = SPEC_ERR_CACHE_LEN;
                else if (need > held) grow[i] = min((int)need - held, kMany);
            }
        }
    }
    block_prefix(grow, a.B, s_pref, s_warp);
    const int need = s_pref[a.B];
    int limit = 0;
    if (need > 0) {
        PoolScan scan(s_warp, s_cta, ranks, rank, a.pages);
        int32_t unused[kPgWords];
        int passes = 0;
        do scan.read<false>(a.ref, passes++, unused);
        while (passes < scan.passes && scan.total < need);
        limit = covered(s_pref, a.B, min(need, scan.total));
        if (passes > 1) scan.total = 0;
        for (int p = 0; p < passes && (passes == 1 || scan.total < limit); ++p) {
            if (passes > 1) scan.read<false>(a.ref, p, unused);  // a pool of several passes is read again
            int upto = scan.before;
#pragma unroll
            for (int j = 0; j < kPgWords; ++j) {
                uint32_t w;
                const int r = scan.rank_of(j, w, upto);
                if (((w >> lane) & 1u) && r < limit) {
                    const int b = owner_of(s_pref, a.B, r);
                    const int page = scan.first + 32 * j + lane;
                    a.table[(size_t)b * a.max_pages + s_num[b] + (r - s_pref[b])] = page;
                    a.ref[page] = 1;
                }
            }
        }
    }
    if (rank != 0) return;
#pragma unroll
    for (int i = 0; i < kPgPer; ++i) {
        const int b = tid * kPgPer + i;
        if (b < a.B) {
            if (err[i] == SPEC_OK && grow[i] > 0) {  // the prefixes may have stopped at kMany, above any limit
                if (s_pref[b + 1] <= limit) a.num[b] = s_num[b] + grow[i];
                else err[i] = SPEC_ERR_POOL;
            }
            a.out_status[b] = err[i];
            if (err[i] != SPEC_OK) set_status(a.status, err[i]);
        }
    }
}

struct CommitArgs {
    int32_t* table;
    int32_t* num;
    int32_t* ref;
    const int32_t* len;
    const int32_t* accept;
    int32_t* out_len;
    int* status;
    int pages, B, max_pages, page_size, window, sinks;
};

// Commit: one warp a request, a lane per slot given back.
__global__ void __launch_bounds__(256) k_commit_pages(CommitArgs a) {
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= a.B) return;
    const int n = a.len[b], acc = a.accept[b], held = a.num[b];
    const long long now = (long long)n + acc + 1;
    int32_t* row = a.table + (size_t)b * a.max_pages;
    if (n < 0 || acc < -1 || held < 0 || held > a.max_pages || now > (long long)held * a.page_size ||
        now > 0x7fffffffll) {
        if (lane == 0) {
            a.out_len[b] = n;
            set_status(a.status, SPEC_ERR_CACHE_LEN);
        }
        return;
    }
    const int keep = (int)((now + a.page_size - 1) / a.page_size);
    for (int s = keep + lane; s < held; s += 32) {
        release(a.ref, a.pages, row[s], a.status);
        row[s] = -1;
    }
    if (a.window > 0) {
        // pages that start at or behind the sinks and end before the first
        // position that the next token sees, now - window + 1
        const int from = (int)(((long long)a.sinks + a.page_size - 1) / a.page_size);
        const long long unseen = now - a.window + 1;
        const int to = unseen > 0 ? (int)(unseen / a.page_size) : 0;
        for (int s = from + lane; s < min(to, keep); s += 32) {
            const int page = row[s];
            if (page != -1) {
                release(a.ref, a.pages, page, a.status);
                row[s] = -1;
            }
        }
    }
    if (lane == 0) {
        a.num[b] = keep;
        a.out_len[b] = (int)now;
    }
}

struct FreeArgs {
    int32_t* table;
    int32_t* num;
    int32_t* ref;
    int32_t* len;
    const int32_t* requests;
    int* status;
    int pages, n, B, max_pages;
};

// Free: one warp an entry of the list.  Each slot is exchanged for -1, so that
// of two warps with the same request one gets its page.
__global__ void __launch_bounds__(256) k_free_pages(FreeArgs a) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (i >= a.n) return;
    const int b = a.requests[i];
    if (b < 0 || b >= a.B) {
        if (lane == 0) set_status(a.status, SPEC_ERR_REQUEST);
        return;
    }
    int32_t* row = a.table + (size_t)b * a.max_pages;
    const int held = min(max(*(volatile int32_t*)(a.num + b), 0), a.max_pages);
    for (int s = lane; s < held; s += 32) release(a.ref, a.pages, atomicExch(row + s, -1), a.status);
    __syncwarp();
    if (lane == 0) {
        a.num[b] = 0;
        a.len[b] = 0;
    }
}

struct ForkArgs {
    int32_t* table;
    int32_t* num;
    int32_t* ref;
    int32_t* len;
    const int32_t* src;
    const int32_t* dst;
    int32_t* out_status;
    int* status;
    int32_t* list;  // [3][n]: page, copy, tokens
    int pages, n, B, max_pages, page_size;
};

constexpr int kForkSrc = 1 << 30;  // flag beside a request's count as a dst

// Fork, the tables: (1) every block checks all forks; (2) the valid ones'
// destinations give their pages back, one warp each; (3) the pool is scanned
// for the copies of partial last pages; (4) the destinations' rows are
// written.  A valid fork's dst is no other fork's dst or src, so nothing that
// is written is read by another fork.
__global__ void __launch_bounds__(kPgThreads) k_fork_tables(ForkArgs a) {
    pdl_trigger();
    pdl_wait();
    __shared__ int s_pref[SPEC_MAX_BATCH + 1];
    __shared__ int s_use[SPEC_MAX_BATCH];
    __shared__ int s_warp[kPgWarps + 1], s_cta[2 * kPgCluster];
    __shared__ signed char s_err[SPEC_MAX_BATCH];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    for (int b = tid; b < a.B; b += kPgThreads) s_use[b] = 0;
    __syncthreads();
    for (int i = tid; i < a.n; i += kPgThreads) {
        const int s = a.src[i], d = a.dst[i];
        if (s >= 0 && s < a.B) atomicOr(&s_use[s], kForkSrc);
        if (d >= 0 && d < a.B) atomicAdd(&s_use[d], 1);
    }
    __syncthreads();
    int part[kPgPer];
#pragma unroll
    for (int q = 0; q < kPgPer; ++q) {
        const int i = tid * kPgPer + q;
        part[q] = 0;
        if (i < a.n) {
            const int s = a.src[i], d = a.dst[i];
            int err = SPEC_OK;
            if (s < 0 || s >= a.B || d < 0 || d >= a.B || s_use[d] != 1) err = SPEC_ERR_REQUEST;
            else {
                const int n = a.len[s], held = a.num[s];
                const long long need = n >= 0 ? ((long long)n + a.page_size - 1) / a.page_size : 0;
                if (n < 0 || held > a.max_pages || need > held) err = SPEC_ERR_CACHE_LEN;
                else if (n % a.page_size) {
                    const int page = a.table[(size_t)s * a.max_pages + need - 1];
                    if (page < 0 || page >= a.pages) err = SPEC_ERR_PAGE;
                    else part[q] = 1;
                }
            }
            s_err[i] = (signed char)err;
        }
    }
    block_prefix(part, a.n, s_pref, s_warp);

    const int warps = ranks * kPgWarps, me = warp * ranks + rank;
    for (int i = me; i < a.n; i += warps) {
        if (s_err[i] != SPEC_OK) continue;
        const int d = a.dst[i];
        const int held = min(max(a.num[d], 0), a.max_pages);
        int32_t* row = a.table + (size_t)d * a.max_pages;
        for (int s = lane; s < held; s += 32) {
            release(a.ref, a.pages, row[s], a.status);
            row[s] = -1;
        }
    }
    cluster.sync();  // what was given back is free for the scan

    const int need = s_pref[a.n];
    int limit = 0;
    if (need > 0) {
        PoolScan scan(s_warp, s_cta, ranks, rank, a.pages);
        int32_t unused[kPgWords];
        int passes = 0;
        do scan.read<false>(a.ref, passes++, unused);
        while (passes < scan.passes && scan.total < need);
        limit = min(need, scan.total);
        if (passes > 1) scan.total = 0;
        for (int p = 0; p < passes && (passes == 1 || scan.total < limit); ++p) {
            if (passes > 1) scan.read<false>(a.ref, p, unused);
            int upto = scan.before;
#pragma unroll
            for (int j = 0; j < kPgWords; ++j) {
                uint32_t w;
                const int r = scan.rank_of(j, w, upto);
                if (((w >> lane) & 1u) && r < limit) {
                    const int i = owner_of(s_pref, a.n, r);
                    const int page = scan.first + 32 * j + lane;
                    const int s = a.src[i];
                    const int whole = a.len[s] / a.page_size;
                    a.table[(size_t)a.dst[i] * a.max_pages + whole] = page;
                    a.ref[page] = 1;
                    a.list[a.n + i] = page;
                }
            }
        }
        cluster.sync();  // the scan of every block is done before references are added
    }
    for (int i = me; i < a.n; i += warps) {
        int err = s_err[i], tokens = 0;
        if (err == SPEC_OK) {
            const int s = a.src[i], d = a.dst[i], n = a.len[s];
            const int whole = n / a.page_size;
            const bool cut = s_pref[i + 1] > s_pref[i];
            if (cut && s_pref[i + 1] > limit) err = SPEC_ERR_POOL;
            const int32_t* from = a.table + (size_t)s * a.max_pages;
            int32_t* to = a.table + (size_t)d * a.max_pages;
            if (err == SPEC_OK) {
                for (int q = lane; q < whole; q += 32) {
                    const int page = from[q];
                    to[q] = page;
                    if (page >= 0 && page < a.pages) atomicAdd(a.ref + page, 1);
                    else if (page != -1) set_status(a.status, SPEC_ERR_PAGE);
                }
                if (cut) tokens = n % a.page_size;
                if (lane == 0 && cut) a.list[i] = from[whole];
            }
            if (lane == 0) {
                a.num[d] = err == SPEC_OK ? whole + (cut ? 1 : 0) : 0;
                a.len[d] = err == SPEC_OK ? n : 0;
            }
        }
        if (lane == 0) {
            a.list[2 * a.n + i] = tokens;
            a.out_status[i] = err;
            if (err != SPEC_OK) set_status(a.status, err);
        }
    }
}

// ------------------------------------------------------------------- copies
// 16-byte vectors of one page's tokens, K or V of one layer.
struct PageShape {
    uint32_t per_row;    // vectors of one (token, head)
    uint32_t per_token;  // vectors of one token
    FastDiv by_token, by_row;
    int flat;  // 1: a token's vectors and the tokens are adjacent
    int whole_flat;  // 1: a whole page's vectors are adjacent, in whatever order
};

__device__ __forceinline__ long long vec_at(const CacheView& c, const PageShape& g, uint32_t i, bool flat) {
    if (flat) return (long long)i * 16;
    const uint32_t t = g.by_token.div(i), r = i - t * g.per_token;
    const uint32_t h = g.by_row.div(r);
    return t * c.token + h * c.head + (long long)(r - h * g.per_row) * 16;
}

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyVecs = kCopyThreads * kCopyUnroll;  // 32 KB an item

// Copies vectors [i0, min(i0 + kCopyVecs, n)) of page `src` to page `dst`,
// all loads of a thread in flight before its first store.
__device__ __forceinline__ void copy_vecs(const CacheView& c, const PageShape& g, char* base, int src, int dst,
                                          uint32_t i0, uint32_t n, bool flat) {
    const char* from = base + (long long)src * c.page;
    char* to = base + (long long)dst * c.page;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        const uint32_t i = i0 + u * kCopyThreads + threadIdx.x;
        if (i < n) v[u] = *(const uint4*)(from + vec_at(c, g, i, flat));
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        const uint32_t i = i0 + u * kCopyThreads + threadIdx.x;
        if (i < n) *(uint4*)(to + vec_at(c, g, i, flat)) = v[u];
    }
}

// Fork, the data: block (i, layer and K or V, 32 KB slice).
__global__ void __launch_bounds__(kCopyThreads) k_fork_copy(CacheView c, PageShape g, const int32_t* list, int n) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x;
    const int tokens = list[2 * n + i];
    const uint32_t vecs = (uint32_t)tokens * g.per_token, i0 = blockIdx.z * kCopyVecs;
    if (i0 >= vecs) return;
    const int layer = blockIdx.y >> 1;
    char* base = ((blockIdx.y & 1) ? c.v : c.k) + layer * c.layer;
    copy_vecs(c, g, base, list[i], list[n + i], i0, vecs, g.flat);
}

struct CompactArgs {
    const int32_t* table;
    const int32_t* num;
    const int32_t* ref;
    int32_t* out_table;
    int32_t* out_ref;
    int32_t* out_total;
    int* status;
    int32_t* name;   // [pages] new id of a referenced page
    int32_t* mover;  // [pages] referenced pages from N on, by their rank among all referenced
    int32_t* count;  // [pages] their counts
    int32_t* hole;   // [pages] free pages below N
    int pages, B, max_pages;
};

// Compact, the plan.  With f(p) free pages before p, a referenced page p is
// number p - f(p) of the N referenced ones.  The free pages below N are the
// holes 0..h-1, the referenced pages from N on are the numbers N-h..N-1, so
// hole k gets number N-h+k: one scan finds N, a second both lists, and h is
// their length.
__global__ void __launch_bounds__(kPgThreads) k_compact_plan(CompactArgs a) {
    pdl_trigger();
    pdl_wait();
    __shared__ int s_warp[kPgWarps + 1], s_cta[2 * kPgCluster], s_holes[kPgCluster];
    __shared__ int s_mine;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) s_mine = 0;
    PoolScan scan(s_warp, s_cta, ranks, rank, a.pages);
    int32_t ref[kPgWords];
    for (int p = 0; p < scan.passes; ++p) scan.read<true>(a.ref, p, ref);
    const int N = a.pages - scan.total;
    if (scan.passes > 1) scan.total = 0;
    int holes = 0;
    for (int p = 0; p < scan.passes; ++p) {
        if (scan.passes > 1) scan.read<true>(a.ref, p, ref);
        int upto = scan.before;
#pragma unroll
        for (int j = 0; j < kPgWords; ++j) {
            uint32_t w;
            const int f = scan.rank_of(j, w, upto);
            const int page = scan.first + 32 * j + lane;
            if (page < a.pages) {
                if (ref[j] == 0) {
                    if (page < N) {
                        a.hole[f] = page;
                        ++holes;
                    } else {
                        a.out_ref[page] = 0;
                    }
                    a.name[page] = -1;
                } else if (page < N) {
                    a.name[page] = page;
                    a.out_ref[page] = ref[j];
                } else {
                    a.mover[page - f] = page;
                    a.count[page - f] = ref[j];
                    a.out_ref[page] = 0;
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) holes += __shfl_xor_sync(0xffffffffu, holes, o);
    if (lane == 0 && holes) atomicAdd(&s_mine, holes);
    __syncthreads();
    if (tid < ranks) *cluster.map_shared_rank(&s_holes[rank], tid) = s_mine;
    cluster.sync();
    int h = 0;
    for (int r = 0; r < ranks; ++r) h += s_holes[r];
    for (int k = rank * kPgThreads + tid; k < h; k += ranks * kPgThreads) {
        const int q = N - h + k;
        const int to = __ldcg(a.hole + k);
        a.out_ref[to] = __ldcg(a.count + q);
        a.name[__ldcg(a.mover + q)] = to;
    }
    if (rank == 0 && tid == 0) {
        *a.out_total = N;
        a.status[kPgMoved] = h;
    }
}

// Compact, the data: first the moved pages in 32 KB items, then the tables.
__global__ void __launch_bounds__(kCopyThreads) k_compact_move(CompactArgs a, CacheView c, PageShape g) {
    pdl_trigger();
    pdl_wait();
    const int h = a.status[kPgMoved], N = *a.out_total;
    const uint32_t vecs = (uint32_t)c.page_size * g.per_token;
    const int slices = (int)((vecs + kCopyVecs - 1) / kCopyVecs);
    const long long items = (long long)h * c.layers * 2 * slices;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const long long kv = it / slices;
        const int slice = (int)(it - kv * slices);
        const int k = (int)(kv / (2 * c.layers)), lk = (int)(kv - (long long)k * 2 * c.layers);
        char* base = ((lk & 1) ? c.v : c.k) + (lk >> 1) * c.layer;
        copy_vecs(c, g, base, a.mover[N - h + k], a.hole[k], (uint32_t)slice * kCopyVecs, vecs, g.whole_flat);
    }
    const long long slots = (long long)a.B * a.max_pages;
    for (long long i = (long long)blockIdx.x * kCopyThreads + threadIdx.x; i < slots;
         i += (long long)gridDim.x * kCopyThreads) {
        const int b = (int)(i / a.max_pages), s = (int)(i - (long long)b * a.max_pages);
        int page = s < a.num[b] ? a.table[i] : -1;
        if (page >= 0) {
            const int to = page < a.pages ? a.name[page] : -1;
            if (to < 0) set_status(a.status, SPEC_ERR_PAGE);
            page = to;
        }
        a.out_table[i] = page;
    }
}

}  // namespace specv

// ===================================================================== host
using namespace specv;

namespace {

std::mutex g_pg_mu;
struct PagesInfo {
    int cluster = 0, sms = 0;
};
PagesInfo g_pg[64];

// Blocks of the cluster kernels: 16 where the GPU can place them, else the
// portable 8.
int pages_info(PagesInfo& out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_pg_mu);
    PagesInfo& d = g_pg[dev];
    if (!d.cluster) {
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SPEC_ERR_CUDA;
        const void* fns[3] = {(const void*)k_reserve_pages, (const void*)k_fork_tables, (const void*)k_compact_plan};
        int cl = kPgCluster;
        for (const void* f : fns) {
            int n = 0;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kPgCluster);
            cfg.blockDim = dim3(kPgThreads);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = kPgCluster;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
                cudaOccupancyMaxActiveClusters(&n, f, &cfg) != cudaSuccess || n < 1) {
                cudaGetLastError();
                cl = 8;
            }
        }
        d.cluster = cl;
    }
    out = d;
    return SPEC_OK;
}

// One block per 16384 pages, in a cluster of a power of two: a small pool is
// scanned by one block, without the launch and the barriers of sixteen.  `least`
// blocks where there is other work for them.
template <typename A>
int launch_cluster(void (*kernel)(A), const A& a, int least, int most, cudaStream_t st) {
    int blocks = 1;
    while (blocks < least && blocks < most) blocks *= 2;
    while (blocks < most && (long long)blocks * kPgWarps * kPgWords * 32 < a.pages) blocks *= 2;
    return launch_dependent(kernel, dim3(blocks), kPgThreads, 0, st, blocks, a);
}

int check_tables(const int32_t* table, const int32_t* num, const int32_t* ref, int pages, int B, int max_pages,
                 void* ws, size_t ws_bytes, size_t need) {
    if (!table || !num || !ref || !ws) return SPEC_ERR_NULL;
    if (((uintptr_t)table | (uintptr_t)num | (uintptr_t)ref) & 3 || ((uintptr_t)ws & 15)) return SPEC_ERR_ALIGN;
    if (ws_bytes < need) return SPEC_ERR_WORKSPACE;
    (void)pages;
    (void)B;
    (void)max_pages;
    return SPEC_OK;
}

bool tables_shape_ok(int pages, int B, int max_pages) {
    return pages >= 1 && pages < kMany && B >= 0 && B <= SPEC_MAX_BATCH && max_pages >= 1;
}

PageShape page_shape(const spec_cache* c) {
    PageShape g;
    const int es = dtype_size(c->dt);
    g.per_row = (uint32_t)(c->head_dim * es / 16);
    g.per_token = g.per_row * (uint32_t)c->kv_heads;
    g.by_token = FastDiv(g.per_token);
    g.by_row = FastDiv(g.per_row);
    const bool heads = c->kv_heads == 1 || c->head_stride == c->head_dim;
    g.flat = heads && (c->page_size == 1 || c->token_stride == (long long)c->kv_heads * c->head_dim);
    g.whole_flat = g.flat || ((c->page_size == 1 || c->token_stride == c->head_dim) &&
                              (c->kv_heads == 1 || c->head_stride == (long long)c->page_size * c->head_dim));
    return g;
}

// vectors of a page must be countable in 31 bits
bool page_size_ok(const spec_cache* c) {
    return (long long)c->page_size * c->kv_heads * c->head_dim * dtype_size(c->dt) / 16 < 0x7fffffffll - kCopyVecs;
}

}  // namespace

extern "C" {

size_t spec_cache_workspace_bytes(int B, int pages) {
    if (B < 0 || B > SPEC_MAX_BATCH || pages < 0) return 0;
    return 256 + ((size_t)B * 12 + 255) / 256 * 256 + (size_t)pages * 16;
}

int spec_reserve_pages(int32_t* page_table, int32_t* num_pages, int32_t* ref_count, int pages,
                       const int32_t* cache_len, const int32_t* verify_len, int B, int gamma, int max_pages,
                       int page_size, int32_t* out_status, void* workspace, size_t workspace_bytes,
                       spec_stream_t stream) {
    TraceRange tr("spec_reserve_pages");
    if (!tables_shape_ok(pages, B, max_pages) || gamma < 0 || gamma > SPEC_MAX_GAMMA || page_size < 1)
        return SPEC_ERR_SHAPE;
    if (B == 0) return SPEC_OK;
    if (!cache_len || !out_status) return SPEC_ERR_NULL;
    int rc = check_tables(page_table, num_pages, ref_count, pages, B, max_pages, workspace, workspace_bytes, 256);
    if (rc != SPEC_OK) return rc;
    if (((uintptr_t)cache_len | (uintptr_t)verify_len | (uintptr_t)out_status) & 3) return SPEC_ERR_ALIGN;
    PagesInfo d;
    if ((rc = pages_info(d)) != SPEC_OK) return rc;
    const ReserveArgs a{page_table, num_pages, ref_count, cache_len, verify_len, out_status,
                        (int*)workspace, pages, B, gamma, max_pages, page_size};
    return launch_cluster(k_reserve_pages, a, 1, d.cluster, (cudaStream_t)stream);
}

int spec_commit_pages(int32_t* page_table, int32_t* num_pages, int32_t* ref_count, int pages,
                      const int32_t* cache_len, const int32_t* accept_len, int B, int max_pages, int page_size,
                      int window, int sinks, int32_t* out_cache_len, void* workspace, size_t workspace_bytes,
                      spec_stream_t stream) {
    TraceRange tr("spec_commit_pages");
    if (!tables_shape_ok(pages, B, max_pages) || page_size < 1 || window < 0 || sinks < 0) return SPEC_ERR_SHAPE;
    if (B == 0) return SPEC_OK;
    if (!cache_len || !accept_len || !out_cache_len) return SPEC_ERR_NULL;
    const int rc = check_tables(page_table, num_pages, ref_count, pages, B, max_pages, workspace, workspace_bytes, 256);
    if (rc != SPEC_OK) return rc;
    if (((uintptr_t)cache_len | (uintptr_t)accept_len | (uintptr_t)out_cache_len) & 3) return SPEC_ERR_ALIGN;
    const CommitArgs a{page_table, num_pages, ref_count, cache_len, accept_len, out_cache_len,
                       (int*)workspace, pages, B, max_pages, page_size, window, sinks};
    return launch_dependent(k_commit_pages, dim3((B + 7) / 8), 256, 0, (cudaStream_t)stream, 0, a);
}

int spec_free_pages(int32_t* page_table, int32_t* num_pages, int32_t* ref_count, int pages, int32_t* cache_len,
                    const int32_t* requests, int n, int B, int max_pages, void* workspace, size_t workspace_bytes,
                    spec_stream_t stream) {
    TraceRange tr("spec_free_pages");
    if (!tables_shape_ok(pages, B, max_pages) || n < 0 || n > SPEC_MAX_BATCH) return SPEC_ERR_SHAPE;
    if (B == 0 || n == 0) return SPEC_OK;
    if (!cache_len || !requests) return SPEC_ERR_NULL;
    const int rc = check_tables(page_table, num_pages, ref_count, pages, B, max_pages, workspace, workspace_bytes, 256);
    if (rc != SPEC_OK) return rc;
    if (((uintptr_t)cache_len | (uintptr_t)requests) & 3) return SPEC_ERR_ALIGN;
    const FreeArgs a{page_table, num_pages, ref_count, cache_len, requests, (int*)workspace, pages, n, B, max_pages};
    return launch_dependent(k_free_pages, dim3((n + 7) / 8), 256, 0, (cudaStream_t)stream, 0, a);
}

int spec_fork_pages(int32_t* page_table, int32_t* num_pages, int32_t* ref_count, int32_t* cache_len,
                    const int32_t* src, const int32_t* dst, int n, int B, int max_pages, const spec_cache* cache,
                    int32_t* out_status, void* workspace, size_t workspace_bytes, spec_stream_t stream) {
    TraceRange tr("spec_fork_pages");
    CacheView c;
    int rc = cache_view(cache, c);
    if (rc != SPEC_OK) return rc;
    if (!tables_shape_ok(c.pages, B, max_pages) || n < 0 || n > B || c.layers > 32767 || !page_size_ok(cache))
        return SPEC_ERR_SHAPE;
    if (n == 0) return SPEC_OK;
    if (!cache_len || !src || !dst || !out_status) return SPEC_ERR_NULL;
    rc = check_tables(page_table, num_pages, ref_count, c.pages, B, max_pages, workspace, workspace_bytes,
                      256 + (size_t)B * 12);
    if (rc != SPEC_OK) return rc;
    if (((uintptr_t)cache_len | (uintptr_t)src | (uintptr_t)dst | (uintptr_t)out_status) & 3) return SPEC_ERR_ALIGN;
    const PageShape g = page_shape(cache);
    const long long slices = ((long long)c.page_size * g.per_token + kCopyVecs - 1) / kCopyVecs;
    if (slices > 65535) return SPEC_ERR_SHAPE;
    PagesInfo d;
    if ((rc = pages_info(d)) != SPEC_OK) return rc;
    int32_t* list = (int32_t*)((char*)workspace + 256);
    const ForkArgs a{page_table, num_pages, ref_count, cache_len, src, dst, out_status, (int*)workspace, list,
                     c.pages, n, B, max_pages, c.page_size};
    if ((rc = launch_cluster(k_fork_tables, a, (n + kPgWarps - 1) / kPgWarps, d.cluster, (cudaStream_t)stream)) != SPEC_OK) return rc;
    return launch_dependent(k_fork_copy, dim3(n, c.layers * 2, (unsigned)slices), kCopyThreads, 0,
                            (cudaStream_t)stream, 0, c, g, list, n);
}

int spec_compact_pages(const int32_t* page_table, const int32_t* num_pages, const int32_t* ref_count, int B,
                       int max_pages, const spec_cache* cache, int32_t* out_page_table, int32_t* out_ref_count,
                       int32_t* out_total, void* workspace, size_t workspace_bytes, spec_stream_t stream) {
    TraceRange tr("spec_compact_pages");
    CacheView c;
    int rc = cache_view(cache, c);
    if (rc != SPEC_OK) return rc;
    if (!tables_shape_ok(c.pages, B, max_pages) || !page_size_ok(cache)) return SPEC_ERR_SHAPE;
    if (!ref_count || !out_ref_count || !out_total || !workspace || (B > 0 && (!page_table || !num_pages ||
                                                                              !out_page_table)))
        return SPEC_ERR_NULL;
    if (((uintptr_t)page_table | (uintptr_t)num_pages | (uintptr_t)ref_count | (uintptr_t)out_page_table |
         (uintptr_t)out_ref_count | (uintptr_t)out_total) & 3 || ((uintptr_t)workspace & 15))
        return SPEC_ERR_ALIGN;
    if (workspace_bytes < spec_cache_workspace_bytes(B, c.pages)) return SPEC_ERR_WORKSPACE;
    PagesInfo d;
    if ((rc = pages_info(d)) != SPEC_OK) return rc;
    int32_t* lists = (int32_t*)((char*)workspace + 256 + ((size_t)B * 12 + 255) / 256 * 256);
    const size_t P = (size_t)c.pages;
    const CompactArgs a{page_table, num_pages, ref_count, out_page_table, out_ref_count, out_total, (int*)workspace,
                        lists, lists + P, lists + 2 * P, lists + 3 * P, c.pages, B, max_pages};
    if ((rc = launch_cluster(k_compact_plan, a, 1, d.cluster, (cudaStream_t)stream)) != SPEC_OK) return rc;
    return launch_dependent(k_compact_move, dim3(d.sms * 4), kCopyThreads, 0, (cudaStream_t)stream, 0, a, c,
                            page_shape(cache));
}

}  // extern "C"
