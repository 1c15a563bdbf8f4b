// Attention of a batch that shares prefixes: the plan that finds the groups, the
// C entries, and the kernel that joins the parts of rows.
//
// A row's keys are two sets: the positions that its request shares with a group,
// and the positions behind them.  Each set's sums (o, l) with their maximum m are
// those of a softmax over that set, and with M = max m_i
//   out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
// The attention kernels take a group's set once, for the rows of all its members,
// as a request of that many rows; a shared key is read once a row tile of the group
// instead of once a request, and from L2 but for the first.
#include <cooperative_groups.h>

#include <math.h>

#include <algorithm>

#include "specv_attend.cuh"
#include "specv_trace.h"

namespace cg = cooperative_groups;

namespace specv {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCluster = 16;
constexpr int kPlanAgain = 32;  // passes until classes are taken apart by the first page too

struct PlanArgs {
    const int32_t* table;
    const int32_t* len;
    const int32_t* ell;
    const int32_t* row;
    int32_t* leader;
    int32_t* shared;
    int* plan;
    ShareItem* items;
    int32_t* list;
    uint8_t* kinds;
    int rows, B, gamma, max_pages, page_size, least;
    int limit;
    int key;   // the last entry of a prefix of `least` positions
    int hash;  // places of the classes' table, a power of two
};

// Leading entries that two rows of the page table have alike, `most` at most; by a
// warp, sixteen words of 32 entries at a time.
__device__ __forceinline__ int common_pages(const int32_t* x, const int32_t* y, int most) {
    constexpr int W = 16;
    const int lane = threadIdx.x & 31;
    for (int i0 = 0; i0 < most; i0 += 32 * W) {
        int32_t p[W], q[W];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int i = i0 + 32 * w + lane;
            p[w] = i < most ? x[i] : -1;
            q[w] = i < most ? y[i] : -1;
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint32_t differ = __ballot_sync(0xffffffffu, p[w] != q[w] || p[w] < 0);
            if (differ) return i0 + 32 * w + __ffs(differ) - 1;
        }
    }
    return most;
}

__device__ __forceinline__ void put_item(ShareItem* to, int n, int ell, int base, int rows, int b, int skip, int kind,
                                         int code) {
    int4* p = (int4*)to;
    p[0] = make_int4(n, ell, base, rows);
    p[1] = make_int4(b, skip, kind, code);
}

// The plan.  Requests with the same page where a prefix of `least` positions ends are
// a class, the lowest of them its head.  Each counts the leading full pages that it has
// like the head; the depth d that saves most reads, (members of depth >= d but the
// head) * d, makes those members and the head a group.  The head leaves its class in
// any case, the others go into the next pass, until none is left: a pass for each group
// of a tree of prompts.  Who shares `least` positions with a head is in its class, so
// how coarse classes are decides the passes and nothing else.  By the first page, chats
// behind a short common prompt were one class: 64 of them with four samples each took
// 106 us for 32 passes and as many groups, now 8.7 for all; 1000 lone requests ahead of a
// group 187 and 11.5.  (By both pages at once: a load more, plan of 1024 alone 7.7 -> 10 us.)
// Passes in number need groups whose own pages save more than the prompt of all, 40 of
// them, 900 pages deep, 160 us, or tables that no call here makes, with a page alike
// behind other ones: those are taken apart by the first page after a while.
// Then the groups' rows are listed and the items written.
//
// The requests' few numbers are in every block's shared memory.  What takes a step
// for each pair of requests, or reads the tables, is divided over the cluster's warps
// (a request each), whose results go to all blocks.  Bound by latency: barriers, and a
// few round trips to the tables a pass.  16 requests 8.5 us, 64 of one prompt 8.5, 64 in a
// tree of 6 prompts 14.6; 1024 in a tree of 96 prompts 36 us (with 8 blocks 48).
template <int PER>  // requests of a thread
__global__ void __launch_bounds__(kPlanThreads) k_share_plan(PlanArgs a) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ unsigned long long s_mem[];
    unsigned long long* s_best = s_mem;               // the best depth's key, by head
    int* s_class = (int*)(s_best + a.B);              // place in the classes' table; -1 placed
    int* s_full = s_class + a.B;                      // full pages
    int* s_head = s_full + a.B;                       // of its last pass
    int* s_shared = s_head + a.B;                     // pages shared; 0 alone
    int* s_rows = s_shared + a.B;                     // rows, 0 of a request with an error
    int* s_depth = s_rows + a.B;                      // [2][B] by pass; then the groups' rows and their places
    int* s_others = s_depth + 2 * a.B;                // members of its depth or more, but the head
    int* s_page = s_others + a.B;                     // [hash] the classes' keys
    int* s_low = s_page + a.hash;                     // [hash] the lowest request of a class
    __shared__ unsigned long long s_scan[kPlanWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int warp0 = warp * ranks + rank, warps = kPlanWarps * ranks;  // among the cluster's
    auto meet = [&] {
        if (ranks > 1) cluster.sync();
        else __syncthreads();
    };

    int code[PER], n[PER], ell[PER], base[PER], from[PER];
    for (int i = tid; i < a.hash; i += kPlanThreads) s_page[i] = -1;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = i * kPlanThreads + tid;
        code[i] = SPEC_OK;
        n[i] = ell[i] = base[i] = 0;
        from[i] = -1;
        if (b < a.B) {
            n[i] = a.len[b];
            ell[i] = a.ell ? a.ell[b] : a.gamma;
            base[i] = a.row ? a.row[b] : b * (a.gamma + 1);
            if (a.key < a.max_pages) from[i] = a.table[(size_t)b * a.max_pages + a.key];
        }
    }
    if (rank == 0 && tid == 0) a.plan[kPlanStatus] = SPEC_OK;
    for (int r = rank * kPlanThreads + tid; r < a.rows; r += ranks * kPlanThreads) a.kinds[r] = 0;
    __syncthreads();
    // the place of a class in the table, of which at least half is free
    auto place_of = [&](int key) {
        int at = (int)((uint32_t)key * 2654435761u >> 12 & (uint32_t)(a.hash - 1));
        for (;; at = (at + 1) & (a.hash - 1)) {
            const int old = atomicCAS(&s_page[at], -1, key);
            if (old == -1 || old == key) return at;
        }
    };
    bool any = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = i * kPlanThreads + tid;
        if (b >= a.B) continue;
        if (ell[i] < 0 || ell[i] > a.gamma) code[i] = SPEC_ERR_VERIFY_LEN;
        else if (base[i] < 0 || base[i] > a.rows - ell[i] - 1) code[i] = SPEC_ERR_ROW_INDEX;
        else if (n[i] < 0 || n[i] >= a.limit - ell[i]) code[i] = SPEC_ERR_CACHE_LEN;
        const int full = code[i] == SPEC_OK ? n[i] / a.page_size : 0;
        int at = -1;
        if (full > a.key && from[i] >= 0) {
            at = place_of(from[i]);
            any = true;
        }
        s_class[b] = at;
        s_full[b] = full;
        s_head[b] = b;
        s_shared[b] = 0;
        s_rows[b] = code[i] == SPEC_OK ? ell[i] + 1 : 0;
        s_best[b] = 0;
    }
    if (ranks > 1) cluster.sync();  // every block runs, and its kinds are zero

    for (int pass = 0; pass < a.B && __syncthreads_or(any); ++pass) {  // a head a pass at least
        int* s_d = s_depth + (pass & 1) * a.B;
        if (pass == kPlanAgain) {
            for (int i = tid; i < a.hash; i += kPlanThreads) s_page[i] = -1;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int b = i * kPlanThreads + tid;
                if (b >= a.B || s_class[b] < 0) continue;
                const uint32_t x = (uint32_t)a.table[(size_t)b * a.max_pages];
                s_class[b] = place_of((int)((x * 2246822519u ^ (uint32_t)from[i]) & 0x7fffffffu));
            }
        }
        for (int i = tid; i < a.hash; i += kPlanThreads) s_low[i] = 0x7fffffff;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int b = i * kPlanThreads + tid;
            if (b < a.B && s_class[b] >= 0) atomicMin(&s_low[s_class[b]], b);
        }
        __syncthreads();
        for (int b = warp0; b < a.B; b += warps) {
            const int c = s_class[b], h = c < 0 ? b : s_low[c];
            if (h == b) continue;
            const int d = common_pages(a.table + (size_t)b * a.max_pages, a.table + (size_t)h * a.max_pages,
                                       min(s_full[b], s_full[h]));
            if (lane < ranks) *cluster.map_shared_rank(s_d + b, lane) = d;
        }
        meet();
        for (int b = warp0; b < a.B; b += warps) {
            const int c = s_class[b], h = c < 0 ? b : s_low[c];
            if (h == b || (long long)s_d[b] * a.page_size < a.least) continue;
            const int d = s_d[b];
            int others = 0;
            for (int x = h + 1 + lane; x < a.B; x += 32) others += s_class[x] == c && s_d[x] >= d;
            others = __reduce_add_sync(0xffffffffu, others);
            if (lane < ranks) *cluster.map_shared_rank(s_others + b, lane) = others;
        }
        meet();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int b = i * kPlanThreads + tid;
            if (b >= a.B || s_class[b] < 0) continue;
            const int h = s_low[s_class[b]], d = s_d[b];
            const unsigned long long others = (unsigned)s_others[b];
            if (h != b && (long long)d * a.page_size >= a.least) atomicMax(&s_best[h], others * d << 13 | others);
        }
        __syncthreads();
        any = false;
        int now[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int b = i * kPlanThreads + tid;
            now[i] = -1;
            if (b >= a.B || s_class[b] < 0) continue;
            const int h = s_low[s_class[b]];
            const unsigned long long best = s_best[h];
            const int d = best ? (int)((best >> 13) / (best & 8191)) : 0;
            if (d > 0 && (b == h || s_d[b] >= d)) {
                s_head[b] = h;
                s_shared[b] = d;
            } else if (b != h) {
                now[i] = s_class[b];
                any = true;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int b = i * kPlanThreads + tid;
            if (b < a.B) s_class[b] = now[i];
        }
    }

    // the groups' rows: their number, and the place of the first in the list
    int* s_sum = s_depth;
    int* s_start = s_depth + a.B;
    __syncthreads();
    for (int b = tid; b < a.B; b += kPlanThreads) s_sum[b] = 0;
    __syncthreads();
    for (int b = tid; b < a.B; b += kPlanThreads)
        if (s_shared[b] > 0) atomicAdd(&s_sum[s_head[b]], s_rows[b]);
    __syncthreads();
    // groups << 32 | rows, before each of PER adjacent requests
    unsigned long long mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        if (b < a.B && s_shared[b] > 0 && s_head[b] == b) mine += 1ull << 32 | (unsigned long long)s_sum[b];
    }
    unsigned long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    unsigned long long before = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const int groups = (int)(total >> 32);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        if (b < a.B && s_shared[b] > 0 && s_head[b] == b) {
            s_start[b] = (int)before;
            if (rank == 0)
                put_item(a.items + (before >> 32), s_shared[b] * a.page_size - 1, 0, (int)before, s_sum[b], b, 0, kPrefix,
                         SPEC_OK);
            before += 1ull << 32 | (unsigned long long)s_sum[b];
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = i * kPlanThreads + tid;
        if (b >= a.B || warp % ranks != rank) continue;
        const int shared = s_shared[b];
        put_item(a.items + groups + b, n[i] - shared * a.page_size, ell[i], base[i], s_rows[b], b, shared,
                 shared > 0 ? kRest : kAlone, code[i]);
        a.leader[b] = s_head[b];
        a.shared[b] = shared;
        if (code[i] != SPEC_OK) set_status(a.plan + kPlanStatus, code[i]);
    }
    __syncthreads();
    // the rows: of a group's members, behind those of the members before
    for (int b = warp0; b < a.B; b += warps) {
        const int rows = s_rows[b], h = s_head[b], row = a.row ? a.row[b] : b * (a.gamma + 1);
        if (s_shared[b] == 0) {
            for (int j = lane; j < rows; j += 32) a.kinds[row + j] = 1;
            continue;
        }
        int at = 0;
        for (int y = h + lane; y < b; y += 32) at += s_shared[y] > 0 && s_head[y] == h ? s_rows[y] : 0;
        at = s_start[h] + __reduce_add_sync(0xffffffffu, at);
        for (int j = lane; j < rows; j += 32) {
            a.kinds[row + j] = 2;
            a.list[at + j] = row + j;
        }
    }
    if (rank == 0 && tid == 0) {
        a.plan[kPlanIs] = kPlanMagic;
        a.plan[kPlanB] = a.B;
        a.plan[kPlanGamma] = a.gamma;
        a.plan[kPlanRows] = a.rows;
        a.plan[kPlanSlots] = a.max_pages;
        a.plan[kPlanPage] = a.page_size;
        a.plan[kPlanItems] = groups + a.B;
    }
}

constexpr int kShareJoinThreads = 256;
constexpr int kShareJoinRows = kShareJoinThreads / 32;
constexpr int kMostSms = 160;
static_assert(kMostSms <= kShareJoinThreads, "a thread of the joining kernel for each block that may have failed");

// The running maximum and sums of parts.
template <int V>
struct Joined {
    float M, L;
    float4 o[V];
};

template <int V>
__device__ __forceinline__ void take_part(Joined<V>& s, float m, float l, const float4 (&o)[V]) {
    const float top = fmaxf(m, s.M), ref = top == -INFINITY ? 0.0f : top;
    const float x = exp2f(s.M - ref), y = exp2f(m - ref);
    s.M = top;
    s.L = s.L * x + y * l;
#pragma unroll
    for (int v = 0; v < V; ++v)
        s.o[v] = make_float4(s.o[v].x * x + y * o[v].x, s.o[v].y * x + y * o[v].y, s.o[v].z * x + y * o[v].z,
                             s.o[v].w * x + y * o[v].w);
}

template <int V>
__device__ __forceinline__ void load_part(const PartRow& p, int dim, float& m, float& l, float4 (&o)[V]) {
    const int lane = threadIdx.x & 31;
    m = *p.m;
    l = *p.l;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        o[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (4 * lane + 128 * v < dim) o[v] = *(const float4*)(p.o + 4 * lane + 128 * v);
    }
}

// Joins the parts of rows that two items have, or that one has in several blocks'
// runs: one warp a row and head, four adjacent columns a lane (V times).  Most parts
// are in `side`, and are read along with the word that says so: a round trip less.
// The order of the parts is fixed.  Once a wait of any block has run out, `where` may
// still be an earlier call's, and rows written directly an earlier call's too: all rows
// become NaN.  34,816 rows and heads 18 us (28 with a round trip
// each for the kind, the place and the parts; 1 us of it for the failed blocks' words),
// 2,048 5.5 us.
template <typename T, int V>
__global__ void __launch_bounds__(kShareJoinThreads) k_share_join(AttendArgs a, CacheView c, int blocks) {
    pdl_trigger();
    pdl_wait();
    const int all = a.rows * a.q_heads, dim = c.head_dim, lane = threadIdx.x & 31;
    const int mine = blockIdx.x * kShareJoinRows + (threadIdx.x >> 5), row = min(mine, all - 1);
    const bool fail = a.failed && (int)threadIdx.x < blocks && a.failed[threadIdx.x];
    // what a row of another kind has here is anything, and not used
    const int kind = a.kinds[a.by_heads.div((uint32_t)row)];
    const int2 x0 = a.where[row], x1 = a.where[(long long)all + row];
    float m0, l0, m1, l1;
    float4 o0[V], o1[V];
    load_part<V>(side_row(a, dim, row), dim, m0, l0, o0);
    load_part<V>(side_row(a, dim, (long long)all + row), dim, m1, l1, o1);
    const bool lost = a.failed && __syncthreads_or(fail);
    if (mine >= all || requests_of<true>(a, c) == 0 || kind == 0 || (x0.x < 0 && !lost)) return;
    // whatever `where` holds, reads stay in range
    auto fits = [&](int2 x) {
        return x.x == 0 || (x.x > 0 && x.x <= blocks && x.y >= 0 && (x.y >> 7) + x.x <= blocks && (x.y & 127) < a.tile_rows);
    };
    Joined<V> s;
    s.M = -INFINITY;
    s.L = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) s.o[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto parts_of = [&](int2 x, float m, float l, const float4 (&o)[V]) {
        if (!fits(x)) {
            s.L = __int_as_float(0x7fc00000);
            return;
        }
        if (x.x == 0) {
            take_part<V>(s, m, l, o);
            return;
        }
        constexpr int BATCH = 4 / V;  // parts under way
#pragma unroll 1
        for (int i0 = 0; i0 < x.x; i0 += BATCH) {
            float mm[BATCH], ll[BATCH];
            float4 oo[BATCH][V];
#pragma unroll
            for (int f = 0; f < BATCH; ++f)
                if (i0 + f < x.x)
                    load_part<V>(part_row(a, part_at(a, (x.y >> 7) + i0 + f, i0 + f == 0 ? 1 : 0), dim, x.y & 127), dim,
                                 mm[f], ll[f], oo[f]);
#pragma unroll
            for (int f = 0; f < BATCH; ++f)
                if (i0 + f < x.x) take_part<V>(s, mm[f], ll[f], oo[f]);
        }
    };
    if (lost) {
        s.L = __int_as_float(0x7fc00000);
    } else {
        parts_of(x0, m0, l0, o0);
        if (kind == 2) parts_of(x1, m1, l1, o1);
    }
    const float inv = 1.0f / s.L;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (4 * lane + 128 * v < dim) {
            Vec<T, 4> four;
            four.x[0] = from_f32<T>(s.o[v].x * inv);
            four.x[1] = from_f32<T>(s.o[v].y * inv);
            four.x[2] = from_f32<T>(s.o[v].z * inv);
            four.x[3] = from_f32<T>(s.o[v].w * inv);
            *(Vec<T, 4>*)((T*)a.out + (long long)row * dim + 4 * lane + 128 * v) = four;
        }
    if (a.lse && lane == 0) a.lse[row] = (s.M + log2f(s.L)) * 0.6931471805599453f;
}

}  // namespace specv

// ===================================================================== host
using namespace specv;

namespace {

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

struct PlanLayout {
    size_t items, list, kinds, total;
    PlanLayout(int B, int gamma, int rows) {
        items = 256;
        list = items + up(sizeof(ShareItem) * 2 * (size_t)B);
        kinds = list + up(sizeof(int32_t) * (size_t)B * (gamma + 1));
        total = kinds + up((size_t)rows);
    }
};

// Blocks of the largest cluster: 16 where the GPU can place them, else the portable 8.
int plan_cluster(const void* kernel, size_t smem, std::atomic<int> (&known)[64], int& blocks) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ERR_CUDA;
    blocks = known[dev].load(std::memory_order_relaxed);
    if (blocks) return SPEC_OK;
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPlanCluster);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPlanCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    blocks = kPlanCluster;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        blocks = 8;
    }
    known[dev].store(blocks, std::memory_order_relaxed);
    return SPEC_OK;
}

// Shared memory of the plan: 10 words a request, two a place of the table (224 KB for
// the largest batch).
template <int PER>
int launch_plan(const PlanArgs& a, cudaStream_t st) {
    auto smem = [](size_t B, size_t hash) { return 4 * (10 * B + 2 * hash); };
    static std::atomic<unsigned long long> done{0};
    if (const int rc = allow_smem((const void*)k_share_plan<PER>,
                                  (int)smem(PER * kPlanThreads, 2 * PER * kPlanThreads), done))
        return rc;
    static std::atomic<int> known[64];
    int most = 0;
    const size_t largest = smem(PER * kPlanThreads, 2 * PER * kPlanThreads);
    if (const int rc = plan_cluster((const void*)k_share_plan<PER>, largest, known, most)) return rc;
    // a warp a request, in a cluster of a power of two
    int blocks = 1;
    while (blocks < most && blocks * kPlanWarps < a.B) blocks *= 2;
    return launch_dependent(k_share_plan<PER>, dim3(blocks), kPlanThreads, smem(a.B, a.hash), st, blocks, a);
}

bool plan_shape_ok(int B, int gamma, int rows) {
    return B >= 0 && B <= SPEC_MAX_BATCH && gamma >= 0 && gamma <= SPEC_MAX_GAMMA && rows >= 0;
}

// The workspace's size may not depend on the GPU, nor on the types.
struct ShareLayout {
    size_t failed, parts, side, side_ml, where, total;
    ShareLayout(int rows, int q_heads, int head_dim) {
        const AttendPlan plans[6] = {
            attend_f32_shared_plan(head_dim, kMostSms),           attend_mma_shared_plan(1, head_dim, false, kMostSms),
            attend_mma_shared_plan(1, head_dim, true, kMostSms),  attend_mma_shared_plan(17, head_dim, false, kMostSms),
            attend_mma_shared_plan(17, head_dim, true, kMostSms), attend_tc_plan(kMostSms)};
        size_t most = 0;
        for (const AttendPlan& p : plans)
            most = std::max(most, sizeof(float) * 2 * (size_t)p.blocks * p.tile_rows * (head_dim + 2));
        const size_t n = 2 * (size_t)rows * q_heads;
        failed = 256;
        parts = failed + up(sizeof(int) * kMostSms);
        side = parts + up(most);
        side_ml = side + up(n * head_dim * sizeof(float));
        where = side_ml + up(n * sizeof(float2));
        total = where + up(n * sizeof(int2));
    }
};

bool heads_ok(int q_heads, int kv_heads) {
    return q_heads >= 1 && kv_heads >= 1 && q_heads <= 65535 && q_heads % kv_heads == 0;
}

// rows and heads countable in 31 bits, as the joining kernel does, and so a group's rows of
// a KV head (rows that two requests have are not allowed, but count twice there)
bool share_shape_ok(int B, int gamma, int rows, int q_heads, int kv_heads) {
    return plan_shape_ok(B, gamma, rows) && heads_ok(q_heads, kv_heads) && (long long)rows * q_heads < 0x7fffff00ll &&
           (long long)B * (gamma + 1) * (q_heads / kv_heads) < 0x7fffff00ll;
}

template <typename T>
int launch_join(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    const int n = (a.rows * a.q_heads + kShareJoinRows - 1) / kShareJoinRows;
    return c.head_dim <= 128 ? launch_dependent(k_share_join<T, 1>, dim3(n), kShareJoinThreads, 0, st, 0, a, c, blocks)
                             : launch_dependent(k_share_join<T, 2>, dim3(n), kShareJoinThreads, 0, st, 0, a, c, blocks);
}

}  // namespace

extern "C" {

size_t spec_share_plan_bytes(int B, int gamma, int rows) {
    return plan_shape_ok(B, gamma, rows) ? PlanLayout(B, gamma, rows).total : 0;
}

int spec_share_plan(const int32_t* page_table, int max_pages, int page_size, const int32_t* cache_len,
                    const int32_t* verify_len, const int32_t* q_row, int rows, int B, int gamma, int least,
                    int32_t* out_leader, int32_t* out_shared, void* plan, size_t plan_bytes, spec_stream_t stream) {
    TraceRange tr("spec_share_plan");
    if (!plan_shape_ok(B, gamma, rows) || max_pages < 1 || page_size < 1 || least < 0) return SPEC_ERR_SHAPE;
    if (!q_row && rows < B * (gamma + 1)) return SPEC_ERR_SHAPE;
    if (B == 0) return SPEC_OK;
    if (!page_table || !cache_len || !out_leader || !out_shared || !plan) return SPEC_ERR_NULL;
    if ((uintptr_t)plan & 15) return SPEC_ERR_ALIGN;
    if (((uintptr_t)page_table | (uintptr_t)cache_len | (uintptr_t)verify_len | (uintptr_t)q_row |
         (uintptr_t)out_leader | (uintptr_t)out_shared) & 3)
        return SPEC_ERR_ALIGN;
    const PlanLayout at(B, gamma, rows);
    if (plan_bytes < at.total) return SPEC_ERR_WORKSPACE;
    PlanArgs a;
    a.table = page_table;
    a.len = cache_len;
    a.ell = verify_len;
    a.row = q_row;
    a.leader = out_leader;
    a.shared = out_shared;
    a.plan = (int*)plan;
    a.items = (ShareItem*)((char*)plan + at.items);
    a.list = (int32_t*)((char*)plan + at.list);
    a.kinds = (uint8_t*)plan + at.kinds;
    a.rows = rows;
    a.B = B;
    a.gamma = gamma;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.least = least;
    a.limit = (int)std::min((long long)max_pages * page_size, 0x7fffffc0ll);
    a.key = std::max(1, (int)(((long long)least + page_size - 1) / page_size)) - 1;
    a.hash = 32;
    while (a.hash < 2 * B) a.hash *= 2;
    cudaStream_t st = (cudaStream_t)stream;
    return B <= kPlanThreads ? launch_plan<1>(a, st) : launch_plan<SPEC_MAX_BATCH / kPlanThreads>(a, st);
}

size_t spec_attend_shared_workspace_bytes(int B, int gamma, int rows, int q_heads, int kv_heads, int head_dim) {
    if (!share_shape_ok(B, gamma, rows, q_heads, kv_heads) || head_dim < 8 || head_dim > SPEC_MAX_HEAD_DIM ||
        (head_dim & 7))
        return 0;
    return ShareLayout(rows, q_heads, head_dim).total;
}

int spec_attend_shared(const void* q, long long q_row_stride, long long q_head_stride, spec_dtype dt, int q_heads,
                       const spec_cache* cache, const int32_t* page_table, int max_pages, const void* plan,
                       size_t plan_bytes, int rows, int B, int gamma, float scale, void* out, float* out_lse,
                       void* workspace, size_t workspace_bytes, spec_stream_t stream) {
    TraceRange tr("spec_attend_shared");
    CacheView c;
    int rc = cache_view(cache, c);
    if (rc != SPEC_OK) return rc;
    if (!share_shape_ok(B, gamma, rows, q_heads, c.kv_heads) || max_pages < 1 || scale - scale != 0.0f)
        return SPEC_ERR_SHAPE;
    if (dt != SPEC_F32 && dt != SPEC_BF16 && dt != SPEC_F16) return SPEC_ERR_SHAPE;
    if (cache->dt != dt && !(cache->dt == SPEC_E4M3 && dt != SPEC_F32)) return SPEC_ERR_SHAPE;
    if (B == 0 || rows == 0) return SPEC_OK;
    if (!q || !out || !page_table || !plan || !workspace) return SPEC_ERR_NULL;
    const long long es = dtype_size(dt);
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace | (uintptr_t)plan) & 15) return SPEC_ERR_ALIGN;
    if (((q_row_stride | q_head_stride) * es) & 15) return SPEC_ERR_ALIGN;
    if (((uintptr_t)page_table | (uintptr_t)out_lse) & 3) return SPEC_ERR_ALIGN;
    const PlanLayout in(B, gamma, rows);
    const ShareLayout at(rows, q_heads, c.head_dim);
    if (plan_bytes < in.total || workspace_bytes < at.total) return SPEC_ERR_WORKSPACE;
    int sms = 0;
    if ((rc = sm_count(sms)) != SPEC_OK) return rc;
    sms = std::min(sms, kMostSms);

    AttendArgs a = {};
    char* ws = (char*)workspace;
    a.q = (const char*)q;
    a.q_row = q_row_stride * es;
    a.q_head = q_head_stride * es;
    a.out = out;
    a.lse = out_lse;
    a.table = page_table;
    a.status = (int*)workspace;
    a.parts = (float*)(ws + at.parts);
    a.q_heads = q_heads;
    a.group = q_heads / c.kv_heads;
    a.rows = rows;
    a.B = B;
    a.gamma = gamma;
    a.max_pages = max_pages;
    a.scale = scale * 1.4426950408889634f;  // log2(e)
    a.by_group = FastDiv((uint32_t)a.group);
    a.by_heads = FastDiv((uint32_t)q_heads);
    a.plan = (const int*)plan;
    a.items = (const ShareItem*)((const char*)plan + in.items);
    a.list = (const int32_t*)((const char*)plan + in.list);
    a.kinds = (const uint8_t*)plan + in.kinds;
    a.side = (float*)(ws + at.side);
    a.side_ml = (float2*)(ws + at.side_ml);
    a.where = (int2*)(ws + at.where);
    cudaStream_t st = (cudaStream_t)stream;

    const bool f8 = cache->dt == SPEC_E4M3;
    const int most = (int)std::min((long long)B * (gamma + 1) * a.group, 1ll << 30);  // of an item
    // the tensor-core kernel whenever it takes the cache, for few rows too: 4 requests of one
    // token behind 30,000 positions, 32/8 heads, bf16 45 us against 52 of the warp-level one
    // (e4m3 41 against 47, heads of 64 35 against 41), 16 requests without grouped heads 35 and 37
    const bool tc = dt != SPEC_F32 && attend_tc_takes(c, kTcLeast + 1);
    const AttendPlan p = dt == SPEC_F32 ? attend_f32_shared_plan(c.head_dim, sms)
                         : tc           ? attend_tc_plan(sms)
                                        : attend_mma_shared_plan(most, c.head_dim, f8, sms);
    a.failed = tc ? (int*)(ws + at.failed) : nullptr;
    a.tile_rows = p.tile_rows;
    while ((1 << a.tile_shift) < p.tile_rows) ++a.tile_shift;
    a.part_floats = (long long)p.tile_rows * (c.head_dim + 2);
    // Tensor-core kernel: of at most 32 rows one softmax warp of a stream has work, and a tile
    // is sooner done; a unit's set-up and end cost as much as four tiles of many rows.  The
    // bench batches in us, 64 chats / three documents / 64 blocks / a tree, by the cost of a
    // tile of few rows, of many, and of a set-up: 1, 1, 3 162 / 147 / 196 / 78; 1, 1, 4 162 /
    // 146 / 188 / 77; 3, 4, 12 148 / 165 / - / -; 4, 5, 20 152 / 145 / 188 / 76.  The others,
    // whose tiles are smaller: fp32, 40 x 9 rows of 16 heads of 256 behind 444 positions by
    // leads of 1, 2, 3 tiles 197, 215, 224 us, 64 single tokens 242, 250, 260; 16 bits, heads
    // of 192 over e4m3 334, 252, 223, of 256 191, 191, 195
    a.few = tc ? 32 : 0;
    a.cost[0] = tc ? 4 : 1;
    a.cost[1] = tc ? 5 : 1;
    a.lead = tc ? 20 : dt == SPEC_F32 ? 1 : 3;
    a.part_cost = (tc ? 0.2f / 1.1f : 0.2f / 0.45f) * a.cost[1];  // as in spec_attend
    if (dt == SPEC_F32) rc = attend_f32_shared(a, c, p.blocks, st);
    else if (tc) rc = attend_tc_shared(a, c, dt, cache->dt, p.blocks, st);
    else rc = attend_mma_shared(a, c, dt, f8, p.blocks, st);
    if (rc != SPEC_OK) return rc;
    if (dt == SPEC_F32) return launch_join<float>(a, c, p.blocks, st);
    if (dt == SPEC_BF16) return launch_join<__nv_bfloat16>(a, c, p.blocks, st);
    return launch_join<__half>(a, c, p.blocks, st);
}

}  // extern "C"
