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
constexpr int kPlanCluster = 8;
constexpr int kPlanPer = SPEC_MAX_BATCH / kPlanThreads;  // requests of a thread
constexpr int kPlanPasses = 32;
constexpr int kPlanInts = 8;  // shared memory of a request

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
};

// Leading entries that two rows of the page table have alike, `most` at most; by a
// warp, eight words of 32 entries at a time.
__device__ __forceinline__ int common_pages(const int32_t* x, const int32_t* y, int most) {
    constexpr int W = 8;
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

// The plan.  Requests that begin with the same page are a class, the lowest of
// them its head.  Each counts the leading full pages that it has like the head;
// the depth d that saves most reads, (members of depth >= d but the head) * d, makes
// those members and the head a group.  The head leaves its class in any case, the
// others go into the next pass: a tree of prompts takes a pass for each of its
// groups.  Then the groups' rows are listed and the items written.
//
// The requests' few numbers are in every block's shared memory, and each block
// takes the same decisions from them; only the page tables' rows are divided over
// the cluster's warps.  Bound by latency: barriers, and a chain of a few round trips
// to the tables a pass.
__global__ void __launch_bounds__(kPlanThreads) k_share_plan(PlanArgs a) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ int s_mem[];
    int* s_first = s_mem;            // class: the first page, -1 placed
    int* s_full = s_first + a.B;     // full pages
    int* s_head = s_full + a.B;      // of this pass; then the leader
    int* s_shared = s_head + a.B;    // pages shared; 0 alone
    int* s_rows = s_shared + a.B;    // rows, 0 of a request with an error
    int* s_leader = s_rows + a.B;
    int* s_depth = s_leader + a.B;   // [2][B] by pass; then the groups' rows, and their places
    // key of the best depth by head; B is not always even
    __shared__ unsigned long long s_best[SPEC_MAX_BATCH];
    __shared__ unsigned long long s_scan[kPlanWarps + 1];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    int code[kPlanPer], n[kPlanPer], ell[kPlanPer], base[kPlanPer];
    bool any = false;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const int b = i * kPlanThreads + tid;
        code[i] = SPEC_OK;
        if (b >= a.B) continue;
        n[i] = a.len[b];
        ell[i] = a.ell ? a.ell[b] : a.gamma;
        base[i] = a.row ? a.row[b] : b * (a.gamma + 1);
        if (ell[i] < 0 || ell[i] > a.gamma) code[i] = SPEC_ERR_VERIFY_LEN;
        else if (base[i] < 0 || base[i] > a.rows - ell[i] - 1) code[i] = SPEC_ERR_ROW_INDEX;
        else if (n[i] < 0 || n[i] >= a.limit - ell[i]) code[i] = SPEC_ERR_CACHE_LEN;
        const bool good = code[i] == SPEC_OK;
        const int full = good ? n[i] / a.page_size : 0;
        const int first = full > 0 ? a.table[(size_t)b * a.max_pages] : -1;
        s_first[b] = first < 0 ? -1 : first;
        s_full[b] = full;
        s_shared[b] = 0;
        s_leader[b] = b;
        s_rows[b] = good ? ell[i] + 1 : 0;
        any |= first >= 0;
    }
    if (rank == 0 && tid == 0) a.plan[kPlanStatus] = SPEC_OK;
    for (int r = rank * kPlanThreads + tid; r < a.rows; r += ranks * kPlanThreads) a.kinds[r] = 0;
    cluster.sync();

    for (int pass = 0; pass < kPlanPasses && __syncthreads_or(any); ++pass) {
        int* s_d = s_depth + (pass & 1) * a.B;
#pragma unroll
        for (int i = 0; i < kPlanPer; ++i) {
            const int b = i * kPlanThreads + tid;
            if (b >= a.B || s_first[b] < 0) continue;
            int h = 0;
            while (s_first[h] != s_first[b]) ++h;
            s_head[b] = h;
            s_best[b] = 0;
        }
        __syncthreads();
        for (int b = warp * ranks + rank; b < a.B; b += kPlanWarps * ranks) {
            const int h = s_first[b] < 0 ? b : s_head[b];
            if (h == b) continue;
            const int d = common_pages(a.table + (size_t)b * a.max_pages, a.table + (size_t)h * a.max_pages,
                                       min(s_full[b], s_full[h]));
            if (lane < ranks) *cluster.map_shared_rank(s_d + b, lane) = d;
        }
        cluster.sync();
#pragma unroll
        for (int i = 0; i < kPlanPer; ++i) {
            const int b = i * kPlanThreads + tid;
            if (b >= a.B || s_first[b] < 0) continue;
            const int h = s_head[b];
            if (h == b || (long long)s_d[b] * a.page_size < a.least) continue;
            unsigned long long others = 0;
            for (int x = h + 1; x < a.B; ++x) others += s_first[x] == s_first[b] && s_d[x] >= s_d[b];
            atomicMax(&s_best[h], others * s_d[b] << 13 | others);
        }
        __syncthreads();
        any = false;
        int now[kPlanPer];
#pragma unroll
        for (int i = 0; i < kPlanPer; ++i) {
            const int b = i * kPlanThreads + tid;
            now[i] = -1;
            if (b >= a.B || s_first[b] < 0) continue;
            const int h = s_head[b];
            const unsigned long long best = s_best[h];
            const int d = best ? (int)((best >> 13) / (best & 8191)) : 0;
            if (d > 0 && (b == h || s_d[b] >= d)) {
                s_leader[b] = h;
                s_shared[b] = d;
            } else if (b != h) {
                now[i] = s_first[b];
                any = true;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPlanPer; ++i) {
            const int b = i * kPlanThreads + tid;
            if (b < a.B) s_first[b] = now[i];
        }
    }

    // the groups' rows: their number, and the place of the first in the list
    int* s_sum = s_depth;
    int* s_start = s_depth + a.B;
    cluster.sync();  // nobody writes another's depths any more
    for (int b = tid; b < a.B; b += kPlanThreads) s_sum[b] = 0;
    __syncthreads();
    for (int b = tid; b < a.B; b += kPlanThreads)
        if (s_shared[b] > 0) atomicAdd(&s_sum[s_leader[b]], s_rows[b]);
    __syncthreads();
    // groups << 32 | rows, before each of four adjacent requests
    unsigned long long mine = 0;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const int b = tid * kPlanPer + i;
        if (b < a.B && s_shared[b] > 0 && s_leader[b] == b) mine += 1ull << 32 | (unsigned long long)s_sum[b];
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
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const int groups = (int)(total >> 32);
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const int b = tid * kPlanPer + i;
        if (b < a.B && s_shared[b] > 0 && s_leader[b] == b) {
            s_start[b] = (int)before;
            if (rank == 0) {
                ShareItem it;
                it.n = s_shared[b] * a.page_size - 1;
                it.ell = 0;
                it.base = (int)before;
                it.rows = s_sum[b];
                it.b = b;
                it.skip = 0;
                it.kind = kPrefix;
                it.code = SPEC_OK;
                a.items[before >> 32] = it;
            }
            before += 1ull << 32 | (unsigned long long)s_sum[b];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const int b = i * kPlanThreads + tid;
        if (b >= a.B || (warp % ranks) != rank) continue;
        ShareItem it;
        const int shared = s_shared[b], leader = s_leader[b];
        it.code = code[i];
        it.n = n[i] - shared * a.page_size;
        it.ell = ell[i];
        it.base = base[i];
        it.rows = s_rows[b];
        it.b = b;
        it.skip = shared;
        it.kind = shared > 0 ? kRest : kAlone;
        a.items[groups + b] = it;
        a.leader[b] = leader;
        a.shared[b] = shared;
        if (code[i] != SPEC_OK) {
            set_status(a.plan + kPlanStatus, code[i]);
            continue;
        }
        int at = 0;
        if (shared > 0) {
            at = s_start[leader];
            for (int y = leader; y < b; ++y) at += s_leader[y] == leader ? s_rows[y] : 0;
        }
        for (int j = 0; j <= ell[i]; ++j) {
            a.kinds[base[i] + j] = shared > 0 ? 2 : 1;
            if (shared > 0) a.list[at + j] = base[i] + j;
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
constexpr int kSharePairs = SPEC_MAX_HEAD_DIM / 64;  // column pairs of a lane

// Joins the parts of rows that two items have, or that one has in several blocks'
// runs: one warp a row and head, up to four parts' loads under way.  The order of
// the parts is fixed.
template <typename T>
__global__ void __launch_bounds__(kShareJoinThreads) k_share_join(AttendArgs a, CacheView c, int blocks) {
    constexpr int BATCH = 4;
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x * kShareJoinRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int all = a.rows * a.q_heads;
    if (row >= all || requests_of<true>(a, c) == 0) return;
    const int kind = a.kinds[row / a.q_heads];
    if (kind == 0) return;
    const int2 x0 = a.where[row], x1 = kind == 2 ? a.where[(long long)all + row] : make_int2(0, 0);
    if (x0.x < 0) return;
    const int dim = c.head_dim;
    const int n0 = max(x0.x, 1), n = n0 + (kind == 2 ? max(x1.x, 1) : 0);
    // a call whose waits ran out may have told nothing of a row
    auto fits = [&](int2 x) {
        return x.x == 0 || (x.x > 0 && x.x <= blocks && x.y >= 0 && (x.y >> 7) + x.x <= blocks && (x.y & 127) < a.tile_rows);
    };
    const bool good = fits(x0) && fits(x1);
    float M = -INFINITY, L = 0.0f;
    float2 sum[kSharePairs];
#pragma unroll
    for (int e = 0; e < kSharePairs; ++e) sum[e] = make_float2(0.0f, 0.0f);
#pragma unroll 1
    for (int i0 = 0; good && i0 < n; i0 += BATCH) {
        float m[BATCH], l[BATCH];
        float2 o[BATCH][kSharePairs];
#pragma unroll
        for (int f = 0; f < BATCH; ++f) {
            const int i = i0 + f;
            m[f] = -INFINITY;
            l[f] = 0.0f;
            if (i < n) {
                const bool rest = i < n0;
                const int2 x = rest ? x0 : x1;
                const int q = rest ? i : i - n0;
                const PartRow p = x.x == 0 ? side_row(a, dim, rest ? row : (long long)all + row)
                                           : part_row(a, part_at(a, (x.y >> 7) + q, q == 0 ? 1 : 0), dim, x.y & 127);
                m[f] = *p.m;
                l[f] = *p.l;
#pragma unroll
                for (int e = 0; e < kSharePairs; ++e)
                    if (2 * lane + 64 * e < dim) o[f][e] = *(const float2*)(p.o + 2 * lane + 64 * e);
            }
        }
        const float top = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), M);
        const float ref = top == -INFINITY ? 0.0f : top, old = exp2f(M - ref);
        M = top;
        L *= old;
#pragma unroll
        for (int e = 0; e < kSharePairs; ++e) {
            sum[e].x *= old;
            sum[e].y *= old;
        }
#pragma unroll
        for (int f = 0; f < BATCH; ++f)
            if (i0 + f < n) {
                const float w = exp2f(m[f] - ref);
                L = fmaf(w, l[f], L);
#pragma unroll
                for (int e = 0; e < kSharePairs; ++e)
                    if (2 * lane + 64 * e < dim) {
                        sum[e].x = fmaf(w, o[f][e].x, sum[e].x);
                        sum[e].y = fmaf(w, o[f][e].y, sum[e].y);
                    }
            }
    }
    const float inv = 1.0f / L;
#pragma unroll
    for (int e = 0; e < kSharePairs; ++e)
        if (2 * lane + 64 * e < dim) {
            Vec<T, 2> two;
            two.x[0] = from_f32<T>(good ? sum[e].x * inv : __int_as_float(0x7fc00000));
            two.x[1] = from_f32<T>(good ? sum[e].y * inv : __int_as_float(0x7fc00000));
            *(Vec<T, 2>*)((T*)a.out + (long long)row * dim + 2 * lane + 64 * e) = two;
        }
    if (a.lse && lane == 0) a.lse[row] = (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace specv

// ===================================================================== host
using namespace specv;

namespace {

constexpr int kMostSms = 160;

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

bool plan_shape_ok(int B, int gamma, int rows) {
    return B >= 0 && B <= SPEC_MAX_BATCH && gamma >= 0 && gamma <= SPEC_MAX_GAMMA && rows >= 0;
}

// The workspace's size may not depend on the GPU, nor on the types.
struct ShareLayout {
    size_t parts, side, side_ml, where, total;
    ShareLayout(int rows, int q_heads, int head_dim) {
        const AttendPlan plans[4] = {attend_simt_plan(1, head_dim, kMostSms),
                                     attend_mma_shared_plan(head_dim, false, kMostSms),
                                     attend_mma_shared_plan(head_dim, true, kMostSms), attend_tc_plan(kMostSms)};
        size_t most = 0;
        for (const AttendPlan& p : plans)
            most = std::max(most, sizeof(float) * 2 * (size_t)p.blocks * p.tile_rows * (head_dim + 2));
        const size_t n = 2 * (size_t)rows * q_heads;
        parts = 256;
        side = parts + up(most);
        side_ml = side + up(n * head_dim * sizeof(float));
        where = side_ml + up(n * sizeof(float2));
        total = where + up(n * sizeof(int2));
    }
};

bool heads_ok(int q_heads, int kv_heads) {
    return q_heads >= 1 && kv_heads >= 1 && q_heads <= 65535 && q_heads % kv_heads == 0;
}

// rows and heads countable in 31 bits, as the joining kernel does
bool share_shape_ok(int B, int gamma, int rows, int q_heads, int kv_heads) {
    return plan_shape_ok(B, gamma, rows) && heads_ok(q_heads, kv_heads) && (long long)rows * q_heads < 0x7fffff00ll;
}

template <typename T>
int launch_join(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    const int n = (a.rows * a.q_heads + kShareJoinRows - 1) / kShareJoinRows;
    return launch_dependent(k_share_join<T>, dim3(n), kShareJoinThreads, 0, st, 0, a, c, blocks);
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
    static std::atomic<unsigned long long> done{0};
    if (const int rc = allow_smem((const void*)k_share_plan, SPEC_MAX_BATCH * kPlanInts * 4, done)) return rc;
    // a warp a request, in a cluster of a power of two
    int blocks = 1;
    while (blocks < kPlanCluster && blocks * kPlanWarps < B) blocks *= 2;
    return launch_dependent(k_share_plan, dim3(blocks), kPlanThreads, sizeof(int) * kPlanInts * (size_t)B,
                            (cudaStream_t)stream, blocks, a);
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
    a.plan = (const int*)plan;
    a.items = (const ShareItem*)((const char*)plan + in.items);
    a.list = (const int32_t*)((const char*)plan + in.list);
    a.kinds = (const uint8_t*)plan + in.kinds;
    a.side = (float*)(ws + at.side);
    a.side_ml = (float2*)(ws + at.side_ml);
    a.where = (int2*)(ws + at.where);
    cudaStream_t st = (cudaStream_t)stream;

    const bool f8 = cache->dt == SPEC_E4M3;
    const bool tc = dt != SPEC_F32 && attend_tc_takes(c, kTcLeast + 1);
    const AttendPlan p = dt == SPEC_F32 ? attend_simt_plan(1, c.head_dim, sms)
                         : tc           ? attend_tc_plan(sms)
                                        : attend_mma_shared_plan(c.head_dim, f8, sms);
    a.tile_rows = p.tile_rows;
    while ((1 << a.tile_shift) < p.tile_rows) ++a.tile_shift;
    a.part_floats = (long long)p.tile_rows * (c.head_dim + 2);
    a.lead = tc ? 3 : 2;
    a.part_cost = tc ? 0.2f / 1.1f : 0.2f / 0.45f;  // as in spec_attend
    if (dt == SPEC_F32) rc = attend_simt_shared(a, c, p.blocks, st);
    else if (tc) rc = attend_tc_shared(a, c, dt, cache->dt, p.blocks, st);
    else rc = attend_mma_shared(a, c, dt, f8, p.blocks, st);
    if (rc != SPEC_OK) return rc;
    if (dt == SPEC_F32) return launch_join<float>(a, c, p.blocks, st);
    if (dt == SPEC_BF16) return launch_join<__nv_bfloat16>(a, c, p.blocks, st);
    return launch_join<__half>(a, c, p.blocks, st);
}

}  // extern "C"
