// Attention over the paged cache: the C entry, the choice of kernel, and the
// kernel that joins the parts of units that were split over blocks.
#include "specv_attend.cuh"

#include <math.h>

#include <algorithm>

#include "specv_trace.h"

namespace specv {

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = kJoinThreads / 32;
constexpr int kJoinPairs = SPEC_MAX_HEAD_DIM / 64;  // column pairs of a lane

// A row's n parts: their maximum M, and sums scaled by 2^-M.
struct Joined {
    float M, L;
    float2 o[kJoinPairs];
};

__device__ __forceinline__ Joined join_parts(const AttendArgs& a, int dim, int r, int n) {
    constexpr int BATCH = 4;  // parts whose values are fetched together
    const int lane = threadIdx.x & 31;
    const float* own = part_at(a, blockIdx.x, 1);
    const float* rest = part_at(a, blockIdx.x + 1, 0);
    Joined s;
    s.M = -INFINITY;
    s.L = 0.0f;
#pragma unroll
    for (int e = 0; e < kJoinPairs; ++e) s.o[e] = make_float2(0.0f, 0.0f);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += BATCH) {
        float m[BATCH], l[BATCH];
        float2 o[BATCH][kJoinPairs];
#pragma unroll
        for (int f = 0; f < BATCH; ++f) {
            const int i = i0 + f;
            m[f] = -INFINITY;
            l[f] = 0.0f;
            if (i < n) {
                const float* p = i == 0 ? own : rest + (i - 1) * 2 * a.part_floats;
                m[f] = p[a.tile_rows * dim + r];
                l[f] = p[a.tile_rows * (dim + 1) + r];
#pragma unroll
                for (int e = 0; e < kJoinPairs; ++e)
                    if (2 * lane + 64 * e < dim) o[f][e] = *(const float2*)(p + r * dim + 2 * lane + 64 * e);
            }
        }
        const float M = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), s.M);
        const float base = M == -INFINITY ? 0.0f : M, old = exp2f(s.M - base);
        s.M = M;
        s.L *= old;
#pragma unroll
        for (int e = 0; e < kJoinPairs; ++e) {
            s.o[e].x *= old;
            s.o[e].y *= old;
        }
#pragma unroll
        for (int f = 0; f < BATCH; ++f)
            if (i0 + f < n) {
                const float w = exp2f(m[f] - base);
                s.L = fmaf(w, l[f], s.L);
#pragma unroll
                for (int e = 0; e < kJoinPairs; ++e)
                    if (2 * lane + 64 * e < dim) {
                        s.o[e].x = fmaf(w, o[f][e].x, s.o[e].x);
                        s.o[e].y = fmaf(w, o[f][e].y, s.o[e].y);
                    }
            }
    }
    return s;
}

// Joins the parts of the unit that block blockIdx.x left open: the block's own
// and those of the blocks after it, in a fixed order.  With each part's maximum
// m_i and sum l_i, M = max m_i: out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
// Bound by its round trips: what is open, then four parts at a time.  One warp a
// row.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(AttendArgs a, CacheView c) {
    pdl_trigger();
    pdl_wait();
    const int4 open = a.open[blockIdx.x];
    const int n = open.x, r = blockIdx.y * kJoinRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (n == 0 || r >= (int)((uint32_t)open.w >> 16)) return;
    const int dim = c.head_dim;
    const Joined s = join_parts(a, dim, r, n);
    const long long row = out_row(a, open.y, open.w & 0xffff, open.z + r);
    const float inv = 1.0f / s.L;
#pragma unroll
    for (int e = 0; e < kJoinPairs; ++e)
        if (2 * lane + 64 * e < dim) {
            Vec<T, 2> two;
            two.x[0] = from_f32<T>(s.o[e].x * inv);
            two.x[1] = from_f32<T>(s.o[e].y * inv);
            *(Vec<T, 2>*)((T*)a.out + row * dim + 2 * lane + 64 * e) = two;
        }
    if (a.lse && lane == 0) a.lse[row] = (s.M + log2f(s.L)) * 0.6931471805599453f;
}

}  // namespace specv

// ===================================================================== host
using namespace specv;

namespace {

bool heads_ok(int q_heads, int kv_heads) {
    return q_heads >= 1 && kv_heads >= 1 && q_heads <= 65535 && q_heads % kv_heads == 0;
}

// The workspace's size may not depend on the GPU, nor on the cache's type (e4m3
// has the most blocks): it is that of the largest
// grid the library launches.
constexpr int kMostSms = 160;

size_t header_bytes() { return 256 + (sizeof(int4) * kMostSms * 4 + 255) / 256 * 256; }

size_t parts_bytes(const AttendPlan& p, int head_dim) {
    return sizeof(float) * 2 * (size_t)p.blocks * p.tile_rows * (head_dim + 2);
}

template <typename T>
int launch_join(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    const int most = min(a.tile_rows, (a.gamma + 1) * a.group);
    return launch_dependent(k_attend_join<T>, dim3(blocks, (most + kJoinRows - 1) / kJoinRows), kJoinThreads, 0, st, 0, a, c);
}

}  // namespace

extern "C" {

size_t spec_attend_workspace_bytes(int B, int gamma, int q_heads, int kv_heads, int head_dim) {
    if (B < 0 || B > SPEC_MAX_BATCH || gamma < 0 || gamma > SPEC_MAX_GAMMA || !heads_ok(q_heads, kv_heads) ||
        head_dim < 8 || head_dim > SPEC_MAX_HEAD_DIM || (head_dim & 7))
        return 0;
    const int rows = (gamma + 1) * (q_heads / kv_heads);
    return header_bytes() + max(parts_bytes(attend_simt_plan(rows, head_dim, kMostSms), head_dim),
                                max(parts_bytes(attend_mma_plan(rows, head_dim, true, kMostSms), head_dim),
                                    parts_bytes(attend_tc_plan(kMostSms), head_dim)));
}

int spec_attend(const void* q, long long q_row_stride, long long q_head_stride, spec_dtype dt, int q_heads,
                const spec_cache* cache, const int32_t* page_table, int max_pages, const int32_t* cache_len,
                const int32_t* verify_len, const int32_t* q_row, int rows, int B, int gamma, float scale,
                int window, int sinks, void* out, float* out_lse, void* workspace, size_t workspace_bytes,
                spec_stream_t stream) {
    TraceRange tr("spec_attend");
    CacheView c;
    int rc = cache_view(cache, c);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || B > SPEC_MAX_BATCH || gamma < 0 || gamma > SPEC_MAX_GAMMA || !heads_ok(q_heads, c.kv_heads) ||
        max_pages < 1 || rows < 0 || window < 0 || sinks < 0 || scale - scale != 0.0f)
        return SPEC_ERR_SHAPE;
    if (dt != SPEC_F32 && dt != SPEC_BF16 && dt != SPEC_F16) return SPEC_ERR_SHAPE;
    if (cache->dt != dt && !(cache->dt == SPEC_E4M3 && dt != SPEC_F32)) return SPEC_ERR_SHAPE;
    if (!q_row && rows < B * (gamma + 1)) return SPEC_ERR_SHAPE;
    if (B == 0) return SPEC_OK;
    if (!q || !out || !page_table || !cache_len || !workspace) return SPEC_ERR_NULL;
    const long long es = dtype_size(dt);
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15) return SPEC_ERR_ALIGN;
    if (((q_row_stride | q_head_stride) * es) & 15) return SPEC_ERR_ALIGN;
    if (((uintptr_t)page_table | (uintptr_t)cache_len | (uintptr_t)verify_len | (uintptr_t)q_row |
         (uintptr_t)out_lse) & 3)
        return SPEC_ERR_ALIGN;
    if (workspace_bytes < spec_attend_workspace_bytes(B, gamma, q_heads, c.kv_heads, c.head_dim))
        return SPEC_ERR_WORKSPACE;
    int sms = 0;
    if ((rc = sm_count(sms)) != SPEC_OK) return rc;
    sms = min(sms, kMostSms);

    AttendArgs a;
    a.q = (const char*)q;
    a.q_row = q_row_stride * es;
    a.q_head = q_head_stride * es;
    a.out = out;
    a.lse = out_lse;
    a.table = page_table;
    a.len = cache_len;
    a.ell = verify_len;
    a.row = q_row;
    a.status = (int*)workspace;
    a.open = (int4*)((char*)workspace + 256);
    a.parts = (float*)((char*)workspace + header_bytes());
    a.q_heads = q_heads;
    a.group = q_heads / c.kv_heads;
    a.rows = rows;
    a.B = B;
    a.gamma = gamma;
    a.max_pages = max_pages;
    a.limit = (int)std::min((long long)max_pages * c.page_size, 0x7fffffc0ll);
    a.window = window;
    a.sinks = sinks;
    a.scale = scale * 1.4426950408889634f;  // log2(e)
    a.by_group = FastDiv((uint32_t)a.group);
    cudaStream_t st = (cudaStream_t)stream;

    const int most = (gamma + 1) * a.group;
    const bool tc = dt != SPEC_F32 && attend_tc_takes(c, most);
    const AttendPlan p = dt == SPEC_F32 ? attend_simt_plan(most, c.head_dim, sms)
                         : tc           ? attend_tc_plan(sms)
                                        : attend_mma_plan(most, c.head_dim, cache->dt == SPEC_E4M3, sms);
    a.tile_rows = p.tile_rows;
    a.tile_shift = 0;
    while ((1 << a.tile_shift) < p.tile_rows) ++a.tile_shift;
    a.part_floats = (long long)p.tile_rows * (c.head_dim + 2);
    a.lead = tc ? 3 : 2;
    // a part costs the joining kernel about 0.2 us a row, a tile its block 0.45 us
    // (64 keys) or 1.1 us (128): a unit of t tiles in parts of sqrt(0.2 / 0.45 t)
    // or sqrt(0.2 / 1.1 t) tiles spends as long on the one as on the other
    a.part_cost = tc ? 0.2f / 1.1f : 0.2f / 0.45f;
    if (dt == SPEC_F32) rc = attend_simt(a, c, p.blocks, st);
    else if (tc) rc = attend_tc(a, c, dt, cache->dt, p.blocks, st);
    else if (cache->dt == SPEC_E4M3) rc = attend_mma8(a, c, dt, p.blocks, st);
    else rc = attend_mma16(a, c, dt, p.blocks, st);
    if (rc != SPEC_OK) return rc;
    if (dt == SPEC_F32) return launch_join<float>(a, c, p.blocks, st);
    if (dt == SPEC_BF16) return launch_join<__nv_bfloat16>(a, c, p.blocks, st);
    return launch_join<__half>(a, c, p.blocks, st);
}

}  // extern "C"
