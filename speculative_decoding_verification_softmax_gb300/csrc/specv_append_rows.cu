// Rotary positions and the append of rows by their slots: the C entry.
#include "specv_append.cuh"
#include "specv_trace.h"

using namespace specv;

extern "C" int spec_append_rows(const void* q, long long q_row_stride, long long q_head_stride, const void* k,
                                const void* v, long long k_row_stride, long long k_head_stride,
                                long long v_row_stride, long long v_head_stride, spec_dtype dt, int q_heads,
                                const spec_cache* cache, const int32_t* position, const int64_t* slot, int rows,
                                const uint64_t* turns, int rotary_dim, int interleaved, float mscale, void* out_q,
                                void* workspace, size_t workspace_bytes, spec_stream_t stream) {
    TraceRange tr("spec_append_rows");
    CacheView c;
    const int rc = cache_view(cache, c);
    if (rc != SPEC_OK) return rc;
    if (rows < 0 || q_heads < 0 || q_heads > 65535) return SPEC_ERR_SHAPE;
    if (dt != SPEC_F32 && dt != SPEC_BF16 && dt != SPEC_F16) return SPEC_ERR_SHAPE;
    if (cache->dt != dt && !(cache->dt == SPEC_E4M3 && dt != SPEC_F32)) return SPEC_ERR_SHAPE;
    const long long es = dtype_size(dt);
    if (rotary_dim < 0 || rotary_dim > c.head_dim || (rotary_dim & 1)) return SPEC_ERR_SHAPE;
    if (mscale - mscale != 0.0f) return SPEC_ERR_SHAPE;
    if (rows == 0) return SPEC_OK;
    if ((q_heads > 0 && (!q || !out_q)) || !k || !v || !position || !slot || !workspace || (rotary_dim > 0 && !turns))
        return SPEC_ERR_NULL;
    if (q_heads == 0) {
        q = out_q = nullptr;
        q_row_stride = q_head_stride = 0;
    }
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out_q | (uintptr_t)workspace) & 15)
        return SPEC_ERR_ALIGN;
    if (((q_row_stride | q_head_stride | k_row_stride | k_head_stride | v_row_stride | v_head_stride) * es) & 15)
        return SPEC_ERR_ALIGN;
    if (((uintptr_t)position & 3) || (((uintptr_t)slot | (uintptr_t)turns) & 7)) return SPEC_ERR_ALIGN;
    if (workspace_bytes < 256) return SPEC_ERR_WORKSPACE;
    AppendArgs a = {};
    a.q = (const char*)q;
    a.k = (const char*)k;
    a.v = (const char*)v;
    a.q_row = q_row_stride * es;
    a.q_head = q_head_stride * es;
    a.k_row = k_row_stride * es;
    a.k_head = k_head_stride * es;
    a.v_row = v_row_stride * es;
    a.v_head = v_head_stride * es;
    a.out_q = (char*)out_q;
    a.turns = (const unsigned long long*)turns;
    a.status = (int*)workspace;
    a.q_heads = q_heads;
    a.rows = rows;
    a.half = rotary_dim / 2;
    a.mscale = mscale;
    a.position = position;
    a.slot = (const long long*)slot;
    a.slots = (long long)c.pages * c.page_size;
    return launch_types<true>(a, c, dt, cache->dt, interleaved != 0, (cudaStream_t)stream);
}
