// Rotary positions and the append of the tested tokens to a paged cache.
//
// Angles.  The angle of position p and pair i is p f_i.  With f_i / (2 pi) held
// as a fraction F of 2^64, p F mod 2^64 is the angle's fraction of a turn, an
// exact wrapping 64-bit product at any position (an fp32 angle of position
// 10^6 would be off by 0.06, and GB300's fp64 pipe is narrow).  Its upper 32
// bits, as a signed number of half turns, go to sincospif.
//
// One block a row: the angles of the row's pairs are computed once into shared
// memory and used by all q and k heads, which then pass as 16-byte vectors.
// Bound by HBM for large batches (each input read once, each output written
// once), by launch and one round trip of the page table for small ones.
#include "specv_cache.cuh"
#include "specv_trace.h"

namespace specv {

struct AppendArgs {
    const char* q;
    const char* k;
    const char* v;
    long long q_row, q_head, k_row, k_head, v_row, v_head;  // strides in bytes
    char* out_q;
    const int32_t* table;
    const int32_t* len;
    const int32_t* ell;
    const int32_t* row;
    const unsigned long long* turns;
    int* status;
    int q_heads, rows, B, gamma, max_pages, half;
    float mscale;
};

constexpr int kAppendThreads = 256;

// The pages' entry of a position, or null (and the status) where there is none.
__device__ __forceinline__ long long entry_at(const AppendArgs& a, const CacheView& c, int b, long long pos) {
    const long long most = (long long)a.max_pages * c.page_size;
    if (pos < 0 || pos >= most || pos > 0x7fffffffll) {
        if (threadIdx.x == 0) set_status(a.status, SPEC_ERR_CACHE_LEN);
        return -1;
    }
    const uint32_t slot = c.by_page.div((uint32_t)pos);
    const int page = a.table[(size_t)b * a.max_pages + slot];
    if (page < 0 || page >= c.pages) {
        if (threadIdx.x == 0) set_status(a.status, SPEC_ERR_PAGE);
        return -1;
    }
    return (long long)page * c.page + ((long long)pos - (long long)slot * c.page_size) * c.token;
}

// E adjacent elements as 32-bit floats.
template <typename T, int E>
__device__ __forceinline__ void load_vec(const char* p, float (&x)[E]) {
    const Vec<T, E> v = *(const Vec<T, E>*)p;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = to_f32(v.x[e]);
}

template <typename T, int E>
__device__ __forceinline__ void store_vec(char* p, const float (&x)[E]) {
    Vec<T, E> v;
#pragma unroll
    for (int e = 0; e < E; ++e) v.x[e] = from_f32<T>(x[e]);
    *(Vec<T, E>*)p = v;
}

// T: rows, C: cache, E: elements of a vector.  Work items of a row: for each q
// and k head, the vectors of its first halves (with their partners, so that one
// thread reads and writes a pair and out_q may be q) or, interleaved, its
// vectors; then the unturned vectors; then v's.  E is 16 bytes' worth where the
// turned part is whole vectors, else a single element (a pair if interleaved).
template <typename T, typename C, bool INTERLEAVED, int E>
__global__ void __launch_bounds__(kAppendThreads) k_append(AppendArgs a, CacheView c) {
    __shared__ float s_cos[SPEC_MAX_HEAD_DIM / 2], s_sin[SPEC_MAX_HEAD_DIM / 2];
    const int G1 = a.gamma + 1;
    const int b = blockIdx.x / G1, j = blockIdx.x - b * G1;
    const int ell = a.ell ? a.ell[b] : a.gamma;
    if (ell < 0 || ell > a.gamma) {
        if (j == 0 && threadIdx.x == 0) set_status(a.status, SPEC_ERR_VERIFY_LEN);
        return;
    }
    if (j > ell) return;
    long long r = (long long)b * G1 + j;
    if (a.row) {
        const int first = a.row[b];
        if (first < 0 || first > a.rows - ell - 1) {
            if (threadIdx.x == 0) set_status(a.status, SPEC_ERR_ROW_INDEX);
            return;
        }
        r = first + j;
    }
    const long long pos = (long long)a.len[b] + j;
    const long long entry = entry_at(a, c, b, pos);
    for (int i = threadIdx.x; i < a.half; i += kAppendThreads) {
        const unsigned long long turn = (unsigned long long)pos * a.turns[i];
        const float half_turns = (float)(int)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
        float s, co;
        sincospif(half_turns, &s, &co);
        s_cos[i] = co * a.mscale;
        s_sin[i] = s * a.mscale;
    }
    __syncthreads();

    const int D = c.head_dim, H = c.kv_heads, heads = a.q_heads + H;
    const int per_head = D / E;                   // vectors of a head
    const int turned = 2 * a.half / E;            // of them turned
    const int pairs = INTERLEAVED ? turned : turned / 2;
    const int items = per_head - turned + pairs;  // work items of a q or k head
    const int all = heads * items + H * per_head;
    const char* q = a.q + r * a.q_row;
    const char* k = a.k + r * a.k_row;
    const char* v = a.v + r * a.v_row;
    char* out_q = a.out_q + r * (long long)a.q_heads * D * (int)sizeof(T);
    for (int it = threadIdx.x; it < all; it += kAppendThreads) {
        if (it >= heads * items) {
            const int h = (it - heads * items) / per_head, w = (it - heads * items) - h * per_head;
            if (entry < 0) continue;
            float x[E];
            load_vec<T, E>(v + h * a.v_head + w * E * (int)sizeof(T), x);
            if (sizeof(C) == 1 && c.v_scale) {
                const float s = c.v_scale[h];
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = x[e] / s;
            }
            store_vec<C, E>(c.v + entry + h * c.head + w * E * (int)sizeof(C), x);
            continue;
        }
        const int head = it / items, w = it - head * items;
        const bool is_q = head < a.q_heads;
        const int h = is_q ? head : head - a.q_heads;
        if (!is_q && entry < 0) continue;
        const char* from = is_q ? q + h * a.q_head : k + h * a.k_head;
        char* to = is_q ? out_q + (long long)h * D * (int)sizeof(T) : c.k + entry + h * c.head;
        const bool scaled = sizeof(C) == 1 && !is_q && c.k_scale;
        const float s = scaled ? c.k_scale[h] : 1.0f;
        float x[E], y[E];
        int at, partner = -1;
        if (w >= pairs) {
            at = (turned + w - pairs) * E;
            load_vec<T, E>(from + at * (int)sizeof(T), x);
        } else if (INTERLEAVED) {
            at = w * E;
            load_vec<T, E>(from + at * (int)sizeof(T), x);
#pragma unroll
            for (int e = 0; e + 1 < E; e += 2) {
                const float co = s_cos[(at + e) >> 1], si = s_sin[(at + e) >> 1];
                const float u = x[e], t = x[e + 1];
                x[e] = u * co - t * si;
                x[e + 1] = u * si + t * co;
            }
        } else {
            at = w * E;
            partner = at + a.half;
            load_vec<T, E>(from + at * (int)sizeof(T), x);
            load_vec<T, E>(from + partner * (int)sizeof(T), y);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float co = s_cos[at + e], si = s_sin[at + e];
                const float u = x[e], t = y[e];
                x[e] = u * co - t * si;
                y[e] = u * si + t * co;
            }
        }
        if (scaled) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x[e] = x[e] / s;
                y[e] = y[e] / s;
            }
        }
        if (is_q) {
            store_vec<T, E>(to + at * (int)sizeof(T), x);
            if (partner >= 0) store_vec<T, E>(to + partner * (int)sizeof(T), y);
        } else {
            store_vec<C, E>(to + at * (int)sizeof(C), x);
            if (partner >= 0) store_vec<C, E>(to + partner * (int)sizeof(C), y);
        }
    }
}

}  // namespace specv

// ===================================================================== host
using namespace specv;

namespace {

template <typename T, typename C>
int launch_append(const AppendArgs& a, const CacheView& c, bool interleaved, cudaStream_t st) {
    const int blocks = a.B * (a.gamma + 1);
    constexpr int E = 16 / sizeof(T);
    if (interleaved) {
        if (2 * a.half % E == 0) k_append<T, C, true, E><<<blocks, kAppendThreads, 0, st>>>(a, c);
        else k_append<T, C, true, 2><<<blocks, kAppendThreads, 0, st>>>(a, c);
    } else {
        if (a.half % E == 0) k_append<T, C, false, E><<<blocks, kAppendThreads, 0, st>>>(a, c);
        else k_append<T, C, false, 1><<<blocks, kAppendThreads, 0, st>>>(a, c);
    }
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" int spec_append_kv(const void* q, long long q_row_stride, long long q_head_stride, const void* k,
                              const void* v, long long k_row_stride, long long k_head_stride,
                              long long v_row_stride, long long v_head_stride, spec_dtype dt, int q_heads,
                              const spec_cache* cache, const int32_t* page_table, int max_pages,
                              const int32_t* cache_len, const int32_t* verify_len, const int32_t* row, int rows,
                              int B, int gamma, const uint64_t* turns, int rotary_dim, int interleaved,
                              float mscale, void* out_q, void* workspace, size_t workspace_bytes,
                              spec_stream_t stream) {
    TraceRange tr("spec_append_kv");
    CacheView c;
    const int rc = cache_view(cache, c);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || B > SPEC_MAX_BATCH || gamma < 0 || gamma > SPEC_MAX_GAMMA || q_heads < 1 || q_heads > 65535 ||
        max_pages < 1 || rows < 0)
        return SPEC_ERR_SHAPE;
    if (dt != SPEC_F32 && dt != SPEC_BF16 && dt != SPEC_F16) return SPEC_ERR_SHAPE;
    if (cache->dt != dt && !(cache->dt == SPEC_E4M3 && dt != SPEC_F32)) return SPEC_ERR_SHAPE;
    const long long es = dtype_size(dt);
    if (rotary_dim < 0 || rotary_dim > c.head_dim || (rotary_dim & 1)) return SPEC_ERR_SHAPE;
    if (!(mscale == mscale) || mscale - mscale != 0.0f) return SPEC_ERR_SHAPE;
    if (!row && rows < B * (gamma + 1)) return SPEC_ERR_SHAPE;
    if (B == 0) return SPEC_OK;
    if (!q || !k || !v || !out_q || !page_table || !cache_len || !workspace || (rotary_dim > 0 && !turns))
        return SPEC_ERR_NULL;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out_q | (uintptr_t)workspace) & 15)
        return SPEC_ERR_ALIGN;
    if (((q_row_stride | q_head_stride | k_row_stride | k_head_stride | v_row_stride | v_head_stride) * es) & 15)
        return SPEC_ERR_ALIGN;
    if (((uintptr_t)page_table | (uintptr_t)cache_len | (uintptr_t)verify_len | (uintptr_t)row) & 3 ||
        ((uintptr_t)turns & 7))
        return SPEC_ERR_ALIGN;
    if (workspace_bytes < 256) return SPEC_ERR_WORKSPACE;
    AppendArgs a;
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
    a.table = page_table;
    a.len = cache_len;
    a.ell = verify_len;
    a.row = row;
    a.turns = (const unsigned long long*)turns;
    a.status = (int*)workspace;
    a.q_heads = q_heads;
    a.rows = rows;
    a.B = B;
    a.gamma = gamma;
    a.max_pages = max_pages;
    a.half = rotary_dim / 2;
    a.mscale = mscale;
    cudaStream_t st = (cudaStream_t)stream;
    const bool il = interleaved != 0;
    if (dt == SPEC_F32) return launch_append<float, float>(a, c, il, st);
    if (dt == SPEC_BF16)
        return cache->dt == SPEC_E4M3 ? launch_append<__nv_bfloat16, __nv_fp8_e4m3>(a, c, il, st)
                                      : launch_append<__nv_bfloat16, __nv_bfloat16>(a, c, il, st);
    return cache->dt == SPEC_E4M3 ? launch_append<__half, __nv_fp8_e4m3>(a, c, il, st)
                                  : launch_append<__half, __half>(a, c, il, st);
}
