// Rotary positions and the append of the tested tokens to a paged cache.
//
// Angles.  The angle of position p and pair i is p f_i.  With f_i / (2 pi) held
// as a fraction F of 2^64, p F mod 2^64 is the angle's fraction of a turn, an
// exact wrapping 64-bit product at any position (an fp32 angle of position
// 10^6 would be off by 0.06, and GB300's fp64 pipe is narrow).  Its upper 32
// bits, as a signed number of half turns, go to sincospif.
//
// The angles of a row's pairs are computed once into shared memory and used by all
// q and k heads, which then pass as 16-byte vectors.
// Bound by HBM for large batches (each input read once, each output written
// once), by launch and one round trip of the page table for small ones.
#include <type_traits>

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
    // work items of a row, see k_append
    int all, qk_items, items, pairs, turned;
    FastDiv by_items, by_head, by_blocks, by_half;
};

// Threads of a block: with one row, two items each where 128 to 512 of them do.
constexpr int kAppendLeast = 128, kAppendMost = 512, kAppendTwo = 128;

// One work item of a row: vector `at` of a q, k or v head, and its partner in a
// half layout.
struct Item {
    int what;  // 0 q, 1 k, 2 v
    int h, at, partner;  // head, first elements
    bool turn;
};

template <bool INTERLEAVED, int E>
__device__ __forceinline__ Item item_of(const AppendArgs& a, int i) {
    Item it;
    it.partner = -1;
    it.turn = false;
    if (i >= a.qk_items) {
        const uint32_t x = (uint32_t)(i - a.qk_items);
        it.what = 2;
        it.h = (int)a.by_head.div(x);
        it.at = ((int)x - it.h * (int)a.by_head.d) * E;
        return it;
    }
    const int head = (int)a.by_items.div((uint32_t)i), w = i - head * a.items;
    it.what = head < a.q_heads ? 0 : 1;
    it.h = head < a.q_heads ? head : head - a.q_heads;
    it.turn = w < a.pairs;
    it.at = (it.turn ? w : a.turned + w - a.pairs) * E;
    if (it.turn && !INTERLEAVED) it.partner = it.at + a.half;
    return it;
}

// The item's vectors in the block's n rows.
template <typename T, int E, int RB>
__device__ __forceinline__ void load_item(const AppendArgs& a, const Item& it, int n, const char* q, const char* k,
                                          const char* v, Vec<T, E> (&x)[RB], Vec<T, E> (&y)[RB]) {
    const char* from = (it.what == 0 ? q + it.h * a.q_head : it.what == 1 ? k + it.h * a.k_head : v + it.h * a.v_head) +
                       it.at * (int)sizeof(T);
    const long long row = it.what == 0 ? a.q_row : it.what == 1 ? a.k_row : a.v_row;
    const int partner = (it.partner - it.at) * (int)sizeof(T);
#pragma unroll
    for (int rr = 0; rr < RB; ++rr)
        if (rr < n) {
            x[rr] = *(const Vec<T, E>*)(from + rr * row);
            if (it.partner >= 0) y[rr] = *(const Vec<T, E>*)(from + rr * row + partner);
        }
}

// E values as T, to nearest even (e4m3: clamped to the largest finite value; a
// NaN stays NaN), converted in pairs.
template <typename T, int E>
__device__ __forceinline__ void store_vec(char* p, const float (&x)[E]) {
    Vec<T, E> v;
    if constexpr (E == 1 || std::is_same<T, float>::value) {
#pragma unroll
        for (int e = 0; e < E; ++e) v.x[e] = from_f32<T>(x[e]);
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 two = make_float2(x[e], x[e + 1]);
            if constexpr (std::is_same<T, __nv_bfloat16>::value)
                *(__nv_bfloat162*)&v.x[e] = __float22bfloat162_rn(two);
            else if constexpr (std::is_same<T, __half>::value) *(__half2*)&v.x[e] = __float22half2_rn(two);
            else *(__nv_fp8x2_storage_t*)&v.x[e] = __nv_cvt_float2_to_fp8x2(two, __NV_SATFINITE, __NV_E4M3);
        }
    }
    *(Vec<T, E>*)p = v;
}

// N adjacent floats of shared memory.
template <int N>
__device__ __forceinline__ void load_angles(const float* s, float (&x)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int n = 0; n < N; n += 4) *(float4*)&x[n] = *(const float4*)(s + n);
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = s[n];
    }
}

template <typename T, typename C, bool INTERLEAVED, int E>
__device__ __forceinline__ void put_item(const AppendArgs& a, const CacheView& c, const Item& it, long long entry,
                                         char* out_q, const float* s_cos, const float* s_sin, const Vec<T, E>& vx,
                                         const Vec<T, E>& vy) {
    if (it.what != 0 && entry < 0) return;
    float x[E], y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        x[e] = to_f32(vx.x[e]);
        y[e] = 0.0f;
    }
    if (it.turn) {
        constexpr int P = INTERLEAVED ? (E + 1) / 2 : E;  // pairs
        float co[P], si[P];
        const int first = INTERLEAVED ? it.at >> 1 : it.at;
        load_angles<P>(s_cos + first, co);
        load_angles<P>(s_sin + first, si);
        if (INTERLEAVED) {
#pragma unroll
            for (int e = 0; e + 1 < E; e += 2) {
                const float u = x[e], t = x[e + 1];
                x[e] = u * co[e >> 1] - t * si[e >> 1];
                x[e + 1] = u * si[e >> 1] + t * co[e >> 1];
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float u = x[e], t = to_f32(vy.x[e]);
                x[e] = u * co[e] - t * si[e];
                y[e] = u * si[e] + t * co[e];
            }
        }
    }
    if (it.what == 0) {
        char* to = out_q + (long long)it.h * c.head_dim * (int)sizeof(T);
        store_vec<T, E>(to + it.at * (int)sizeof(T), x);
        if (it.partner >= 0) store_vec<T, E>(to + it.partner * (int)sizeof(T), y);
        return;
    }
    const float* scales = it.what == 1 ? c.k_scale : c.v_scale;
    if (sizeof(C) == 1 && scales) {
        const float inv = 1.0f / scales[it.h];  // one division a vector
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] *= inv;
            y[e] *= inv;
        }
    }
    char* to = (it.what == 1 ? c.k : c.v) + entry + it.h * c.head;
    store_vec<C, E>(to + it.at * (int)sizeof(C), x);
    if (it.partner >= 0) store_vec<C, E>(to + it.partner * (int)sizeof(C), y);
}

// T: rows, C: cache, E: elements of a vector.  Work items of a row: for each q
// and k head, the vectors of its first halves (with their partners, so that one
// thread reads and writes a pair and out_q may be q) or, interleaved, its
// vectors; then the unturned vectors; then v's.  E is 16 bytes' worth where the
// turned part is whole vectors, else a single element (a pair if interleaved).
//
// A block has RB adjacent rows of one request: a thread works its items' places
// out once and takes them in every row, all rows' loads in flight together.  One
// row a block (RB = 1) is for batches that would not fill the GPU otherwise; a
// large batch with one row a block was bound by instructions.  A block's first
// loads are on their way before the angles and the pages are known.
//
// 4,600 rows of 40 + 8 heads of 128, bf16 (e4m3 cache, 103 MB), by rows a block and
// blocks of 128 threads an SM: interleaved, 64 values turned, one row 38 us, two rows
// 24 us (12 blocks), 25 (10), 26 (8), four rows 27 to 38 (their registers leave fewer
// warps).  The half layout, whose items have two vectors a row, 128 values turned: one
// row 38 us, two rows 32 (12 blocks, spilling at 40 registers), 28 (10), 27 (8); 1,700
// rows 13, 18, 16 and 13 us.  fp32 rows (206 MB): one row 58, 38 (12), 38 (10), 40 (8).
template <typename T, bool INTERLEAVED>
constexpr int kAppendBlocks = sizeof(T) == 2 && !INTERLEAVED ? 8 : 12;

template <typename T, typename C, bool INTERLEAVED, int E, int RB>
__global__ void __launch_bounds__(RB == 1 ? kAppendMost : kAppendTwo, RB == 1 ? 1 : kAppendBlocks<T, INTERLEAVED>)
    k_append(AppendArgs a, CacheView c) {
    __shared__ __align__(16) float s_cos[RB][SPEC_MAX_HEAD_DIM / 2], s_sin[RB][SPEC_MAX_HEAD_DIM / 2];
    __shared__ long long s_entry[RB];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, threads = blockDim.x;
    const int b = (int)a.by_blocks.div(blockIdx.x), j0 = (blockIdx.x - b * (int)a.by_blocks.d) * RB;
    const int ell = a.ell ? a.ell[b] : a.gamma;
    const int len = a.len[b];
    const int first = a.row ? a.row[b] : b * (a.gamma + 1);
    if (ell < 0 || ell > a.gamma) {
        if (j0 == 0 && tid == 0) set_status(a.status, SPEC_ERR_VERIFY_LEN);
        return;
    }
    const int n = min(RB, ell + 1 - j0);  // rows of the block
    if (n <= 0) return;
    if (first < 0 || first > a.rows - ell - 1) {
        if (tid == 0) set_status(a.status, SPEC_ERR_ROW_INDEX);
        return;
    }
    const long long r = (long long)first + j0;
    const char* q = a.q + r * a.q_row;
    const char* k = a.k + r * a.k_row;
    const char* v = a.v + r * a.v_row;
    Vec<T, E> x[RB], y[RB];
    Item it = item_of<INTERLEAVED, E>(a, min(tid, a.all - 1));
    load_item<T, E, RB>(a, it, n, q, k, v, x, y);

    for (int i = tid; i < RB * a.half; i += threads) {
        const int rr = RB == 1 ? 0 : (int)a.by_half.div((uint32_t)i), pair = i - rr * a.half;
        const unsigned long long turn = (unsigned long long)((long long)len + j0 + rr) * a.turns[pair];
        const float half_turns = (float)(int)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
        float s, co;
        sincospif(half_turns, &s, &co);
        s_cos[rr][pair] = co * a.mscale;
        s_sin[rr][pair] = s * a.mscale;
    }
    if (tid < n) {  // the positions' places in the pages
        const long long pos = (long long)len + j0 + tid;
        long long entry = -1;
        if (pos < 0 || pos >= (long long)a.max_pages * c.page_size || pos > 0x7fffffffll) {
            set_status(a.status, SPEC_ERR_CACHE_LEN);
        } else {
            const uint32_t slot = c.by_page.div((uint32_t)pos);
            const int page = a.table[(size_t)b * a.max_pages + slot];
            if (page >= 0 && page < c.pages)
                entry = (long long)page * c.page + (pos - (long long)slot * c.page_size) * c.token;
            else
                set_status(a.status, SPEC_ERR_PAGE);
        }
        s_entry[tid] = entry;
    }
    __syncthreads();
    const long long out_row = (long long)a.q_heads * c.head_dim * (int)sizeof(T);
    char* out_q = a.out_q + r * out_row;
    for (int i = tid; i < a.all;) {
#pragma unroll
        for (int rr = 0; rr < RB; ++rr)
            if (rr < n)
                put_item<T, C, INTERLEAVED, E>(a, c, it, s_entry[rr], out_q + rr * out_row, s_cos[rr], s_sin[rr], x[rr],
                                               y[rr]);
        i += threads;
        if (i >= a.all) break;
        it = item_of<INTERLEAVED, E>(a, i);
        load_item<T, E, RB>(a, it, n, q, k, v, x, y);
    }
}

}  // namespace specv

// ===================================================================== host
using namespace specv;

namespace {

template <typename T, typename C, bool INTERLEAVED, int E>
int launch_vectors(AppendArgs a, const CacheView& c, cudaStream_t st) {
    const int per_head = c.head_dim / E, heads = a.q_heads + c.kv_heads;
    a.turned = 2 * a.half / E;
    a.pairs = INTERLEAVED ? a.turned : a.turned / 2;
    a.items = per_head - a.turned + a.pairs;
    a.qk_items = heads * a.items;
    a.all = a.qk_items + c.kv_heads * per_head;
    a.by_items = FastDiv((uint32_t)a.items);
    a.by_head = FastDiv((uint32_t)per_head);
    a.by_half = FastDiv((uint32_t)max(a.half, 1));
    // two rows a block where the blocks still fill the GPU four times over
    int sms = 0;
    if (const int rc = sm_count(sms)) return rc;
    const int two = (a.gamma + 2) / 2;
    if ((long long)a.B * two >= 4ll * sms) {
        a.by_blocks = FastDiv((uint32_t)two);
        return launch_dependent(k_append<T, C, INTERLEAVED, E, 2>, dim3(a.B * two), kAppendTwo, 0, st, 0, a, c);
    }
    a.by_blocks = FastDiv((uint32_t)a.gamma + 1);
    const int threads = min(kAppendMost, max(kAppendLeast, (a.all + 63) / 64 * 32));
    return launch_dependent(k_append<T, C, INTERLEAVED, E, 1>, dim3(a.B * (a.gamma + 1)), threads, 0, st, 0, a, c);
}

template <typename T, typename C>
int launch_append(const AppendArgs& a, const CacheView& c, bool interleaved, cudaStream_t st) {
    constexpr int E = 16 / sizeof(T);
    if (interleaved)
        return 2 * a.half % E == 0 ? launch_vectors<T, C, true, E>(a, c, st) : launch_vectors<T, C, true, 2>(a, c, st);
    return a.half % E == 0 ? launch_vectors<T, C, false, E>(a, c, st) : launch_vectors<T, C, false, 1>(a, c, st);
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
