// The tensor-core attention kernels: tensor maps of the cache and the launch.
#pragma once

#include "specv_attend_tc.cuh"

namespace specv {

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return (EncodeTiled) nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

// The cache as {head_dim, page_size, kv_heads, pages}, in boxes of 64 16-bit
// values (a swizzled panel) or of whole e4m3 rows, and `box` tokens; values
// behind head_dim read as zero.
bool make_map(CUtensorMap& map, void* at, const CacheView& c, spec_dtype dt, int box) {
    const EncodeTiled fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                                (cuuint64_t)c.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token, (cuuint64_t)c.head, (cuuint64_t)c.page};
    // L2 fetches no more around a row than the row itself: other heads' values
    // beside it are used by other units, at other times
    const int row = c.head_dim * dtype_size(dt);
    const CUtensorMapL2promotion fetch = row >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                         : row >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                      : CU_TENSOR_MAP_L2_PROMOTION_NONE;
    const cuuint32_t extent[4] = {dt == SPEC_E4M3 && c.head_dim > 64 ? 128u : 64u, (cuuint32_t)box, 1, 1}, step[4] = {1, 1, 1, 1};
    return fn(&map,
              dt == SPEC_E4M3  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
              : dt == SPEC_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                               : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              4, at, dims, strides, extent, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              dt == SPEC_E4M3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int box_tokens(int page_size) {
    int box = kTcKeys;
    while (page_size % box) box >>= 1;
    return box;
}

template <typename T, typename O, bool F8, int D, bool SH>
int launch_dim(const AttendArgs& a, const CacheView& c, const TcArgs& tc, const CUtensorMap& mk,
               const CUtensorMap& mv, int blocks, cudaStream_t st) {
    using Sh = TcShape<F8, D>;
    auto* f = k_attend_tc<T, O, F8, D, SH>;
    static std::atomic<unsigned long long> done{0};
    if (const int rc = allow_smem((const void*)f, Sh::kSmem, done)) return rc;
    return launch_dependent(f, dim3(blocks), kTcThreads, Sh::kSmem, st, 0, a, c, tc, mk, mv);
}

template <typename T, typename O, bool F8, bool SH>
int launch(const AttendArgs& a, const CacheView& c, const TcArgs& tc, const CUtensorMap& mk, const CUtensorMap& mv,
           int blocks, cudaStream_t st) {
    return c.head_dim <= 64 ? launch_dim<T, O, F8, 64, SH>(a, c, tc, mk, mv, blocks, st)
                            : launch_dim<T, O, F8, 128, SH>(a, c, tc, mk, mv, blocks, st);
}

template <bool SH>
int tc_launch(const AttendArgs& a, const CacheView& c, spec_dtype dt, spec_dtype cache_dt, int blocks,
              cudaStream_t st) {
    TcArgs tc;
    tc.box = box_tokens(c.page_size);
    tc.shift = 0;
    while ((1 << tc.shift) < tc.box) ++tc.shift;
    tc.expire_first = expire_first_wait();
    CUtensorMap mk, mv;
    if (!make_map(mk, c.k, c, cache_dt, tc.box) || !make_map(mv, c.v, c, cache_dt, tc.box)) return SPEC_ERR_CUDA;
    if (cache_dt == SPEC_E4M3)
        return dt == SPEC_F16 ? launch<__half, __half, true, SH>(a, c, tc, mk, mv, blocks, st)
                              : launch<__half, __nv_bfloat16, true, SH>(a, c, tc, mk, mv, blocks, st);
    return dt == SPEC_F16 ? launch<__half, __half, false, SH>(a, c, tc, mk, mv, blocks, st)
                          : launch<__nv_bfloat16, __nv_bfloat16, false, SH>(a, c, tc, mk, mv, blocks, st);
}

}  // namespace

}  // namespace specv
