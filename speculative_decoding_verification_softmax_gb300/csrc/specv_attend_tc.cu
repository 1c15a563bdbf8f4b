// The tensor-core attention kernels: tensor maps of the cache and the launch.
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

// The cache as {head_dim, page_size, kv_heads, pages}, in boxes of 64 values
// and `box` tokens; values behind head_dim read as zero.
bool make_map(CUtensorMap& map, void* at, const CacheView& c, bool half, int box) {
    const EncodeTiled fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                                (cuuint64_t)c.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token, (cuuint64_t)c.head, (cuuint64_t)c.page};
    const cuuint32_t extent[4] = {64, (cuuint32_t)box, 1, 1}, step[4] = {1, 1, 1, 1};
    return fn(&map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, at, dims, strides,
              extent, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int box_tokens(int page_size) {
    int box = kTcKeys;
    while (page_size % box) box >>= 1;
    return box;
}

template <typename T, int D>
int launch(const AttendArgs& a, const CacheView& c, const TcArgs& tc, const CUtensorMap& mk, const CUtensorMap& mv,
           int blocks, cudaStream_t st) {
    auto* f = k_attend_tc<T, D>;
    if (cudaFuncSetAttribute((const void*)f, cudaFuncAttributeMaxDynamicSharedMemorySize, TcShape<D>::kSmem) !=
        cudaSuccess)
        return SPEC_ERR_CUDA;
    f<<<blocks, kTcThreads, TcShape<D>::kSmem, st>>>(a, c, tc, mk, mv);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

// Boxes of 8 tokens (one swizzle atom) or more must lie within a page, and the
// strides within what a tensor map holds.
bool attend_tc_takes(const CacheView& c, int rows) {
    const long long most = 1ll << 40;
    return rows > 16 && c.head_dim <= 128 && c.page_size % 8 == 0 && c.page > 0 && c.token > 0 && c.head > 0 &&
           c.page < most && c.token < most && c.head < most;
}

AttendPlan attend_tc_plan(int sms) {
    AttendPlan p;
    p.blocks = sms;
    p.tile_rows = kTcRows;
    return p;
}

int attend_tc(const AttendArgs& a, const CacheView& c, spec_dtype dt, int blocks, cudaStream_t st) {
    TcArgs tc;
    tc.box = box_tokens(c.page_size);
    tc.shift = 0;
    while ((1 << tc.shift) < tc.box) ++tc.shift;
    CUtensorMap mk, mv;
    const bool half = dt == SPEC_F16;
    if (!make_map(mk, c.k, c, half, tc.box) || !make_map(mv, c.v, c, half, tc.box)) return SPEC_ERR_CUDA;
    if (c.head_dim <= 64)
        return half ? launch<__half, 64>(a, c, tc, mk, mv, blocks, st)
                    : launch<__nv_bfloat16, 64>(a, c, tc, mk, mv, blocks, st);
    return half ? launch<__half, 128>(a, c, tc, mk, mv, blocks, st)
                : launch<__nv_bfloat16, 128>(a, c, tc, mk, mv, blocks, st);
}

}  // namespace specv
