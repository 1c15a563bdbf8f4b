// The warp-level attention kernels over e4m3 caches: products in fp16.
#include "specv_attend_mma.cuh"

namespace specv {

int attend_mma8(const AttendArgs& a, const CacheView& c, spec_dtype dt, int blocks, cudaStream_t st) {
    return dt == SPEC_BF16 ? mma_launch_dim<__half, __nv_bfloat16, true>(a, c, blocks, st)
                           : mma_launch_dim<__half, __half, true>(a, c, blocks, st);
}

}  // namespace specv
