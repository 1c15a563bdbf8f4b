// The warp-level attention kernels over 16-bit caches.
#include "specv_attend_mma.cuh"

namespace specv {

// Rows of a unit: 16 for each of the warps that split them.
AttendPlan attend_mma_plan(int rows, int head_dim, bool f8, int sms) {
    const int wr = rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 64 ? 4 : 8;
    AttendPlan p;
    p.blocks = sms * mma_per_sm(f8, head_dim, wr);
    p.tile_rows = 16 * wr;
    return p;
}

int attend_mma16(const AttendArgs& a, const CacheView& c, spec_dtype dt, int blocks, cudaStream_t st) {
    return dt == SPEC_BF16 ? mma_launch_dim<__nv_bfloat16, __nv_bfloat16, false>(a, c, blocks, st)
                           : mma_launch_dim<__half, __half, false>(a, c, blocks, st);
}

}  // namespace specv
