// The warp-level attention kernels over the items of a plan: heads of more than
// 128, and pages that are not a multiple of 8 tokens.
#include "specv_attend_mma.cuh"

namespace specv {

namespace {

constexpr int kWr = 8;

template <typename T, typename O, bool F8>
int launch(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    if (c.head_dim <= 64) return mma_launch<T, O, F8, 64, kWr, 1, true>(a, c, blocks, st);
    if (c.head_dim <= 128) return mma_launch<T, O, F8, 128, kWr, 1, true>(a, c, blocks, st);
    return mma_launch<T, O, F8, 256, kWr, 1, true>(a, c, blocks, st);
}

}  // namespace

AttendPlan attend_mma_shared_plan(int head_dim, bool f8, int sms) {
    AttendPlan p;
    p.blocks = sms * mma_per_sm(f8, head_dim, kWr);
    p.tile_rows = 16 * kWr;
    return p;
}

int attend_mma_shared(const AttendArgs& a, const CacheView& c, spec_dtype dt, bool f8, int blocks, cudaStream_t st) {
    if (f8)
        return dt == SPEC_BF16 ? launch<__half, __nv_bfloat16, true>(a, c, blocks, st)
                               : launch<__half, __half, true>(a, c, blocks, st);
    return dt == SPEC_BF16 ? launch<__nv_bfloat16, __nv_bfloat16, false>(a, c, blocks, st)
                           : launch<__half, __half, false>(a, c, blocks, st);
}

}  // namespace specv
