// The tensor-core attention kernels over the items of a plan.
#include "specv_attend_tc_launch.cuh"

namespace specv {

int attend_tc_shared(const AttendArgs& a, const CacheView& c, spec_dtype dt, spec_dtype cache_dt, int blocks,
                     cudaStream_t st) {
    return tc_launch<true>(a, c, dt, cache_dt, blocks, st);
}

}  // namespace specv
