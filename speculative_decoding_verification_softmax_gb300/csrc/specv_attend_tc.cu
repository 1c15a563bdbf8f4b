// The tensor-core attention kernels over the requests of a call.
#include "specv_attend_tc_launch.cuh"

namespace specv {

// Boxes of 8 tokens (one swizzle atom) or more must lie within a page, and the
// strides within what a tensor map holds.
bool attend_tc_takes(const CacheView& c, int rows) {
    const long long most = 1ll << 40;
    return rows > kTcLeast && c.head_dim <= 128 && c.page_size % 8 == 0 && c.page > 0 && c.token > 0 && c.head > 0 &&
           c.page < most && c.token < most && c.head < most;
}

AttendPlan attend_tc_plan(int sms) {
    AttendPlan p;
    p.blocks = sms;
    p.tile_rows = kTcRows;
    return p;
}

int attend_tc(const AttendArgs& a, const CacheView& c, spec_dtype dt, spec_dtype cache_dt, int blocks,
              cudaStream_t st) {
    return tc_launch<false>(a, c, dt, cache_dt, blocks, st);
}

}  // namespace specv
