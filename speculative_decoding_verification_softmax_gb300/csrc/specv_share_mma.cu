// The warp-level attention kernels over the items of a plan: heads of more than
// 128, and pages that are not a multiple of 8 tokens.
#include "specv_attend_mma.cuh"

namespace specv {

namespace {

// Eight warps of 16 rows each, or one of them with the keys split over four.  Measured,
// bf16, 64 requests behind 8192 positions, 4 KV heads of 256: 8 rows of each in units of
// 64 rows 257 us, of 128 193 us; 36 rows 706 and 398 us.  8 requests of 2 rows behind 4092
// positions, 8 KV heads of 256: 62 us with eight warps of rows, 45 with the keys split.
constexpr int kWr = 8;

template <typename T, typename O, bool F8, int D>
int launch_rows(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    return a.tile_rows == 16 ? mma_launch<T, O, F8, D, 1, 4, true>(a, c, blocks, st)
                             : mma_launch<T, O, F8, D, kWr, 1, true>(a, c, blocks, st);
}

template <typename T, typename O, bool F8>
int launch(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    if (c.head_dim <= 64) return launch_rows<T, O, F8, 64>(a, c, blocks, st);
    if (c.head_dim <= 128) return launch_rows<T, O, F8, 128>(a, c, blocks, st);
    return launch_rows<T, O, F8, 256>(a, c, blocks, st);
}

}  // namespace

AttendPlan attend_mma_shared_plan(int rows, int head_dim, bool f8, int sms) {
    const int wr = rows <= 16 ? 1 : kWr;
    AttendPlan p;
    p.blocks = sms * mma_per_sm(f8, head_dim, wr);
    p.tile_rows = 16 * wr;
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
