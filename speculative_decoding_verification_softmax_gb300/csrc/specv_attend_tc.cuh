// Attention over the paged cache with the 5th-generation tensor cores
// (tcgen05.mma, accumulators in TMEM), for units of many query rows.
//
// The unit's rows are the 128 lanes of the accumulators: S = Q K^T and O += P V
// with M = 128, tiles of 128 keys.  A key's bytes are used for up to 128 rows'
// products, 128 FLOP a byte of a 16-bit cache: at HBM's rate that is half of
// what these instructions do, and twice what the warp-level ones do.
//
// Two streams of key tiles (even and odd) run against one another: while the
// four warps of one stream take the softmax of their scores, the tensor cores
// work for the other.  Each stream has its own S and O columns in TMEM and its
// own running maximum and sum; the unit's end joins them.  P overlays S.
//   warps 0-3, 4-7   softmax of the even and odd tiles, a row a thread; the
//                    query rows' load and the unit's output
//   warps 8-11       loads: K and V tiles, in the order of their use, through a
//                    ring of shared-memory slots that runs on over the units
//   warp 12          one thread issues all matrix instructions
// The loads are TMA boxes of as many tokens as always lie in one page.  V rows
// that some query row must not see (the cache's end, the window's edges) are
// loaded by the warps themselves instead: what nobody sees becomes zero, and a
// value that is not finite is left out and added by itself to its rows.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "specv_attend.cuh"

namespace specv {

constexpr int kTcKeys = 128;
constexpr int kTcRows = 128;
constexpr int kTcThreads = 13 * 32;
constexpr int kTcUnits = 8;  // flags of units under way

// A running maximum stays the reference until it is passed by this much (to
// base 2): weights reach 2^8 instead of 1, exactly as well in 16 bits, and the
// output in TMEM is scaled again a few times a unit instead of every tile.
constexpr float kTcSlack = 8.0f;

template <int D>
struct TcShape {
    static constexpr int kPanel = kTcKeys * 128;       // 64 columns of a tile, 128-byte rows
    static constexpr int kTile = kPanel * (D / 64);    // K or V of a tile
    static constexpr int kSlots = D == 64 ? 10 : 6;
    static constexpr int kQ = kTcRows * 128 * (D / 64);
    static constexpr int kSmem = 1024 + kQ + kSlots * kTile;
    static constexpr int kCols = 512;                  // TMEM columns: S0, S1, O0, O1 (a power of two)
};

struct TcArgs {
    int box, shift;  // tokens of a TMA box, 2^shift
};

// ------------------------------------------------------------------- PTX
__device__ __forceinline__ void tc_alloc(uint32_t* at, int cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(at)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tc_dealloc(uint32_t base, int cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}
// 32 columns of the warp's 32 lanes, and the wait for them.
__device__ __forceinline__ void tc_ld32(float (&x)[32], uint32_t at) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t at, const float (&x)[32]) {
    const uint32_t* r = reinterpret_cast<const uint32_t*>(x);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Box of {64 columns, `box` tokens, 1 head, 1 page} into shared memory.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int col, int token, int head, int page,
                                        uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(map), "r"(smem_u32(bar)), "r"(col), "r"(token), "r"(head), "r"(page)
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Operand descriptors: 128-byte swizzle, eight 128-byte rows an atom.  K-major
// (Q, K: the columns of a product adjacent): atoms of further rows 1024 bytes on.
// MN-major (V: a key's row is the product's N): atoms of further keys 1024 bytes
// on, further 64 columns a panel on.
__device__ __forceinline__ uint64_t desc_k(uint32_t at) {
    return (uint64_t)((at >> 4) & 0x3fff) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t at, uint32_t panel) {
    return (uint64_t)((at >> 4) & 0x3fff) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Waits for phase `parity`.  A wait that runs out of time sets `fail`, and all
// other waits of the block then end at once: every role runs its loops to their
// ends, without results, and the block returns.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* fail) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*fail) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *fail = 1;
            return false;
        }
    }
}

__device__ __forceinline__ uint32_t panel_at(int row, int chunk) {  // byte of a 16-byte chunk, 8 a panel row
    return (uint32_t)((chunk >> 3) * (128 * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

template <typename T>
__device__ __forceinline__ bool tc_nonfinite(uint32_t w, uint32_t half_mask) {
    const uint32_t e = (std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u) & half_mask;
    return (w & e) == e;
}

// The segments of a block's run, the same for every role.
struct Walk {
    Request req;
    int b, unit, t0, nt, h, r0, R;
    long long at, left, step;

    __device__ void start(const AttendArgs& a, const CacheView& c, const Run& run) {
        b = run.b;
        at = run.at;
        left = run.left;
        step = run.step;
        nt = 0;
        if (left > 0) req = request_of<kTcKeys>(a, c, b);
    }
    __device__ bool next(const AttendArgs& a, const CacheView& c) {
        at += nt;
        left -= nt;
        if (left <= 0) return false;
        if (at == (long long)req.units * req.tiles) {
            do req = request_of<kTcKeys>(a, c, ++b);
            while (req.units == 0);
            at = 0;
        }
        unit = (int)(at / req.tiles);
        t0 = (int)(at - (long long)unit * req.tiles);
        nt = (int)min((long long)(req.tiles - t0), left);
        h = unit / req.row_tiles;
        r0 = (unit - h * req.row_tiles) * kTcRows;
        R = min((req.ell + 1) * a.group - r0, kTcRows);
        return true;
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_attend_tc(AttendArgs a, CacheView c, TcArgs tc, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv) {
    using Sh = TcShape<D>;
    constexpr int KT = kTcKeys, NS = Sh::kSlots, CW = D / 8;  // chunks of a row
    extern __shared__ char smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], empty[NS], s_full[2], p_full[2], o_done[2], q_full, drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail, s_flags[kTcUnits];
    __shared__ long long s_scan[kTcThreads / 32 + 1];
    __shared__ Run s_run;
    __shared__ float s_ml[2][kTcRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    const uint32_t sq = base, ring = base + Sh::kQ;

    if (warp == 12) tc_alloc(&s_tmem, Sh::kCols);
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 4);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
        }
        mbar_init(&q_full, 8);
        mbar_init(&drain, 1);
        fence_mbar_init();
        s_fail = 0;
    }
    if (tid < kTcUnits) s_flags[tid] = 0;
    tc_fence_before();
    const Run run = run_of<KT, kTcThreads>(a, c, s_scan, &s_run);  // also the barrier behind the set-up
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int* fail = &s_fail;
    Walk w;
    w.start(a, c, run);
    int4 open = make_int4(0, 0, 0, 0);

    if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------------ loads
        // Items of a unit, in the order of their use: K0, K1, V0, K2, V1, ...
        const int lw = warp - 8, lt = tid - 8 * 32;
        const int boxes = KT / tc.box;
        uint32_t item = 0, issued = 0;
        int u = 0;
        while (w.next(a, c)) {
            const int32_t* pages = a.table + (size_t)w.b * a.max_pages;
            const int end = w.req.n + w.req.ell;
            bool bad = false;
            for (int i = 0; i < 2 * w.nt; ++i) {
                // item i: K of tile i for i < 2 (or the only one), then V and K in turn
                bool is_v;
                int t;
                if (w.nt == 1) {
                    is_v = i == 1;
                    t = 0;
                } else if (i < 2) {
                    is_v = false;
                    t = i;
                } else {
                    const int x = i - 2;
                    if (x < 2 * (w.nt - 2)) {
                        is_v = (x & 1) == 0;
                        t = is_v ? x >> 1 : (x >> 1) + 2;
                    } else {
                        is_v = true;
                        t = w.nt - 2 + (x - 2 * (w.nt - 2));
                    }
                }
                const int key0 = tile_key<KT>(w.req, w.t0 + t);
                const int slot = (int)(item % NS);
                const uint32_t dst = ring + slot * Sh::kTile;
                const bool whole = all_see<KT>(a, w.req, key0);
                const bool by_hand = is_v && !whole;
                // the lane's box of the tile: where it lies, looked up before the
                // slot is free; -1 if nobody sees any of it
                long long at = -1;
                int page = -1, token = 0;
                if ((by_hand || lw == 0) && lane < boxes) {
                    const int k = key0 + (lane << tc.shift);
                    bool need = k <= end;
                    if (need && !whole) {
                        need = false;
                        for (int x = 0; x < tc.box; ++x) need |= any_sees(a, w.req, k + x);
                    }
                    if (need) {
                        const uint32_t place = c.by_page.div((uint32_t)k);
                        token = k - (int)place * c.page_size;
                        page = pages[place];
                        if (page < 0 || page >= c.pages) {
                            bad = true;
                            page = -1;
                        } else {
                            at = (long long)page * c.page + (long long)token * c.token + w.h * c.head;
                        }
                    }
                }
                if (bad) atomicOr(&s_flags[u & (kTcUnits - 1)], 1);
                const bool ok =
                    __all_sync(0xffffffffu, item < NS || tc_wait(&empty[slot], ((item / NS) & 1) ^ 1, fail));
                if (by_hand) {
                    if (ok) {
                        bool dirty = false;
                        constexpr int RS = 128 / CW, BATCH = 8;  // rows of a step, steps in flight
                        const int ch = lt % CW;
#pragma unroll 1
                        for (int i0 = 0; i0 < KT / RS; i0 += BATCH) {
                            uint4 v[BATCH];
#pragma unroll
                            for (int q = 0; q < BATCH; ++q) {
                                const int k = lt / CW + (i0 + q) * RS;
                                const long long from = __shfl_sync(0xffffffffu, at, k >> tc.shift);
                                v[q] = make_uint4(0u, 0u, 0u, 0u);
                                if (from >= 0 && ch * 8 < c.head_dim && any_sees(a, w.req, key0 + k))
                                    v[q] = *(const uint4*)(c.v + from + (k & (tc.box - 1)) * c.token + ch * 16);
                            }
#pragma unroll
                            for (int q = 0; q < BATCH; ++q) {
                                uint32_t e[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    if (tc_nonfinite<T>(e[z], 0xffffu)) {
                                        e[z] &= 0xffff0000u;
                                        dirty = true;
                                    }
                                    if (tc_nonfinite<T>(e[z], 0xffff0000u)) {
                                        e[z] &= 0xffffu;
                                        dirty = true;
                                    }
                                }
                                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                                 dst + panel_at(lt / CW + (i0 + q) * RS, ch)),
                                             "r"(e[0]), "r"(e[1]), "r"(e[2]), "r"(e[3])
                                             : "memory");
                            }
                        }
                        if (dirty) atomicOr(&s_flags[u & (kTcUnits - 1)], 2);
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[slot]);
                } else if (lw == 0) {
                    const bool have = ok && page >= 0;
                    const int n = __popc(__ballot_sync(0xffffffffu, have));
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)n * tc.box * 128 * (D / 64));
                    __syncwarp();
                    if (have) {
#pragma unroll
                        for (int p = 0; p < D / 64; ++p)
                            tma_box(dst + p * Sh::kPanel + (lane << tc.shift) * 128, is_v ? &mv : &mk, p * 64, token, w.h,
                                    page, &full[slot]);
                    }
                    if (ok) issued = item + 1;
                } else if (lane == 0) {
                    mbar_arrive(&full[slot]);
                }
                __syncwarp();
                ++item;
            }
            ++u;
        }
        if (*fail && warp == 8) {  // copies under way land before the block ends
            for (uint32_t k = issued > NS ? issued - NS : 0; k < issued; ++k)
                mbar_wait_bounded(&full[k % NS], (k / NS) & 1);
        }
    } else if (warp == 12) {
        // ------------------------------------------------- matrix instructions
        constexpr uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
        constexpr uint32_t head = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(kTcRows >> 4) << 24);
        constexpr uint32_t id_s = head | ((uint32_t)(KT >> 3) << 17);
        constexpr uint32_t id_o = head | ((uint32_t)(D >> 3) << 17) | (1u << 16);
        if (lane == 0) {
            uint32_t item = 0, pn[2] = {0, 0};
            int u = 0;
            while (w.next(a, c)) {
                tc_wait(&q_full, u & 1, fail);
                ++u;
                tc_fence_after();
                auto scores = [&](int t) {
                    const int slot = (int)(item % NS);
                    tc_wait(&full[slot], (item / NS) & 1, fail);
                    tc_fence_after();
                    const uint32_t k = ring + slot * Sh::kTile;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * Sh::kPanel + (kk & 3) * 32;
                        tc_mma_ss(tmem + (t & 1) * KT, desc_k(sq + off), desc_k(k + off), id_s, kk > 0);
                    }
                    tc_commit(&empty[slot]);
                    tc_commit(&s_full[t & 1]);
                    ++item;
                };
                scores(0);
                if (w.nt > 1) scores(1);
                for (int t = 0; t < w.nt; ++t) {
                    const int s = t & 1;
                    tc_wait(&p_full[s], pn[s]++ & 1, fail);
                    const int slot = (int)(item % NS);
                    tc_wait(&full[slot], (item / NS) & 1, fail);
                    tc_fence_after();
                    const uint32_t v = ring + slot * Sh::kTile;
#pragma unroll
                    for (int kk = 0; kk < KT / 16; ++kk)
                        tc_mma_ts(tmem + 2 * KT + s * D, tmem + s * KT + kk * 8, desc_mn(v + kk * 2048, Sh::kPanel), id_o,
                                  t > 1 || kk > 0);
                    tc_commit(&empty[slot]);
                    tc_commit(&o_done[s]);
                    ++item;
                    if (t + 2 < w.nt) scores(t + 2);
                }
            }
            if (*fail) {
                tc_commit(&drain);
                mbar_wait_bounded(&drain, 0);
            }
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------- softmax and output
        const int s = warp >> 2;
        const int row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + s * KT, to = tmem + lanes + 2 * KT;
        const float scale = fabsf(a.scale);
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
        uint32_t seen = 0;  // tiles of the stream so far
        int u = 0;
        while (w.next(a, c)) {
            // query rows, 16 bytes a step
            for (int x = tid; x < kTcRows * CW; x += 256) {
                const int r = x / CW, ch = x - r * CW;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (r < w.R && ch * 8 < c.head_dim) {
                    const int j = (int)a.by_group.div((uint32_t)(w.r0 + r));
                    const int hq = w.h * a.group + (w.r0 + r - j * a.group);
                    v = *(const uint4*)(a.q + (long long)(w.req.base + j) * a.q_row + hq * a.q_head + ch * 16);
                    v.x ^= flip;
                    v.y ^= flip;
                    v.z ^= flip;
                    v.w ^= flip;
                }
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(sq + panel_at(r, ch)), "r"(v.x), "r"(v.y),
                             "r"(v.z), "r"(v.w)
                             : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);

            const bool active = (warp & 3) * 32 < w.R;  // the warp has rows
            const int pos = w.req.n + (row < w.R ? (int)a.by_group.div((uint32_t)(w.r0 + row)) : w.req.ell);
            float m = -INFINITY, l = 0.0f;
            for (int t = s; t < w.nt; t += 2) {
                tc_wait(&s_full[s], seen & 1, fail);
                tc_fence_after();
                if (active) {
                    const int key0 = tile_key<KT>(w.req, w.t0 + t);
                    const bool cut = !all_see<KT>(a, w.req, key0);
                    float x[32], top = -INFINITY;
                    if (!cut) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            tc_ld32(x, ts + q * 32);
#pragma unroll
                            for (int e = 0; e < 32; ++e) top = fmaxf(top, x[e]);
                        }
                        top *= scale;
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            tc_ld32(x, ts + q * 32);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (sees(a, pos, key0 + q * 32 + e)) top = fmaxf(top, x[e] * scale);
                        }
                    }
                    const bool up = top > m + kTcSlack;
                    if (__any_sync(0xffffffffu, up)) {
                        const float now = up ? top : m;
                        const float corr = up ? ex2_approx(m - now) : 1.0f;
                        l *= corr;
                        m = now;
                        if (t >= 2) {
                            tc_wait(&o_done[s], (seen - 1) & 1, fail);
                            tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < D / 32; ++q) {
                                tc_ld32(x, to + s * D + q * 32);
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[e] *= corr;
                                tc_st32(to + s * D + q * 32, x);
                            }
                        }
                    }
                    // weights: their sum is of the unrounded ones; for the
                    // product they are rounded to T, 2^-9 (bf16) or 2^-12 of
                    // each at most, as much as the output's own rounding
                    const float ref = m == -INFINITY ? 0.0f : m;
                    float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        tc_ld32(x, ts + q * 32);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            x[e] = fmaf(x[e], scale, -ref);
                            if (cut && !sees(a, pos, key0 + q * 32 + e)) x[e] = -INFINITY;
                            x[e] = ex2_approx(x[e]);
                            if (e & 1) sum1 += x[e];
                            else sum0 += x[e];
                        }
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (std::is_same<T, __half>::value)
                                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p[e]) : "f"(x[2 * e + 1]), "f"(x[2 * e]));
                            else
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[e]) : "f"(x[2 * e + 1]), "f"(x[2 * e]));
                        }
                        tc_st16(ts + q * 16, p);
                    }
                    l += sum0 + sum1;
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s]);
                ++seen;
            }
            if (s < w.nt) tc_wait(&o_done[s], (seen - 1) & 1, fail);
            if (s == 1) {
                s_ml[0][row] = m;
                s_ml[1][row] = l;
            }
            tc_fence_before();
            asm volatile("bar.sync 1, 256;" ::: "memory");
            tc_fence_after();

            // the two streams' weights, for both of them; the parts' maximum and
            // sum, or the reciprocal of the sum in the weights
            const int flags = s_flags[u & (kTcUnits - 1)];
            const bool complete = w.nt == w.req.tiles;
            float* part = part_at(a, blockIdx.x, w.t0 == 0 ? 1 : 0);
            int j = 0;
            long long orow = 0;
            if (row < w.R) orow = out_row(a, w.req, w.h, w.r0 + row, &j);
            if (s == 0) {
                const float m1 = s_ml[0][row];
                const float M = fmaxf(m, m1), ref = M == -INFINITY ? 0.0f : M;
                const float w0 = ex2_approx(m - ref), w1 = ex2_approx(m1 - ref);
                float L = l * w0 + s_ml[1][row] * w1;
                if ((flags & 1) || *fail) L = __int_as_float(0x7fc00000);
                const float inv = complete ? 1.0f / L : 1.0f;
                s_ml[0][row] = w0 * inv;
                s_ml[1][row] = w1 * inv;
                if (row < w.R) {
                    if (!complete) {
                        part[a.tile_rows * c.head_dim + row] = M;
                        part[a.tile_rows * (c.head_dim + 1) + row] = L;
                    } else if (a.lse) {
                        a.lse[orow] = (M + log2f(L)) * 0.6931471805599453f;
                    }
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");

            // output: stream s's warps write columns [s D/2, (s+1) D/2)
            if (active) {
                const float w0 = s_ml[0][row], w1 = s_ml[1][row];
#pragma unroll 1
                for (int q = 0; q < D / 64; ++q) {
                    const int col = s * (D / 2) + q * 32;
                    float x[32];
                    tc_ld32(x, to + col);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] *= w0;
                    if (w.nt > 1) {
                        float y[32];
                        tc_ld32(y, to + D + col);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = fmaf(w1, y[e], x[e]);
                    }
                    if (flags & 2) {  // values that are not finite, by themselves
                        const int32_t* pages = a.table + (size_t)w.b * a.max_pages;
                        for (int t = 0; t < w.nt; ++t) {
                            const int key0 = tile_key<KT>(w.req, w.t0 + t);
                            if (all_see<KT>(a, w.req, key0)) continue;
                            for (int k = key0; k < key0 + KT && k <= pos; ++k) {
                                if (!sees(a, pos, k)) continue;
                                const long long at = key_at(a, c, pages, k);
                                if (at < 0) continue;
                                const T* v = (const T*)(c.v + at + w.h * c.head);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (col + e < c.head_dim) {
                                        const float y = to_f32(v[col + e]);
                                        if (!(fabsf(y) <= 3.4e38f)) x[e] += y;
                                    }
                            }
                        }
                    }
                    if (row < w.R) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            if (col + e >= c.head_dim) break;
                            if (complete) {
                                uint32_t o[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    const float lo = x[e + 2 * z], hi = x[e + 2 * z + 1];
                                    if (std::is_same<T, __half>::value)
                                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[z]) : "f"(hi), "f"(lo));
                                    else
                                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[z]) : "f"(hi), "f"(lo));
                                }
                                *(uint4*)((char*)a.out + (orow * c.head_dim + col + e) * 2) =
                                    make_uint4(o[0], o[1], o[2], o[3]);
                            } else {
                                float4* p = (float4*)(part + row * c.head_dim + col + e);
                                p[0] = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                                p[1] = make_float4(x[e + 4], x[e + 5], x[e + 6], x[e + 7]);
                            }
                        }
                    }
                }
            }
            if (tid == 0 && (flags & 1)) set_status(a.status, SPEC_ERR_PAGE);
            if (w.t0 == 0 && !complete)
                open = make_int4(1 + (int)((w.req.tiles - w.nt + w.step - 1) / w.step), w.b, w.unit, 0);
            tc_fence_before();
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (tid == 0) s_flags[u & (kTcUnits - 1)] = 0;
            ++u;
        }
        if (tid == 0) a.open[blockIdx.x] = open;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tc_dealloc(tmem, Sh::kCols);
    }
    if (tid == 0 && s_fail) set_status(a.status, SPEC_ERR_TIMEOUT);
    report_requests<T, KT>(a, c);
}

}  // namespace specv
