// Attention over the paged cache with warp-level matrix instructions
// (mma.sync m16n8k16, 16-bit operands, fp32 sums).
//
// With few query rows a key's bytes are used for few products: one row of a
// head group needs 2 FLOP a byte of cache, 16 rows 32, far below what even the
// warp-level instructions do per byte that HBM brings, so the kernel is built
// around the stream of keys and values:
//   - the unit's keys pass through shared memory in tiles of 64, in a ring of
//     cp.async stages that keeps two or more tiles in flight per block;
//   - WR warps split the query rows, 16 each, and WK warps split a tile's keys;
//     each warp has its own running maximum, sum and output in registers, so a
//     tile costs one barrier; the WK parts are joined when the unit ends;
//   - S = Q K^T has its accumulators laid out as the next product's A operand,
//     so the weights never leave the registers.
// An e4m3 cache is widened to fp16 (exact) on the way from shared memory to the
// operands: its keys' bytes are read 16 at a time in an order that the query rows
// share, and its values are transposed as pairs of bytes.
//
// Measured: one token of 32 requests of 4096 to 32768 positions, 32/8 heads of 128,
// bf16: 357 us for 2.40 GB, 6.7 TB/s (HBM).  Up to 16384 positions: bf16 212 us,
// 6.5 TB/s; e4m3 126 us, 4.5 TB/s, where the widening's instructions are the bound;
// heads of 256 579 us, 4.5 TB/s (one block an SM).  The tensor-core kernel takes 217
// and 150 us for the first two of these.
#pragma once

#include <type_traits>

#include "specv_attend.cuh"

namespace specv {

constexpr int kMmaKeys = 64;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// True if one of the two 16-bit values is an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool any_nonfinite(uint32_t w);
template <>
__device__ __forceinline__ bool any_nonfinite<__nv_bfloat16>(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
template <>
__device__ __forceinline__ bool any_nonfinite<__half>(uint32_t w) {
    return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
}

// Weights are rounded to T for the product with V.  fp16 has a least step of 2^-24:
// the weights are taken times 2^15 (the largest, 1, stays below its 65504), so that
// those down to 2^-29 are rounded to 2^-11 of their own, and the sums of all smaller
// ones are off by 2^-40 of the largest for each.  A long rest far below a few
// dominant keys would be lost otherwise, in the product but not in the sum.  bf16
// has fp32's exponents.  What the weights refer to is the running maximum less 15,
// rounded up: they stay at or below 2^15 where fp32 has steps of more than one.
template <typename T>
__device__ __forceinline__ float reference_of(float top) {
    return std::is_same<T, __half>::value ? __fsub_ru(top, 15.0f) : top;
}

// Four e4m3 values to fp16 (exact).
__device__ __forceinline__ void widen4(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

// Byte offset of 16-byte chunk `ch` of key row `k` in a tile with CH chunks a
// row: the chunk is exchanged within its 128 bytes so that eight adjacent rows
// have the same chunk in eight different bank groups, and (the order of the
// exchange) two adjacent rows have four adjacent chunks in eight.
template <int CH>
__device__ __forceinline__ uint32_t tile_at(int k, int ch) {
    if (CH >= 8) return (uint32_t)(k * CH + (ch ^ (((k & 1) << 2) | ((k >> 1) & 3)))) * 16;
    return (uint32_t)(k * CH + (ch ^ ((k >> 1) & 3))) * 16;
}

// Blocks of an SM, by registers and shared memory.
constexpr int mma_per_sm(bool f8, int dim, int wr) {
    return dim <= 64    ? (wr == 8 ? 2 : f8 ? 4 : 3)
           : dim <= 128 ? (wr == 8 ? 1 : f8 ? 3 : 2)
                        : (wr == 8 || !f8 ? 1 : 2);
}

template <bool F8, int D, int WR, int WK>
struct MmaShape {
    static constexpr int kThreads = 32 * WR * WK;
    static constexpr int kRows = 16 * WR;
    static constexpr int kCh = D * (F8 ? 1 : 2) / 16;              // chunks of a cache row
    static constexpr int kStage = 2 * kMmaKeys * kCh * 16;         // K and V of a tile
    static constexpr int kPerSm = mma_per_sm(F8, D, WR);
    static constexpr int kBudget = 226 * 1024 / kPerSm - 2048;
    static constexpr int kFit = kBudget / kStage;
    static constexpr int kStages = kFit < 6 ? kFit : 6;
    static constexpr int kJoin = 4 * WK * kRows * (D + 4);         // outputs of all warps, fp32
    static constexpr int kSmem = kStages * kStage > kJoin ? kStages * kStage : kJoin;
    static_assert(kStages >= 2, "the ring needs two stages");
};

// T: type of the products, O: type of q and out, F8: e4m3 cache.
template <typename T, typename O, bool F8, int D, int WR, int WK>
__global__ void __launch_bounds__(32 * WR * WK, MmaShape<F8, D, WR, WK>::kPerSm) k_attend_mma(AttendArgs a,
                                                                                            CacheView c) {
    using Sh = MmaShape<F8, D, WR, WK>;
    constexpr int KT = kMmaKeys, THREADS = Sh::kThreads, CH = Sh::kCh, NS = Sh::kStages;
    constexpr int KW = KT / WK;               // keys of a warp
    constexpr int CK = KW < 32 ? KW : 32;     // keys of a softmax step
    constexpr int RG = THREADS / CH, RP = KT / RG;  // loads: row groups, adjacent rows of a thread
    extern __shared__ __align__(128) char smem[];
    __shared__ RunShared<THREADS> s_run;
    __shared__ float s_m[WK][Sh::kRows], s_l[WK][Sh::kRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wr = warp % WR, wk = warp / WR;
    const int g = lane >> 2, t4 = lane & 3;
    const uint32_t sbase = smem_u32(smem);
    const int lch = tid % CH, lrow = tid / CH * RP;  // loads: chunk and first row

    pdl_trigger();
    pdl_wait();
    run_of<KT>(a, c, s_run);
    int4 open = make_int4(0, 0, 0, 0);
    const int dim = c.head_dim;
    const bool has_chunk = lch * 16 < dim * (F8 ? 1 : 2);
    const bool by_group = c.page_size % RP == 0;  // a thread's rows share a page
    Walk<KT> w(a, c, s_run.run);
    while (w.next(a, c)) {
        const Request& req = w.req;
        const int t0 = w.t0, nt = w.nt, h = w.h, r0 = w.r0, R = w.R;
        const int32_t* pages = a.table + (size_t)w.b * a.max_pages;
        bool bad = false;

        // ---- loads of tile t into stage s; `page`: the group's page, fetched a tile ahead
        auto page_of = [&](int t) {
            const int key = tile_key<KT>(req, t) + lrow;
            // a group may begin before the window or behind the end; none of
            // its rows is loaded then
            return key <= req.n + req.ell ? pages[c.by_page.div((uint32_t)key)] : 0;
        };
        auto load = [&](int t, int s, int page) {
            const int key0 = tile_key<KT>(req, t) + lrow;
            const uint32_t dk = sbase + s * Sh::kStage, dv = dk + Sh::kStage / 2;
            const char* src0 = c.k;
            long long off = 0;
            if (by_group) {
                const uint32_t slot = c.by_page.div((uint32_t)min(key0, req.n + req.ell));
                off = (long long)page * c.page + (long long)(key0 - (int)slot * c.page_size) * c.token;
            }
            off += h * c.head + lch * 16;
#pragma unroll
            for (int i = 0; i < RP; ++i) {
                const int key = key0 + i;
                bool take = has_chunk && any_sees(a, req, key);
                long long at = off + i * c.token;
                if (!by_group) {
                    if (take) {
                        const uint32_t slot = c.by_page.div((uint32_t)key);
                        page = pages[slot];
                        at = (long long)page * c.page + (long long)(key - (int)slot * c.page_size) * c.token +
                             h * c.head + lch * 16;
                    }
                }
                if (take && (page < 0 || page >= c.pages)) {
                    bad = true;
                    take = false;
                }
                const uint32_t to = tile_at<CH>(lrow + i, lch);
                cp_async16(dk + to, take ? c.k + at : src0, take);
                cp_async16(dv + to, take ? c.v + at : src0, take);
            }
        };

        int page = page_of(t0);
#pragma unroll
        for (int s = 0; s < NS - 1; ++s) {
            if (s < nt) {
                const int now = page;
                if (s + 1 < nt) page = page_of(t0 + s + 1);
                load(t0 + s, s, now);
            }
            cp_async_commit();
        }

        // ---- query rows of the warp, as A operands; rows behind the last are zero
        uint32_t qf[D / 16][4];
        float rs[2];
        int pos[2];
        {
            const int row_a = r0 + wr * 16 + g;
            const char* qp[2];
            bool have[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = row_a + 8 * i;
                have[i] = wr * 16 + g + 8 * i < R;
                const int j = have[i] ? (int)a.by_group.div((uint32_t)r) : 0;
                const int head = h * a.group + (have[i] ? r - j * a.group : 0);
                qp[i] = a.q + (long long)(req.base + j) * a.q_row + head * a.q_head;
                pos[i] = have[i] ? req.n + j : req.n + req.ell;
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // e4m3: a thread's 16 adjacent bytes of a key are its operands of
                    // four products, four bytes each
                    const int d = F8 ? (kk >> 2) * 64 + t4 * 16 + (kk & 3) * 4 + (i >> 1) * 2
                                     : kk * 16 + 2 * t4 + (i >> 1) * 8;
                    qf[kk][i] = have[i & 1] && d < dim ? *(const uint32_t*)(qp[i & 1] + d * 2) : 0u;
                }
            rs[0] = rs[1] = a.scale * (F8 && c.k_scale ? c.k_scale[h] : 1.0f);
            if (!std::is_same<T, O>::value) {
                // bf16 rows under fp16 products: each row is scaled by a power of
                // two that brings its largest value into [1, 2), exactly but for
                // values 2^-14 below it, which lose bits that are 2^-25 of it
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = 0.0f;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int x = i; x < 4; x += 2)
                            top = fmaxf(top, fmaxf(fabsf(bf16_lo(qf[kk][x])), fabsf(bf16_hi(qf[kk][x]))));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // exponent of the largest value, kept where its inverse is a normal number
                    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -126), 126);
                    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                    rs[i] *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int x = i; x < 4; x += 2)
                            qf[kk][x] = pack2<__half>(bf16_lo(qf[kk][x]) * down, bf16_hi(qf[kk][x]) * down);
                }
            }
        }

        float acc[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        for (int t = 0; t < nt; ++t) {
            cp_async_wait<NS - 2>();
            __syncthreads();  // tile t is there, and stage (t - 1) % NS is free
            {
                const int nx = t + NS - 1;
                if (nx < nt) {
                    const int now = page;
                    if (nx + 1 < nt) page = page_of(t0 + nx + 1);
                    load(t0 + nx, nx % NS, now);
                }
                cp_async_commit();
            }
            const int key0 = tile_key<KT>(req, t0 + t);
            const uint32_t sk = sbase + (t % NS) * Sh::kStage, sv = sk + Sh::kStage / 2;

            const bool part = !all_see<KT>(a, req, key0);
            bool dirty = false;
            if (part) {
                // values that are not finite, at keys that only some rows see,
                // must not meet a weight of zero: they are taken out of the
                // product and added by themselves to the rows that see them
                for (int i = tid; i < KT * CH; i += THREADS) {
                    uint32_t x[4];
                    const uint32_t at = sv + tile_at<CH>(i / CH, i % CH);
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                 : "r"(at)
                                 : "memory");
                    bool any = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (F8) {  // the bytes 7f and ff
                            const uint32_t nan = ((x[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                            any |= nan != 0;
                            x[e] &= ~((nan >> 7) * 0xffu);
                        } else if (any_nonfinite<T>(x[e])) {
                            any = true;
                            if (any_nonfinite<T>(x[e] & 0xffffu)) x[e] &= 0xffff0000u;
                            if (any_nonfinite<T>(x[e] & 0xffff0000u)) x[e] &= 0xffffu;
                        }
                    if (any) {
                        dirty = true;
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x[0]), "r"(x[1]),
                                     "r"(x[2]), "r"(x[3])
                                     : "memory");
                    }
                }
                dirty = __syncthreads_or(dirty);
            }

#pragma unroll
            for (int ck = 0; ck < KW; ck += CK) {
                const int k0 = wk * KW + ck;  // first key of the step within the tile
                float s[CK / 8][4];
#pragma unroll
                for (int n = 0; n < CK / 8; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
                if (F8) {
#pragma unroll
                    for (int j = 0; j < D / 64; ++j)
#pragma unroll
                        for (int n = 0; n < CK / 8; ++n) {
                            uint32_t x[4];
                            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                         : "r"(sk + tile_at<CH>(k0 + n * 8 + g, 4 * j + t4))
                                         : "memory");
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                uint32_t b0, b1;
                                widen4(x[q], b0, b1);
                                mma16816<T>(s[n], qf[4 * j + q], b0, b1);
                            }
                        }
                } else {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int n = 0; n < CK / 16; ++n) {
                            uint32_t b[4];
                            const int i = lane >> 3;
                            ldsm4(b, sk + tile_at<CH>(k0 + n * 16 + (i >> 1) * 8 + (lane & 7), kk * 2 + (i & 1)));
                            mma16816<T>(s[2 * n], qf[kk], b[0], b[1]);
                            mma16816<T>(s[2 * n + 1], qf[kk], b[2], b[3]);
                        }
                }
                // scores to base 2, masked where the tile is cut by a border
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < CK / 8; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[n][i] *= rs[i >> 1];
                        if (part && !sees(a, pos[i >> 1], key0 + k0 + n * 8 + 2 * t4 + (i & 1))) s[n][i] = -INFINITY;
                        top[i >> 1] = fmaxf(top[i >> 1], s[n][i]);
                    }
                float base[2];
                bool up = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                    top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
                    up |= top[i] > m[i];
                    top[i] = fmaxf(top[i], m[i]);
                    base[i] = top[i] == -INFINITY ? 0.0f : reference_of<T>(top[i]);
                }
                if (__any_sync(0xffffffffu, up)) {  // a new maximum: what there is shrinks
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float corr = ex2_approx(reference_of<T>(m[i]) - base[i]);
                        l[i] *= corr;
                        m[i] = top[i];
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            acc[n][2 * i] *= corr;
                            acc[n][2 * i + 1] *= corr;
                        }
                    }
                }
                // weights (see reference_of); their sum is of the unrounded ones.  For
                // the product they are rounded to T: 2^-8 (bf16) or 2^-11 of each at
                // most, as much as the output's own rounding
#pragma unroll
                for (int n = 0; n < CK / 8; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[n][i] = ex2_approx(s[n][i] - base[i >> 1]);
                        l[i >> 1] += s[n][i];
                    }
#pragma unroll
                for (int n = 0; n < CK / 16; ++n) {
                    const uint32_t p[4] = {pack2<T>(s[2 * n][0], s[2 * n][1]), pack2<T>(s[2 * n][2], s[2 * n][3]),
                                           pack2<T>(s[2 * n + 1][0], s[2 * n + 1][1]),
                                           pack2<T>(s[2 * n + 1][2], s[2 * n + 1][3])};
                    const int i = lane >> 3, row = k0 + n * 16 + (i & 1) * 8 + (lane & 7);
                    if (F8) {
                        // pairs of bytes transposed: a register has two keys' values of
                        // two adjacent columns, which go to two products
#pragma unroll
                        for (int dt = 0; dt < D / 32; ++dt) {
                            uint32_t b[4], even[4], odd[4];
                            ldsm4_t(b, sv + tile_at<CH>(row, dt * 2 + (i >> 1)));
#pragma unroll
                            for (int q = 0; q < 4; ++q) widen4(__byte_perm(b[q], 0, 0x3120), even[q], odd[q]);
                            mma16816<T>(acc[4 * dt], p, even[0], even[1]);
                            mma16816<T>(acc[4 * dt + 1], p, odd[0], odd[1]);
                            mma16816<T>(acc[4 * dt + 2], p, even[2], even[3]);
                            mma16816<T>(acc[4 * dt + 3], p, odd[2], odd[3]);
                        }
                    } else {
#pragma unroll
                        for (int dt = 0; dt < D / 16; ++dt) {
                            uint32_t b[4];
                            ldsm4_t(b, sv + tile_at<CH>(row, dt * 2 + (i >> 1)));
                            mma16816<T>(acc[2 * dt], p, b[0], b[1]);
                            mma16816<T>(acc[2 * dt + 1], p, b[2], b[3]);
                        }
                    }
                }
                if (dirty) {
                    for (int k = 0; k < CK; ++k) {
                        const int key = key0 + k0 + k;
                        if (!any_sees(a, req, key)) continue;
                        const long long at = key_at(a, c, pages, key);
                        if (at < 0) continue;
                        const char* v = c.v + at + h * c.head;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int d = F8 ? (n >> 1) * 16 + 4 * t4 + 2 * (i & 1) + (n & 1)
                                                 : n * 8 + 2 * t4 + (i & 1);
                                if (d >= dim || !sees(a, pos[i >> 1], key)) continue;
                                const float x = F8 ? to_f32(((const __nv_fp8_e4m3*)v)[d]) : to_f32(((const T*)v)[d]);
                                if (!(fabsf(x) <= 3.4e38f)) acc[n][i] += x;
                            }
                    }
                }
            }
        }

        // ---- the unit's end: join the WK warps of each row through shared memory
        cp_async_wait<0>();
        if (__syncthreads_or(bad)) {
            l[0] = l[1] = __int_as_float(0x7fc00000);
            if (tid == 0) set_status(a.status, SPEC_ERR_PAGE);
        }
        float* so = (float*)smem + (size_t)wk * Sh::kRows * (D + 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            const int r = wr * 16 + g + 8 * i;
            if (t4 == 0) {
                s_m[wk][r] = reference_of<T>(m[i]);
                s_l[wk][r] = l[i];
            }
            if (F8) {
#pragma unroll
                for (int n = 0; n < D / 8; n += 2)
                    *(float4*)(so + r * (D + 4) + n * 8 + 4 * t4) =
                        make_float4(acc[n][2 * i], acc[n + 1][2 * i], acc[n][2 * i + 1], acc[n + 1][2 * i + 1]);
            } else {
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *(float2*)(so + r * (D + 4) + n * 8 + 2 * t4) = make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
            }
        }
        __syncthreads();
        const bool whole = w.whole();
        float* out = part_at(a, blockIdx.x, t0 == 0 ? 1 : 0);
        const float vs = F8 && c.v_scale ? c.v_scale[h] : 1.0f;
        for (int r = warp; r < R; r += THREADS / 32) {
            float M = -INFINITY, L = 0.0f, part[WK];
#pragma unroll
            for (int k = 0; k < WK; ++k) M = fmaxf(M, s_m[k][r]);
            const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
            for (int k = 0; k < WK; ++k) {
                part[k] = WK == 1 ? 1.0f : ex2_approx(s_m[k][r] - base);
                L += part[k] * s_l[k][r];
            }
            const long long row = out_row(a, req.base, h, r0 + r);
            const float inv = whole ? vs / L : vs;
            for (int d = 2 * lane; d < dim; d += 64) {
                float x = 0.0f, y = 0.0f;
#pragma unroll
                for (int k = 0; k < WK; ++k) {
                    const float2 o = *(const float2*)((float*)smem + ((size_t)k * Sh::kRows + r) * (D + 4) + d);
                    x += part[k] * o.x;
                    y += part[k] * o.y;
                }
                if (whole) *(uint32_t*)((char*)a.out + (row * dim + d) * 2) = pack2<O>(x * inv, y * inv);
                else *(float2*)(out + r * dim + d) = make_float2(x * inv, y * inv);
            }
            if (lane == 0) {
                if (!whole) {
                    out[a.tile_rows * dim + r] = M;
                    out[a.tile_rows * (dim + 1) + r] = L;
                } else if (a.lse) {
                    a.lse[row] = (M + log2f(L)) * 0.6931471805599453f;
                }
            }
        }
        __syncthreads();  // the stages are free for the next unit
        if (t0 == 0 && !whole) open = w.open();
    }
    if (tid == 0) a.open[blockIdx.x] = open;
    report_requests<O, KT>(a, c, THREADS);
}

// ------------------------------------------------------------------- launch
template <typename T, typename O, bool F8, int D, int WR, int WK>
int mma_launch(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    using Sh = MmaShape<F8, D, WR, WK>;
    auto* f = k_attend_mma<T, O, F8, D, WR, WK>;
    static std::atomic<unsigned long long> done{0};
    if (const int rc = allow_smem((const void*)f, Sh::kSmem, done)) return rc;
    return launch_dependent(f, dim3(blocks), Sh::kThreads, Sh::kSmem, st, 0, a, c);
}

template <typename T, typename O, bool F8, int D>
int mma_launch_rows(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    switch (a.tile_rows) {
        case 16: return mma_launch<T, O, F8, D, 1, 4>(a, c, blocks, st);
        case 32: return mma_launch<T, O, F8, D, 2, 2>(a, c, blocks, st);
        case 64: return mma_launch<T, O, F8, D, 4, 1>(a, c, blocks, st);
        default: return mma_launch<T, O, F8, D, 8, 1>(a, c, blocks, st);
    }
}

template <typename T, typename O, bool F8>
int mma_launch_dim(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    if (c.head_dim <= 64) return mma_launch_rows<T, O, F8, 64>(a, c, blocks, st);
    if (c.head_dim <= 128) return mma_launch_rows<T, O, F8, 128>(a, c, blocks, st);
    return mma_launch_rows<T, O, F8, 256>(a, c, blocks, st);
}

}  // namespace specv
