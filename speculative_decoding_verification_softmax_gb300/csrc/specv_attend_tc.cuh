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
// work for the other.  Each stream has its own O columns in TMEM and its own
// running maximum and sum; the unit's end joins them.  Scores have two places (three
// for heads of 64, for which TMEM has room), taken by the tiles in turn; P overlays S.
//   warps 0-3, 4-7   softmax of the even and odd tiles, a row a thread; the
//                    unit's output
//   warps 8-11       the next unit's query rows; 16-bit cache: repair of V tiles
//                    that a border cuts; e4m3 cache: the widening of all tiles
//                    to fp16 (exact; an item takes 700 to 1500 cycles, mostly latency,
//                    so two pairs or four warps have one each under way)
//   warp 13          the block's units, told to all others through a ring, so
//                    that none waits for a request's lengths between two units
//   warps 14, 12     K and V tiles by TMA, in the order of their use, through a
//                    ring of shared-memory slots that runs on over the units
//                    (two warps: a box takes 100 cycles to issue, and a tile of
//                    pages of 16 tokens is 8 boxes or 16)
//   warp 15          one thread issues all matrix instructions
// A TMA box is as many tokens as always lie in one page.  In V tiles that some
// query row must not see whole (the cache's end, the window's edges), rows that
// nobody sees become zero, and a value that is not finite is taken out and added
// by itself to the rows that see it.
//
// Measured: 64 requests of 500 to 8192 positions, blocks of 16 drafts, 32/8 heads
// of 128, bf16: 200 us for 1.22 GB, 6.1 TB/s (HBM; 10% go to the switches between
// units).  19 requests of 16384 positions: 190 us, 6.7 TB/s; heads of 64 100 us,
// 6.4 TB/s (127 with two places for scores).  e4m3 is bound by the softmax and the
// widening instead: 106 us (heads of 64) and 148 to 167 us (128) there; ragged windows
// of 4000, 28/4 heads of 64, pages of 16: 62 us for 116 MB (fp16 cache 55 us).
//
// SH: the units are those of a plan's items (specv_share.cu), whose query rows may be any
// requests'.  64 x 17 rows behind 8192 shared positions, 32/8 heads of 128, bf16: 163 us,
// 1,006 TFLOP/s; 240 x 4 rows over three prefixes of 32768: 128 us, 945.  Bound by the two
// streams' chains: of the 1,700 to 1,800 cycles of a tile the products are 1,024, and a
// stream has scores 1,400 cycles after it has handed its weights over and weights
// 2,000 cycles after that.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "specv_attend.cuh"

namespace specv {

constexpr int kTcKeys = 128;
constexpr int kTcRows = 128;
constexpr int kTcThreads = 16 * 32;
constexpr int kTcUnits = 8;  // ring of units under way

// The weights' reference is the running maximum, and stays until it is passed by
// kTcSlack (to base 2): weights reach 2^kTcSlack instead of 1, exactly as well in 16
// bits, and the output in TMEM is scaled again a few times a unit instead of every
// tile.  fp16 weights (the least step is 2^-24) have a reference kTcUp below it, and
// reach 2^15: those down to 2^-25 of the maximum are rounded to 2^-11 of their own,
// smaller ones to 2^-36 of it.  Without it a long rest far below a few dominant keys
// was lost, in the product but not in the sum.  Maximum and reference are rounded up,
// the limit down: no weight passes 2^15 where fp32 has steps of more than one.
template <typename T>
constexpr float kTcSlack = std::is_same<T, __half>::value ? 4.0f : 8.0f;
template <typename T>
constexpr float kTcUp = std::is_same<T, __half>::value ? 11.0f : 0.0f;
// From this score on (fp32 has steps of 2^-4 there, for bf16 of 2) the products of the
// matrix instructions are scaled and rounded before the reference is taken from them:
// in one fused operation with it they would differ from their rounded maximum by more
// than the weights' type holds (beyond 2^28, bf16 2^31).
template <typename T>
constexpr float kTcFine = std::is_same<T, __half>::value ? 1048576.0f : 33554432.0f;

// Shared memory: query rows, slots of 16-bit K or V tiles, and for an e4m3
// cache the slots in which its tiles arrive.  The copies in flight cover HBM's
// latency: 96 KB or more of 16-bit tiles, 64 KB or more of e4m3 ones.
template <bool F8, int D>
struct TcShape {
    static constexpr int kPanel = kTcKeys * 128;     // 64 columns of a tile, 128-byte rows
    static constexpr int kTile = kPanel * (D / 64);  // K or V of a tile
    static constexpr int kRawTile = kTcKeys * D;
    static constexpr int kSlots = F8 ? (D == 64 ? 6 : 3) : (D == 64 ? 12 : 6);
    static constexpr int kRaw = F8 ? (D == 64 ? 10 : 5) : 0;
    static constexpr int kQ = kTcRows * 128 * (D / 64);
    // threads that widen or repair a tile: with slots enough for four tiles under
    // way, each warp has its own
    static constexpr int kWideners = F8 && kSlots >= 6 ? 32 : 64;
    static constexpr int kTeams = 128 / kWideners;
    static constexpr int kSmem = 1024 + kQ + kSlots * kTile + kRaw * kRawTile;
    // beside it, barriers, units and weights have to fit 227 KB: 1,808 to 1,968 bytes,
    // over e4m3 (with the rows' scales of bf16) 2,816 to 2,960
    static_assert(kSmem + (F8 ? 3 : 2) * 1024 <= 227 * 1024, "shared memory of an SM");
    // Tiles whose scores are under way, each in TMEM columns of its own: the scores
    // of tile i are taken before the products with V of tile i - kAhead.  A third
    // one, for which heads of 64 leave room, lets a stream find its next scores
    // ready when it has handed over its weights.
    static constexpr int kAhead = D == 64 ? 3 : 2;
    // A wait on a slot's parity passes at once while the slot is two uses behind, so
    // whoever waits has to know that the use before is over.  A team of wideners
    // knows it of items kSlots before its last one (the products take items in order),
    // which is enough if there are no more teams than slots; a loader of what the
    // wideners gave back before its own last item, which is up to kAhead + 1 items
    // ago (2 within a unit): with two teams, its slot's own team among them.
    // The same holds for o_done: a stream that scales its output at tile t waits for
    // its product of tile t - 2, and knows that of t - 4 to be over from the scores of
    // t, which follow the product of t - kAhead, or from the end of the unit before.
    static_assert(kAhead <= 4, "phases of o_done");
    static_assert(!F8 || kTeams <= kSlots, "slots of the wideners");
    static_assert(F8 || kAhead + 1 <= kSlots, "slots of the loaders");
    static_assert(!F8 || kRaw >= kSlots + kAhead + 1 || (kTeams == 2 && kAhead == 2 && kRaw >= kSlots + 2),
                  "slots of the loaders");
    static constexpr int kCols = 512;  // TMEM columns: scores, O0, O1 (a power of two)
    static_assert(kAhead * kTcKeys + 2 * D <= kCols, "columns of TMEM");
};

struct TcArgs {
    int box, shift;    // tokens of a TMA box, 2^shift
    int expire_first;  // test hook: the products' first wait counts as run out (0 in normal use)
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
// Matrix instructions, called by a whole warp and issued by the one thread with
// `issue`: the operands stay in the warp's uniform registers.
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void tc_mma_ss(uint32_t issue, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u), "r"(issue)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t issue, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u), "r"(issue)
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t issue, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(issue)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// 32 columns of the warp's 32 lanes; the values are there after tc_wait32.
__device__ __forceinline__ void tc_ld32(float (&x)[32], uint32_t at) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
// Waits for the warp's loads; names the values, so that no use moves above it.
__device__ __forceinline__ void tc_wait32(float (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]),
          "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15]),
          "+f"(x[16]), "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]), "+f"(x[22]), "+f"(x[23]),
          "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29]), "+f"(x[30]), "+f"(x[31])
        :
        : "memory");
}
// Eight columns from each of two places, and the wait for them.
__device__ __forceinline__ void tc_ld8(float (&x)[8], float (&y)[8], uint32_t at, uint32_t at2) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(y[0]),
          "=f"(y[1]), "=f"(y[2]), "=f"(y[3]), "=f"(y[4]), "=f"(y[5]), "=f"(y[6]), "=f"(y[7])
        : "r"(at), "r"(at2)
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

template <int N>
__device__ __forceinline__ void tc_more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void tc_fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
// ends, without results, and the block returns.  No slot that TMA fills is loaded
// again then: one that looked free while its copy is under way would get an arrival
// too many.  Wideners and loaders remember the first such wait of their own (a phase
// that was skipped lets a later wait on its parity pass); the products go on giving
// slots back (to end them cost 4% at 119 rows), so over a 16-bit cache the loaders,
// who take those, look at `fail` behind each wait.  The waiting thread is suspended
// for up to 20 us at a time and looks at the clock every 16th time only:
// spinning on the clock slowed the softmax warps' exponentials several times over.
__device__ __forceinline__ bool tc_try(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* fail) {
    if (tc_try(bar, parity)) return true;
    unsigned long long t0 = 0;
    for (uint32_t n = 1;; ++n) {
        if (tc_try(bar, parity)) return true;
        if (*fail) return false;
        if ((n & 15) == 0) {
            const unsigned long long now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) {
                *fail = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ uint32_t panel_at(int row, int chunk) {  // byte of a 16-byte chunk, 8 a panel row
    return (uint32_t)((chunk >> 3) * (128 * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

// Item i of a unit of nt tiles, in the order of use: K0, K1, V0, K2, V1, ... where
// K is two tiles ahead.
template <int AHEAD>
__device__ __forceinline__ void item_of(int i, int nt, bool& is_v, int& t) {
    const int first = min(AHEAD, nt), x = i - first, pairs = 2 * (nt - first);
    is_v = x >= pairs || (x >= 0 && (x & 1) == 0);
    t = x < 0 ? i : x >= pairs ? nt - first + (x - pairs) : is_v ? x >> 1 : (x >> 1) + first;
}

// Bits lo .. hi - 1 of a word, for any lo and hi.
__device__ __forceinline__ uint32_t bits_of(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 32);
    return lo >= hi ? 0u : (0xffffffffu << lo) & (0xffffffffu >> (32 - hi));
}
// Which of the 32 positions from `key` the row at position p sees.
__device__ __forceinline__ uint32_t seen_bits(const AttendArgs& a, int p, int key) {
    const int hi = min(p - key + 1, 32);
    if (a.window == 0) return bits_of(0, hi);
    // p - t < window, without an overflow for any window
    const int lo = p >= a.window ? p - a.window + 1 - key : 0;
    return bits_of(lo, hi) | bits_of(0, min(hi, a.sinks > key ? min(a.sinks - key, 32) : 0));
}

template <typename T>
__device__ __forceinline__ uint32_t tc_pack(float lo, float hi) {
    uint32_t r;
    if (std::is_same<T, __half>::value) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Sets the values of a word that are not finite (two 16-bit or four e4m3 ones: all
// bits of the exponent, or of all but the sign, set) to zero.  Adding the lowest of
// these bits carries into the sign's place, and no further.
template <typename T, bool F8>
__device__ __forceinline__ uint32_t finite_of(uint32_t w) {
    constexpr uint32_t bits = F8 ? 0x7f7f7f7fu : std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    constexpr uint32_t low = F8 ? 0x01010101u : std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    const uint32_t m = ((w & bits) + low) & (F8 ? 0x80808080u : 0x80008000u);
    return w & ~(F8 ? (m >> 7) * 0xffu : (m >> 15) * 0xffffu);
}

// The part of a V tile from key key0 on that a thread has in shared memory: of the
// rows k, k + STEP, ... 16 bytes each, at at(row).  What no query row sees becomes
// zero, and so do values that are not finite where only some see them; true if
// there were such.  Short loops over just these rows: the tile waits for them.
template <typename T, bool F8, int KT, int STEP, typename At>
__device__ __forceinline__ bool repair(const AttendArgs& a, const Request& req, int key0, int k, At at) {
    const int end = req.n + req.ell;
    bool dirty = false;
    // behind the end, and between the sinks and the window; then what only some of
    // the rows see: their own positions, and the first ones of their windows
#pragma unroll 1
    for (int i = 0; i < (a.window > 0 ? 4 : 2); ++i) {
        const bool some = i & 1;
        int from, to;  // in the tile
        if (i < 2) {
            from = (some ? req.n : end) + 1 - key0;
            to = some ? end + 1 - key0 : KT;
        } else {
            from = max(a.sinks, some ? req.n - a.window + 1 : 0) - key0;
            to = max((some ? end : req.n) - a.window + 1, 0) - key0;
        }
        from = max(from, 0);
        to = min(to, KT);
        from += (k - from) & (STEP - 1);  // the thread's first row from there on
#pragma unroll 1
        for (int r = from; r < to; r += STEP) {
            uint4 z = make_uint4(0u, 0u, 0u, 0u);
            if (some) {
                const uint4 v = lds16(at(r));
                z = make_uint4(finite_of<T, F8>(v.x), finite_of<T, F8>(v.y), finite_of<T, F8>(v.z),
                               finite_of<T, F8>(v.w));
                if (z.x == v.x && z.y == v.y && z.z == v.z && z.w == v.w) continue;
                dirty = true;
            }
            sts16(at(r), z);
        }
    }
    return dirty;
}

// Two fp32 operations of one instruction.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 of_two(Two v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The weights of 32 scores: their sums (four, so that few additions wait for one
// another), and rounded to T into 16 columns.
template <typename T>
__device__ __forceinline__ void weigh(float (&x)[32], Two scale, Two ref, Two& sum0, Two& sum1, uint32_t to) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const float2 v = of_two(fma2(two(x[e], x[e + 1]), scale, ref));
        x[e] = v.x;
        x[e + 1] = v.y;
    }
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const float v0 = ex2_approx(x[e]), v1 = ex2_approx(x[e + 1]);
        Two& sum = e & 2 ? sum1 : sum0;
        sum = add2(sum, two(v0, v1));
        p[e >> 1] = tc_pack<T>(v0, v1);
    }
    tc_st16(to, p);
}

// Four e4m3 values to fp16 (exact).
__device__ __forceinline__ void tc_widen(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

// A unit (a segment of the block's run) as the roles read it; nt = 0 ends the
// run.
struct Unit {
    int n, ell, base, b;
    int sink_tiles, first_tile, t0, nt;
    int h, r0, skip;  // SH: skip, and b | kind << 16
    int rows_parts;  // rows R, and the parts if the unit is left open here << 8, -1 if it is whole

    __device__ __forceinline__ int rows() const { return rows_parts & 255; }
    __device__ __forceinline__ int parts() const { return rows_parts >> 8; }

    __device__ __forceinline__ Request request() const {
        Request r;
        r.n = n;
        r.ell = ell;
        r.base = base;
        r.b = b & 0xffff;
        r.kind = b >> 16;
        r.skip = skip;
        r.sink_tiles = sink_tiles;
        r.first_tile = first_tile;
        return r;
    }
};

// True in all `threads` threads of named barrier `id` if it is in each: roles of
// several warps that meet at barriers go on to the next unit, or end, together.
__device__ __forceinline__ bool all_agree(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(x ? 1u : 0u)
        : "memory");
    return r != 0;
}

// A role's view of the ring: next() waits for the next unit, done() gives the
// last one's place back (each role's warps once).  After a wait that ran out of
// time there is no next unit.
struct Units {
    const Unit* ring;
    uint64_t* full;
    uint64_t* empty;
    volatile int* fail;
    int u;
    Request req;
    int b, t0, nt, h, r0, R;

    __device__ __forceinline__ Units(const Unit* r, uint64_t* f, uint64_t* e, volatile int* x)
        : ring(r), full(f), empty(e), fail(x), u(-1) {}
    __device__ __forceinline__ bool next() {
        ++u;
        if (!__all_sync(0xffffffffu, tc_wait(&full[u % kTcUnits], (u / kTcUnits) & 1, fail))) return false;
        const Unit& s = ring[u % kTcUnits];
        nt = s.nt;
        if (nt == 0) return false;
        req = s.request();
        b = s.b;
        t0 = s.t0;
        h = s.h;
        r0 = s.r0;
        R = s.rows();
        return true;
    }
    __device__ __forceinline__ const Unit& now() const { return ring[u % kTcUnits]; }
    __device__ __forceinline__ void done() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[u % kTcUnits]);
    }
};

struct Eight {
    float x[8];
};

// The sums of the values that are not finite, of columns col .. col + 7, of the
// keys that the row at position p sees in the tiles of a segment that a border
// cuts.
template <typename T, bool F8, int KT, bool SH>
__device__ __noinline__ Eight sum_nonfinite(const AttendArgs& a, const CacheView& c, Unit w, int p, int col) {
    const Request req = w.request();
    Eight sum = {};
    const int32_t* pages = pages_of<SH>(a, req, w.b);
    for (int t = 0; t < w.nt; ++t) {
        const int key0 = tile_key<KT>(req, w.t0 + t);
        if (all_see<KT>(a, req, key0)) continue;
        for (int k = key0; k < key0 + KT && k <= p; ++k) {
            if (!sees(a, p, k)) continue;
            const long long at = key_at(a, c, pages, k);
            if (at < 0) continue;
            const char* v = c.v + at + w.h * c.head;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = F8 ? to_f32(((const __nv_fp8_e4m3*)v)[col + e]) : to_f32(((const T*)v)[col + e]);
                if (!(fabsf(z) <= 3.4e38f)) sum.x[e] += z;
            }
        }
    }
    return sum;
}

// Scales a row's scores where they are; the largest one.
static __device__ __noinline__ float scale_scores(uint32_t ts, float by) {
    float x[32], top = -INFINITY;
#pragma unroll 1
    for (int q = 0; q < kTcKeys / 32; ++q) {
        tc_ld32(x, ts + q * 32);
        tc_wait32(x);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            x[e] *= by;
            top = fmaxf(top, x[e]);
        }
        tc_st32(ts + q * 32, x);
    }
    tc_wait_st();
    return top;
}

// T: type of the products, O: type of q and out, F8: e4m3 cache.
template <typename T, typename O, bool F8, int D, bool SH>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_attend_tc(const __grid_constant__ AttendArgs a, const __grid_constant__ CacheView c, TcArgs tc,
                const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv) {
    using Sh = TcShape<F8, D>;
    constexpr int KT = kTcKeys, NS = Sh::kSlots, NB = Sh::kAhead, CW = D / 8;  // CW: 16-byte chunks of a row
    constexpr int NR = F8 ? Sh::kRaw : NS;                    // slots that TMA fills
    extern __shared__ char smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], empty[NS], raw_full[NR], raw_empty[F8 ? NR : 1];
    __shared__ __align__(8) uint64_t s_full[NB], p_full[NB], o_done[2], o_all, q_full, q_empty, drain;
    __shared__ __align__(8) uint64_t unit_full[kTcUnits], unit_empty[kTcUnits];
    __shared__ __align__(16) Unit s_units[kTcUnits];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail, s_flags[kTcUnits];
    // the run, until warp 13 has read it; then (a unit has come from it and ended)
    // the second stream's maxima and sums, the streams' weights
    __shared__ union {
        RunShared<kTcThreads> run;
        float ml[2][kTcRows];
    } s_of;
    auto& s_ml = s_of.ml;
    __shared__ float s_row[2][std::is_same<T, O>::value ? 1 : kTcRows];  // scales of two units' query rows
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    const uint32_t sq = base, ring = base + Sh::kQ, raws = ring + NS * Sh::kTile;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NR; ++i) {
            mbar_init(&raw_full[i], 1);
            if (F8) mbar_init(&raw_empty[i], 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&o_done[i], 1);
        mbar_init(&o_all, 1);
        mbar_init(&q_full, 4);
        for (int i = 0; i < kTcUnits; ++i) {
            mbar_init(&unit_full[i], 1);
            mbar_init(&unit_empty[i], 15);
        }
        mbar_init(&q_empty, 1);
        mbar_init(&drain, 1);
        fence_mbar_init();
        s_fail = 0;
    }
    // TMEM is taken behind the wait, and the next kernel may be placed only then:
    // kernels beside one another, of which one waits for the other, could each
    // hold columns that the other needs
    pdl_wait();
    if (warp == 15) tc_alloc(&s_tmem, Sh::kCols);
    tc_fence_before();
    run_of<KT, SH>(a, c, s_of.run);  // also the barrier behind the set-up
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = s_tmem;
    volatile int* fail = &s_fail;

    // registers: the softmax warps' shares are 168, the others' 88, together
    // what the block was launched with (512 threads of 128).  No warp takes
    // registers again afterwards: one that finished early could take those that
    // the softmax warps still wait for
    if (warp >= 8) {
    tc_fewer_registers<88>();
    if (warp == 12 || warp == 14) {
        // --------------------------------- TMA: K by warp 14, V by warp 12
        // The warp's lanes are the boxes of a group of tiles, whose pages are read
        // while those of the group before are used: the table's round trip would
        // otherwise be the rate of the tiles.
        const bool is_v = warp == 12;
        const int boxes = KT >> tc.shift, group = 32 / boxes;  // boxes of a tile, tiles of a group
        const int of = lane / boxes, row = (lane & (boxes - 1)) << tc.shift;  // the lane's tile and first row
        const CUtensorMap* map = is_v ? &mv : &mk;
        uint32_t before = 0, issued = 0;  // items of the units before, items issued
        bool ok = true;  // no wait for a slot has run out, see tc_wait
        Units w(s_units, unit_full, unit_empty, fail);
        while (w.next()) {
            const int32_t* pages = pages_of<SH>(a, w.req, w.b);
            const int end = w.req.n + w.req.ell, first = min(NB, w.nt);
            int page = 0, token = 0, page1 = 0, token1 = 0;
            bool need = false, need1 = false;  // some row sees some of the box
            auto fetch = [&](int t) {
                need1 = t < w.nt;
                if (!need1) return;
                const int k = tile_key<KT>(w.req, w.t0 + t) + row;
                const int last = min(k + tc.box - 1, end);
                need1 = k <= end && (a.window == 0 || w.req.n - last < a.window || k < a.sinks);
                if (!need1) return;
                const int p = (int)c.by_page.div((uint32_t)k);
                token1 = k - p * c.page_size;
                page1 = pages[p];
            };
            fetch(of);
#pragma unroll 1
            for (int t = 0; t < w.nt; ++t) {
                if ((t & (group - 1)) == 0) {
                    page = page1;
                    token = token1;
                    need = need1;
                    fetch(t + group + of);
                }
                // the tile's place in the order of the items
                const uint32_t item =
                    before + (is_v ? t < w.nt - first ? first + 2 * t : w.nt + t : t < first ? t : 2 * t - first + 1);
                const int slot = (int)(item % NR);
                bool have = need && of == (t & (group - 1));
                if (have && (uint32_t)page >= (uint32_t)c.pages) {
                    atomicOr(&s_flags[w.u % kTcUnits], 1);
                    have = false;
                }
                uint64_t* freed = F8 ? &raw_empty[slot] : &empty[slot];
                ok = ok && __all_sync(0xffffffffu, (item < NR || tc_wait(freed, ((item / NR) & 1) ^ 1, fail)) &&
                                                       (F8 || !*fail));
                // a 16-bit tile is ready when it has landed, unless it is to be repaired
                uint64_t* bar = F8 || (is_v && !all_see<KT>(a, w.req, tile_key<KT>(w.req, w.t0 + t)))
                                    ? &raw_full[slot]
                                    : &full[slot];
                have = have && ok;
                const int n = __popc(__ballot_sync(0xffffffffu, have));
                __syncwarp();  // what the lanes said of their pages is known before the tile is there
                // without its slot a tile is left out: an arrival on a barrier that waits for
                // an earlier copy would be one too many
                if (lane == 0 && ok) mbar_arrive_expect_tx(bar, (uint32_t)n * tc.box * (F8 ? D : 2 * D));
                __syncwarp();
                if (have) {
                    if (F8) {
                        tma_box(raws + slot * Sh::kRawTile + row * D, map, 0, token, w.h, page, bar);
                    } else {
#pragma unroll
                        for (int p = 0; p < D / 64; ++p)
                            tma_box(ring + slot * Sh::kTile + p * Sh::kPanel + row * 128, map, p * 64, token, w.h,
                                    page, bar);
                    }
                }
                if (ok) issued = item + 1;
                __syncwarp();
            }
            before += 2 * w.nt;
            w.done();
        }
        if (*fail) {  // copies under way land before the block ends: their time is far below the limit
            const unsigned long long t0 = globaltimer_ns();
            while (issued > 0 && globaltimer_ns() - t0 < 1000000ull) {}
        }
    } else if (warp >= 8 && warp < 12) {
        // ------------------------------------- repair of V, or widening of K and V
        // warps, or pairs of warps, take the items in turn
        constexpr int WT = Sh::kWideners, TEAMS = Sh::kTeams;
        const int team = (tid & 127) / WT, lt = tid % WT;
        auto meet = [&] {
            __syncwarp();
            if (WT > 32) asm volatile("bar.sync %0, 64;" ::"r"(3 + team) : "memory");
        };
        uint32_t item = 0, turns = 0;  // turns: phases of raw_full by slot (16-bit cache)
        bool ok = true;                // no wait for a tile has run out
        int u = 0;
        Units w(s_units, unit_full, unit_empty, fail);
        while (all_agree(2, 128, w.next())) {
            // a negative scale turns the rows' signs
            const uint32_t flip = (a.scale < 0.0f) != (F8 && c.k_scale && c.k_scale[w.h] < 0.0f) ? 0x80008000u : 0u;
            // the products of the unit before are done with the query rows
            if (u > 0) tc_wait(&q_empty, (u - 1) & 1, fail);
            __syncwarp();
            constexpr int QSTEP = 128 / CW;  // rows of a step
            const int qt = tid & 127, qch = qt % CW;
            const bool inside = qch * 8 < c.head_dim;
            if constexpr (SH) {
                // a group's rows are in a list: the reads of eight entries under way together
                // (one by one they took 10,000 cycles a unit of 128 rows)
                constexpr int QIN = 8;
#pragma unroll 1
                for (int rb = qt / CW; rb < w.R; rb += QSTEP * QIN) {
                    const char* from[QIN];
#pragma unroll
                    for (int i = 0; i < QIN; ++i) {
                        const int r = rb + i * QSTEP;
                        from[i] = a.q;
                        if (r < w.R && inside) {
                            const int j = (int)a.by_group.div((uint32_t)(w.r0 + r));
                            const int hq = w.h * a.group + (w.r0 + r - j * a.group);
                            from[i] += (long long)row_of<true>(a, w.req, j) * a.q_row + hq * a.q_head + qch * 16;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < QIN; ++i)
                        if (rb + i * QSTEP < w.R)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sq + panel_at(rb + i * QSTEP, qch)),
                                         "l"(from[i]), "r"(inside ? 16 : 0)
                                         : "memory");
                }
            } else {
#pragma unroll 1
                for (int r = qt / CW; r < w.R; r += QSTEP) {
                    const int j = (int)a.by_group.div((uint32_t)(w.r0 + r));
                    const int hq = w.h * a.group + (w.r0 + r - j * a.group);
                    const char* from = a.q + (long long)(w.req.base + j) * a.q_row + hq * a.q_head + qch * 16;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sq + panel_at(r, qch)),
                                 "l"(inside ? from : a.q), "r"(inside ? 16 : 0)
                                 : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (!std::is_same<T, O>::value || flip) {
                // each thread has its own chunks again, in place
#pragma unroll 1
                for (int r = qt / CW; r < (w.R + QSTEP - 1) / QSTEP * QSTEP; r += QSTEP) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (r < w.R) v = lds16(sq + panel_at(r, qch));
                    if (!std::is_same<T, O>::value) {
                        // bf16 rows under fp16 products: each row is scaled by a power
                        // of two that brings its largest value into [1, 2), exactly but
                        // for values 2^-14 below it, which lose bits that are 2^-25 of it
                        float top = fmaxf(fmaxf(fmaxf(fabsf(bf16_lo(v.x)), fabsf(bf16_hi(v.x))),
                                                fmaxf(fabsf(bf16_lo(v.y)), fabsf(bf16_hi(v.y)))),
                                          fmaxf(fmaxf(fabsf(bf16_lo(v.z)), fabsf(bf16_hi(v.z))),
                                                fmaxf(fabsf(bf16_lo(v.w)), fabsf(bf16_hi(v.w)))));
#pragma unroll
                        for (int o = CW / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -126), 126);
                        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
                        v.x = tc_pack<__half>(bf16_lo(v.x) * down, bf16_hi(v.x) * down);
                        v.y = tc_pack<__half>(bf16_lo(v.y) * down, bf16_hi(v.y) * down);
                        v.z = tc_pack<__half>(bf16_lo(v.z) * down, bf16_hi(v.z) * down);
                        v.w = tc_pack<__half>(bf16_lo(v.w) * down, bf16_hi(v.w) * down);
                        if (r < w.R && qch == 0) s_row[u & 1][r] = __uint_as_float((uint32_t)(127 + ex) << 23);
                    }
                    if (r < w.R) sts16(sq + panel_at(r, qch), make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);

            for (int i = 0; i < 2 * w.nt; ++i, ++item) {
                bool is_v;
                int t;
                item_of<NB>(i, w.nt, is_v, t);
                const int key0 = tile_key<KT>(w.req, w.t0 + t);
                const bool cut = is_v && !all_see<KT>(a, w.req, key0);
                if (!F8 && !cut) continue;
                const int slot = (int)(item % NS);
                if ((int)(item % TEAMS) != team) {
                    turns ^= 1u << slot;
                    continue;
                }
                const uint32_t to = ring + slot * Sh::kTile;
                bool dirty = false;
                if (F8) {
                    const int rs = (int)(item % NR);
                    ok = tc_wait(&raw_full[rs], (item / NR) & 1, fail) && ok;
                    const uint32_t from = raws + rs * Sh::kRawTile;
                    constexpr int STEP = WT / (D / 16), N = KT / STEP, IN = 8;  // rows of a step, steps, loads in flight
                    if (cut) {  // each thread's own chunks, as below
                        dirty = repair<T, true, KT, STEP>(a, w.req, key0, lt / (D / 16), [&](int r) {
                            return from + (uint32_t)(r * D + lt % (D / 16) * 16);
                        });
                        if (dirty) atomicOr(&s_flags[u % kTcUnits], 2);  // before the team meets
                        __syncwarp();
                    }
                    if (item >= NS) tc_wait(&empty[slot], ((item / NS) & 1) ^ 1, fail);
                    const int ch = lt % (D / 16), k0 = lt / (D / 16);
#pragma unroll 1
                    for (int i0 = 0; i0 < N; i0 += IN) {
                        uint4 v[IN];
#pragma unroll
                        for (int q = 0; q < IN; ++q) v[q] = lds16(from + (lt + (i0 + q) * WT) * 16);
#pragma unroll
                        for (int q = 0; q < IN; ++q) {
                            const uint32_t at = to + panel_at(k0 + (i0 + q) * STEP, 2 * ch);
                            uint4 lo, hi;
                            tc_widen(v[q].x, lo.x, lo.y);
                            tc_widen(v[q].y, lo.z, lo.w);
                            tc_widen(v[q].z, hi.x, hi.y);
                            tc_widen(v[q].w, hi.z, hi.w);
                            sts16(at, lo);
                            sts16(at ^ 16, hi);  // the chunk beside it, in the swizzle too
                        }
                    }
                    fence_proxy_async_smem();
                    meet();
                    if (lt == 0 && ok) mbar_arrive(&raw_empty[rs]);
                } else {
                    tc_wait(&raw_full[slot], (turns >> slot) & 1, fail);
                    turns ^= 1u << slot;
                    constexpr int STEP = WT / CW;
                    dirty = repair<T, false, KT, STEP>(a, w.req, key0, lt / CW,
                                                       [&](int r) { return to + panel_at(r, lt % CW); });
                    if (dirty) atomicOr(&s_flags[u % kTcUnits], 2);
                    fence_proxy_async_smem();
                    meet();
                }
                __syncwarp();  // the warp stays together: without it e4m3, heads of 128, 150 -> 168 us
                if (lt == 0 && (F8 || !*fail)) mbar_arrive(&full[slot]);  // 16 bits: see the loaders
            }
            ++u;
            w.done();
        }
    } else if (warp == 13) {
        // -------------------------------------------------------------- units
        Walk<KT, SH> w(a, c, s_of.run.run);
        for (int u = 0;; ++u) {
            const bool more = w.next(a, c);
            const int at = u % kTcUnits;
            // a place that is not given back in time is not written over
            if (!__all_sync(0xffffffffu,
                            u < kTcUnits || tc_wait(&unit_empty[at], ((u / kTcUnits) & 1) ^ 1, fail)))
                break;
            if (lane == 0) {
                Unit s;
                s.nt = 0;
                if (more) {
                    s.n = w.req.n;
                    s.ell = w.req.ell;
                    s.base = w.req.base;
                    s.b = SH ? w.req.b | w.req.kind << 16 : w.b;
                    if (SH) s.skip = w.req.skip;
                    s.sink_tiles = w.req.sink_tiles;
                    s.first_tile = w.req.first_tile;
                    s.t0 = w.t0;
                    s.nt = w.nt;
                    s.h = w.h;
                    s.r0 = w.r0;
                    s.rows_parts = w.R + 256 * (w.whole() ? -1 : w.t0 == 0 ? w.open().x : 0);
                }
                s_units[at] = s;
                s_flags[at] = 0;
                mbar_arrive(&unit_full[at]);
            }
            __syncwarp();
            if (!more) break;
        }
    } else if (warp == 15) {
        // ------------------------------------------------- matrix instructions
        constexpr uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
        constexpr uint32_t head = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(kTcRows >> 4) << 24);
        constexpr uint32_t id_s = head | ((uint32_t)(KT >> 3) << 17);
        constexpr uint32_t id_o = head | ((uint32_t)(D >> 3) << 17) | (1u << 16);
        const uint32_t one = elect_one();
        uint32_t item = 0, first = 0;  // first: tiles of the units before
        Units w(s_units, unit_full, unit_empty, fail);
        while (w.next()) {
            if (tc.expire_first) *fail = 1;
            tc_wait(&q_full, w.u & 1, fail);
            __syncwarp();
            tc_fence_after();
            // O of tile i - NB, then S of tile i in the columns that its weights leave
#pragma unroll 1
            for (int i = 0; i < w.nt + NB; ++i) {
                if (i >= NB) {
                    const uint32_t slot = item % NS, g = first + i - NB, s = (i - NB) & 1;
                    tc_wait(&full[slot], (item / NS) & 1, fail);
                    tc_wait(&p_full[g % NB], (g / NB) & 1, fail);
                    __syncwarp();
                    tc_fence_after();
                    const uint64_t v = desc_mn(ring + slot * Sh::kTile, Sh::kPanel);
                    const uint32_t from = tmem + (g % NB) * KT, out = tmem + NB * KT + s * D;
#pragma unroll
                    for (int kk = 0; kk < KT / 16; ++kk)
                        tc_mma_ts(one, out, from + kk * 8, v + kk * (2048 >> 4), id_o, i >= NB + 2 || kk > 0);
                    tc_commit(one, &o_done[s]);
                    tc_commit(one, &empty[slot]);
                    ++item;
                }
                if (i < w.nt) {
                    const uint32_t slot = item % NS, at = (first + i) % NB;
                    tc_wait(&full[slot], (item / NS) & 1, fail);
                    __syncwarp();
                    tc_fence_after();
                    const uint64_t q = desc_k(sq), k = desc_k(ring + slot * Sh::kTile);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * Sh::kPanel + (kk & 3) * 32) >> 4;
                        tc_mma_ss(one, tmem + at * KT, q + off, k + off, id_s, kk > 0);
                    }
                    tc_commit(one, &s_full[at]);
                    tc_commit(one, &empty[slot]);
                    if (i == w.nt - 1) tc_commit(one, &q_empty);
                    ++item;
                }
            }
            tc_commit(one, &o_all);
            first += w.nt;
            w.done();
        }
        if (*fail) {
            tc_commit(one, &drain);
            mbar_wait_bounded(&drain, 0);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();  // every product and every use of TMEM is done
    if (warp == 15) {
        tc_fence_after();
        tc_dealloc(tmem, Sh::kCols);
    }
    } else {
        tc_more_registers<168>();
        // ------------------------------------------------- softmax and output
        const int s = warp >> 2;
        const int row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t to = tmem + lanes + NB * KT;
        int4 open = make_int4(0, 0, 0, 0);
        uint32_t seen = 0, first = 0;  // tiles of the stream so far, tiles of the units before
        int u = 0;
        Units w(s_units, unit_full, unit_empty, fail);
        while (all_agree(1, 256, w.next())) {
            const bool active = (warp & 3) * 32 < w.R;  // the warp has rows
            const int pos = row < w.R ? position_of<SH>(w.req, (int)a.by_group.div((uint32_t)(w.r0 + row)))
                                      : w.req.n + w.req.ell;
            float scale = fabsf(a.scale) * (F8 && c.k_scale ? fabsf(c.k_scale[w.h]) : 1.0f);
            float m = -INFINITY, l = 0.0f;  // the reference and the sum
            bool coarse = false;            // a score of the warp has been beyond kTcFine
            for (int t = s; t < w.nt; t += 2) {
                const uint32_t g = first + t, ts = tmem + lanes + (g % NB) * KT;
                tc_wait(&s_full[g % NB], (g / NB) & 1, fail);
                __syncwarp();
                tc_fence_after();
                if (active) {
                    if (!std::is_same<T, O>::value && t == s) scale *= s_row[u & 1][row];
                    const int key0 = tile_key<KT>(w.req, w.t0 + t);
                    float by = scale;
                    // The loops over 32 columns stay loops: the roles' code together has
                    // to fit the instruction cache (unrolled, they were 2.5 times slower)
                    float x[32], y[32], top = -INFINITY, top1 = -INFINITY;
                    if (coarse || !all_see<KT>(a, w.req, key0)) {
                        // scores that the row does not see, in a pass of its own: a tile
                        // that a border cuts is rare, and this code cold.  The others are
                        // scaled here (at a scale of zero, infinity times it is no number)
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            tc_ld32(x, ts + q * 32);
                            tc_wait32(x);
                            const uint32_t see = seen_bits(a, pos, key0 + q * 32);
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = (see >> e) & 1u ? x[e] * scale : -INFINITY;
                            tc_st32(ts + q * 32, x);
                        }
                        tc_wait_st();
                        by = 1.0f;
                    }
#pragma unroll 1
                    for (int q = 0; q < 4; q += 2) {
                        tc_ld32(x, ts + q * 32);
                        tc_ld32(y, ts + q * 32 + 32);
                        tc_wait32(x);
                        tc_wait32(y);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            top = fmaxf(top, fmaxf(x[e], x[e + 1]));
                            top1 = fmaxf(top1, fmaxf(y[e], y[e + 1]));
                        }
                    }
                    top = fmaxf(top, top1);
                    // nothing seen stays below everything, at a scale of zero too
                    if (top != -INFINITY) top = __fmul_ru(top, by);
                    bool up = top > __fadd_rd(m, kTcUp<T> + kTcSlack<T>);
                    if (__any_sync(0xffffffffu, up)) {
                        if (!coarse && __any_sync(0xffffffffu, up && row < w.R && fabsf(top) >= kTcFine<T>)) {
                            // the first such tile: its scores are scaled now, see kTcFine
                            coarse = true;
                            top = scale_scores(ts, by);
                            by = 1.0f;
                            up = top > __fadd_rd(m, kTcUp<T> + kTcSlack<T>);
                        }
                        const float now = up ? __fsub_ru(top, kTcUp<T>) : m;
                        const float corr = up ? ex2_approx(m - now) : 1.0f;
                        l *= corr;
                        m = now;
                        if (t >= 2) {  // see TcShape
                            tc_wait(&o_done[s], (seen - 1) & 1, fail);
                            __syncwarp();
                            tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < D / 32; ++q) {
                                tc_ld32(x, to + s * D + q * 32);
                                tc_wait32(x);
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[e] *= corr;
                                tc_st32(to + s * D + q * 32, x);
                            }
                        }
                    }
                    // weights: their sum is of the unrounded ones; for the
                    // product they are rounded to T, 2^-8 (bf16) or 2^-11 of
                    // each at most, as much as the output's own rounding
                    const float ref = m == -INFINITY ? 0.0f : m;
                    const Two by2 = two(by, by), ref2 = two(-ref, -ref);
                    Two sum0 = two(0.0f, 0.0f), sum1 = sum0;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        tc_ld32(x, ts + q * 32);
                        tc_wait32(x);
                        weigh<T>(x, by2, ref2, sum0, sum1, ts + q * 16);
                    }
                    const float2 sums = of_two(add2(sum0, sum1));
                    l += sums.x + sums.y;
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[g % NB]);
                ++seen;
            }
            first += w.nt;
            // all products of the unit, by a barrier with one phase a unit.  The
            // stream's own o_done would not do: three tiles ahead, the scores of its
            // last tile say nothing of its product before, and while that one is not
            // over the wait for the last one's parity passes at once
            tc_wait(&o_all, u & 1, fail);
            if (s == 1) {
                s_ml[0][row] = m;
                s_ml[1][row] = l;
            }
            __syncwarp();
            tc_fence_before();
            asm volatile("bar.sync 1, 256;" ::: "memory");
            tc_fence_after();

            // the two streams' weights, for both of them; the parts' maximum and
            // sum, or the reciprocal of the sum in the weights
            const int flags = s_flags[u % kTcUnits];
            const bool whole = w.now().parts() < 0;
            const bool complete = whole && (!SH || w.req.kind == kAlone);
            float* part = part_at(a, blockIdx.x, w.t0 == 0 ? 1 : 0);
            long long orow = 0, at = 0;
            if (row < w.R) orow = SH ? shared_out_row(a, w.req, w.h, w.r0 + row) : out_row(a, w.req.base, w.h, w.r0 + row);
            if (SH) at = where_of(a, w.req.kind, orow);
            const PartRow to_part = SH && whole ? side_row(a, c.head_dim, at) : part_row(a, part, c.head_dim, row);
            if (s == 0) {
                const float m1 = s_ml[0][row];
                const float M = fmaxf(m, m1), ref = M == -INFINITY ? 0.0f : M;
                const float w0 = ex2_approx(m - ref), w1 = ex2_approx(m1 - ref);
                float L = l * w0 + s_ml[1][row] * w1;
                if ((flags & 1) || *fail) L = __int_as_float(0x7fc00000);
                const float inv = (complete ? 1.0f / L : 1.0f) * (F8 && c.v_scale ? c.v_scale[w.h] : 1.0f);
                s_ml[0][row] = w0 * inv;
                s_ml[1][row] = w1 * inv;
                if (row < w.R) {
                    if (!complete) {
                        *to_part.m = M;
                        *to_part.l = L;
                    } else if (a.lse) {
                        a.lse[orow] = (M + log2f(L)) * 0.6931471805599453f;
                    }
                    if (SH && w.t0 == 0) tell(a, at, whole, complete, w.now().parts(), row);
                }
            }
            __syncwarp();
            asm volatile("bar.sync 1, 256;" ::: "memory");

            // output: stream s's warps write columns [s D/2, (s+1) D/2), eight at a
            // time (a short loop: this code is cold when it is reached)
            if (active) {
                const float w0 = s_ml[0][row], w1 = s_ml[1][row];
#pragma unroll 1
                for (int col = s * (D / 2); col < (s + 1) * (D / 2) && col < c.head_dim; col += 8) {
                    float x[8], y[8];
                    tc_ld8(x, y, to + col, to + D + col);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] *= w0;
                        // without an odd tile its columns hold anything
                        if (w.nt > 1) x[e] = fmaf(w1, y[e], x[e]);
                    }
                    if (flags & 2) {
                        const Eight more = sum_nonfinite<T, F8, KT, SH>(a, c, w.now(), pos, col);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] += more.x[e];
                    }
                    if (row < w.R) {
                        if (complete) {
                            *(uint4*)((char*)a.out + (orow * c.head_dim + col) * 2) =
                                make_uint4(tc_pack<O>(x[0], x[1]), tc_pack<O>(x[2], x[3]), tc_pack<O>(x[4], x[5]),
                                           tc_pack<O>(x[6], x[7]));
                        } else {
                            float4* p = (float4*)(to_part.o + col);
                            p[0] = make_float4(x[0], x[1], x[2], x[3]);
                            p[1] = make_float4(x[4], x[5], x[6], x[7]);
                        }
                    }
                }
            }
            if (tid == 0 && (flags & 1)) set_status(a.status, SPEC_ERR_PAGE);
            if (!SH && w.now().parts() > 0) open = open_of(w.now().parts(), w.req.base, w.r0, w.R, w.h);
            __syncwarp();
            tc_fence_before();  // the barrier on the way to the next unit: both halves are written
            ++u;
            w.done();
        }
        if (!SH && tid == 0) a.open[blockIdx.x] = open;
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        if (tid == 0 && s_fail) set_status(a.status, SPEC_ERR_TIMEOUT);
        if (SH && tid == 0) a.failed[blockIdx.x] = s_fail;
        report_requests<O, KT, SH>(a, c, 256);
    }
}

}  // namespace specv
