// Attention over the paged cache: arguments, the split of the work over the
// blocks, and the parts that blocks leave for the joining kernel.
#pragma once

#include <atomic>

#include "specv_cache.cuh"

namespace specv {

// A batch that shares prefixes (SH below) is split into items by a plan made once
// for all layers (specv_share.cu): of each group the shared positions, for the
// rows of all its members, and of each request the positions behind them.  An item
// is to the kernels what a request is otherwise.
enum { kAlone = 0, kRest = 1, kPrefix = 2 };  // an item: a whole request, one's rest, a group's prefix
struct alignas(16) ShareItem {
    int n, ell;      // as a request's, without the positions of `skip` (a prefix: its last position, and 0)
    int base, rows;  // first row; of a prefix, its place in the plan's list of rows
    int b, skip;     // row of the page table, and its entries left out
    int kind, code;
};

struct AttendArgs {
    const char* q;
    long long q_row, q_head;  // strides in bytes
    void* out;
    float* lse;
    const int32_t* table;
    const int32_t* len;
    const int32_t* ell;
    const int32_t* row;
    int* status;
    int4* open;    // [blocks]: of the unit that a block left open its parts (0: none), first
                   // row of q, first row of the unit, rows << 16 | KV head
    float* parts;  // [blocks][2][tile rows * (D + 2)]
    long long part_floats;
    int q_heads, group, rows, B, gamma, max_pages;
    int window, sinks;
    int tile_rows;    // rows of a unit at most, 2^tile_shift
    int tile_shift;
    int limit;        // positions of a request: pages of the table, and below 2^31
    int lead;         // what a unit costs beside its tiles, in tiles
    float part_cost;  // of a part when joined, in tiles
    float scale;      // of the scores, to base 2
    FastDiv by_group;
    // SH: the plan, and the parts of rows that two items have (each side: [rows][q_heads])
    const int* plan;  // its header
    const ShareItem* items;
    const int32_t* list;
    const uint8_t* kinds;
    float* side;      // [2][rows][q_heads][D], sums scaled by 2^-M
    float2* side_ml;  // [2][rows][q_heads]: M and the sum of weights
    int2* where;      // [2][rows][q_heads]: parts of a unit that was cut, and block << 7 | row of the unit
                      // of the first; 0 in `side`, -1 nothing to join
    FastDiv by_heads;
    int* failed;  // [blocks], by every call: 1 if a wait of the block ran out; NULL: the kernel has no waits
    int few, cost[2];  // what a tile costs, in the measure of `lead`: of items of at most `few` rows a KV head, of others
};

// ---------------------------------------------------------------- the work
// Request b has (ell+1) * group query rows for each KV head.  A unit is up to
// tile_rows of them against the request's visible keys, cut into tiles of KT
// adjacent keys: tiles of the sinks, then tiles from the window's first key on.
// All units' tiles, in order, are dealt to the blocks in equal runs, so that
// ragged lengths leave no block idle; a run may end inside a unit, whose parts
// are then joined.  A unit counts `lead` tiles more than it has, before its
// first: its set-up and its end take time, and runs of short requests would
// otherwise take up to twice as long as others.
struct Request {
    int code;      // SPEC_OK or why there is no work
    int n, ell;    // cache length, drafts
    int base;      // first row
    int sink_tiles, first_tile, tiles, row_tiles, units;
    int rows, b, skip, kind;  // SH, see ShareItem
};

// Items of a plan, or requests.  A plan made for other sizes has none.
constexpr int kPlanMagic = 0x73706c6e;
enum { kPlanStatus, kPlanIs, kPlanB, kPlanGamma, kPlanRows, kPlanSlots, kPlanPage, kPlanItems, kPlanWords };
template <bool SH>
__device__ __forceinline__ int requests_of(const AttendArgs& a, const CacheView& c) {
    if constexpr (SH) {
        const bool fits = a.plan[kPlanIs] == kPlanMagic && a.plan[kPlanB] == a.B && a.plan[kPlanGamma] == a.gamma &&
                          a.plan[kPlanRows] == a.rows && a.plan[kPlanSlots] == a.max_pages &&
                          a.plan[kPlanPage] == c.page_size;
        return fits ? a.plan[kPlanItems] : 0;
    }
    return a.B;
}

template <int KT, bool SH>
__device__ __forceinline__ Request request_of(const AttendArgs& a, const CacheView& c, int b) {
    Request r;
    if constexpr (SH) {
        const int4* p = (const int4*)(a.items + b);
        const int4 x = p[0], y = p[1];
        r.n = x.x;
        r.ell = x.y;
        r.base = x.z;
        r.rows = x.w;
        r.b = y.x;
        r.skip = y.y;
        r.kind = y.z;
        r.code = y.w;
        r.sink_tiles = r.first_tile = 0;
        r.tiles = r.code == SPEC_OK ? (int)((uint32_t)(r.n + r.ell) / KT) + 1 : 0;
        r.row_tiles = r.code == SPEC_OK ? (r.rows * a.group + a.tile_rows - 1) >> a.tile_shift : 0;
        r.units = r.row_tiles * c.kv_heads;
        return r;
    }
    r.n = a.len[b];
    r.ell = a.ell ? a.ell[b] : a.gamma;
    r.base = a.row ? a.row[b] : b * (a.gamma + 1);
    r.tiles = r.units = r.row_tiles = r.sink_tiles = r.first_tile = 0;
    r.code = SPEC_OK;
    if (r.ell < 0 || r.ell > a.gamma) r.code = SPEC_ERR_VERIFY_LEN;
    else if (r.base < 0 || r.base > a.rows - r.ell - 1) r.code = SPEC_ERR_ROW_INDEX;
    else if (r.n < 0 || r.n >= a.limit - r.ell)
        r.code = SPEC_ERR_CACHE_LEN;
    if (r.code != SPEC_OK) return r;
    const int last = (int)((uint32_t)(r.n + r.ell) / KT) + 1;
    if (a.window > 0) {
        const int first = max(0, r.n - a.window + 1);
        r.first_tile = (int)((uint32_t)first / KT);
        r.sink_tiles = min((int)(((uint32_t)a.sinks + KT - 1) / KT), r.first_tile);
    }
    r.tiles = r.sink_tiles + last - r.first_tile;
    r.row_tiles = ((r.ell + 1) * a.group + a.tile_rows - 1) >> a.tile_shift;
    r.units = r.row_tiles * c.kv_heads;
    return r;
}

// Rows (of a head) of a request, and of them row j: its row in q and out, its
// position.
template <bool SH>
__device__ __forceinline__ int rows_of(const Request& r) { return SH ? r.rows : r.ell + 1; }
template <bool SH>
__device__ __forceinline__ int row_of(const AttendArgs& a, const Request& r, int j) {
    if constexpr (SH)
        if (r.kind == kPrefix) return a.list[r.base + j];
    return r.base + j;
}
template <bool SH>
__device__ __forceinline__ int position_of(const Request& r, int j) { return r.n + (SH ? min(j, r.ell) : j); }

// The pages of a request (or item) b.
template <bool SH>
__device__ __forceinline__ const int32_t* pages_of(const AttendArgs& a, const Request& r, int b) {
    return SH ? a.table + (size_t)r.b * a.max_pages + r.skip : a.table + (size_t)b * a.max_pages;
}

// What a tile, and a unit with its set-up, cost in the measure of the runs.
template <bool SH>
__device__ __forceinline__ int cost_of(const AttendArgs& a, const Request& r) {
    return SH ? a.cost[r.rows * a.group > a.few] : 1;
}
template <bool SH>
__device__ __forceinline__ int length_of(const AttendArgs& a, const Request& r) {
    return r.tiles * cost_of<SH>(a, r) + a.lead;
}

// First key of tile t of a request.
template <int KT>
__device__ __forceinline__ int tile_key(const Request& r, int t) {
    return (t < r.sink_tiles ? t : t - r.sink_tiles + r.first_tile) * KT;
}

// Whether position t is one that any row of the request sees (the rows' own
// order, t <= p, apart), and whether the row at position p sees it.
__device__ __forceinline__ bool any_sees(const AttendArgs& a, const Request& r, int t) {
    return t <= r.n + r.ell && (a.window == 0 || r.n - t < a.window || t < a.sinks);
}
__device__ __forceinline__ bool sees(const AttendArgs& a, int p, int t) {
    return t <= p && (a.window == 0 || p - t < a.window || t < a.sinks);
}

// True if every row of the request sees all KT keys of the tile.
template <int KT>
__device__ __forceinline__ bool all_see(const AttendArgs& a, const Request& r, int key) {
    return key + KT - 1 <= r.n && (a.window == 0 || r.n + r.ell - key < a.window || key + KT <= a.sinks);
}

struct Run {
    Request req;     // of the run's first tile
    int b;
    long long at;    // tile within the request (unit-major, leads included)
    long long left;  // tiles of the run
    long long step;  // tiles of every block's run
};

template <int THREADS>
struct RunShared {
    long long sum[THREADS / 32];
    int longest[THREADS / 32];
    Run run;
};

// n / d; the 64-bit division is long, and its case rare.
__device__ __forceinline__ long long quotient(long long n, uint32_t d) {
    return n >> 32 ? n / (long long)d : (long long)((uint32_t)n / d);
}

// The block's run, in s.run.  All threads call it.
template <int KT, bool SH, int THREADS>
__device__ __forceinline__ void run_of(const AttendArgs& a, const CacheView& c, RunShared<THREADS>& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int count = requests_of<SH>(a, c);
    const int per = (count + THREADS - 1) / THREADS;
    const int b0 = tid * per, b1 = min(count, b0 + per);
    long long mine = 0;
    int longest = 0;
    Request r = {};
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        r = request_of<KT, SH>(a, c, b);
        mine += (long long)r.units * length_of<SH>(a, r);
        longest = max(longest, r.tiles * cost_of<SH>(a, r));
    }
    longest = (int)__reduce_max_sync(0xffffffffu, (unsigned)longest);
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) {
        s.sum[warp] = x;
        s.longest[warp] = longest;
    }
    if (tid == 0) s.run.left = 0;
    __syncthreads();
    long long before = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const long long y = s.sum[w];
        if (w < warp) before += y;
        total += y;
        longest = max(longest, s.longest[w]);
    }
    // few long units are not cut into more parts than joining them is worth
    const int least = max(SH ? max(2, max(a.cost[0], a.cost[1])) : 2, (int)sqrtf(a.part_cost * (float)longest));
    const long long step = max(quotient(total + gridDim.x - 1, gridDim.x), (long long)least);
    const long long start = (long long)blockIdx.x * step;
    if (start >= before && start < before + mine) {
        long long at = start - before;
        int b = b0;
        if (per > 1) {
#pragma unroll 1
            for (;; ++b) {
                r = request_of<KT, SH>(a, c, b);
                const long long w = (long long)r.units * length_of<SH>(a, r);
                if (at < w) break;
                at -= w;
            }
        }
        s.run.req = r;
        s.run.b = b;
        s.run.at = at;
        s.run.left = min(step, total - start);
        s.run.step = step;
    }
    __syncthreads();
}

__device__ __forceinline__ int4 open_of(int parts, int base, int r0, int R, int h) {
    return make_int4(parts, base, r0, (int)((uint32_t)R << 16 | (uint32_t)h));
}

// The segments of a run: tiles t0 .. t0 + nt - 1 of a unit, for the rows r0 ..
// r0 + R - 1 of KV head h.
template <int KT, bool SH>
struct Walk {
    Request req;
    int b, unit, t0, nt, h, r0, R;
    int place;  // in the unit, leads included
    int rest;   // of the unit behind the segment
    long long left, step;

    __device__ __forceinline__ Walk(const AttendArgs& a, const CacheView& c, const Run& run) {
        b = run.b;
        left = run.left;
        step = run.step;
        unit = place = 0;
        if (left > 0) {
            req = run.req;
            unit = (int)quotient(run.at, (uint32_t)length_of<SH>(a, req));
            place = (int)(run.at - (long long)unit * length_of<SH>(a, req));
        }
    }
    __device__ __forceinline__ bool next(const AttendArgs& a, const CacheView& c) {
        for (;;) {
            if (left <= 0) return false;
            if (place == length_of<SH>(a, req)) {
                place = 0;
                if (++unit == req.units) {
                    unit = 0;
#pragma unroll 1
                    do req = request_of<KT, SH>(a, c, ++b);
                    while (req.units == 0);
                }
            }
            const int length = length_of<SH>(a, req);
            const int take = (int)min((long long)(length - place), left);
            // a tile belongs to the run that its cost ends in: a unit's last run has at least
            // one, and so have those between (step is no less than a tile's cost)
            t0 = max(place - a.lead, 0);
            nt = max(place + take - a.lead, 0);
            if constexpr (SH) {
                t0 /= cost_of<SH>(a, req);
                nt /= cost_of<SH>(a, req);
            }
            nt -= t0;
            rest = length - place - take;
            place += take;
            left -= take;
            if (nt > 0) break;
        }
        h = unit / req.row_tiles;
        r0 = (unit - h * req.row_tiles) * a.tile_rows;
        R = min(rows_of<SH>(req) * a.group - r0, a.tile_rows);
        return true;
    }
    // True if the segment is the whole unit; else its parts are joined, and the
    // block with tile 0 says how many there are.
    __device__ __forceinline__ bool whole() const { return nt == req.tiles; }
    __device__ __forceinline__ int4 open() const {
        const int parts = rest <= step ? rest > 0 : (int)((uint32_t)(rest - 1) / (uint32_t)step) + 1;
        return open_of(1 + parts, req.base, r0, R, h);
    }
};

// Where a block's part of a unit goes: slot 1 if the unit begins in the block,
// slot 0 if it began in an earlier one.
__device__ __forceinline__ float* part_at(const AttendArgs& a, int block, int slot) {
    return a.parts + ((long long)block * 2 + slot) * a.part_floats;
}

// SH: a row's part of a unit, where it goes.  `i` is the index of the row (its own
// of out, or behind all of these for a prefix).
struct PartRow {
    float* o;
    float* m;
    float* l;
};
__device__ __forceinline__ PartRow part_row(const AttendArgs& a, float* part, int dim, int r) {
    return {part + r * dim, part + a.tile_rows * dim + r, part + a.tile_rows * (dim + 1) + r};
}
__device__ __forceinline__ PartRow side_row(const AttendArgs& a, int dim, long long i) {
    float* ml = (float*)(a.side_ml + i);
    return {a.side + i * dim, ml, ml + 1};
}
// Row r of KV head h of a request in out, and its index in `where`.
__device__ __forceinline__ long long shared_out_row(const AttendArgs& a, const Request& q, int h, int r) {
    const int j = (int)a.by_group.div((uint32_t)r);
    return (long long)row_of<true>(a, q, j) * a.q_heads + h * a.group + (r - j * a.group);
}
__device__ __forceinline__ long long where_of(const AttendArgs& a, int kind, long long row) {
    return kind == kPrefix ? row + (long long)a.rows * a.q_heads : row;
}
// What the joining kernel is told of row r of a unit, by the block with its tile 0:
// `parts` of a unit that was cut.
__device__ __forceinline__ void tell(const AttendArgs& a, long long i, bool whole, bool direct, int parts, int r) {
    a.where[i] = whole ? make_int2(direct ? -1 : 0, 0) : make_int2(parts, (int)(blockIdx.x << 7) | r);
}

// The row of out (and the index of lse) of row r of KV head h of a request whose
// first row is `base`.
__device__ __forceinline__ long long out_row(const AttendArgs& a, int base, int h, int r) {
    const int j = (int)a.by_group.div((uint32_t)r);
    return (long long)(base + j) * a.q_heads + h * a.group + (r - j * a.group);
}

// Byte offset of a key's first value (head 0) in the pages, or -1 if its entry
// is no page.
__device__ __forceinline__ long long key_at(const AttendArgs& a, const CacheView& c, const int32_t* pages, int t) {
    const uint32_t slot = c.by_page.div((uint32_t)t);
    const int page = pages[slot];
    if (page < 0 || page >= c.pages) return -1;
    return (long long)page * c.page + (long long)(t - (int)slot * c.page_size) * c.token;
}

// After its run, a block reports requests without work, and fills the rows of
// those whose positions do not fit (blocks share the requests).  Called by the
// first `threads` threads of the block.
template <typename T, int KT, bool SH>
__device__ __forceinline__ void report_requests(const AttendArgs& a, const CacheView& c, int threads) {
    const int count = requests_of<SH>(a, c);
    if (SH && count == 0 && blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, SPEC_ERR_PLAN);
#pragma unroll 1
    for (int b = blockIdx.x; b < count; b += gridDim.x) {
        const Request r = request_of<KT, SH>(a, c, b);
        if (r.code == SPEC_OK) continue;
        if (threadIdx.x == 0) set_status(a.status, r.code);
        if (r.code != SPEC_ERR_CACHE_LEN) continue;
        const long long first = (long long)r.base * a.q_heads, n = (long long)(r.ell + 1) * a.q_heads;
        const float nan = __int_as_float(0x7fc00000);
        T* out = (T*)a.out + first * c.head_dim;
        for (long long i = threadIdx.x; i < n * c.head_dim; i += threads) out[i] = from_f32<T>(nan);
        if (a.lse)
            for (long long i = threadIdx.x; i < n; i += threads) a.lse[first + i] = nan;
    }
}

// Lets a kernel use `bytes` of dynamic shared memory, once per device (a bit
// each in `done`, which belongs to the kernel).
inline int allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ERR_CUDA;
    if ((done.load(std::memory_order_relaxed) >> dev) & 1ull) return SPEC_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return SPEC_ERR_CUDA;
    done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return SPEC_OK;
}

// ------------------------------------------------------------------ kernels
struct AttendPlan {
    int blocks;     // of the grid, at most
    int tile_rows;  // rows of a unit
};

// fp32 rows: products on the CUDA cores.
AttendPlan attend_simt_plan(int rows, int head_dim, int sms);
int attend_simt(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st);

// The same over the items of a plan, for units of many rows.
AttendPlan attend_f32_shared_plan(int head_dim, int sms);
int attend_f32_shared(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st);

// 16-bit rows: warp-level matrix instructions, over 16-bit and e4m3 caches.
AttendPlan attend_mma_plan(int rows, int head_dim, bool f8, int sms);
int attend_mma16(const AttendArgs& a, const CacheView& c, spec_dtype dt, int blocks, cudaStream_t st);
int attend_mma8(const AttendArgs& a, const CacheView& c, spec_dtype dt, int blocks, cudaStream_t st);
AttendPlan attend_mma_shared_plan(int rows, int head_dim, bool f8, int sms);
int attend_mma_shared(const AttendArgs& a, const CacheView& c, spec_dtype dt, bool f8, int blocks, cudaStream_t st);

// 16-bit rows, many of them a KV head: the tensor cores, over 16-bit and e4m3 caches.
constexpr int kTcLeast = 16;  // rows that the warp-level kernels take as well
bool attend_tc_takes(const CacheView& c, int rows);
AttendPlan attend_tc_plan(int sms);
int attend_tc(const AttendArgs& a, const CacheView& c, spec_dtype dt, spec_dtype cache_dt, int blocks,
              cudaStream_t st);
int attend_tc_shared(const AttendArgs& a, const CacheView& c, spec_dtype dt, spec_dtype cache_dt, int blocks,
                     cudaStream_t st);

}  // namespace specv
