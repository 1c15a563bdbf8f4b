// Attention over the paged cache: arguments, the split of the work over the
// blocks, and the parts that blocks leave for the joining kernel.
#pragma once

#include <atomic>

#include "specv_cache.cuh"

namespace specv {

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
};

template <int KT>
__device__ __forceinline__ Request request_of(const AttendArgs& a, const CacheView& c, int b) {
    Request r;
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
template <int KT, int THREADS>
__device__ __forceinline__ void run_of(const AttendArgs& a, const CacheView& c, RunShared<THREADS>& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + THREADS - 1) / THREADS;
    const int b0 = tid * per, b1 = min(a.B, b0 + per);
    long long mine = 0;
    int longest = 0;
    Request r = {};
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        r = request_of<KT>(a, c, b);
        mine += (long long)r.units * (r.tiles + a.lead);
        longest = max(longest, r.tiles);
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
    const int least = max(2, (int)sqrtf(a.part_cost * (float)longest));
    const long long step = max(quotient(total + gridDim.x - 1, gridDim.x), (long long)least);
    const long long start = (long long)blockIdx.x * step;
    if (start >= before && start < before + mine) {
        long long at = start - before;
        int b = b0;
        if (per > 1) {
#pragma unroll 1
            for (;; ++b) {
                r = request_of<KT>(a, c, b);
                const long long w = (long long)r.units * (r.tiles + a.lead);
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
template <int KT>
struct Walk {
    Request req;
    int b, unit, t0, nt, h, r0, R;
    int place;  // in the unit, leads included
    long long left, step;

    __device__ __forceinline__ Walk(const AttendArgs& a, const CacheView& c, const Run& run) {
        b = run.b;
        left = run.left;
        step = run.step;
        unit = place = 0;
        if (left > 0) {
            req = run.req;
            unit = (int)quotient(run.at, (uint32_t)(req.tiles + a.lead));
            place = (int)(run.at - (long long)unit * (req.tiles + a.lead));
        }
    }
    __device__ __forceinline__ bool next(const AttendArgs& a, const CacheView& c) {
        for (;;) {
            if (left <= 0) return false;
            if (place == req.tiles + a.lead) {
                place = 0;
                if (++unit == req.units) {
                    unit = 0;
#pragma unroll 1
                    do req = request_of<KT>(a, c, ++b);
                    while (req.units == 0);
                }
            }
            const int take = (int)min((long long)(req.tiles + a.lead - place), left);
            t0 = max(place - a.lead, 0);
            nt = max(place + take - a.lead, 0) - t0;
            place += take;
            left -= take;
            if (nt > 0) break;
        }
        h = unit / req.row_tiles;
        r0 = (unit - h * req.row_tiles) * a.tile_rows;
        R = min((req.ell + 1) * a.group - r0, a.tile_rows);
        return true;
    }
    // True if the segment is the whole unit; else its parts are joined, and the
    // block with tile 0 says how many there are.
    __device__ __forceinline__ bool whole() const { return nt == req.tiles; }
    __device__ __forceinline__ int4 open() const {
        const int rest = req.tiles - nt;
        const int parts = rest <= step ? rest > 0 : (int)((uint32_t)(rest - 1) / (uint32_t)step) + 1;
        return open_of(1 + parts, req.base, r0, R, h);
    }
};

// Where a block's part of a unit goes: slot 1 if the unit begins in the block,
// slot 0 if it began in an earlier one.
__device__ __forceinline__ float* part_at(const AttendArgs& a, int block, int slot) {
    return a.parts + ((long long)block * 2 + slot) * a.part_floats;
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
template <typename T, int KT>
__device__ __forceinline__ void report_requests(const AttendArgs& a, const CacheView& c, int threads) {
#pragma unroll 1
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const Request r = request_of<KT>(a, c, b);
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

// 16-bit rows: warp-level matrix instructions, over 16-bit and e4m3 caches.
AttendPlan attend_mma_plan(int rows, int head_dim, bool f8, int sms);
int attend_mma16(const AttendArgs& a, const CacheView& c, spec_dtype dt, int blocks, cudaStream_t st);
int attend_mma8(const AttendArgs& a, const CacheView& c, spec_dtype dt, int blocks, cudaStream_t st);

// 16-bit rows, many of them a KV head: the tensor cores, over 16-bit and e4m3 caches.
bool attend_tc_takes(const CacheView& c, int rows);
AttendPlan attend_tc_plan(int sms);
int attend_tc(const AttendArgs& a, const CacheView& c, spec_dtype dt, spec_dtype cache_dt, int blocks,
              cudaStream_t st);

}  // namespace specv
