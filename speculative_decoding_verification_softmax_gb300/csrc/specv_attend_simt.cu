// Attention over the paged cache on the CUDA cores: the path of fp32 rows,
// whose products keep 32 bits.
//
// A block takes one unit at a time: 16 query rows against tiles of 64 keys.
// One pass over the keys with the running maximum m and sum l of each row's
// softmax, to base 2: a tile's scores s give m' = max(m, max s), p = 2^(s - m'),
// l' = l 2^(m - m') + sum p and o' = o 2^(m - m') + p V.
//
// Bound by the warps that work in the products: two of a block's eight have each
// four of the 16 rows, and those whose rows a unit lacks wait at the barriers.  One
// token of 32 requests of 2000 to 4000 positions, 32/8 heads of 128 (four rows, so
// six warps wait), takes 354 us for 820 MB, 2.3 TB/s.
#include "specv_attend.cuh"

namespace specv {

constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 16;
constexpr int kSimtKeys = 64;
constexpr int kSimtPad = 20;  // floats of a key's weights (16 rows): conflict-free 16-byte stores

// Blocks of an SM, by shared memory: 43, 80 and 154 KB each.
constexpr int simt_per_sm(int dim) { return dim <= 64 ? 3 : dim <= 128 ? 2 : 1; }

template <int D>
constexpr size_t simt_smem() {
    return sizeof(float) * (kSimtRows * D + kSimtKeys * (D + 4) + kSimtKeys * D + kSimtKeys * kSimtPad);
}

template <int D>
__global__ void __launch_bounds__(kSimtThreads, simt_per_sm(D)) k_attend_simt(AttendArgs a, CacheView c) {
    using T = float;
    constexpr int KT = kSimtKeys, CN = D / 64;
    extern __shared__ float4 smem4[];
    float* s_q = (float*)smem4;             // [16][D]
    float* s_k = s_q + kSimtRows * D;       // [64][D + 4]
    float* s_v = s_k + KT * (D + 4);        // [64][D]
    float* s_p = s_v + KT * D;              // [64][20]: scores, then weights, by key
    __shared__ float s_corr[kSimtRows], s_l[kSimtRows], s_m[kSimtRows];
    __shared__ RunShared<kSimtThreads> s_run;
    const int tid = threadIdx.x;
    const int col = tid & 63, rg = tid >> 6;     // products: a key or column, and 4 rows
    const int srow = tid >> 4, slane = tid & 15;  // softmax: 16 threads a row

    pdl_trigger();
    pdl_wait();
    run_of<KT>(a, c, s_run);
    int4 open = make_int4(0, 0, 0, 0);
    const int dim = c.head_dim;
    Walk<KT> w(a, c, s_run.run);
    while (w.next(a, c)) {
        const Request& req = w.req;
        const int t0 = w.t0, nt = w.nt, h = w.h, r0 = w.r0, R = w.R;
        const int32_t* pages = a.table + (size_t)w.b * a.max_pages;

        __syncthreads();
        for (int i = tid; i < kSimtRows * D; i += kSimtThreads) {
            const int r = i / D, d = i - r * D;
            float x = 0.0f;
            if (r < R && d < dim) {
                const int j = (int)a.by_group.div((uint32_t)(r0 + r));
                const int head = h * a.group + (r0 + r - j * a.group);
                x = ((const T*)(a.q + (long long)(req.base + j) * a.q_row + head * a.q_head))[d];
            }
            s_q[i] = x;
        }
        const float scale = a.scale;
        float acc[4][CN];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < CN; ++n) acc[i][n] = 0.0f;
        float m = -INFINITY, l = 0.0f;
        bool bad = false;
        const int myrow = r0 + srow;
        const int mypos = req.n + (int)a.by_group.div((uint32_t)myrow);

        for (int t = t0; t < t0 + nt; ++t) {
            const int key0 = tile_key<KT>(req, t);
            __syncthreads();
            for (int i = tid; i < KT * (D / 4); i += kSimtThreads) {
                const int k = i / (D / 4), d = (i - k * (D / 4)) * 4;
                float4 kx = make_float4(0.0f, 0.0f, 0.0f, 0.0f), vx = kx;
                if (d < dim && any_sees(a, req, key0 + k)) {
                    const long long at = key_at(a, c, pages, key0 + k);
                    if (at < 0) {
                        bad = true;
                    } else {
                        kx = *(const float4*)(c.k + at + h * c.head + d * 4);
                        vx = *(const float4*)(c.v + at + h * c.head + d * 4);
                    }
                }
                *(float4*)(s_k + k * (D + 4) + d) = kx;
                *(float4*)(s_v + k * D + d) = vx;
            }
            __syncthreads();
            if (rg * 4 < R) {
                float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int d = 0; d < D; d += 4) {
                    const float4 kk = *(const float4*)(s_k + col * (D + 4) + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 qq = *(const float4*)(s_q + (rg * 4 + i) * D + d);
                        s[i] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, s[i]))));
                    }
                }
                *(float4*)(s_p + col * kSimtPad + rg * 4) =
                    make_float4(s[0] * scale, s[1] * scale, s[2] * scale, s[3] * scale);
            }
            __syncthreads();
            {
                float s[KT / 16], top = -INFINITY;
#pragma unroll
                for (int i = 0; i < KT / 16; ++i) {
                    const int k = slane + 16 * i;
                    s[i] = srow < R && sees(a, mypos, key0 + k) ? s_p[k * kSimtPad + srow] : -INFINITY;
                    top = fmaxf(top, s[i]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o, 16));
                const float m2 = fmaxf(m, top), base = m2 == -INFINITY ? 0.0f : m2;
                const float corr = exp2f(m - base);
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < KT / 16; ++i) {
                    const float p = exp2f(s[i] - base);
                    sum += p;
                    s_p[(slane + 16 * i) * kSimtPad + srow] = p;
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o, 16);
                l = l * corr + sum;
                m = m2;
                if (slane == 0) s_corr[srow] = corr;
            }
            __syncthreads();
            if (rg * 4 < R) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float corr = s_corr[rg * 4 + i];
#pragma unroll
                    for (int n = 0; n < CN; ++n) acc[i][n] *= corr;
                }
                for (int k = 0; k < KT; ++k) {
                    const float4 p = *(const float4*)(s_p + k * kSimtPad + rg * 4);
#pragma unroll
                    for (int n = 0; n < CN; ++n) {
                        const float v = s_v[k * D + col + 64 * n];
                        // a weight of zero takes nothing, whatever the value
                        acc[0][n] = p.x == 0.0f ? acc[0][n] : fmaf(p.x, v, acc[0][n]);
                        acc[1][n] = p.y == 0.0f ? acc[1][n] : fmaf(p.y, v, acc[1][n]);
                        acc[2][n] = p.z == 0.0f ? acc[2][n] : fmaf(p.z, v, acc[2][n]);
                        acc[3][n] = p.w == 0.0f ? acc[3][n] : fmaf(p.w, v, acc[3][n]);
                    }
                }
            }
        }
        if (__syncthreads_or(bad)) {
            l = __int_as_float(0x7fc00000);
            if (tid == 0) set_status(a.status, SPEC_ERR_PAGE);
        }
        if (slane == 0) {
            s_l[srow] = l;
            s_m[srow] = m;
        }
        __syncthreads();
        const bool whole = w.whole();
        float* part = part_at(a, blockIdx.x, t0 == 0 ? 1 : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rg * 4 + i;
            if (r >= R) break;
            if (whole) {
                const long long row = out_row(a, req.base, h, r0 + r);
                const float inv = 1.0f / s_l[r];
#pragma unroll
                for (int n = 0; n < CN; ++n)
                    if (col + 64 * n < dim) ((T*)a.out)[row * dim + col + 64 * n] = acc[i][n] * inv;
                if (a.lse && col == 0) a.lse[row] = (s_m[r] + log2f(s_l[r])) * 0.6931471805599453f;
            } else {
#pragma unroll
                for (int n = 0; n < CN; ++n)
                    if (col + 64 * n < dim) part[r * dim + col + 64 * n] = acc[i][n];
                if (col == 0) {
                    part[a.tile_rows * dim + r] = s_m[r];
                    part[a.tile_rows * (dim + 1) + r] = s_l[r];
                }
            }
        }
        if (t0 == 0 && !whole) open = w.open();
    }
    if (tid == 0) a.open[blockIdx.x] = open;
    report_requests<T, KT>(a, c, kSimtThreads);
}

AttendPlan attend_simt_plan(int rows, int head_dim, int sms) {
    (void)rows;
    AttendPlan p;
    p.blocks = sms * simt_per_sm(head_dim);
    p.tile_rows = kSimtRows;
    return p;
}

namespace {

template <int D>
int launch(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    auto* f = k_attend_simt<D>;
    static std::atomic<unsigned long long> done{0};
    if (const int rc = allow_smem((const void*)f, (int)simt_smem<D>(), done)) return rc;
    return launch_dependent(f, dim3(blocks), kSimtThreads, simt_smem<D>(), st, 0, a, c);
}

}  // namespace

int attend_simt(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    if (c.head_dim <= 64) return launch<64>(a, c, blocks, st);
    if (c.head_dim <= 128) return launch<128>(a, c, blocks, st);
    return launch<256>(a, c, blocks, st);
}

}  // namespace specv
