// Attention over the items of a plan on the CUDA cores: fp32 rows, whose products
// keep 32 bits.
//
// A block takes one unit at a time: 64 query rows against tiles of KT keys, which
// two buffers of cp.async bring.  A thread has 4 rows and KT / 16 keys of the scores,
// and the same 4 rows and D / 16 columns of the output: 16 bytes of shared memory feed
// 5 to 8 multiplications a lane, where the 16-row kernel's feed 3.  A row's 16 threads
// are half a warp, which takes its softmax by shuffles and passes its weights through
// shared memory among itself: a tile costs one barrier.  One pass over the keys with
// the running maximum and sum, to base 2.
//
// 75 x 33 rows behind 1333 positions, 32/2 heads of 128: 1.82 ms, 35 TFLOP/s (the 16-row
// kernel 3.78 ms), bound by the multiplications and the loads that feed them alike.  One
// token of 64 requests, of whose 64 rows a unit has 4: 253 us for 272 MB.
#include <type_traits>

#include "specv_attend.cuh"

namespace specv {

constexpr int kF32Threads = 256;
constexpr int kF32Rows = 64;

constexpr int f32_keys(int dim) { return dim <= 64 ? 64 : 32; }
// Blocks of an SM, by shared memory: 102, 109 and 207 KB each.
constexpr int f32_per_sm(int dim) { return dim <= 128 ? 2 : 1; }

template <int D>
struct F32Shape {
    static constexpr int kKeys = f32_keys(D);
    static constexpr int kQ = D + 4;          // floats of a row of Q and K: conflict-free 16-byte loads
    static constexpr int kP = kF32Rows + 4;   // of a key's weights
    static constexpr int kSmem = 4 * (kF32Rows * kQ + 2 * kKeys * (kQ + D) + kKeys * kP);
};

__device__ __forceinline__ void f32_fetch(float* to, const char* from, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(take ? 16 : 0)
                 : "memory");
}

// c += a b, two of them in one instruction.
__device__ __forceinline__ void fma_two(float2& c, float2 a, float2 b) {
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "+f"(c.x), "+f"(c.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
}

template <int D>
__global__ void __launch_bounds__(kF32Threads, f32_per_sm(D)) k_attend_f32(AttendArgs a, CacheView c) {
    using Sh = F32Shape<D>;
    constexpr int KT = Sh::kKeys, QS = Sh::kQ, PS = Sh::kP, KN = KT / 16, CN = D / 64;
    extern __shared__ float4 smem4[];
    float* s_q = (float*)smem4;               // [64][QS]
    float* s_k = s_q + kF32Rows * QS;         // [2][KT][QS]
    float* s_v = s_k + 2 * KT * QS;           // [2][KT][D]
    float* s_p = s_v + 2 * KT * D;            // [KT][PS]: weights, by key
    __shared__ RunShared<kF32Threads> s_run;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;

    pdl_trigger();
    pdl_wait();
    run_of<KT, true>(a, c, s_run);
    const int dim = c.head_dim;
    const float scale = a.scale;
    Walk<KT, true> w(a, c, s_run.run);
    while (w.next(a, c)) {
        const Request& req = w.req;
        const int t0 = w.t0, nt = w.nt, h = w.h, r0 = w.r0, R = w.R;
        const int32_t* pages = pages_of<true>(a, req, w.b);
        bool bad = false;
        auto fetch = [&](int t) {
            const int key0 = tile_key<KT>(req, t);
            float* k = s_k + (t & 1) * KT * QS;
            float* v = s_v + (t & 1) * KT * D;
#pragma unroll
            for (int u = 0; u < KT * (D / 4) / kF32Threads; ++u) {
                const int i = u * kF32Threads + tid, row = i / (D / 4), d = (i - row * (D / 4)) * 4;
                bool take = d < dim && any_sees(a, req, key0 + row);
                long long at = 0;
                if (take) {
                    at = key_at(a, c, pages, key0 + row);
                    if (at < 0) {
                        bad = true;
                        take = false;
                    }
                }
                at = take ? at + h * c.head + d * 4 : 0;
                f32_fetch(k + row * QS + d, c.k + at, take);
                f32_fetch(v + row * D + d, c.v + at, take);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        __syncthreads();  // the unit before is done with its buffers
        fetch(t0);
#pragma unroll 4
        for (int i = tid; i < kF32Rows * (D / 4); i += kF32Threads) {
            const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < R && d < dim) {
                const int j = (int)a.by_group.div((uint32_t)(r0 + r));
                const int head = h * a.group + (r0 + r - j * a.group);
                x = *(const float4*)(a.q + (long long)row_of<true>(a, req, j) * a.q_row + head * a.q_head + d * 4);
            }
            *(float4*)(s_q + r * QS + d) = x;
        }
        const bool active = (ty & ~1) * 4 < R;  // the warp has rows
        int pos[4];
        float m[4], l[4];
        float4 acc[4][CN];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pos[i] = position_of<true>(req, (int)a.by_group.div((uint32_t)(r0 + ty * 4 + i)));
            m[i] = -INFINITY;
            l[i] = 0.0f;
#pragma unroll
            for (int n = 0; n < CN; ++n) acc[i][n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }

        for (int t = t0; t < t0 + nt; ++t) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();  // tile t is there, and tile t - 1 is done with
            if (t + 1 < t0 + nt) fetch(t + 1);
            if (!active) continue;
            const int key0 = tile_key<KT>(req, t);
            const float* k = s_k + (t & 1) * KT * QS + tx * QS;
            const float* q = s_q + ty * 4 * QS;
            float s[4][KN];
            float2 s2[4][KN];  // the sums of even and odd columns
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < KN; ++n) s2[i][n] = make_float2(0.0f, 0.0f);
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 qq[4], kk[KN];
#pragma unroll
                for (int i = 0; i < 4; ++i) qq[i] = *(const float4*)(q + i * QS + d);
#pragma unroll
                for (int n = 0; n < KN; ++n) kk[n] = *(const float4*)(k + n * 16 * QS + d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n = 0; n < KN; ++n) {
                        fma_two(s2[i][n], make_float2(qq[i].x, qq[i].y), make_float2(kk[n].x, kk[n].y));
                        fma_two(s2[i][n], make_float2(qq[i].z, qq[i].w), make_float2(kk[n].z, kk[n].w));
                    }
            }
            const bool part = !all_see<KT>(a, req, key0);
            float corr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < KN; ++n) {
                    s[i][n] = (s2[i][n].x + s2[i][n].y) * scale;
                    if (part && !sees(a, pos[i], key0 + tx + 16 * n)) s[i][n] = -INFINITY;
                    top = fmaxf(top, s[i][n]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o, 16));
                const float now = fmaxf(m[i], top), ref = now == -INFINITY ? 0.0f : now;
                corr[i] = exp2f(m[i] - ref);
                m[i] = now;
                l[i] *= corr[i];
#pragma unroll
                for (int n = 0; n < KN; ++n) {
                    s[i][n] = exp2f(s[i][n] - ref);
                    l[i] += s[i][n];
                }
#pragma unroll
                for (int n = 0; n < CN; ++n) {
                    acc[i][n].x *= corr[i];
                    acc[i][n].y *= corr[i];
                    acc[i][n].z *= corr[i];
                    acc[i][n].w *= corr[i];
                }
            }
            float* p = s_p + ty * 4;
            __syncwarp();  // the weights of the tile before have been read
#pragma unroll
            for (int n = 0; n < KN; ++n)
                *(float4*)(p + (tx + 16 * n) * PS) = make_float4(s[0][n], s[1][n], s[2][n], s[3][n]);
            __syncwarp();
            const float* v = s_v + (t & 1) * KT * D + tx * 4;
            auto products = [&](auto cut) {
#pragma unroll 4
                for (int key = 0; key < KT; ++key) {
                    const float4 pp = *(const float4*)(p + key * PS);
                    const float x[4] = {pp.x, pp.y, pp.z, pp.w};
#pragma unroll
                    for (int n = 0; n < CN; ++n) {
                        const float4 vv = *(const float4*)(v + key * D + 64 * n);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // where a border cuts, a weight of zero takes nothing, whatever the value
                            if (decltype(cut)::value && x[i] == 0.0f) continue;
                            float2* o = (float2*)&acc[i][n];
                            fma_two(o[0], make_float2(x[i], x[i]), make_float2(vv.x, vv.y));
                            fma_two(o[1], make_float2(x[i], x[i]), make_float2(vv.z, vv.w));
                        }
                    }
                }
            };
            if (part) products(std::true_type{});
            else products(std::false_type{});
        }
        const bool missing = __syncthreads_or(bad);
        if (missing && tid == 0) set_status(a.status, SPEC_ERR_PAGE);
        const bool whole = w.whole(), direct = whole && req.kind == kAlone;
        float* parts = part_at(a, blockIdx.x, t0 == 0 ? 1 : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o, 16);
            const int r = ty * 4 + i;
            if (r >= R) continue;
            if (missing) l[i] = __int_as_float(0x7fc00000);
            const long long row = shared_out_row(a, req, h, r0 + r), at = where_of(a, req.kind, row);
            const PartRow to = whole ? side_row(a, dim, at) : part_row(a, parts, dim, r);
            float* o = direct ? (float*)a.out + row * dim : to.o;
            const float inv = direct ? 1.0f / l[i] : 1.0f;
#pragma unroll
            for (int n = 0; n < CN; ++n)
                if (tx * 4 + 64 * n < dim)
                    *(float4*)(o + tx * 4 + 64 * n) =
                        make_float4(acc[i][n].x * inv, acc[i][n].y * inv, acc[i][n].z * inv, acc[i][n].w * inv);
            if (tx == 0) {
                if (!direct) {
                    *to.m = m[i];
                    *to.l = l[i];
                } else if (a.lse) {
                    a.lse[row] = (m[i] + log2f(l[i])) * 0.6931471805599453f;
                }
                if (t0 == 0) tell(a, at, whole, direct, w.open().x, r);
            }
        }
    }
    report_requests<float, KT, true>(a, c, kF32Threads);
}

AttendPlan attend_f32_shared_plan(int head_dim, int sms) {
    AttendPlan p;
    p.blocks = sms * f32_per_sm(head_dim);
    p.tile_rows = kF32Rows;
    return p;
}

namespace {

template <int D>
int launch(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    auto* f = k_attend_f32<D>;
    static std::atomic<unsigned long long> done{0};
    if (const int rc = allow_smem((const void*)f, F32Shape<D>::kSmem, done)) return rc;
    return launch_dependent(f, dim3(blocks), kF32Threads, F32Shape<D>::kSmem, st, 0, a, c);
}

}  // namespace

int attend_f32_shared(const AttendArgs& a, const CacheView& c, int blocks, cudaStream_t st) {
    if (c.head_dim <= 64) return launch<64>(a, c, blocks, st);
    if (c.head_dim <= 128) return launch<128>(a, c, blocks, st);
    return launch<256>(a, c, blocks, st);
}

}  // namespace specv
