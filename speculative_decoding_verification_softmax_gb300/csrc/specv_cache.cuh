// What the paged key-value cache calls share: the cache as the kernels see it,
// its checks on the host, and conversions between the element types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "specv_common.cuh"

namespace specv {

// Division by a positive constant of numbers below 2^31 (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994):
// with 2^(s-1) < d <= 2^s and m = floor(2^32 (2^s - d) / d) + 1 the quotient is
// (floor(n m / 2^32) + n) >> s.
struct FastDiv {
    uint32_t d, m, s;
    FastDiv() = default;
    explicit FastDiv(uint32_t divisor) : d(divisor), s(0) {
        while ((1ull << s) < d) ++s;
        m = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

// Strides in bytes.
struct CacheView {
    char* k;
    char* v;
    long long layer, page, token, head;
    int layers, pages, page_size, kv_heads, head_dim;
    FastDiv by_page;
    const float* k_scale;
    const float* v_scale;
};

inline int dtype_size(spec_dtype dt) {
    return dt == SPEC_F32 ? 4 : dt == SPEC_E4M3 ? 1 : 2;
}

// Host checks of a cache; `data`: its storage is read or written.
inline int cache_view(const spec_cache* c, CacheView& o) {
    if (!c) return SPEC_ERR_NULL;
    if (c->dt != SPEC_F32 && c->dt != SPEC_BF16 && c->dt != SPEC_F16 && c->dt != SPEC_E4M3) return SPEC_ERR_SHAPE;
    if (c->layers < 1 || c->pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->kv_heads > 65535 ||
        c->head_dim < 8 || c->head_dim > SPEC_MAX_HEAD_DIM || (c->head_dim & 7))
        return SPEC_ERR_SHAPE;
    const long long es = dtype_size(c->dt);
    if ((c->head_dim * es) & 15) return SPEC_ERR_SHAPE;
    if (!c->k || !c->v) return SPEC_ERR_NULL;
    if (((uintptr_t)c->k | (uintptr_t)c->v) & 15) return SPEC_ERR_ALIGN;
    if (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3) return SPEC_ERR_ALIGN;
    o.layer = c->layer_stride * es;
    o.page = c->page_stride * es;
    o.token = c->token_stride * es;
    o.head = c->head_stride * es;
    if ((o.layer | o.page | o.token | o.head) & 15) return SPEC_ERR_ALIGN;
    o.k = (char*)c->k;
    o.v = (char*)c->v;
    o.layers = c->layers;
    o.pages = c->pages;
    o.page_size = c->page_size;
    o.kv_heads = c->kv_heads;
    o.head_dim = c->head_dim;
    o.by_page = FastDiv((uint32_t)c->page_size);
    o.k_scale = c->dt == SPEC_E4M3 ? c->k_scale : nullptr;
    o.v_scale = c->dt == SPEC_E4M3 ? c->v_scale : nullptr;
    return SPEC_OK;
}

// SMs of the current device.
inline int sm_count(int& sms) {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ERR_CUDA;
    sms = known[dev].load(std::memory_order_relaxed);
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SPEC_ERR_CUDA;
        known[dev].store(sms, std::memory_order_relaxed);
    }
    return SPEC_OK;
}

// Launches a programmatic dependent of the kernel before it in the stream: its
// blocks may be placed while that one drains.  Every kernel launched so waits
// (pdl_wait) before it touches memory, and lets the next one be placed at once
// (pdl_trigger).  `cluster` > 0: one cluster of so many blocks.
template <typename... P, typename... A>
int launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster,
                     A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// ------------------------------------------------------------- element types
template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_fp8_e4m3>(__nv_fp8_e4m3 x) { return (float)x; }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half(x); }
// to nearest even, clamped to the largest finite value (a NaN stays NaN)
template <>
__device__ __forceinline__ __nv_fp8_e4m3 from_f32<__nv_fp8_e4m3>(float x) { return __nv_fp8_e4m3(x); }

// N adjacent elements as one access (N * sizeof(T) = 4, 8, 16 or 32 bytes).
template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Vec {
    T x[N];
};

}  // namespace specv
