// Building blocks of the kernels that go over rows of bf16 or fp32: checked
// loads and stores of a few elements, sums over a row's threads, launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "common.cuh"

namespace ql {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// W consecutive elements, moved as one or two 16-byte words (W * sizeof(T) a
// multiple of 16, 16-byte aligned) or one by one.
template <typename T, int W>
struct alignas(W * sizeof(T) >= 16 ? 16 : W * sizeof(T)) Pack {
    T v[W];
};
template <typename T, int W>
__device__ __forceinline__ Pack<T, W> zero_pack() {
    Pack<T, W> r;
#pragma unroll
    for (int i = 0; i < W; ++i) r.v[i] = from_f32<T>(0.0f);
    return r;
}
template <typename T, int W, typename B>
__device__ __forceinline__ Pack<T, W> load_pack(const T* p, const B& b, int span) {
    Pack<T, W> r = zero_pack<T, W>();
    if (QL_IN(b, span, p, sizeof(T) * W)) {
        if constexpr (sizeof(T) * W > 16) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T) * W / 16); ++i)
                reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(p)[i];
        } else {
            r = *reinterpret_cast<const Pack<T, W>*>(p);
        }
    }
    return r;
}
template <typename T, int W, typename B>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, W>& r, const B& b, int span) {
    if (QL_IN(b, span, p, sizeof(T) * W)) {
        if constexpr (sizeof(T) * W > 16) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T) * W / 16); ++i)
                reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(&r)[i];
        } else {
            *reinterpret_cast<Pack<T, W>*>(p) = r;
        }
    }
}
template <typename T, typename B>
__device__ __forceinline__ T load_one(const T* p, const B& b, int span, T other) {
    return QL_IN(b, span, p, sizeof(T)) ? *p : other;
}
template <typename T, typename B>
__device__ __forceinline__ void store_one(T* p, T v, const B& b, int span) {
    if (QL_IN(b, span, p, sizeof(T))) *p = v;
}

// W elements of a vector of bf16 or fp32 that may be missing (then `other`), from
// element c on; 16-byte aligned where W > 1.
template <int W, typename B>
__device__ __forceinline__ void load_weights(float (&w)[W], const void* p, bool bf16, int64_t c, float other, const B& b, int span) {
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = other;
    } else if (bf16) {
        const Pack<__nv_bfloat16, W> v = load_pack<__nv_bfloat16, W>(static_cast<const __nv_bfloat16*>(p) + c, b, span);
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = to_f32(v.v[i]);
    } else {
        const Pack<float, W> v = load_pack<float, W>(static_cast<const float*>(p) + c, b, span);
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = v.v[i];
    }
}

// v[0 .. N) summed over the threads of a row: a warp, or a whole block by way of
// s [N * 32] in shared memory (which the caller may use again only after a barrier).
// Every thread gets the sums; their order does not depend on timing.
template <int N, bool WARP>
__device__ __forceinline__ void sum_over_row(float (&v)[N], float* s) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (!WARP) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i * 32 + warp] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = lane < warps ? s[i * 32 + lane] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        }
    }
}

// Asynchronous copies into a thread's own place in shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    if constexpr (BYTES > 16) {
        copy_async<16>(to, from);
        copy_async<BYTES - 16>(static_cast<uint8_t*>(to) + 16, static_cast<const uint8_t*>(from) + 16);
    } else if constexpr (BYTES == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(to)), "l"(from), "n"(BYTES) : "memory");
    }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of the thread's groups are on their way; `stages` - 1 of them.
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void copy_wait(int stages) {
    if (stages >= 4) copy_wait<3>();
    else if (stages == 3) copy_wait<2>();
    else if (stages == 2) copy_wait<1>();
    else copy_wait<0>();
}
// Launch with programmatic stream serialization: the kernel may start before its
// predecessor ends and waits for it (griddepcontrol.wait) before its first access.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster_after(void (*kern)(KArgs...), dim3 grid, int threads, unsigned cluster, size_t smem, cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t st, const Args&... args) {
    return launch_cluster_after(kern, grid, threads, 1, smem, st, args...);
}

__host__ __device__ inline bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }
// Rows of es-byte elements, row stride in elements, that start on multiples of `bytes`.
inline bool rows_aligned(const void* p, int64_t es, int64_t stride, int64_t rows, int64_t bytes) {
    return aligned_to(p, bytes) && (rows <= 1 || (stride * es) % bytes == 0);
}

}  // namespace ql
