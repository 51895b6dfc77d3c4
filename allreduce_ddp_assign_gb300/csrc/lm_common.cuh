// Definitions shared by the language-model kernels (clip.cu, embedding.cu,
// vocab_loss.cu): element types, 16-byte vectors, ids, the status word.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "common.h"

namespace ddplm {

constexpr int kErrWait = 1;  // a wait ran out
constexpr int kErrId = 2;    // a token id or target out of range

// Address of the status word of ddp_lm_status on the current device (nullptr if unavailable).
int* lm_status_word();

template <int DT> struct Elem;
template <> struct Elem<DDP_F32> {
    using T = float;
    __device__ __forceinline__ static float to_f(T x) { return x; }
    __device__ __forceinline__ static T from_f(float x) { return x; }
};
template <> struct Elem<DDP_BF16> {
    using T = __nv_bfloat16;
    __device__ __forceinline__ static float to_f(T x) { return __bfloat162float(x); }
    __device__ __forceinline__ static T from_f(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Elem<DDP_F16> {
    using T = __half;
    __device__ __forceinline__ static float to_f(T x) { return __half2float(x); }
    __device__ __forceinline__ static T from_f(float x) { return __float2half_rn(x); }
};

// 16 bytes of elements
template <int DT> struct __align__(16) Vec {
    static constexpr int N = 16 / static_cast<int>(sizeof(typename Elem<DT>::T));
    typename Elem<DT>::T v[N];
};

__host__ __device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline int elem_size(int dt) { return dt == DDP_F32 ? 4 : 2; }
inline bool known_dtype(int dt) { return dt == DDP_F32 || dt == DDP_BF16 || dt == DDP_F16; }

__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, int64_t i)
{
    return id_bytes == 8 ? __ldg(static_cast<const long long*>(ids) + i)
                         : static_cast<int64_t>(__ldg(static_cast<const int*>(ids) + i));
}

// Launched so that it may start while the kernel before it ends: everything that
// kernel wrote is read after this.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may be started (it still waits for this one's end before it reads anything).
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_plain(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A&&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, A&&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace ddplm
