// Global gradient norm and clipping over many tensors.
//
//   n = sqrt(sum_k sum_i g_k[i]^2)  or  max |g_k[i]|,   c = min(1, max_norm / (n + 1e-6)),   g_k[i] <- c g_k[i]
//
// The tensors are laid end to end in one element space (their lengths' prefix
// sums); each CTA takes an equal contiguous slice and walks the tensors in it,
// so hundreds of small tensors cost no more launches than one large one.
//
// HBM-bound: one pass reads every element for the norm, a second reads and
// writes it.  The factor is known only when the last element has been read.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "lm_common.cuh"

namespace ddplm {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxGrid = DDP_CLIP_WORKSPACE_BYTES / 8;  // one double of partial result a CTA

struct ClipArgs {
    const void* const* grads;
    void* const* out;  // nullptr: in place
    const int64_t* offset;
    const int32_t* dtypes;
    int32_t ntensors;
    int64_t total;
    double* part;
    float* norm;
    float max_norm;
};

// the last tensor that starts at or before element e (empty tensors before it are skipped over)
__device__ __forceinline__ int find_tensor(const int64_t* offset, int n, int64_t e)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offset[mid] <= e) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A value's square is exact enough in fp32 while it stays well inside its range:
// a vector whose largest magnitude lies outside [2^-40, 2^60] is squared in fp64.
__device__ __forceinline__ bool fp32_square_range(float m) { return m >= 0x1p-40f && m <= 0x1p60f; }

template <int DT, bool INF> struct Accum {
    // sum of squares (fp64) or largest magnitude of N values
    template <int N> __device__ __forceinline__ static void add(double& acc, const float (&x)[N])
    {
        if (INF) {
            float m = static_cast<float>(acc);
#pragma unroll
            for (int j = 0; j < N; ++j) m = (fabsf(x[j]) > m || x[j] != x[j]) ? fabsf(x[j]) : m;  // a NaN stays
            acc = m;
        } else {
            float m = 0.f, s = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                m = fmaxf(m, fabsf(x[j]));
                s = fmaf(x[j], x[j], s);
            }
            if (fp32_square_range(m)) {
                acc += static_cast<double>(s);
            } else if (!(s == 0.f && m == 0.f)) {
#pragma unroll
                for (int j = 0; j < N; ++j) acc += static_cast<double>(x[j]) * static_cast<double>(x[j]);
            }
        }
    }
};

// largest magnitude where a NaN beats everything
__device__ __forceinline__ double pick_max(double a, double b) { return (b > a || b != b) ? b : a; }

template <bool INF> __device__ __forceinline__ double join(double a, double b)
{
    if (INF) return a != a ? a : pick_max(a, b);
    return a + b;
}

// Every thread gets the CTA's joined value; the order is fixed.
template <bool INF> __device__ double block_join(double v)
{
    __shared__ double sh[32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v = join<INF>(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    double r = 0.0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) r = join<INF>(r, sh[w]);
    __syncthreads();
    return r;
}

template <int DT, bool INF>
__device__ __forceinline__ void norm_piece(const void* base, int64_t i0, int64_t n, double& acc)
{
    using T = typename Elem<DT>::T;
    constexpr int N = Vec<DT>::N;
    const T* p = static_cast<const T*>(base) + i0;
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
    if (head > n) head = n;
    const int64_t nv = (n - head) / N;
    const int64_t tail = head + nv * N;
    for (int64_t i = threadIdx.x; i < head; i += blockDim.x) {
        const float x[1] = {Elem<DT>::to_f(p[i])};
        Accum<DT, INF>::template add<1>(acc, x);
    }
    const Vec<DT>* pv = reinterpret_cast<const Vec<DT>*>(p + head);
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < nv; i += blockDim.x) {
        const Vec<DT> v = pv[i];
        float x[N];
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = Elem<DT>::to_f(v.v[j]);
        Accum<DT, INF>::template add<N>(acc, x);
    }
    for (int64_t i = tail + threadIdx.x; i < n; i += blockDim.x) {
        const float x[1] = {Elem<DT>::to_f(p[i])};
        Accum<DT, INF>::template add<1>(acc, x);
    }
}

template <bool INF> __global__ void __launch_bounds__(kThreads) norm_kernel(ClipArgs a)
{
    const int64_t e0 = a.total / gridDim.x * blockIdx.x + min(static_cast<int64_t>(blockIdx.x), a.total % gridDim.x);
    const int64_t e1 = e0 + a.total / gridDim.x + (blockIdx.x < a.total % gridDim.x);
    double acc = 0.0;
    if (e0 < e1) {
        int k = find_tensor(a.offset, a.ntensors, e0);
        for (int64_t e = e0; e < e1 && k < a.ntensors; ++k) {
            const int64_t lo = a.offset[k], hi = a.offset[k + 1];
            const int64_t end = hi < e1 ? hi : e1;
            if (end <= e) continue;
            const void* g = a.grads[k];
            if (g) {
                const int dt = a.dtypes[k];
                if (dt == DDP_F32) norm_piece<DDP_F32, INF>(g, e - lo, end - e, acc);
                else if (dt == DDP_BF16) norm_piece<DDP_BF16, INF>(g, e - lo, end - e, acc);
                else norm_piece<DDP_F16, INF>(g, e - lo, end - e, acc);
            }
            e = end;
        }
    }
    const double r = block_join<INF>(acc);
    if (threadIdx.x == 0) a.part[blockIdx.x] = r;
}

// every CTA joins the partial results again, in the same order
template <bool INF> __device__ float total_norm(const double* part, int n)
{
    double acc = 0.0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) acc = join<INF>(acc, part[i]);
    acc = block_join<INF>(acc);
    return INF ? static_cast<float>(acc) : static_cast<float>(sqrt(acc));
}

template <bool INF> __global__ void __launch_bounds__(kThreads) norm_end_kernel(const double* part, int n, float* norm)
{
    const float r = total_norm<INF>(part, n);
    if (threadIdx.x == 0) *norm = r;
}

template <int DT>
__device__ __forceinline__ void scale_piece(const void* src, void* dst, int64_t i0, int64_t n, float c)
{
    using T = typename Elem<DT>::T;
    constexpr int N = Vec<DT>::N;
    const T* p = static_cast<const T*>(src) + i0;
    T* q = static_cast<T*>(dst) + i0;
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
    // vectors where both sides share their place within 16 bytes
    if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) || head > n) head = n;
    const int64_t nv = (n - head) / N;
    const int64_t tail = head + nv * N;
    for (int64_t i = threadIdx.x; i < head; i += blockDim.x) q[i] = Elem<DT>::from_f(Elem<DT>::to_f(p[i]) * c);
    const Vec<DT>* pv = reinterpret_cast<const Vec<DT>*>(p + head);
    Vec<DT>* qv = reinterpret_cast<Vec<DT>*>(q + head);
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < nv; i += blockDim.x) {
        Vec<DT> v = pv[i];
#pragma unroll
        for (int j = 0; j < N; ++j) v.v[j] = Elem<DT>::from_f(Elem<DT>::to_f(v.v[j]) * c);
        qv[i] = v;
    }
    for (int64_t i = tail + threadIdx.x; i < n; i += blockDim.x) q[i] = Elem<DT>::from_f(Elem<DT>::to_f(p[i]) * c);
}

template <bool INF> __global__ void __launch_bounds__(kThreads) scale_kernel(ClipArgs a, int nparts)
{
    const float norm = total_norm<INF>(a.part, nparts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
    const float ratio = a.max_norm / (norm + 1e-6f);
    const float c = ratio > 1.f ? 1.f : ratio;  // a NaN stays
    if (c == 1.f && !a.out) return;
    const int64_t e0 = a.total / gridDim.x * blockIdx.x + min(static_cast<int64_t>(blockIdx.x), a.total % gridDim.x);
    const int64_t e1 = e0 + a.total / gridDim.x + (blockIdx.x < a.total % gridDim.x);
    if (e0 >= e1) return;
    int k = find_tensor(a.offset, a.ntensors, e0);
    for (int64_t e = e0; e < e1 && k < a.ntensors; ++k) {
        const int64_t lo = a.offset[k], hi = a.offset[k + 1];
        const int64_t end = hi < e1 ? hi : e1;
        if (end <= e) continue;
        const void* g = a.grads[k];
        void* o = a.out ? a.out[k] : const_cast<void*>(g);
        if (g && o) {
            const int dt = a.dtypes[k];
            if (dt == DDP_F32) scale_piece<DDP_F32>(g, o, e - lo, end - e, c);
            else if (dt == DDP_BF16) scale_piece<DDP_BF16>(g, o, e - lo, end - e, c);
            else scale_piece<DDP_F16>(g, o, e - lo, end - e, c);
        }
        e = end;
    }
}

// one wave of CTAs at most, 4096 elements a CTA at least
int grid_for(int64_t total)
{
    const int64_t want = (total + 4095) / 4096;
    const int64_t wave = static_cast<int64_t>(ddp::device_sm_count()) * 4;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, wave, kMaxGrid})));
}

ddp_status check(const char* fn, const ClipArgs& a, int32_t norm_type, const void* workspace, int64_t workspace_bytes)
{
    using ddp::fail;
    if (a.ntensors < 0) return fail(DDP_E_INVAL, "%s: ntensors = %d < 0", fn, a.ntensors);
    if (a.total < 0) return fail(DDP_E_INVAL, "%s: total = %lld < 0", fn, static_cast<long long>(a.total));
    if (a.ntensors == 0 && a.total > 0) return fail(DDP_E_INVAL, "%s: elements without tensors", fn);
    if (norm_type != DDP_NORM_L2 && norm_type != DDP_NORM_INF)
        return fail(DDP_E_INVAL, "%s: unknown norm_type %d", fn, norm_type);
    if (!a.norm) return fail(DDP_E_INVAL, "%s: norm is NULL", fn);
    if (a.total > 0 && (!a.grads || !a.offset || !a.dtypes)) return fail(DDP_E_INVAL, "%s: a table is NULL", fn);
    if (!workspace) return fail(DDP_E_INVAL, "%s: workspace is NULL", fn);
    if (workspace_bytes < DDP_CLIP_WORKSPACE_BYTES)
        return fail(DDP_E_INVAL, "%s: workspace of %lld bytes, needs %d", fn, static_cast<long long>(workspace_bytes),
                    static_cast<int>(DDP_CLIP_WORKSPACE_BYTES));
    if (!aligned16(workspace)) return fail(DDP_E_INVAL, "%s: workspace is not 16-byte aligned", fn);
    return DDP_OK;
}

ddp_status launch(const char* fn, const ClipArgs& a, bool inf, bool clip, void* stream)
{
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int grid = grid_for(a.total);
    if (inf) norm_kernel<true><<<grid, kThreads, 0, s>>>(a);
    else norm_kernel<false><<<grid, kThreads, 0, s>>>(a);
    if (clip) {
        if (inf) scale_kernel<true><<<grid, kThreads, 0, s>>>(a, grid);
        else scale_kernel<false><<<grid, kThreads, 0, s>>>(a, grid);
    } else {
        if (inf) norm_end_kernel<true><<<1, kThreads, 0, s>>>(a.part, grid, a.norm);
        else norm_end_kernel<false><<<1, kThreads, 0, s>>>(a.part, grid, a.norm);
    }
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return ddp::fail(DDP_E_CUDA, "%s: kernel launch failed: %s", fn, cudaGetErrorString(err));
    return ddp::ok();
}

}  // namespace
}  // namespace ddplm

extern "C" ddp_status ddp_grad_norm(const void* const* grads, const int64_t* offset, const int32_t* dtypes,
                                    int32_t ntensors, int64_t total, int32_t norm_type, float* norm, void* workspace,
                                    int64_t workspace_bytes, void* stream)
{
    const ddplm::ClipArgs a{grads, nullptr, offset, dtypes, ntensors, total, static_cast<double*>(workspace), norm, 0.f};
    const ddp_status st = ddplm::check("ddp_grad_norm", a, norm_type, workspace, workspace_bytes);
    if (st != DDP_OK) return st;
    return ddplm::launch("ddp_grad_norm", a, norm_type == DDP_NORM_INF, false, stream);
}

extern "C" ddp_status ddp_clip_grads(const void* const* grads, void* const* out, const int64_t* offset,
                                     const int32_t* dtypes, int32_t ntensors, int64_t total, int32_t norm_type,
                                     float max_norm, float* norm, void* workspace, int64_t workspace_bytes,
                                     void* stream)
{
    const char* fn = "ddp_clip_grads";
    const ddplm::ClipArgs a{grads, out, offset, dtypes, ntensors, total, static_cast<double*>(workspace), norm,
                            max_norm};
    const ddp_status st = ddplm::check(fn, a, norm_type, workspace, workspace_bytes);
    if (st != DDP_OK) return st;
    if (!(max_norm >= 0.f)) return ddp::fail(DDP_E_INVAL, "%s: max_norm = %g is negative or NaN", fn, max_norm);
    return ddplm::launch(fn, a, norm_type == DDP_NORM_INF, true, stream);
}
