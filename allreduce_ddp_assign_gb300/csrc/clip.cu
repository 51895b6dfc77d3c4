// Global gradient norm and clipping over many tensors.
//
//   n = sqrt(sum_k sum_i g_k[i]^2)  or  max |g_k[i]|,   c = min(1, max_norm / (n + 1e-6)),   g_k[i] <- c g_k[i]
//
// The tensors are laid end to end in one element space (their lengths' prefix
// sums).  A CTA takes a contiguous slice of it, its warps take turns of some elements,
// and each walks the tensors in its turn by itself, so that hundreds of small tensors
// cost neither more launches nor a wait for each.
//
// HBM-bound: one pass reads every element for the norm, a second reads and writes
// it; the factor is known only when the last element has been read.  The second
// pass goes backwards, where the first one's last elements are still in L2.
//
// Measured on a GB300: 334M fp32 elements in 385 tensors 657 us (4.0 GB, 6.1 TB/s: the
// norm's pass 210 us, 6.3 TB/s); 124M bf16 in 193 tensors 151 us (0.74 GB, 4.9 TB/s; the
// norm's pass 59 us, 4.2 TB/s, where half of the time goes into the squares between the
// loads); 0.33M fp32 in 17 tensors 13 us, which is two launches and their dependent reads.
// Sums of squares: fp32 over at most 32 values, fp64 beyond.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "lm_common.cuh"

namespace ddplm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerSm = 3;        // CTAs of the two passes on an SM
constexpr int kBatch = 4;        // vectors a lane keeps in flight
constexpr int kWindow = kThreads;  // tensors whose tables a CTA holds at a time
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
    int32_t clip;
    int32_t turn;  // elements of a warp's turn (set by the launcher)
};

// A CTA's view of the tables: `count` tensors from `first`.
template <int N> struct Window {
    int64_t offset[N + 1];
    const void* grad[N];
    void* out[N];
    int32_t dtype[N];
    int32_t first, count;
};

// Loads the tables from tensor `first` on; every thread calls it.
template <int N> __device__ __forceinline__ void load_window(Window<N>& w, const ClipArgs& a, int first)
{
    __syncthreads();
    const int i = threadIdx.x;
    const int count = min(N, a.ntensors - first);
    if (i < count) {
        w.offset[i] = a.offset[first + i];
        w.grad[i] = a.grads[first + i];
        w.out[i] = a.out ? a.out[first + i] : const_cast<void*>(w.grad[i]);
        w.dtype[i] = a.dtypes[first + i];
        if (i == count - 1) w.offset[count] = a.offset[first + count];
    }
    if (i == 0) {
        w.first = first;
        w.count = count;
    }
    __syncthreads();
}

// The last tensor that starts at or before element e, found by all threads together.
__device__ __forceinline__ int find_tensor(const ClipArgs& a, int64_t e)
{
    int k = -1;
    for (int base = 0; base < a.ntensors; base += blockDim.x) {
        const int i = base + threadIdx.x;
        k += __syncthreads_count(i < a.ntensors && a.offset[i] <= e);
    }
    return k;
}

// A value's square is exact enough in fp32 while it stays well inside its range:
// values whose largest magnitude lies outside [2^-40, 2^60] are scaled first.
__device__ __forceinline__ bool fp32_square_range(float m) { return m >= 0x1p-40f && m <= 0x1p60f; }

// larger magnitude where a NaN beats everything
__device__ __forceinline__ double pick_max(double a, double b) { return (b > a || b != b) ? b : a; }
template <bool INF> __device__ __forceinline__ double join(double a, double b)
{
    if (INF) return a != a ? a : pick_max(a, b);
    return a + b;
}

// N values (at most 32) into the sum of squares, in fp32 and then once in fp64, or into the largest magnitude.
template <bool INF, int N> __device__ __forceinline__ void add_values(double& acc, const float (&x)[N])
{
    // (four chains each: the loads of the next values wait for these)
    float mm[4] = {0.f, 0.f, 0.f, 0.f};
    if (INF) {
        float bad = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            mm[j & 3] = fmaxf(mm[j & 3], fabsf(x[j]));
            bad = x[j] != x[j] ? x[j] : bad;
        }
        acc = join<true>(acc, bad != bad ? bad : fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3])));
        return;
    }
    float ss[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < N; ++j) {
        mm[j & 3] = fmaxf(mm[j & 3], fabsf(x[j]));
        ss[j & 3] = fmaf(x[j], x[j], ss[j & 3]);
    }
    const float m = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3]));
    float s = (ss[0] + ss[1]) + (ss[2] + ss[3]);
    if (fp32_square_range(m)) {
        acc += static_cast<double>(s);
    } else if (!(s == 0.f && m == 0.f)) {
        // moved into the range by a power of two, whose square is taken out again in fp64
        const bool large = m > 1.f;
        const float f = large ? 0x1p-68f : 0x1p100f;
        s = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) s = fmaf(x[j] * f, x[j] * f, s);
        acc += static_cast<double>(s) * (large ? 0x1p136 : 0x1p-200);
    }
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

// elements before the first 16-byte boundary, at most n
template <typename T> __device__ __forceinline__ int head_of(const T* p, int n)
{
    return min(n, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T)));
}

// one warp, n values (a turn's or fewer) of one tensor
template <int DT, bool INF> __device__ __forceinline__ void norm_piece(const void* base, int64_t i0, int n, int lane, double& acc)
{
    using T = typename Elem<DT>::T;
    constexpr int N = Vec<DT>::N;
    const T* p = static_cast<const T*>(base) + i0;
    const int head = head_of(p, n), nv = (n - head) / N, tail = head + nv * N;
    // the ragged ends: fewer than 32 values each
    float e[2] = {lane < head ? Elem<DT>::to_f(p[lane]) : 0.f, tail + lane < n ? Elem<DT>::to_f(p[tail + lane]) : 0.f};
    const Vec<DT>* pv = reinterpret_cast<const Vec<DT>*>(p + head);
    int i = lane;
    for (; i + 32 * (kBatch - 1) < nv; i += 32 * kBatch) {
        Vec<DT> v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) v[u] = pv[i + 32 * u];
        float x[kBatch * N];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
            for (int j = 0; j < N; ++j) x[u * N + j] = Elem<DT>::to_f(v[u].v[j]);
        add_values<INF>(acc, x);
    }
    for (; i < nv; i += 32) {
        const Vec<DT> v = pv[i];
        float x[N];
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = Elem<DT>::to_f(v.v[j]);
        add_values<INF>(acc, x);
    }
    add_values<INF>(acc, e);
}

template <int DT> __device__ __forceinline__ void scale_piece(const void* src, void* dst, int64_t i0, int n, int lane, float c)
{
    using T = typename Elem<DT>::T;
    constexpr int N = Vec<DT>::N;
    const T* p = static_cast<const T*>(src) + i0;
    T* q = static_cast<T*>(dst) + i0;
    if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) {
        // vectors need both sides at the same place within 16 bytes
        for (int i = lane; i < n; i += 32 * kBatch) {
            T v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (i + 32 * u < n) v[u] = p[i + 32 * u];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (i + 32 * u < n) q[i + 32 * u] = Elem<DT>::from_f(Elem<DT>::to_f(v[u]) * c);
        }
        return;
    }
    const int head = head_of(p, n), nv = (n - head) / N, tail = head + nv * N;
    if (lane < head) q[lane] = Elem<DT>::from_f(Elem<DT>::to_f(p[lane]) * c);
    if (tail + lane < n) q[tail + lane] = Elem<DT>::from_f(Elem<DT>::to_f(p[tail + lane]) * c);
    const Vec<DT>* pv = reinterpret_cast<const Vec<DT>*>(p + head);
    Vec<DT>* qv = reinterpret_cast<Vec<DT>*>(q + head);
    for (int i = lane; i < nv; i += 32 * kBatch) {
        Vec<DT> v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i + 32 * u < nv) v[u] = pv[i + 32 * u];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i + 32 * u >= nv) continue;
#pragma unroll
            for (int j = 0; j < N; ++j) v[u].v[j] = Elem<DT>::from_f(Elem<DT>::to_f(v[u].v[j]) * c);
            // the results are not read again here: they leave L2 first
            __stcs(reinterpret_cast<uint4*>(qv + i + 32 * u), *reinterpret_cast<const uint4*>(&v[u]));
        }
    }
}

// What a walk over the elements does with a piece of a tensor.
template <bool INF> struct NormWalk {
    double acc = 0.0;
    template <int N> __device__ __forceinline__ void piece(const Window<N>& w, int k, int64_t i0, int n, int lane)
    {
        if (!w.grad[k]) return;
        if (w.dtype[k] == DDP_F32) norm_piece<DDP_F32, INF>(w.grad[k], i0, n, lane, acc);
        else if (w.dtype[k] == DDP_BF16) norm_piece<DDP_BF16, INF>(w.grad[k], i0, n, lane, acc);
        else norm_piece<DDP_F16, INF>(w.grad[k], i0, n, lane, acc);
    }
};
struct ScaleWalk {
    float c;
    template <int N> __device__ __forceinline__ void piece(const Window<N>& w, int k, int64_t i0, int n, int lane)
    {
        if (!w.grad[k] || !w.out[k]) return;
        if (w.dtype[k] == DDP_F32) scale_piece<DDP_F32>(w.grad[k], w.out[k], i0, n, lane, c);
        else if (w.dtype[k] == DDP_BF16) scale_piece<DDP_BF16>(w.grad[k], w.out[k], i0, n, lane, c);
        else scale_piece<DDP_F16>(w.grad[k], w.out[k], i0, n, lane, c);
    }
};

// One CTA's walk over [e0, e1), in strides of `warps` turns of `turn` elements, from the
// end where BACK.  The window holds the tensors of the slice; where it does not hold all
// of them the slice is walked in parts, a window each.
template <bool BACK, typename F, int N>
__device__ __forceinline__ void walk(Window<N>& w, const ClipArgs& a, int first, int64_t e0, int64_t e1, F& f)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, turn = a.turn;
    if (w.first != first) load_window(w, a, first);
    for (int64_t s0 = e0; s0 < e1;) {
        const int64_t s1 = min(e1, w.offset[w.count]);
        const int64_t turns = (s1 - s0 + turn - 1) / turn;
        int k = BACK ? w.count - 1 : 0;
        for (int64_t j = warp; j < turns; j += warps) {
            const int64_t t0 = s0 + (BACK ? turns - 1 - j : j) * turn, t1 = min(s1, t0 + turn);
            // the tensor of the turn's first element (k only ever moves one way)
            if (BACK)
                while (w.offset[k] > t0) --k;
            else
                while (w.offset[k + 1] <= t0) ++k;
            int kk = k;
            for (int64_t e = t0; e < t1; ++kk) {
                const int64_t end = min(t1, w.offset[kk + 1]);
                if (end <= e) continue;
                f.piece(w, kk, e - w.offset[kk], static_cast<int>(end - e), lane);
                e = end;
            }
        }
        s0 = s1;
        if (s0 >= e1 || w.first + w.count >= a.ntensors) break;
        load_window(w, a, w.first + w.count);
    }
}

__device__ __forceinline__ void slice_of(const ClipArgs& a, int cta, int ctas, int64_t* e0, int64_t* e1)
{
    const int64_t per = a.total / ctas, more = a.total % ctas;
    *e0 = per * cta + min(static_cast<int64_t>(cta), more);
    *e1 = *e0 + per + (cta < more);
}

__device__ __forceinline__ float factor(const ClipArgs& a, float norm)
{
    const float ratio = a.max_norm / (norm + 1e-6f);
    return ratio > 1.f ? 1.f : ratio;  // a NaN stays
}

template <bool INF> __global__ void __launch_bounds__(kThreads, kPerSm) norm_kernel(const __grid_constant__ ClipArgs a)
{
    __shared__ Window<kWindow> w;
    wait_for_previous();
    allow_next();
    int64_t e0, e1;
    slice_of(a, blockIdx.x, gridDim.x, &e0, &e1);
    NormWalk<INF> f;
    if (threadIdx.x == 0) w.first = -1;
    __syncthreads();
    if (e0 < e1) walk<false>(w, a, a.ntensors <= kWindow ? 0 : find_tensor(a, e0), e0, e1, f);
    const double r = block_join<INF>(f.acc);
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
    wait_for_previous();
    const float r = total_norm<INF>(part, n);
    if (threadIdx.x == 0) *norm = r;
}

template <bool INF> __global__ void __launch_bounds__(kThreads, kPerSm) scale_kernel(const __grid_constant__ ClipArgs a)
{
    __shared__ Window<kWindow> w;
    int64_t e0, e1;
    slice_of(a, blockIdx.x, gridDim.x, &e0, &e1);
    // The tables are older than the norm pass, which let this kernel start: they are read
    // before that pass has ended.
    const int first = e0 < e1 && a.ntensors > kWindow ? find_tensor(a, e0) : 0;
    if (e0 < e1) load_window(w, a, first);
    wait_for_previous();
    const float norm = total_norm<INF>(a.part, gridDim.x);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
    const float c = factor(a, norm);
    if (e0 >= e1 || (c == 1.f && !a.out)) return;
    ScaleWalk f{c};
    walk<true>(w, a, first, e0, e1, f);
}

// Elements of a warp's turn, a multiple of 256.  Long turns keep a lane's loads in batches
// (124M bf16 elements: 171 us with 2048, 156 with 4096, 158 with 8192); few elements
// are spread over the machine's warps (1M elements: 21.5 us with 2048, 24.6 with 4096).
constexpr int kMaxTurn = 4096;
int turn_for(int64_t total)
{
    const int64_t warps = static_cast<int64_t>(ddp::device_sm_count()) * kPerSm * kWarps;
    return static_cast<int>(std::min<int64_t>(kMaxTurn, (total / warps + 256) / 256 * 256));
}

// one wave of CTAs at most, a turn for each warp at least
int grid_for(int64_t total, int turn)
{
    const int64_t want = (total + turn * kWarps - 1) / (turn * kWarps);
    const int64_t wave = static_cast<int64_t>(ddp::device_sm_count()) * kPerSm;
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

template <bool INF> cudaError_t launch_as(const ClipArgs& a, cudaStream_t s)
{
    const dim3 grid(grid_for(a.total, a.turn));
    const cudaError_t e = launch_chained(norm_kernel<INF>, grid, kThreads, 0, s, a);
    if (e != cudaSuccess) return e;
    if (a.clip) return launch_chained(scale_kernel<INF>, grid, kThreads, 0, s, a);
    return launch_chained(norm_end_kernel<INF>, dim3(1), kThreads, 0, s, static_cast<const double*>(a.part),
                          static_cast<int>(grid.x), a.norm);
}

ddp_status launch(const char* fn, ClipArgs a, bool inf, void* stream)
{
    a.turn = turn_for(a.total);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err = inf ? launch_as<true>(a, s) : launch_as<false>(a, s);
    if (err != cudaSuccess) return ddp::fail(DDP_E_CUDA, "%s: kernel launch failed: %s", fn, cudaGetErrorString(err));
    return ddp::ok();
}

}  // namespace
}  // namespace ddplm

extern "C" ddp_status ddp_grad_norm(const void* const* grads, const int64_t* offset, const int32_t* dtypes,
                                    int32_t ntensors, int64_t total, int32_t norm_type, float* norm, void* workspace,
                                    int64_t workspace_bytes, void* stream)
{
    const ddplm::ClipArgs a{grads, nullptr, offset, dtypes, ntensors, total, static_cast<double*>(workspace), norm, 0.f, 0, 0};
    const ddp_status st = ddplm::check("ddp_grad_norm", a, norm_type, workspace, workspace_bytes);
    if (st != DDP_OK) return st;
    return ddplm::launch("ddp_grad_norm", a, norm_type == DDP_NORM_INF, stream);
}

extern "C" ddp_status ddp_clip_grads(const void* const* grads, void* const* out, const int64_t* offset,
                                     const int32_t* dtypes, int32_t ntensors, int64_t total, int32_t norm_type,
                                     float max_norm, float* norm, void* workspace, int64_t workspace_bytes,
                                     void* stream)
{
    const char* fn = "ddp_clip_grads";
    const ddplm::ClipArgs a{grads, out, offset, dtypes, ntensors, total, static_cast<double*>(workspace), norm,
                            max_norm, 1, 0};
    const ddp_status st = ddplm::check(fn, a, norm_type, workspace, workspace_bytes);
    if (st != DDP_OK) return st;
    if (!(max_norm >= 0.f)) return ddp::fail(DDP_E_INVAL, "%s: max_norm = %g is negative or NaN", fn, max_norm);
    return ddplm::launch(fn, a, norm_type == DDP_NORM_INF, stream);
}
