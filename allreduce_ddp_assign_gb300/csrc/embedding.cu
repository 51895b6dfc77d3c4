// Token embedding: lookup with a scale, and the table's gradient by sorted tokens.
//
//   out[t] = s * W[id_t]                      dW[v] = s * sum over t with id_t = v of dY[t]
//
// The gradient is a segmented sum.  Tokens are sorted by id (equal ids in token
// order) and each row of dW is the fp32 sum of its run, taken in that order: no
// atomics, the same bits every time.  HBM-bound: dY is read once, dW written once.
//
// Sort: one launch in which every CTA owns a range of ids, reads all the tokens
// and keeps those of its range.  A token's place is (tokens with smaller ids) +
// (earlier tokens with its id); the first count covers the ranges before the CTA's
// too, so no CTA needs a result of another.
#include <algorithm>
#include <atomic>

#include "lm_common.cuh"

namespace ddplm {
namespace {

__device__ int g_lm_status = 0;

}  // namespace

int* lm_status_word()
{
    static std::atomic<int*> cached[ddp::kMaxDevices] = {};
    const int dev = ddp::current_device();
    int* p = dev >= 0 ? cached[dev].load(std::memory_order_acquire) : nullptr;
    if (!p) {
        void* a = nullptr;
        if (cudaGetSymbolAddress(&a, g_lm_status) != cudaSuccess) return nullptr;
        p = static_cast<int*>(a);
        if (dev >= 0) cached[dev].store(p, std::memory_order_release);
    }
    return p;
}

namespace {

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
template <int DT, bool VEC>
__global__ void __launch_bounds__(256)
lookup_kernel(const void* weight, int64_t ws, int64_t vocab, int64_t dim, const void* ids, int id_bytes, int64_t ntokens,
              float scale, void* out, int64_t os, int* status)
{
    using T = typename Elem<DT>::T;
    constexpr int N = VEC ? Vec<DT>::N : 1;
    const int64_t per_row = dim / N;  // VEC: dim is a multiple of N
    const int64_t n = ntokens * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = i / per_row, c = (i - t * per_row) * N;
        const int64_t id = load_id(ids, id_bytes, t);
        const bool good = id >= 0 && id < vocab;
        if (!good && c == 0) atomicOr(status, kErrId);
        const T* src = static_cast<const T*>(weight) + (good ? id : 0) * ws + c;
        T* dst = static_cast<T*>(out) + t * os + c;
        if (VEC) {
            Vec<DT> v = *reinterpret_cast<const Vec<DT>*>(src);
#pragma unroll
            for (int j = 0; j < N; ++j) v.v[j] = Elem<DT>::from_f(good ? Elem<DT>::to_f(v.v[j]) * scale : 0.f);
            *reinterpret_cast<Vec<DT>*>(dst) = v;
        } else {
            *dst = Elem<DT>::from_f(good ? Elem<DT>::to_f(*src) * scale : 0.f);
        }
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxRange = 1024;  // ids a sorting CTA owns at most (its counters: 4 bytes an id and warp)

struct SortArgs {
    const void* ids;
    int32_t id_bytes;
    int32_t ntokens;
    int64_t vocab, padding_idx;
    int32_t range;   // ids per CTA
    int32_t* order;  // [ntokens] tokens sorted by id
    int32_t* start;  // [vocab + 1] first place of each id in `order`
    int* status;
};

__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortArgs a)
{
    extern __shared__ int32_t sh[];
    int32_t* cnt = sh;                          // [warp][range]
    int32_t* row = sh + kSortWarps * a.range;   // [range] first place of the row, within this CTA's tokens
    __shared__ int32_t less_w[kSortWarps], part[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.range;
    const int64_t hi = lo + a.range < a.vocab ? lo + a.range : a.vocab;
    const int nr = static_cast<int>(hi - lo);
    for (int i = tid; i < kSortWarps * a.range; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    // each warp counts a contiguous stretch of tokens
    const int per = (a.ntokens + kSortWarps - 1) / kSortWarps;
    const int t0 = min(warp * per, a.ntokens), t1 = min(t0 + per, a.ntokens);
    int32_t less = 0;
    for (int t = t0 + lane; t < t1; t += 32) {
        const int64_t id = load_id(a.ids, a.id_bytes, t);
        if (id < 0 || id >= a.vocab) {
            if (blockIdx.x == 0) atomicOr(a.status, kErrId);
        } else if (id != a.padding_idx) {
            less += id < lo;
            if (id >= lo && id < hi) atomicAdd(&cnt[warp * a.range + static_cast<int>(id - lo)], 1);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) less += __shfl_xor_sync(0xffffffffu, less, o);
    if (lane == 0) less_w[warp] = less;
    __syncthreads();
    int32_t base = 0;
    for (int w = 0; w < kSortWarps; ++w) base += less_w[w];
    // per id: total over the warps, then an exclusive scan over the ids
    int32_t total = 0;
    if (tid < nr)
        for (int w = 0; w < kSortWarps; ++w) total += cnt[w * a.range + tid];
    int32_t inc = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int32_t before = base;
    for (int w = 0; w < warp; ++w) before += part[w];
    if (tid < nr) {
        int32_t at = before + inc - total;
        row[tid] = at;
        a.start[lo + tid] = at;
        if (lo + tid + 1 == a.vocab) a.start[a.vocab] = at + total;
        // cnt becomes the first place of this id's tokens from warp w's stretch
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = cnt[w * a.range + tid];
            cnt[w * a.range + tid] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int t = t0; t < t1; t += 32) {
        int64_t id = -1;
        if (t + lane < t1) id = load_id(a.ids, a.id_bytes, t + lane);
        const bool mine = id >= lo && id < hi && id != a.padding_idx;
        const uint32_t any = __ballot_sync(0xffffffffu, mine);
        if (!any) continue;
        if (mine) {
            const int r = static_cast<int>(id - lo);
            const uint32_t same = __match_any_sync(any, r);
            int32_t* c = &cnt[warp * a.range + r];
            const int32_t at = *c + __popc(same & ((1u << lane) - 1u));
            a.order[at] = t + lane;
            __syncwarp(same);
            if (lane == __ffs(same) - 1) *c += __popc(same);
        }
        __syncwarp();
    }
}

struct GradArgs {
    const void* g;
    int64_t gs;
    const int32_t* order;
    const int32_t* start;
    int64_t vocab, dim;
    float scale;
    void* gw;
    int64_t ws;
    int32_t accumulate;
};

// one CTA a table row
template <int DT, int WT> __global__ void __launch_bounds__(128) rows_kernel(GradArgs a)
{
    using T = typename Elem<DT>::T;
    using O = typename Elem<WT>::T;
    for (int64_t v = blockIdx.x; v < a.vocab; v += gridDim.x) {
        const int s0 = a.start[v], s1 = a.start[v + 1];
        if (s0 == s1 && a.accumulate) continue;
        O* dst = static_cast<O*>(a.gw) + v * a.ws;
        for (int64_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
            float acc = 0.f;
            for (int i = s0; i < s1; ++i)
                acc += Elem<DT>::to_f(static_cast<const T*>(a.g)[static_cast<int64_t>(a.order[i]) * a.gs + c]);
            acc *= a.scale;
            if (a.accumulate) acc += Elem<WT>::to_f(dst[c]);
            dst[c] = Elem<WT>::from_f(acc);
        }
    }
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

struct EmbeddingSpace {
    int64_t order, start, total;  // byte offsets
};
EmbeddingSpace space_for(int64_t ntokens, int64_t vocab)
{
    EmbeddingSpace e{};
    e.order = 0;
    e.start = round_up(4 * ntokens, 256);
    e.total = e.start + round_up(4 * (vocab + 1), 256);
    return e;
}

ddp_status check_common(const char* fn, int64_t ntokens, int64_t vocab, int64_t dim, int32_t dtype, int32_t id_bytes,
                        const void* ids, const void* mat, int64_t mat_stride, const char* mat_name)
{
    using ddp::fail;
    if (ntokens < 0) return fail(DDP_E_INVAL, "%s: ntokens = %lld < 0", fn, static_cast<long long>(ntokens));
    if (ntokens >= (int64_t{1} << 31)) return fail(DDP_E_INVAL, "%s: ntokens = %lld is 2^31 or more", fn, static_cast<long long>(ntokens));
    if (vocab < 1 || vocab >= (int64_t{1} << 31))
        return fail(DDP_E_INVAL, "%s: vocab = %lld outside [1, 2^31)", fn, static_cast<long long>(vocab));
    if (dim < 1) return fail(DDP_E_INVAL, "%s: dim = %lld < 1", fn, static_cast<long long>(dim));
    if (!known_dtype(dtype)) return fail(DDP_E_INVAL, "%s: unknown dtype %d", fn, dtype);
    if (id_bytes != 4 && id_bytes != 8) return fail(DDP_E_INVAL, "%s: id_bytes = %d is neither 4 nor 8", fn, id_bytes);
    if (mat_stride < dim)
        return fail(DDP_E_INVAL, "%s: %s's stride %lld < dim = %lld", fn, mat_name, static_cast<long long>(mat_stride),
                    static_cast<long long>(dim));
    if (ntokens > 0 && !ids) return fail(DDP_E_INVAL, "%s: ids is NULL", fn);
    if (ntokens > 0 && !mat) return fail(DDP_E_INVAL, "%s: %s is NULL", fn, mat_name);
    return DDP_OK;
}

template <int DT> void launch_lookup(bool vec, int grid, cudaStream_t s, const void* weight, int64_t ws, int64_t vocab,
                                     int64_t dim, const void* ids, int id_bytes, int64_t ntokens, float scale, void* out,
                                     int64_t os, int* status)
{
    if (vec) lookup_kernel<DT, true><<<grid, 256, 0, s>>>(weight, ws, vocab, dim, ids, id_bytes, ntokens, scale, out, os, status);
    else lookup_kernel<DT, false><<<grid, 256, 0, s>>>(weight, ws, vocab, dim, ids, id_bytes, ntokens, scale, out, os, status);
}

template <int DT> void launch_rows(int grid, cudaStream_t s, const GradArgs& g, int gw_dtype)
{
    if (gw_dtype == DT) rows_kernel<DT, DT><<<grid, 128, 0, s>>>(g);
    else rows_kernel<DT, DDP_F32><<<grid, 128, 0, s>>>(g);
}

}  // namespace
}  // namespace ddplm

using namespace ddplm;

extern "C" ddp_status ddp_embedding_forward(const void* weight, int64_t weight_stride, int32_t dtype, int64_t vocab,
                                            int64_t dim, const void* ids, int32_t id_bytes, int64_t ntokens, float scale,
                                            void* out, int64_t out_stride, void* stream)
{
    const char* fn = "ddp_embedding_forward";
    const ddp_status st = check_common(fn, ntokens, vocab, dim, dtype, id_bytes, ids, weight, weight_stride, "weight");
    if (st != DDP_OK) return st;
    if (out_stride < dim)
        return ddp::fail(DDP_E_INVAL, "%s: out's stride %lld < dim = %lld", fn, static_cast<long long>(out_stride),
                         static_cast<long long>(dim));
    if (ntokens == 0) return ddp::ok();
    if (!out) return ddp::fail(DDP_E_INVAL, "%s: out is NULL", fn);
    int* status = lm_status_word();
    if (!status) return ddp::fail(DDP_E_CUDA, "%s: the status word is unavailable", fn);
    const int n = 16 / elem_size(dtype);
    const bool vec = dim % n == 0 && weight_stride % n == 0 && out_stride % n == 0 && aligned16(weight) && aligned16(out);
    const int64_t items = ntokens * (vec ? dim / n : dim);
    const int grid = static_cast<int>(std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(ddp::device_sm_count()) * 16));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == DDP_F32)
        launch_lookup<DDP_F32>(vec, grid, s, weight, weight_stride, vocab, dim, ids, id_bytes, ntokens, scale, out, out_stride, status);
    else if (dtype == DDP_BF16)
        launch_lookup<DDP_BF16>(vec, grid, s, weight, weight_stride, vocab, dim, ids, id_bytes, ntokens, scale, out, out_stride, status);
    else
        launch_lookup<DDP_F16>(vec, grid, s, weight, weight_stride, vocab, dim, ids, id_bytes, ntokens, scale, out, out_stride, status);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return ddp::fail(DDP_E_CUDA, "%s: kernel launch failed: %s", fn, cudaGetErrorString(err));
    return ddp::ok();
}

extern "C" ddp_status ddp_embedding_workspace(int64_t ntokens, int64_t vocab, int64_t dim, int64_t* bytes)
{
    const char* fn = "ddp_embedding_workspace";
    if (!bytes) return ddp::fail(DDP_E_INVAL, "%s: bytes is NULL", fn);
    if (ntokens < 0 || ntokens >= (int64_t{1} << 31) || vocab < 1 || vocab >= (int64_t{1} << 31) || dim < 1)
        return ddp::fail(DDP_E_INVAL, "%s: ntokens = %lld, vocab = %lld, dim = %lld out of range", fn,
                         static_cast<long long>(ntokens), static_cast<long long>(vocab), static_cast<long long>(dim));
    *bytes = space_for(ntokens, vocab).total;
    return ddp::ok();
}

extern "C" ddp_status ddp_embedding_backward(const void* grad_out, int64_t grad_stride, int32_t dtype, const void* ids,
                                             int32_t id_bytes, int64_t ntokens, float scale, int64_t padding_idx,
                                             int64_t vocab, int64_t dim, void* grad_weight, int64_t gw_stride,
                                             int32_t gw_dtype, int32_t accumulate, void* workspace,
                                             int64_t workspace_bytes, void* stream)
{
    using ddp::fail;
    const char* fn = "ddp_embedding_backward";
    const ddp_status st = check_common(fn, ntokens, vocab, dim, dtype, id_bytes, ids, grad_out, grad_stride, "grad_out");
    if (st != DDP_OK) return st;
    if (!grad_weight) return fail(DDP_E_INVAL, "%s: grad_weight is NULL", fn);
    if (gw_stride < dim)
        return fail(DDP_E_INVAL, "%s: grad_weight's stride %lld < dim = %lld", fn, static_cast<long long>(gw_stride),
                    static_cast<long long>(dim));
    if (gw_dtype != dtype && gw_dtype != DDP_F32) return fail(DDP_E_INVAL, "%s: gw_dtype %d is neither dtype nor DDP_F32", fn, gw_dtype);
    const EmbeddingSpace sp = space_for(ntokens, vocab);
    if (!workspace || !aligned16(workspace) || workspace_bytes < sp.total)
        return fail(DDP_E_INVAL, "%s: workspace of %lld bytes (16-byte aligned), needs %lld", fn,
                    static_cast<long long>(workspace ? workspace_bytes : 0), static_cast<long long>(sp.total));
    if (ntokens == 0 && accumulate) return ddp::ok();
    int* status = lm_status_word();
    if (!status) return fail(DDP_E_CUDA, "%s: the status word is unavailable", fn);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* w = static_cast<char*>(workspace);
    SortArgs a{ids, id_bytes, static_cast<int32_t>(ntokens), vocab, padding_idx, 0, reinterpret_cast<int32_t*>(w + sp.order),
               reinterpret_cast<int32_t*>(w + sp.start), status};
    const int sms = ddp::device_sm_count();
    a.range = static_cast<int32_t>(std::min<int64_t>(kMaxRange, std::max<int64_t>(1, (vocab + sms - 1) / sms)));
    const int grid = static_cast<int>((vocab + a.range - 1) / a.range);
    const int smem = (kSortWarps + 1) * a.range * 4;
    cudaError_t err = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kSortWarps + 1) * kMaxRange * 4);
    if (err != cudaSuccess) return fail(DDP_E_CUDA, "%s: shared memory: %s", fn, cudaGetErrorString(err));
    sort_kernel<<<grid, kSortThreads, smem, s>>>(a);
    const GradArgs g{grad_out, grad_stride, a.order, a.start, vocab, dim, scale, grad_weight, gw_stride, accumulate != 0};
    const int rows = static_cast<int>(std::min<int64_t>(vocab, int64_t{1} << 20));
    if (dtype == DDP_F32) launch_rows<DDP_F32>(rows, s, g, gw_dtype);
    else if (dtype == DDP_BF16) launch_rows<DDP_BF16>(rows, s, g, gw_dtype);
    else launch_rows<DDP_F16>(rows, s, g, gw_dtype);
    err = cudaGetLastError();
    if (err != cudaSuccess) return fail(DDP_E_CUDA, "%s: kernel launch failed: %s", fn, cudaGetErrorString(err));
    return ddp::ok();
}

extern "C" ddp_status ddp_lm_status(void* stream, int32_t* status, int32_t reset)
{
    if (!status) return ddp::fail(DDP_E_INVAL, "ddp_lm_status: status is NULL");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_lm_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && reset && v != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbolAsync(g_lm_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    if (e != cudaSuccess) return ddp::fail(DDP_E_CUDA, "ddp_lm_status: %s", cudaGetErrorString(e));
    *status = v;
    return ddp::ok();
}
