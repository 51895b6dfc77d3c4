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
constexpr int kBatch = 8;        // loads a thread keeps in flight

struct SortArgs {
    const void* ids;
    int32_t id_bytes;
    int32_t ntokens;
    int64_t vocab, padding_idx;
    int32_t range;   // ids per CTA
    int32_t* order;  // [ntokens] tokens sorted by id
    int32_t* key;    // [ntokens] their ids
    int32_t* start;  // [vocab + 1] first place of each id in `order`
    int* status;
    // rows of ids that do not occur (nullptr: left alone)
    uint8_t* clear;
    int64_t clear_stride, clear_bytes;
};

__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortArgs a)
{
    extern __shared__ int32_t sh[];  // [warp][range] counters, then places
    __shared__ int32_t less_w[kSortWarps], part[kSortWarps];
    __shared__ uint8_t seen[kMaxRange];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* cnt = sh + warp * a.range;
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.range;
    const int64_t hi = lo + a.range < a.vocab ? lo + a.range : a.vocab;
    const int nr = static_cast<int>(hi - lo);
    for (int i = tid; i < kSortWarps * a.range; i += kSortThreads) sh[i] = 0;
    __syncthreads();
    wait_for_previous();
    // each warp counts a contiguous stretch of tokens
    const int per = (a.ntokens + kSortWarps - 1) / kSortWarps;
    const int t0 = min(warp * per, a.ntokens), t1 = min(t0 + per, a.ntokens);
    int32_t less = 0;
    for (int t = t0 + lane; t < t1; t += 32 * kBatch) {
        int64_t id[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) id[j] = t + 32 * j < t1 ? load_id(a.ids, a.id_bytes, t + 32 * j) : -1;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (t + 32 * j >= t1 || (a.padding_idx >= 0 && id[j] == a.padding_idx)) continue;
            if (id[j] < 0 || id[j] >= a.vocab) {
                if (blockIdx.x == 0) atomicOr(a.status, kErrId);
                continue;
            }
            less += id[j] < lo;
            if (id[j] >= lo && id[j] < hi) atomicAdd(&cnt[static_cast<int>(id[j] - lo)], 1);
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
        for (int w = 0; w < kSortWarps; ++w) total += sh[w * a.range + tid];
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
        seen[tid] = total > 0;
        a.start[lo + tid] = at;
        if (lo + tid + 1 == a.vocab) a.start[a.vocab] = at + total;
        // the counters become the first places of the id's tokens from each warp's stretch
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = sh[w * a.range + tid];
            sh[w * a.range + tid] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int t = t0; t < t1; t += 32 * kBatch) {
        int64_t id[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            id[j] = t + 32 * j + lane < t1 ? load_id(a.ids, a.id_bytes, t + 32 * j + lane) : -1;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const bool mine = id[j] >= lo && id[j] < hi && id[j] != a.padding_idx;
            const uint32_t any = __ballot_sync(0xffffffffu, mine);
            if (!any) continue;
            if (mine) {
                const int r = static_cast<int>(id[j] - lo);
                const uint32_t same = __match_any_sync(any, r);
                const int at = cnt[r] + __popc(same & ((1u << lane) - 1u));
                a.order[at] = t + 32 * j + lane;
                a.key[at] = static_cast<int32_t>(id[j]);
                __syncwarp(same);
                if (lane == __ffs(same) - 1) cnt[r] += __popc(same);
            }
            __syncwarp();
        }
    }
    // the rest of the range's rows: nothing to wait for
    if (a.clear) {
        for (int r = warp; r < nr; r += kSortWarps) {
            if (seen[r]) continue;
            uint8_t* row = a.clear + (lo + r) * a.clear_stride;
            const int64_t head = min(a.clear_bytes, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15));
            const int64_t body = head + (a.clear_bytes - head) / 16 * 16;
            if (lane * 2 < head) *reinterpret_cast<uint16_t*>(row + lane * 2) = 0;
            for (int64_t c = head + lane * 16; c < body; c += 512) *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
            if (body + lane * 2 < a.clear_bytes) *reinterpret_cast<uint16_t*>(row + body + lane * 2) = 0;
        }
    }
}

// Runs of equal ids are cut into chunks of the sorted order, so that a frequent word's
// run is summed by many warps.  A warp sums one chunk in 32 lanes' columns; runs that
// lie within the chunk go to the table, a run's part that reaches over the chunk's
// edge goes to the workspace: `head` of a chunk is the part of a run that began before
// it, `tail` the part of one that begins in it and goes on.
struct GradArgs {
    const void* g;
    int64_t gs;
    const int32_t* order;
    const int32_t* key;
    const int32_t* start;
    int64_t vocab, dim;
    int32_t chunk;
    float* edge;  // [chunks][head, tail][dim]
    float scale;
    void* gw;
    int64_t ws;
    int32_t accumulate;
};

// A lane's columns: one 16-byte vector of the input, or four single ones 32 apart.
template <int DT, bool VEC> struct Columns {
    static constexpr int N = VEC ? Vec<DT>::N : 4;
    static constexpr int kSlab = 32 * N;
    __device__ __forceinline__ static int64_t at(int64_t slab, int lane, int j)
    {
        return slab * kSlab + (VEC ? lane * N + j : lane + 32 * j);
    }
    __device__ __forceinline__ static void load(const void* g, int64_t row, int64_t dim, int64_t slab, int lane, float (&x)[N])
    {
        using T = typename Elem<DT>::T;
        const T* p = static_cast<const T*>(g) + row;
        if (VEC) {
            Vec<DT> v{};
            if (at(slab, lane, 0) < dim) v = *reinterpret_cast<const Vec<DT>*>(p + at(slab, lane, 0));
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = Elem<DT>::to_f(v.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = at(slab, lane, j) < dim ? Elem<DT>::to_f(p[at(slab, lane, j)]) : 0.f;
        }
    }
    // fp32 rows of `dim` values in the workspace (VEC: dim is a multiple of N, which is one of 4)
    __device__ __forceinline__ static void load_edge(const float* p, int64_t dim, int64_t slab, int lane, float (&x)[N])
    {
#pragma unroll
        for (int j = 0; j < N; j += VEC ? 4 : 1) {
            const bool in = at(slab, lane, j) < dim;
            if (VEC) {
                const float4 v = in ? *reinterpret_cast<const float4*>(p + at(slab, lane, j)) : make_float4(0.f, 0.f, 0.f, 0.f);
                x[j] = v.x; x[j + (VEC ? 1 : 0)] = v.y; x[j + (VEC ? 2 : 0)] = v.z; x[j + (VEC ? 3 : 0)] = v.w;
            } else {
                x[j] = in ? p[at(slab, lane, j)] : 0.f;
            }
        }
    }
    __device__ __forceinline__ static void store_edge(float* p, int64_t dim, int64_t slab, int lane, const float (&x)[N])
    {
#pragma unroll
        for (int j = 0; j < N; j += VEC ? 4 : 1) {
            if (at(slab, lane, j) >= dim) continue;
            if (VEC) *reinterpret_cast<float4*>(p + at(slab, lane, j)) = make_float4(x[j], x[j + (VEC ? 1 : 0)], x[j + (VEC ? 2 : 0)], x[j + (VEC ? 3 : 0)]);
            else p[at(slab, lane, j)] = x[j];
        }
    }
    template <int WT> __device__ __forceinline__ static void store(const GradArgs& a, int64_t v, int64_t slab, int lane, const float (&x)[N])
    {
        using O = typename Elem<WT>::T;
        O* p = static_cast<O*>(a.gw) + v * a.ws;
        if (VEC) {
            if (at(slab, lane, 0) >= a.dim) return;
            p += at(slab, lane, 0);
            constexpr int M = Vec<WT>::N;  // N is a multiple of M
#pragma unroll
            for (int k = 0; k < N; k += M) {
                Vec<WT> o{};
                if (a.accumulate) o = *reinterpret_cast<const Vec<WT>*>(p + k);
#pragma unroll
                for (int j = 0; j < M; ++j) o.v[j] = Elem<WT>::from_f(x[k + j] * a.scale + (a.accumulate ? Elem<WT>::to_f(o.v[j]) : 0.f));
                *reinterpret_cast<Vec<WT>*>(p + k) = o;
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (at(slab, lane, j) >= a.dim) continue;
                O* o = p + at(slab, lane, j);
                *o = Elem<WT>::from_f(x[j] * a.scale + (a.accumulate ? Elem<WT>::to_f(*o) : 0.f));
            }
        }
    }
};

constexpr int kSumWarps = 4;
template <int DT, int WT, bool VEC> __global__ void __launch_bounds__(32 * kSumWarps) chunk_kernel(GradArgs a)
{
    using C = Columns<DT, VEC>;
    const int lane = threadIdx.x & 31;
    const int64_t slabs = (a.dim + C::kSlab - 1) / C::kSlab;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kSumWarps + (threadIdx.x >> 5);
    const int64_t chunk = unit / slabs, slab = unit - chunk * slabs;
    wait_for_previous();
    const int64_t n = a.start[a.vocab];
    const int64_t c0 = chunk * a.chunk, c1 = min(n, c0 + a.chunk);
    if (c0 >= n) return;
    float* edge = a.edge + chunk * 2 * a.dim;
    float acc[C::N];
#pragma unroll
    for (int j = 0; j < C::N; ++j) acc[j] = 0.f;
    int32_t now = a.key[c0];
    bool began_before = c0 > 0 && a.key[c0 - 1] == now;
    for (int64_t i = c0; i < c1; i += kBatch) {
        int32_t tok = 0, key = -1;
        if (lane <= kBatch && i + lane < n) {  // the batch's tokens, and the id after it
            tok = a.order[i + lane];
            key = a.key[i + lane];
        }
        float x[kBatch][C::N];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t row = static_cast<int64_t>(__shfl_sync(0xffffffffu, tok, j)) * a.gs;
            if (i + j < c1) C::load(a.g, row, a.dim, slab, lane, x[j]);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int32_t next = __shfl_sync(0xffffffffu, key, j + 1);
            if (i + j >= c1) continue;
#pragma unroll
            for (int k = 0; k < C::N; ++k) acc[k] += x[j][k];
            const bool at_end = i + j + 1 == c1;
            if (next == now && !at_end) continue;
            if (began_before) C::store_edge(edge, a.dim, slab, lane, acc);
            else if (next == now) C::store_edge(edge + a.dim, a.dim, slab, lane, acc);
            else C::template store<WT>(a, now, slab, lane, acc);
#pragma unroll
            for (int k = 0; k < C::N; ++k) acc[k] = 0.f;
            began_before = false;
            now = next;
        }
    }
}

// Runs that reach over chunks' edges: the tail where a run begins, then the heads of
// the chunks it goes on in.  Eight warps take a stretch of them each; the stretches
// are added in order.
constexpr int kJoinWarps = 8;
template <int DT, int WT, bool VEC> __global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(GradArgs a)
{
    using C = Columns<DT, VEC>;
    __shared__ float sh[kJoinWarps][32][C::N + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t slabs = (a.dim + C::kSlab - 1) / C::kSlab;
    const int64_t chunk = blockIdx.x / slabs, slab = blockIdx.x - chunk * slabs;
    wait_for_previous();
    const int64_t n = a.start[a.vocab];
    const int64_t c1 = (chunk + 1) * a.chunk;
    if (c1 >= n) return;
    const int32_t v = a.key[c1 - 1];
    const int64_t s0 = a.start[v], s1 = a.start[v + 1];
    if (s1 <= c1 || s0 < c1 - a.chunk) return;  // ends here, or began before this chunk
    const int64_t last = (s1 - 1) / a.chunk;    // the heads are those of chunks (chunk, last]
    const int64_t parts = last - chunk + 1;
    const int64_t per = (parts + kJoinWarps - 1) / kJoinWarps;
    const int64_t p0 = warp * per, p1 = min(parts, p0 + per);
    float acc[C::N];
#pragma unroll
    for (int k = 0; k < C::N; ++k) acc[k] = 0.f;
    for (int64_t p = p0; p < p1; p += 4) {
        float x[4][C::N];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (p + j < p1) C::load_edge(a.edge + ((chunk + p + j) * 2 + (p + j == 0)) * a.dim, a.dim, slab, lane, x[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (p + j < p1)
#pragma unroll
                for (int k = 0; k < C::N; ++k) acc[k] += x[j][k];
    }
#pragma unroll
    for (int k = 0; k < C::N; ++k) sh[warp][lane][k] = acc[k];
    __syncthreads();
    if (warp == 0) {
        const int used = static_cast<int>(min(static_cast<int64_t>(kJoinWarps), (parts + per - 1) / per));
        for (int w = 1; w < used; ++w)
#pragma unroll
            for (int k = 0; k < C::N; ++k) acc[k] += sh[w][lane][k];
        C::template store<WT>(a, v, slab, lane, acc);
    }
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Tokens a warp sums: short chunks spread few tokens over the SMs, longer ones write fewer edges.
int32_t chunk_for(int64_t ntokens) { return ntokens <= 16384 ? 16 : 32; }

struct EmbeddingSpace {
    int64_t order, key, start, edge, total;  // byte offsets
};
EmbeddingSpace space_for(int64_t ntokens, int64_t vocab, int64_t dim)
{
    EmbeddingSpace e{};
    const int64_t chunk = chunk_for(ntokens);
    e.order = 0;
    e.key = e.order + round_up(4 * ntokens, 256);
    e.start = e.key + round_up(4 * ntokens, 256);
    e.edge = e.start + round_up(4 * (vocab + 1), 256);
    e.total = e.edge + round_up((ntokens + chunk - 1) / chunk * 8 * dim, 256);
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

template <int DT, int WT, bool VEC> cudaError_t launch_sums_as(const GradArgs& g, int64_t ntokens, cudaStream_t s)
{
    const int64_t slabs = (g.dim + Columns<DT, VEC>::kSlab - 1) / Columns<DT, VEC>::kSlab;
    const int64_t units = (ntokens + g.chunk - 1) / g.chunk * slabs;
    const cudaError_t e = launch_chained(chunk_kernel<DT, WT, VEC>, dim3(static_cast<unsigned>((units + kSumWarps - 1) / kSumWarps)),
                                         32 * kSumWarps, 0, s, g);
    if (e != cudaSuccess) return e;
    return launch_chained(join_kernel<DT, WT, VEC>, dim3(static_cast<unsigned>(units)), 32 * kJoinWarps, 0, s, g);
}
template <int DT> cudaError_t launch_sums(const GradArgs& g, int64_t ntokens, int gw_dtype, bool vec, cudaStream_t s)
{
    if (gw_dtype == DT) return vec ? launch_sums_as<DT, DT, true>(g, ntokens, s) : launch_sums_as<DT, DT, false>(g, ntokens, s);
    return vec ? launch_sums_as<DT, DDP_F32, true>(g, ntokens, s) : launch_sums_as<DT, DDP_F32, false>(g, ntokens, s);
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
    *bytes = space_for(ntokens, vocab, dim).total;
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
    const EmbeddingSpace sp = space_for(ntokens, vocab, dim);
    if (!workspace || !aligned16(workspace) || workspace_bytes < sp.total)
        return fail(DDP_E_INVAL, "%s: workspace of %lld bytes (16-byte aligned), needs %lld", fn,
                    static_cast<long long>(workspace ? workspace_bytes : 0), static_cast<long long>(sp.total));
    if (ntokens == 0 && accumulate) return ddp::ok();
    int* status = lm_status_word();
    if (!status) return fail(DDP_E_CUDA, "%s: the status word is unavailable", fn);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* w = static_cast<char*>(workspace);
    const int64_t es = elem_size(gw_dtype);
    SortArgs a{};
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.ntokens = static_cast<int32_t>(ntokens);
    a.vocab = vocab;
    a.padding_idx = padding_idx;
    a.order = reinterpret_cast<int32_t*>(w + sp.order);
    a.key = reinterpret_cast<int32_t*>(w + sp.key);
    a.start = reinterpret_cast<int32_t*>(w + sp.start);
    a.status = status;
    if (!accumulate) {
        a.clear = static_cast<uint8_t*>(grad_weight);
        a.clear_stride = gw_stride * es;
        a.clear_bytes = dim * es;
    }
    const int sms = ddp::device_sm_count();
    a.range = static_cast<int32_t>(std::min<int64_t>(kMaxRange, std::max<int64_t>(1, (vocab + sms - 1) / sms)));
    static std::atomic<bool> ready[ddp::kMaxDevices] = {};
    const int dev = ddp::current_device();
    cudaError_t err = cudaSuccess;
    if (dev < 0 || !ready[dev].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortWarps * kMaxRange * 4);
        if (err != cudaSuccess) return fail(DDP_E_CUDA, "%s: shared memory: %s", fn, cudaGetErrorString(err));
        if (dev >= 0) ready[dev].store(true, std::memory_order_relaxed);
    }
    err = launch_chained(sort_kernel, dim3(static_cast<unsigned>((vocab + a.range - 1) / a.range)), kSortThreads,
                         kSortWarps * a.range * 4, s, a);
    if (err == cudaSuccess && ntokens > 0) {
        const GradArgs g{grad_out, grad_stride, a.order, a.key, a.start, vocab, dim, chunk_for(ntokens),
                         reinterpret_cast<float*>(w + sp.edge), scale, grad_weight, gw_stride, accumulate != 0};
        const int n = 16 / elem_size(dtype);
        const bool vec = dim % n == 0 && grad_stride % n == 0 && gw_stride % n == 0 && aligned16(grad_out) && aligned16(grad_weight);
        if (dtype == DDP_F32) err = launch_sums<DDP_F32>(g, ntokens, gw_dtype, vec, s);
        else if (dtype == DDP_BF16) err = launch_sums<DDP_BF16>(g, ntokens, gw_dtype, vec, s);
        else err = launch_sums<DDP_F16>(g, ntokens, gw_dtype, vec, s);
    }
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
