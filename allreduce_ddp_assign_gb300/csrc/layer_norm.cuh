// What the two passes of layer norm share (layer_norm.cu, layer_norm_grad.cu).
//
// Layer norm over the rows of a matrix, with the residual addition before it, and its backward pass.
//
//   s = round(x + r),  mu = mean(s),  var = mean((s - mu)^2),  rho = 1 / sqrt(var + eps)
//   y = (s - mu) rho w + b
//   n = (s - mu) rho,  g = dy w,  dx = rho (g - mean(g) - n mean(g n)) + ds
//   dw = sum_t dy n,  db = sum_t dy
//
// HBM-bound: a row is read once into registers, where its sums are taken (the mean first,
// then the squares around it), and written once.  A team of 1, 2, 4, 8 or 16 warps takes a
// row, the fewest whose lanes hold it.  In the backward pass a thread has the same columns
// in every row of its team, so that dw and db are kept in its registers until the rows are
// done; a CTA's teams join theirs in shared memory, and a second kernel joins the CTAs', both
// in a fixed order.  The team follows from the width and from where the rows lie, so that a row's
// result does not depend on the values beside it.  (Rows whose stride is off 16-byte boundaries are taken
// in single elements; one row alone has no stride, and may be taken in vectors, in another order of sums.)
//
// Measured on a GB300 (graph replays, more inputs than L2 holds).  Forward: 8192 x 768 bf16 with fp32
// weights 7.6 us (3.3 TB/s: three or four rows a team between its start and its end), 65536 x 768 33 us (6.1 TB/s),
// 16384 x 1024 fp16 with residual 23.7 us (5.7 TB/s), fp32 without 21.9 (6.1), 65536 x 4096 bf16 with residual
// 378 us (5.7).
// Backward with the gradient past the norm: 8192 x 768 bf16 18.4 us (2.7 TB/s: 15 and 5 for the join,
// cold), 65536 x 1024 89 us (6.0), 65536 x 4096 373 us (5.8); 16384 x 1024 fp32 39 us (5.2).
// Rows in single elements: 20000 x 1001 fp16 22 us forward (3.6 TB/s), 45 backward (2.7), bound by the
// instructions of an element at a time (35 and 58 with a team's size known only at run time).
// Rows that no team holds, which a CTA goes over in passes: odd ones above 8192 values (8192 x 12001 bf16 with
// residual 704 us, backward with ds 762; the floor is 116), any above 16384 (8192 x 20480 bf16 1052 and 1398; 198),
// and forward fp32 ones with a residual above 8192 (4096 x 12288: 160; 119).
#pragma once

#include <algorithm>

#include "lm_common.cuh"

namespace ddplm {
namespace {

constexpr int kWarps = 8;            // warps of a CTA, whose teams take a row each
constexpr int kMaxTeam = 16;         // warps of the largest team, which is a CTA
constexpr int kPerSm = 2;            // CTAs of kWarps warps an SM in the backward pass
constexpr int kLoopThreads = 512;    // threads of a CTA where no team holds a row
constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kLoopPartials = int64_t(1) << 23;   // values of a partial sum that those CTAs write at most

// ---------------------------------------------------------------------------
// rows in registers
// ---------------------------------------------------------------------------
// N elements, as they lie in memory.
template <int DT, int N> struct __align__(N * sizeof(typename Elem<DT>::T)) Pack {
    typename Elem<DT>::T v[N];
};

// A weight or bias: fp32 (wide) or in the rows' type, anywhere or on 16-byte boundaries (vectors).
struct Columns {
    const void* p;
    bool wide, vectors;
};
// Columns N i to N i + N - 1, as they lie in memory.
template <int WDT, int N> __device__ __forceinline__ Pack<WDT, N> load_columns(const Columns& c, int i)
{
    using T = typename Elem<WDT>::T;
    const T* q = static_cast<const T*>(c.p) + static_cast<int64_t>(i) * N;
    constexpr int M = N * sizeof(T) > 16 ? 16 / static_cast<int>(sizeof(T)) : N;
    Pack<WDT, N> out;
#pragma unroll
    for (int u = 0; u < N; u += M) {
        if (c.vectors) {
            const Pack<WDT, M> v = *reinterpret_cast<const Pack<WDT, M>*>(q + u);
#pragma unroll
            for (int e = 0; e < M; ++e) out.v[u + e] = v.v[e];
        } else {
#pragma unroll
            for (int e = 0; e < M; ++e) out.v[u + e] = q[u + e];
        }
    }
    return out;
}
// Keeps 16-bit columns as they lie in memory through a loop: widened ahead of it they would take twice the registers.
template <int WDT, int N> __device__ __forceinline__ void stay_packed(Pack<WDT, N>& c)
{
    if constexpr (sizeof(c) / N == 2) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) asm volatile("" : "+r"(reinterpret_cast<uint32_t*>(c.v)[i]));
    }
}
// One column.
template <int DT> __device__ __forceinline__ float column(const Columns& c, int i)
{
    return c.wide ? static_cast<const float*>(c.p)[i] : Elem<DT>::to_f(static_cast<const typename Elem<DT>::T*>(c.p)[i]);
}

// Rings in shared memory: of S rows, A arrays each, of which a thread holds K vectors of 16 bytes.  At most five rows:
// more were not faster.
__host__ __device__ constexpr int ring_rows(int bytes, int row_bytes) { return bytes / row_bytes < 2 ? 2 : bytes / row_bytes > 5 ? 5 : bytes / row_bytes; }

struct Pair {
    float a, b;
};

__device__ __forceinline__ Pair warp_sum(Pair v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        v.a += __shfl_xor_sync(0xffffffffu, v.a, o);
        v.b += __shfl_xor_sync(0xffffffffu, v.b, o);
    }
    return v;
}

// A team of warps, and sums over it.  The sums alternate between two rows of shared memory:
// a row is written again only behind the barrier of the sum between, which every reader of it
// has passed.
template <bool MULTI> struct Team {
    Pair (*sh)[kMaxTeam];
    int warps;   // of a team
    int index;   // the CTA's teams are numbered
    int me, size;   // the thread in its team, the team's threads
    int turn = 0;
    __device__ __forceinline__ Team(Pair (*shared)[kMaxTeam], int team_warps)
        : sh(shared), warps(MULTI ? team_warps : 1), index((threadIdx.x >> 5) / (MULTI ? team_warps : 1)),
          me(MULTI ? threadIdx.x - index * team_warps * 32 : threadIdx.x & 31), size(MULTI ? 32 * team_warps : 32)
    {
    }
    __device__ __forceinline__ int count() const { return (blockDim.x >> 5) / warps; }
    __device__ __forceinline__ void barrier() const
    {
        if (MULTI) asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(size) : "memory");
        else __syncwarp();
    }
    __device__ __forceinline__ float sum(float v)
    {
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (!MULTI) return v;
        if ((threadIdx.x & 31) == 0) sh[turn][threadIdx.x >> 5].a = v;
        barrier();
        v = sh[turn][index * warps].a;
        for (int w = 1; w < warps; ++w) v += sh[turn][index * warps + w].a;
        turn ^= 1;
        return v;
    }
    __device__ __forceinline__ Pair sum(Pair v)
    {
        v = warp_sum(v);
        if (!MULTI) return v;
        if ((threadIdx.x & 31) == 0) sh[turn][threadIdx.x >> 5] = v;
        barrier();
        v = sh[turn][index * warps];
        for (int w = 1; w < warps; ++w) {
            v.a += sh[turn][index * warps + w].a;
            v.b += sh[turn][index * warps + w].b;
        }
        turn ^= 1;
        return v;
    }
};

// Rows anywhere: a team copies the 16-byte pieces of memory that a row lies in into a ring, and its threads pick single
// elements there, behind a barrier.  A piece's other elements, of the rows beside it, are not used; one that leaves the
// matrix is copied element by element.
template <int DT> struct Rows {
    using T = typename Elem<DT>::T;
    const T* base;
    int64_t stride;
    const char* end;   // of the last row
    __device__ __forceinline__ Rows(const void* p, int64_t row_stride, int rows, int dim)
        : base(static_cast<const T*>(p)), stride(row_stride), end(reinterpret_cast<const char*>(base + (rows - 1) * row_stride + dim))
    {
    }
    __device__ __forceinline__ int skip(int64_t row) const { return (reinterpret_cast<uintptr_t>(base + row * stride) & 15) / sizeof(T); }
    __device__ __forceinline__ void fetch(int64_t row, int rows, int dim, unsigned char* to, int me, int step) const
    {
        const T* begin = base + row * stride;
        const char* at = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(begin) & ~uintptr_t{15});
        const int pieces = (skip(row) + dim + Vec<DT>::N - 1) / Vec<DT>::N;
        const uint32_t to_at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
        if (row > 0 && row + 1 < rows && stride >= Vec<DT>::N) {
            for (int c = me; c < pieces; c += step) copy16(to_at + 16 * c, at + 16 * c);
            return;
        }
        for (int c = me; c < pieces; c += step) {
            const char* from = at + 16 * c;
            if (from >= reinterpret_cast<const char*>(base) && from + 16 <= end) {
                copy16(to_at + 16 * c, from);
            } else {
                const T* q = reinterpret_cast<const T*>(from);
                for (int e = 0; e < Vec<DT>::N; ++e)
                    if (q + e >= begin && q + e < begin + dim) reinterpret_cast<T*>(to)[c * Vec<DT>::N + e] = q[e];
            }
        }
    }
};
// Bytes of a row in the ring, wherever it starts.
template <int DT> __host__ __device__ __forceinline__ int row_room(int dim)
{
    return (dim * static_cast<int>(sizeof(typename Elem<DT>::T)) + 15) / 16 * 16 + 16;
}

// In single elements a thread has kElements of a row at most; the rings of a CTA's teams are `rows` deep, of `arrays`
// rows each.
constexpr int kElements = 16;
template <int DT, int arrays> __host__ __device__ constexpr int element_rows()
{
    constexpr int s = (108 << 10) / (arrays * 32 * kWarps * (kElements * static_cast<int>(sizeof(typename Elem<DT>::T)) + 1));
    return s < 2 ? 2 : s > 4 ? 4 : s;
}
template <int DT, int arrays> constexpr int elements_room(int threads)   // (31 bytes of a row at most are not its own)
{
    return element_rows<DT, arrays>() * arrays * (threads * kElements * static_cast<int>(sizeof(typename Elem<DT>::T)) + threads / 32 * 32);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Warps of a team for rows of `packs` vectors (elements); 0: no team holds them.
int team_for(int64_t packs, int share)
{
    for (int w = 1; w <= kMaxTeam; w *= 2)
        if (packs <= static_cast<int64_t>(32) * w * share) return w;
    return 0;
}

int cta_warps(int team) { return std::max(team, kWarps); }

// CALL<DT> for the type at hand
#define DDP_FOR_TYPE(dtype, CALL) ((dtype) == DDP_F32 ? CALL<DDP_F32> : (dtype) == DDP_BF16 ? CALL<DDP_BF16> : CALL<DDP_F16>)

Columns columns_of(const void* p, int w_dtype) { return {p, w_dtype == DDP_F32, aligned16(p)}; }

bool row_vectors(const void* p, int64_t stride, int dtype) { return aligned16(p) && stride % (16 / elem_size(dtype)) == 0; }

ddp_status check_sizes(const char* fn, int64_t ntokens, int64_t dim)
{
    using ddp::fail;
    if (ntokens < 0 || ntokens >= (int64_t(1) << 31) - 4096)
        return fail(DDP_E_INVAL, "%s: ntokens = %lld", fn, static_cast<long long>(ntokens));
    if (dim < 1 || dim > kMaxDim) return fail(DDP_E_INVAL, "%s: dim = %lld", fn, static_cast<long long>(dim));
    return DDP_OK;
}
ddp_status check_types(const char* fn, int32_t dtype, int32_t w_dtype)
{
    if (!known_dtype(dtype)) return ddp::fail(DDP_E_INVAL, "%s: unknown dtype %d", fn, dtype);
    if (w_dtype != dtype && w_dtype != DDP_F32)
        return ddp::fail(DDP_E_INVAL, "%s: w_dtype %d is neither the dtype nor DDP_F32", fn, w_dtype);
    return DDP_OK;
}
ddp_status check_rows(const char* fn, const char* name, const void* p, int64_t stride, int64_t ntokens, int64_t dim)
{
    if (!p) return ddp::fail(DDP_E_INVAL, "%s: %s is NULL", fn, name);
    if (ntokens > 1 && stride < dim)
        return ddp::fail(DDP_E_INVAL, "%s: %s's stride %lld is below dim", fn, name, static_cast<long long>(stride));
    return DDP_OK;
}
ddp_status launched(const char* fn, cudaError_t e)
{
    if (e != cudaSuccess) return ddp::fail(DDP_E_CUDA, "%s: kernel launch failed: %s", fn, cudaGetErrorString(e));
    return ddp::ok();
}

}  // namespace
}  // namespace ddplm
