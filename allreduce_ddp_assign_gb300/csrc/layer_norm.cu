// Layer norm, forward (the formulas and the teams of warps: layer_norm.cuh).
#include <cmath>

#include "layer_norm.cuh"

namespace ddplm {
namespace {

struct FwdArgs {
    const void *x, *residual;
    Columns weight, bias;   // bias.p: nullptr where there is none
    void *out, *sum;
    float *mean, *rstd;
    int64_t x_stride, r_stride, out_stride, sum_stride;
    int32_t rows, dim, team_warps;
    float eps, inv_dim;
};

// Rows on 16-byte boundaries.  Each thread copies its own vectors of the rows to come into a ring in shared memory,
// asynchronously, and reads only what it copied itself: the loads of the rows to come are on their way while one is
// worked on, and cost neither registers nor a barrier.  The columns' weights and biases stay in registers.
// K: vectors of a thread; W: the type of the weights.
template <int DT, int W, int K> __host__ __device__ constexpr int per_sm()
{
    // registers that hold weights and biases: with more than 24 of them two CTAs share an SM, else three (16384 x 1024
    // fp16 with residual, 32 of them: 23.7 us with two, 30.4 with three, which spill)
    return 2 * K * Vec<DT>::N * (W == DDP_F32 ? 4 : 2) / 4 > 24 ? 2 : 3;
}
template <int DT, int W, int K, bool RES> __host__ __device__ constexpr int stages()
{
    return ring_rows((224 << 10) / per_sm<DT, W, K>() - 2048, (RES ? 2 : 1) * K * 16 * 32 * kWarps);
}

template <int DT, int W, int K, bool RES, bool MULTI, bool BIG>
__global__ void __launch_bounds__(32 * (BIG ? kMaxTeam : kWarps), BIG ? 1 : per_sm<DT, W, K>()) norm_ring_kernel(const __grid_constant__ FwdArgs a)
{
    using E = Elem<DT>;
    constexpr int N = Vec<DT>::N, S = stages<DT, W, K, RES>(), A = RES ? 2 : 1, kThreads = 32 * (BIG ? kMaxTeam : kWarps);
    using P = Pack<DT, N>;
    __shared__ Pair sh[2][kMaxTeam];
    extern __shared__ __align__(16) uint4 ring[];   // [S][A][K][kThreads]
    Team<MULTI> team(sh, a.team_warps);
    const int me = team.me, step = team.size, packs = a.dim / N;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * team.count() + team.index;
    const int64_t every = static_cast<int64_t>(gridDim.x) * team.count();
    const P* mine = reinterpret_cast<const P*>(ring) + threadIdx.x;
    const uint32_t mine_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + 16 * threadIdx.x;
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.rows) {
            const P* x = reinterpret_cast<const P*>(static_cast<const typename E::T*>(a.x) + row * a.x_stride);
            const P* r = RES ? reinterpret_cast<const P*>(static_cast<const typename E::T*>(a.residual) + row * a.r_stride) : nullptr;
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (me + j * step < packs) {
                    copy16(mine_at + (stage * A * K + j) * 16 * kThreads, x + me + j * step);
                    if (RES) copy16(mine_at + ((stage * A + 1) * K + j) * 16 * kThreads, r + me + j * step);
                }
        }
        copies_commit();
    };
    wait_for_previous();
    allow_next();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(first + s * every, s);
    Pack<W, N> weight[K], bias[K];
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (me + j * step < packs && first < a.rows) {
            weight[j] = load_columns<W, N>(a.weight, me + j * step);
            if (a.bias.p) {
                bias[j] = load_columns<W, N>(a.bias, me + j * step);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) bias[j].v[e] = Elem<W>::from_f(0.f);
            }
        }
    int stage = 0;
    for (int64_t row = first; row < a.rows; row += every) {
        fetch(row + (S - 1) * every, stage == 0 ? S - 1 : stage - 1);
        copies_wait<S - 1>();
        const P* at = mine + stage * A * K * kThreads;
        float acc = 0.f;
        P s[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (me + j * step >= packs) continue;
            s[j] = at[j * kThreads];
            if (RES) {
                // what is normalised is the sum as it is stored: the backward pass reads that
                const P r = at[(A - 1) * K * kThreads + j * kThreads];
#pragma unroll
                for (int e = 0; e < N; ++e) s[j].v[e] = E::from_f(E::to_f(s[j].v[e]) + E::to_f(r.v[e]));
                reinterpret_cast<P*>(static_cast<typename E::T*>(a.sum) + row * a.sum_stride)[me + j * step] = s[j];
            }
#pragma unroll
            for (int e = 0; e < N; ++e) acc += E::to_f(s[j].v[e]);
        }
        const float mean = team.sum(acc) * a.inv_dim;
        acc = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (me + j * step >= packs) continue;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = E::to_f(s[j].v[e]) - mean;
                acc = fmaf(d, d, acc);
            }
        }
        const float rstd = 1.f / sqrtf(team.sum(acc) * a.inv_dim + a.eps);
        if (me == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        P* to = reinterpret_cast<P*>(static_cast<typename E::T*>(a.out) + row * a.out_stride);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (me + j * step >= packs) continue;
            stay_packed(weight[j]);
            stay_packed(bias[j]);
            P y;
#pragma unroll
            for (int e = 0; e < N; ++e)
                y.v[e] = E::from_f(fmaf((E::to_f(s[j].v[e]) - mean) * rstd, Elem<W>::to_f(weight[j].v[e]), Elem<W>::to_f(bias[j].v[e])));
            to[me + j * step] = y;
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    copies_wait<0>();
}

// Rows anywhere, in single elements, K of them a thread, TW warps a team (known here, so that a thread's elements are at
// fixed distances).
template <int DT, int K, bool RES, int TW>
__global__ void __launch_bounds__(TW > kWarps ? 32 * TW : 32 * kWarps, TW > kWarps ? 1 : 2) norm_kernel(const __grid_constant__ FwdArgs a)
{
    using E = Elem<DT>;
    using T = typename E::T;
    constexpr int S = element_rows<DT, RES ? 2 : 1>();
    __shared__ Pair sh[2][kMaxTeam];
    extern __shared__ __align__(16) unsigned char bytes[];   // [teams][S][1 or 2][row_room]
    Team<(TW > 1)> team(sh, TW);
    const int me = team.me, room = row_room<DT>(a.dim), left = a.dim - me;
    constexpr int step = 32 * TW;
    // (half of the elements of a larger team's thread are there: half the team would not hold the row)
    auto holds = [&](int j) { return (TW > 1 && j < K / 2) || j * step < left; };
    unsigned char* ring = bytes + team.index * S * (RES ? 2 : 1) * room;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * team.count() + team.index;
    const int64_t every = static_cast<int64_t>(gridDim.x) * team.count();
    const Rows<DT> x(a.x, a.x_stride, a.rows, a.dim), r(RES ? a.residual : a.x, RES ? a.r_stride : a.x_stride, a.rows, a.dim);
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.rows) {
            x.fetch(row, a.rows, a.dim, ring + stage * (RES ? 2 : 1) * room, me, step);
            if (RES) r.fetch(row, a.rows, a.dim, ring + (stage * 2 + 1) * room, me, step);
        }
        copies_commit();
    };
    wait_for_previous();
    allow_next();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(first + s * every, s);
    float weight[K], bias[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        weight[j] = bias[j] = 0.f;
        if (holds(j) && first < a.rows) {
            weight[j] = column<DT>(a.weight, me + j * step);
            if (a.bias.p) bias[j] = column<DT>(a.bias, me + j * step);
        }
    }
    int stage = 0;
    for (int64_t row = first; row < a.rows; row += every) {
        copies_wait<S - 2>();
        team.barrier();   // every thread's pieces are there, and the row before has been read
        fetch(row + (S - 1) * every, stage == 0 ? S - 1 : stage - 1);
        const T* xs = reinterpret_cast<const T*>(ring + stage * (RES ? 2 : 1) * room) + x.skip(row) + me;
        const T* rs = reinterpret_cast<const T*>(ring + (stage * 2 + 1) * room) + r.skip(row) + me;
        float s[K], acc = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            s[j] = 0.f;
            if (holds(j)) {
                s[j] = E::to_f(xs[j * step]);
                if (RES) s[j] = E::to_f(E::from_f(s[j] + E::to_f(rs[j * step])));
            }
            acc += s[j];
        }
        const float mean = team.sum(acc) * a.inv_dim;
        acc = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (holds(j)) acc = fmaf(s[j] - mean, s[j] - mean, acc);
        const float rstd = 1.f / sqrtf(team.sum(acc) * a.inv_dim + a.eps);
        if (me == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        T* yr = static_cast<T*>(a.out) + row * a.out_stride + me;
        T* sr = RES ? static_cast<T*>(a.sum) + row * a.sum_stride + me : nullptr;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (!holds(j)) continue;
            if (RES) sr[j * step] = E::from_f(s[j]);
            yr[j * step] = E::from_f(fmaf((s[j] - mean) * rstd, weight[j], bias[j]));
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    copies_wait<0>();
}

// Rows that no team holds: three passes over the row, which L2 keeps, in batches of columns whose loads are on their way
// together.  Bound by the instructions and latencies of single elements: 1.1 TB/s in 16 bits (8192 x 12001 with residual
// 704 us), 5.0 in fp32 (4096 x 12288 with residual 160).
constexpr int kBatch = 8;
template <int DT> __global__ void __launch_bounds__(kLoopThreads) norm_loop_kernel(const __grid_constant__ FwdArgs a)
{
    using E = Elem<DT>;
    using T = typename E::T;
    __shared__ Pair sh[2][kMaxTeam];
    Team<true> team(sh, kLoopThreads / 32);
    wait_for_previous();
    allow_next();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* xr = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* rr = a.residual ? static_cast<const T*>(a.residual) + row * a.r_stride : nullptr;
        T* sr = a.residual ? static_cast<T*>(a.sum) + row * a.sum_stride : nullptr;
        const T* from = sr ? sr : xr;   // after the first pass: each thread reads what it wrote itself
        T* yr = static_cast<T*>(a.out) + row * a.out_stride;
        float mean = 0.f, rstd = 0.f;
        for (int pass = 0; pass < 3; ++pass) {
            float acc = 0.f;
            for (int i0 = threadIdx.x; i0 < a.dim; i0 += kBatch * kLoopThreads) {
                float s[kBatch], more[kBatch], b[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = i0 + u * kLoopThreads;
                    s[u] = more[u] = b[u] = 0.f;
                    if (i >= a.dim) continue;
                    s[u] = E::to_f((pass == 0 ? xr : from)[i]);
                    if (pass == 0 && rr) more[u] = E::to_f(rr[i]);
                    if (pass == 2) {
                        more[u] = column<DT>(a.weight, i);
                        if (a.bias.p) b[u] = column<DT>(a.bias, i);
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = i0 + u * kLoopThreads;
                    if (i >= a.dim) continue;
                    if (pass == 0) {
                        if (rr) {
                            sr[i] = E::from_f(s[u] + more[u]);
                            s[u] = E::to_f(E::from_f(s[u] + more[u]));
                        }
                        acc += s[u];
                    } else if (pass == 1) {
                        acc = fmaf(s[u] - mean, s[u] - mean, acc);
                    } else {
                        yr[i] = E::from_f(fmaf((s[u] - mean) * rstd, more[u], b[u]));
                    }
                }
            }
            if (pass == 0) mean = team.sum(acc) * a.inv_dim;
            else if (pass == 1) rstd = 1.f / sqrtf(team.sum(acc) * a.inv_dim + a.eps);
        }
        if (threadIdx.x == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

template <int DT, int W, int K, bool RES, bool MULTI, bool BIG> cudaError_t ring_as(const FwdArgs& a, cudaStream_t s)
{
    constexpr int threads = 32 * (BIG ? kMaxTeam : kWarps), smem = stages<DT, W, K, RES>() * (RES ? 2 : 1) * K * 16 * threads;
    static std::atomic<bool> ready[ddp::kMaxDevices] = {};
    const int teams = threads / 32 / a.team_warps;
    const int grid = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(a.rows) + teams - 1) / teams,
                                                        static_cast<int64_t>(ddp::device_sm_count()) * (BIG ? 1 : per_sm<DT, W, K>())));
    return launch_with_room(norm_ring_kernel<DT, W, K, RES, MULTI, BIG>, ready, grid, threads, smem, smem, a, s);
}
template <int DT, int W, int K, bool RES> cudaError_t ring_team(const FwdArgs& a, cudaStream_t s)
{
    if (a.team_warps == 1) return ring_as<DT, W, K, RES, false, false>(a, s);
    if (a.team_warps <= kWarps) return ring_as<DT, W, K, RES, true, false>(a, s);
    return ring_as<DT, W, K, RES, true, true>(a, s);
}
template <int DT, int W, bool RES> cudaError_t ring_share(const FwdArgs& a, int share, cudaStream_t s)
{
    if (share <= 1) return ring_team<DT, W, 1, RES>(a, s);
    if (share <= 2) return ring_team<DT, W, 2, RES>(a, s);
    if (share <= 3) return ring_team<DT, W, 3, RES>(a, s);
    if (share <= 4) return ring_team<DT, W, 4, RES>(a, s);
    // (fp32 rows of more than 8192 values; with a residual their ring would not fit)
    if constexpr (DT == DDP_F32 && !RES) return ring_as<DT, W, 8, RES, true, true>(a, s);
    return cudaErrorInvalidValue;
}
template <int DT, int K, bool RES, int TW> cudaError_t elements_as(const FwdArgs& a, cudaStream_t s)
{
    constexpr int threads = 32 * (TW > kWarps ? TW : kWarps), arrays = RES ? 2 : 1, most = elements_room<DT, arrays>(threads);
    static std::atomic<bool> ready[ddp::kMaxDevices] = {};
    const int teams = threads / 32 / TW, smem = teams * element_rows<DT, arrays>() * arrays * row_room<DT>(a.dim);
    const int grid = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(a.rows) + teams - 1) / teams,
                                                        static_cast<int64_t>(ddp::device_sm_count()) * (TW > kWarps ? 1 : 2)));
    return launch_with_room(norm_kernel<DT, K, RES, TW>, ready, grid, threads, smem, most, a, s);
}
template <int DT, bool RES> cudaError_t elements_team(const FwdArgs& a, cudaStream_t s)
{
    switch (a.team_warps) {
        case 1:
            if (a.dim <= 32 * 4) return elements_as<DT, 4, RES, 1>(a, s);
            if (a.dim <= 32 * 8) return elements_as<DT, 8, RES, 1>(a, s);
            return a.dim <= 32 * 12 ? elements_as<DT, 12, RES, 1>(a, s) : elements_as<DT, kElements, RES, 1>(a, s);
        case 2: return elements_as<DT, kElements, RES, 2>(a, s);
        case 4: return elements_as<DT, kElements, RES, 4>(a, s);
        case 8: return elements_as<DT, kElements, RES, 8>(a, s);
        default: return elements_as<DT, kElements, RES, 16>(a, s);
    }
}

template <int DT, bool RES> cudaError_t forward_as(FwdArgs a, bool vectors, cudaStream_t s)
{
    if (vectors) {
        const int packs = a.dim / Vec<DT>::N;
        a.team_warps = team_for(packs, 4);
        if (a.team_warps == 0 && DT == DDP_F32 && !RES) a.team_warps = team_for(packs, 8);
        if (a.team_warps) {
            const int share = (packs + 32 * a.team_warps - 1) / (32 * a.team_warps);
            return a.weight.wide ? ring_share<DT, DDP_F32, RES>(a, share, s) : ring_share<DT, DT, RES>(a, share, s);
        }
    } else if ((a.team_warps = team_for(a.dim, kElements)) != 0) {
        return elements_team<DT, RES>(a, s);
    }
    return launch_chained(norm_loop_kernel<DT>, dim3(std::min(a.rows, 4 * ddp::device_sm_count())), kLoopThreads, 0, s, a);
}
template <int DT> cudaError_t forward(const FwdArgs& a, bool vectors, cudaStream_t s)
{
    return a.residual ? forward_as<DT, true>(a, vectors, s) : forward_as<DT, false>(a, vectors, s);
}

}  // namespace
}  // namespace ddplm

extern "C" ddp_status ddp_layer_norm_forward(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                             int32_t dtype, int64_t ntokens, int64_t dim, const void* weight,
                                             const void* bias, int32_t w_dtype, float eps, void* out, int64_t out_stride,
                                             void* sum, int64_t sum_stride, float* mean, float* rstd, void* stream)
{
    using namespace ddplm;
    const char* fn = "ddp_layer_norm_forward";
    ddp_status st = check_sizes(fn, ntokens, dim);
    if (st == DDP_OK) st = check_types(fn, dtype, w_dtype);
    if (st != DDP_OK) return st;
    if (!(eps >= 0.f) || std::isinf(eps)) return ddp::fail(DDP_E_INVAL, "%s: eps = %g", fn, eps);
    if (!residual != !sum) return ddp::fail(DDP_E_INVAL, "%s: a residual and a sum come together", fn);
    if (ntokens == 0) return ddp::ok();
    if ((st = check_rows(fn, "x", x, x_stride, ntokens, dim)) != DDP_OK) return st;
    if ((st = check_rows(fn, "out", out, out_stride, ntokens, dim)) != DDP_OK) return st;
    if (residual) {
        if ((st = check_rows(fn, "residual", residual, residual_stride, ntokens, dim)) != DDP_OK) return st;
        if ((st = check_rows(fn, "sum", sum, sum_stride, ntokens, dim)) != DDP_OK) return st;
        if (out == sum) return ddp::fail(DDP_E_INVAL, "%s: out is sum", fn);
    }
    if (!weight) return ddp::fail(DDP_E_INVAL, "%s: weight is NULL", fn);
    if (!mean || !rstd) return ddp::fail(DDP_E_INVAL, "%s: mean or rstd is NULL", fn);
    if (ntokens == 1) x_stride = residual_stride = out_stride = sum_stride = 0;
    const bool vectors = dim % (16 / elem_size(dtype)) == 0 && row_vectors(x, x_stride, dtype) && row_vectors(out, out_stride, dtype) &&
                         (!residual || (row_vectors(residual, residual_stride, dtype) && row_vectors(sum, sum_stride, dtype)));
    const FwdArgs a{x, residual, columns_of(weight, w_dtype), columns_of(bias, w_dtype), out, sum, mean, rstd, x_stride, residual_stride, out_stride, sum_stride,
                    static_cast<int32_t>(ntokens), static_cast<int32_t>(dim), 0, eps, 1.f / static_cast<float>(dim)};
    return launched(fn, DDP_FOR_TYPE(dtype, forward)(a, vectors, static_cast<cudaStream_t>(stream)));
}
