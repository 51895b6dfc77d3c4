// Layer norm, backward (the formulas and the teams of warps: layer_norm.cuh).
#include "layer_norm.cuh"

namespace ddplm {
namespace {

struct BwdArgs {
    const void *dy, *x, *ds;
    Columns weight;
    const float *mean, *rstd;
    void* dx;
    float* part;   // [2][parts][dim]: sums of dw, then of db; nullptr: not wanted
    int64_t dy_stride, x_stride, ds_stride, dx_stride;
    int32_t rows, dim, team_warps;
    float inv_dim;
};

// A thread's sums of dw and db: the columns of packs me, me + step, ... of every row of its team.
template <int K, int N> struct Sums {
    float w[K][N], b[K][N];
    __device__ __forceinline__ Sums()
    {
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e) w[j][e] = b[j][e] = 0.f;
    }
    // The CTA's, in the order of its teams, to its row of the partial sums, where element e of pack p is at
    // e packs + p.  room: 8 K N bytes a thread where there are several teams; every thread calls it.
    __device__ __forceinline__ void store(float* part, int64_t dim, float* room, int packs, int me, int step)
    {
        float* pw = part + blockIdx.x * dim;
        float* pb = pw + gridDim.x * dim;
        const int threads = blockDim.x;
        if (step == threads) {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (me + j * step < packs)
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        pw[e * packs + me + j * step] = w[j][e];
                        pb[e * packs + me + j * step] = b[j][e];
                    }
            return;
        }
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                room[(e * K + j) * threads + threadIdx.x] = w[j][e];
                room[((N + e) * K + j) * threads + threadIdx.x] = b[j][e];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * N * packs; i += threads) {
            const int e = i / packs, p = i - e * packs, j = p / step;
            const float* from = room + (e * K + j) * threads + (p - j * step);
            float v = from[0];
            for (int t = step; t < threads; t += step) v += from[t];
            (e < N ? pw : pb)[(e < N ? e : e - N) * packs + p] = v;
        }
    }
};

// One pack of a row, first for the row's sums, then for dx.
template <int DT, int W, int N>
__device__ __forceinline__ void add_pack(const Pack<DT, N>& x, const Pack<DT, N>& g, const Pack<W, N>& w, float mean, float rstd,
                                         float (&dw)[N], float (&db)[N], Pair& acc)
{
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float y = Elem<DT>::to_f(g.v[e]), n = (Elem<DT>::to_f(x.v[e]) - mean) * rstd;
        dw[e] = fmaf(y, n, dw[e]);
        db[e] += y;
        const float gw = y * Elem<W>::to_f(w.v[e]);
        acc.a += gw;
        acc.b = fmaf(gw, n, acc.b);
    }
}
template <bool DS, int DT, int W, int N>
__device__ __forceinline__ Pack<DT, N> dx_pack(const Pack<DT, N>& x, const Pack<DT, N>& g, const Pack<DT, N>& d, const Pack<W, N>& w,
                                               float mean, float rstd, float m1, float m2)
{
    Pack<DT, N> o;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float n = (Elem<DT>::to_f(x.v[e]) - mean) * rstd;
        float v = rstd * (fmaf(Elem<DT>::to_f(g.v[e]), Elem<W>::to_f(w.v[e]), -m1) - n * m2);
        if (DS) v += Elem<DT>::to_f(d.v[e]);
        o.v[e] = Elem<DT>::from_f(v);
    }
    return o;
}

// Rows on 16-byte boundaries, through a ring in shared memory as in the forward pass.
template <int K, bool DS> __host__ __device__ constexpr int stages()
{
    return ring_rows((224 << 10) / kPerSm - 2048, (DS ? 3 : 2) * K * 16 * 32 * kWarps);
}

template <int DT, int W, int K, bool DS, bool MULTI, bool BIG>
__global__ void __launch_bounds__(32 * (BIG ? kMaxTeam : kWarps), BIG ? 1 : kPerSm) norm_grad_ring_kernel(const __grid_constant__ BwdArgs a)
{
    using E = Elem<DT>;
    using T = typename E::T;
    constexpr int N = Vec<DT>::N, S = stages<K, DS>(), A = DS ? 3 : 2, kThreads = 32 * (BIG ? kMaxTeam : kWarps);
    // the weights stay in registers beside the sums where they take 24 at most
    constexpr bool HOLD = K * N * (W == DDP_F32 ? 4 : 2) / 4 <= 24;
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
            const P* x = reinterpret_cast<const P*>(static_cast<const T*>(a.x) + row * a.x_stride);
            const P* g = reinterpret_cast<const P*>(static_cast<const T*>(a.dy) + row * a.dy_stride);
            const P* d = DS ? reinterpret_cast<const P*>(static_cast<const T*>(a.ds) + row * a.ds_stride) : nullptr;
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (me + j * step < packs) {
                    const uint32_t to = mine_at + (stage * A * K + j) * 16 * kThreads;
                    copy16(to, x + me + j * step);
                    copy16(to + K * 16 * kThreads, g + me + j * step);
                    if (DS) copy16(to + 2 * K * 16 * kThreads, d + me + j * step);
                }
        }
        copies_commit();
    };
    wait_for_previous();
    allow_next();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(first + s * every, s);
    Pack<W, N> weight[HOLD ? K : 1];
    if (HOLD && first < a.rows)
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (me + j * step < packs) weight[HOLD ? j : 0] = load_columns<W, N>(a.weight, me + j * step);
    Sums<K, N> sums;
    int stage = 0;
    float mean = 0.f, rstd = 0.f;
    if (first < a.rows) {
        mean = a.mean[first];
        rstd = a.rstd[first];
    }
    for (int64_t row = first; row < a.rows; row += every) {
        fetch(row + (S - 1) * every, stage == 0 ? S - 1 : stage - 1);
        float next_mean = 0.f, next_rstd = 0.f;
        if (row + every < a.rows) {
            next_mean = a.mean[row + every];
            next_rstd = a.rstd[row + every];
        }
        copies_wait<S - 1>();
        const P* at = mine + stage * A * K * kThreads;
        Pair acc{0.f, 0.f};
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (me + j * step >= packs) continue;
            if (HOLD) stay_packed(weight[HOLD ? j : 0]);
            else weight[0] = load_columns<W, N>(a.weight, me + j * step);
            add_pack(at[j * kThreads], at[(K + j) * kThreads], weight[HOLD ? j : 0], mean, rstd, sums.w[j], sums.b[j], acc);
        }
        acc = team.sum(acc);
        const float m1 = acc.a * a.inv_dim, m2 = acc.b * a.inv_dim;
        P* to = reinterpret_cast<P*>(static_cast<T*>(a.dx) + row * a.dx_stride);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (me + j * step >= packs) continue;
            if (HOLD) stay_packed(weight[HOLD ? j : 0]);
            else weight[0] = load_columns<W, N>(a.weight, me + j * step);
            to[me + j * step] = dx_pack<DS>(at[j * kThreads], at[(K + j) * kThreads], at[((A - 1) * K + j) * kThreads], weight[HOLD ? j : 0],
                                            mean, rstd, m1, m2);
        }
        mean = next_mean;
        rstd = next_rstd;
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    copies_wait<0>();
    if (!a.part) return;
    __syncthreads();   // the ring becomes the room where the teams' sums meet
    sums.store(a.part, a.dim, reinterpret_cast<float*>(ring), packs, me, step);
}

// Rows anywhere, in single elements, K of them a thread, TW warps a team (known here, so that a thread's elements are at
// fixed distances).
template <int DT, int K, bool DS, int TW>
__global__ void __launch_bounds__(TW > kWarps ? 32 * TW : 32 * kWarps, TW > kWarps ? 1 : kPerSm) norm_grad_kernel(const __grid_constant__ BwdArgs a)
{
    using E = Elem<DT>;
    using T = typename E::T;
    using P = Pack<DT, 1>;
    constexpr int A = DS ? 3 : 2, S = element_rows<DT, A>();
    __shared__ Pair sh[2][kMaxTeam];
    extern __shared__ __align__(16) unsigned char bytes[];   // [teams][S][A][row_room]
    Team<(TW > 1)> team(sh, TW);
    const int me = team.me, room = row_room<DT>(a.dim), left = a.dim - me;
    constexpr int step = 32 * TW;
    // (half of the elements of a larger team's thread are there: half the team would not hold the row)
    auto holds = [&](int j) { return (TW > 1 && j < K / 2) || j * step < left; };
    unsigned char* ring = bytes + team.index * S * A * room;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * team.count() + team.index;
    const int64_t every = static_cast<int64_t>(gridDim.x) * team.count();
    const Rows<DT> x(a.x, a.x_stride, a.rows, a.dim), dy(a.dy, a.dy_stride, a.rows, a.dim);
    const Rows<DT> ds(DS ? a.ds : a.x, DS ? a.ds_stride : a.x_stride, a.rows, a.dim);
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.rows) {
            unsigned char* to = ring + stage * A * room;
            x.fetch(row, a.rows, a.dim, to, me, step);
            dy.fetch(row, a.rows, a.dim, to + room, me, step);
            if (DS) ds.fetch(row, a.rows, a.dim, to + 2 * room, me, step);
        }
        copies_commit();
    };
    wait_for_previous();
    allow_next();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(first + s * every, s);
    Pack<DDP_F32, 1> weight[K];
#pragma unroll
    for (int j = 0; j < K; ++j) weight[j].v[0] = holds(j) && first < a.rows ? column<DT>(a.weight, me + j * step) : 0.f;
    Sums<K, 1> sums;
    int stage = 0;
    float mean = 0.f, rstd = 0.f;
    if (first < a.rows) {
        mean = a.mean[first];
        rstd = a.rstd[first];
    }
    for (int64_t row = first; row < a.rows; row += every) {
        copies_wait<S - 2>();
        team.barrier();   // every thread's pieces are there, and the row before has been read
        fetch(row + (S - 1) * every, stage == 0 ? S - 1 : stage - 1);
        float next_mean = 0.f, next_rstd = 0.f;
        if (row + every < a.rows) {
            next_mean = a.mean[row + every];
            next_rstd = a.rstd[row + every];
        }
        const unsigned char* at = ring + stage * A * room;
        const P* xs = reinterpret_cast<const P*>(at) + x.skip(row) + me;
        const P* gs = reinterpret_cast<const P*>(at + room) + dy.skip(row) + me;
        const P* dd = DS ? reinterpret_cast<const P*>(at + 2 * room) + ds.skip(row) + me : xs;
        Pair acc{0.f, 0.f};
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (holds(j)) add_pack(xs[j * step], gs[j * step], weight[j], mean, rstd, sums.w[j], sums.b[j], acc);
        acc = team.sum(acc);
        const float m1 = acc.a * a.inv_dim, m2 = acc.b * a.inv_dim;
        P* to = reinterpret_cast<P*>(static_cast<T*>(a.dx) + row * a.dx_stride) + me;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (holds(j)) to[j * step] = dx_pack<DS>(xs[j * step], gs[j * step], dd[j * step], weight[j], mean, rstd, m1, m2);
        mean = next_mean;
        rstd = next_rstd;
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    copies_wait<0>();
    if (!a.part) return;
    __syncthreads();
    sums.store(a.part, a.dim, reinterpret_cast<float*>(bytes), a.dim, me, step);
}

// fp32 rows of more than 8192 values, on 16-byte boundaries, whose ring would not fit: in registers, a CTA each, whose loads
// have nothing beside them to hide behind (4096 x 12288 with ds 252 us, 3.2 TB/s).
template <int K, bool DS> __global__ void __launch_bounds__(32 * kMaxTeam) norm_grad_wide_kernel(const __grid_constant__ BwdArgs a)
{
    using P = Pack<DDP_F32, 4>;
    constexpr int kStep = 32 * kMaxTeam;
    __shared__ Pair sh[2][kMaxTeam];
    Team<true> team(sh, kMaxTeam);
    const int me = threadIdx.x, packs = a.dim / 4;
    wait_for_previous();
    allow_next();
    Sums<K, 4> sums;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        P x[K], g[K];
        const P* xr = reinterpret_cast<const P*>(static_cast<const float*>(a.x) + row * a.x_stride);
        const P* gr = reinterpret_cast<const P*>(static_cast<const float*>(a.dy) + row * a.dy_stride);
        const P* dr = DS ? reinterpret_cast<const P*>(static_cast<const float*>(a.ds) + row * a.ds_stride) : xr;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (me + j * kStep < packs) {
                x[j] = xr[me + j * kStep];
                g[j] = gr[me + j * kStep];
            }
        const float mean = a.mean[row], rstd = a.rstd[row];
        Pair acc{0.f, 0.f};
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (me + j * kStep < packs)
                add_pack(x[j], g[j], load_columns<DDP_F32, 4>(a.weight, me + j * kStep), mean, rstd, sums.w[j], sums.b[j], acc);
        acc = team.sum(acc);
        const float m1 = acc.a * a.inv_dim, m2 = acc.b * a.inv_dim;
        P* to = reinterpret_cast<P*>(static_cast<float*>(a.dx) + row * a.dx_stride);
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (me + j * kStep < packs)
                to[me + j * kStep] = dx_pack<DS>(x[j], g[j], dr[me + j * kStep], load_columns<DDP_F32, 4>(a.weight, me + j * kStep), mean, rstd, m1, m2);
    }
    if (a.part) sums.store(a.part, a.dim, nullptr, packs, me, kStep);
}

// Rows that no team holds: two passes over the row, which L2 keeps, in batches of columns whose loads are on their way
// together.  The sums of a column, which belongs to one thread, are in the workspace.  8192 x 12001 bf16 with ds 762 us
// (1.0 TB/s): single elements, and each column's sums read and written for every row.
constexpr int kBatch = 8;
template <int DT> __global__ void __launch_bounds__(kLoopThreads) norm_grad_loop_kernel(const __grid_constant__ BwdArgs a)
{
    using E = Elem<DT>;
    using T = typename E::T;
    __shared__ Pair sh[2][kMaxTeam];
    Team<true> team(sh, kLoopThreads / 32);
    wait_for_previous();
    allow_next();
    float* pw = a.part ? a.part + static_cast<int64_t>(blockIdx.x) * a.dim : nullptr;
    float* pb = a.part ? pw + static_cast<int64_t>(gridDim.x) * a.dim : nullptr;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* xr = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* gr = static_cast<const T*>(a.dy) + row * a.dy_stride;
        const T* dr = a.ds ? static_cast<const T*>(a.ds) + row * a.ds_stride : nullptr;
        T* to = static_cast<T*>(a.dx) + row * a.dx_stride;
        const float mean = a.mean[row], rstd = a.rstd[row];
        const bool begin = row == blockIdx.x;
        Pair acc{0.f, 0.f};
        for (int i0 = threadIdx.x; i0 < a.dim; i0 += kBatch * kLoopThreads) {
            float x[kBatch], y[kBatch], w[kBatch], sw[kBatch], sb[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u * kLoopThreads;
                x[u] = y[u] = w[u] = sw[u] = sb[u] = 0.f;
                if (i >= a.dim) continue;
                x[u] = E::to_f(xr[i]);
                y[u] = E::to_f(gr[i]);
                w[u] = column<DT>(a.weight, i);
                if (pw && !begin) {
                    sw[u] = pw[i];
                    sb[u] = pb[i];
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u * kLoopThreads;
                if (i >= a.dim) continue;
                const float n = (x[u] - mean) * rstd, gw = y[u] * w[u];
                acc.a += gw;
                acc.b = fmaf(gw, n, acc.b);
                if (pw) {
                    pw[i] = fmaf(y[u], n, sw[u]);
                    pb[i] = y[u] + sb[u];
                }
            }
        }
        acc = team.sum(acc);
        const float m1 = acc.a * a.inv_dim, m2 = acc.b * a.inv_dim;
        for (int i0 = threadIdx.x; i0 < a.dim; i0 += kBatch * kLoopThreads) {
            float x[kBatch], y[kBatch], w[kBatch], d[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u * kLoopThreads;
                x[u] = y[u] = w[u] = d[u] = 0.f;
                if (i >= a.dim) continue;
                x[u] = E::to_f(xr[i]);
                y[u] = E::to_f(gr[i]);
                w[u] = column<DT>(a.weight, i);
                if (dr) d[u] = E::to_f(dr[i]);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u * kLoopThreads;
                if (i < a.dim) to[i] = E::from_f(rstd * (fmaf(y[u], w[u], -m1) - (x[u] - mean) * rstd * m2) + d[u]);
            }
        }
    }
}

// The partial sums of dw (blockIdx.y 0) and db (1), joined: 32 columns a CTA, 32 threads a column.
struct JoinArgs {
    const float* part;
    void* out[2];
    int32_t parts, dim, packs, accumulate;   // element e of pack p of a row: e packs + p
};
template <int GDT> __global__ void __launch_bounds__(1024) join_columns_kernel(const __grid_constant__ JoinArgs a)
{
    using E = Elem<GDT>;
    __shared__ float sh[32][33];
    wait_for_previous();
    allow_next();
    typename E::T* out = static_cast<typename E::T*>(a.out[blockIdx.y]);
    if (!out) return;
    const int mine = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
    const float* p = a.part + static_cast<int64_t>(blockIdx.y) * a.parts * a.dim;
    float acc = 0.f;
    if (mine < a.dim) {
#pragma unroll 8
        for (int i = lane; i < a.parts; i += 32) acc += p[static_cast<int64_t>(i) * a.dim + mine];
    }
    sh[lane][threadIdx.x & 31] = acc;
    __syncthreads();
    // a warp a column: its 32 sums, joined as a tree
    acc = sh[threadIdx.x & 31][lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    const int at = blockIdx.x * 32 + lane;
    if ((threadIdx.x & 31) || at >= a.dim) return;
    const int each = a.dim / a.packs, e = at / a.packs, col = (at - e * a.packs) * each + e;
    if (a.accumulate) acc += E::to_f(out[col]);
    out[col] = E::from_f(acc);
}

// CTAs that write partial sums (and so the workspace): each has two dim values.
int64_t most_parts(int64_t rows, int64_t dim)
{
    const int64_t ctas = std::min<int64_t>(rows, static_cast<int64_t>(ddp::device_sm_count()) * kPerSm);
    return dim > 32 * kMaxTeam * 32 ? std::min(ctas, std::max<int64_t>(1, kLoopPartials / dim)) : ctas;
}

template <int DT, int W, int K, bool DS, bool MULTI, bool BIG> cudaError_t ring_as(const BwdArgs& a, int parts, cudaStream_t s)
{
    constexpr int threads = 32 * (BIG ? kMaxTeam : kWarps), smem = stages<K, DS>() * (DS ? 3 : 2) * K * 16 * threads;
    static std::atomic<bool> ready[ddp::kMaxDevices] = {};
    return launch_with_room(norm_grad_ring_kernel<DT, W, K, DS, MULTI, BIG>, ready, parts, threads, smem, smem, a, s);
}
template <int DT, int W, int K, bool DS> cudaError_t ring_team(const BwdArgs& a, int parts, cudaStream_t s)
{
    if (a.team_warps == 1) return ring_as<DT, W, K, DS, false, false>(a, parts, s);
    if (a.team_warps <= kWarps) return ring_as<DT, W, K, DS, true, false>(a, parts, s);
    return ring_as<DT, W, K, DS, true, true>(a, parts, s);
}
template <int DT, int W, bool DS> cudaError_t ring_share(const BwdArgs& a, int share, int parts, cudaStream_t s)
{
    if (share <= 1) return ring_team<DT, W, 1, DS>(a, parts, s);
    if (share <= 2) return ring_team<DT, W, 2, DS>(a, parts, s);
    return share <= 3 ? ring_team<DT, W, 3, DS>(a, parts, s) : ring_team<DT, W, 4, DS>(a, parts, s);
}

template <int DT, int K, bool DS, int TW> cudaError_t elements_as(const BwdArgs& a, int parts, cudaStream_t s)
{
    constexpr int threads = 32 * (TW > kWarps ? TW : kWarps), arrays = DS ? 3 : 2, most = elements_room<DT, arrays>(threads);
    static std::atomic<bool> ready[ddp::kMaxDevices] = {};
    constexpr int teams = threads / 32 / TW;
    // (the teams' sums meet where the rings were)
    const int smem = std::max(teams * element_rows<DT, arrays>() * arrays * row_room<DT>(a.dim), teams > 1 ? 8 * K * threads : 0);
    return launch_with_room(norm_grad_kernel<DT, K, DS, TW>, ready, parts, threads, smem, most, a, s);
}
template <int DT, bool DS> cudaError_t elements_team(const BwdArgs& a, int parts, cudaStream_t s)
{
    switch (a.team_warps) {
        case 1:
            if (a.dim <= 32 * 4) return elements_as<DT, 4, DS, 1>(a, parts, s);
            if (a.dim <= 32 * 8) return elements_as<DT, 8, DS, 1>(a, parts, s);
            return a.dim <= 32 * 12 ? elements_as<DT, 12, DS, 1>(a, parts, s) : elements_as<DT, kElements, DS, 1>(a, parts, s);
        case 2: return elements_as<DT, kElements, DS, 2>(a, parts, s);
        case 4: return elements_as<DT, kElements, DS, 4>(a, parts, s);
        case 8: return elements_as<DT, kElements, DS, 8>(a, parts, s);
        default: return elements_as<DT, kElements, DS, 16>(a, parts, s);
    }
}

// *parts: the CTAs, whose sums are in a.part; *packs: how they lie there
template <int DT, bool DS> cudaError_t backward_as(BwdArgs a, bool vectors, int* parts, int* packs, cudaStream_t s)
{
    const int sms = ddp::device_sm_count();
    *packs = vectors ? a.dim / Vec<DT>::N : a.dim;
    a.team_warps = vectors ? team_for(*packs, 4) : team_for(a.dim, kElements);
    if (a.team_warps) {
        const int warps = cta_warps(a.team_warps), teams = warps / a.team_warps;
        *parts = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(a.rows) + teams - 1) / teams,
                                                    static_cast<int64_t>(sms) * (warps > kWarps ? 1 : kPerSm)));
        if (!vectors) return elements_team<DT, DS>(a, *parts, s);
        const int share = (*packs + 32 * a.team_warps - 1) / (32 * a.team_warps);
        return a.weight.wide ? ring_share<DT, DDP_F32, DS>(a, share, *parts, s) : ring_share<DT, DT, DS>(a, share, *parts, s);
    }
    if (vectors && DT == DDP_F32 && team_for(*packs, 8)) {
        *parts = std::min(a.rows, sms);
        return launch_chained(norm_grad_wide_kernel<8, DS>, dim3(*parts), 32 * kMaxTeam, 0, s, a);
    }
    *packs = a.dim;
    *parts = static_cast<int>(most_parts(a.rows, a.dim));
    return launch_chained(norm_grad_loop_kernel<DT>, dim3(*parts), kLoopThreads, 0, s, a);
}
template <int DT> cudaError_t backward(const BwdArgs& a, bool vectors, int* parts, int* packs, cudaStream_t s)
{
    return a.ds ? backward_as<DT, true>(a, vectors, parts, packs, s) : backward_as<DT, false>(a, vectors, parts, packs, s);
}

}  // namespace
}  // namespace ddplm

extern "C" ddp_status ddp_layer_norm_workspace(int64_t ntokens, int64_t dim, int64_t* bytes)
{
    using namespace ddplm;
    const char* fn = "ddp_layer_norm_workspace";
    const ddp_status st = check_sizes(fn, ntokens, dim);
    if (st != DDP_OK) return st;
    if (!bytes) return ddp::fail(DDP_E_INVAL, "%s: bytes is NULL", fn);
    *bytes = 256 + 8 * dim * most_parts(ntokens, dim);
    return ddp::ok();
}

extern "C" ddp_status ddp_layer_norm_backward(const void* grad_out, int64_t grad_stride, const void* x, int64_t x_stride,
                                              const float* mean, const float* rstd, const void* grad_sum,
                                              int64_t grad_sum_stride, int32_t dtype, int64_t ntokens, int64_t dim,
                                              const void* weight, int32_t w_dtype, void* grad_x, int64_t grad_x_stride,
                                              void* grad_weight, void* grad_bias, int32_t gw_dtype, int32_t accumulate,
                                              void* workspace, int64_t workspace_bytes, void* stream)
{
    using namespace ddplm;
    using ddp::fail;
    const char* fn = "ddp_layer_norm_backward";
    ddp_status st = check_sizes(fn, ntokens, dim);
    if (st == DDP_OK) st = check_types(fn, dtype, w_dtype);
    if (st != DDP_OK) return st;
    const bool columns = grad_weight || grad_bias;
    if (columns) {
        if (gw_dtype != dtype && gw_dtype != DDP_F32)
            return fail(DDP_E_INVAL, "%s: gw_dtype %d is neither the dtype nor DDP_F32", fn, gw_dtype);
        if (grad_weight == grad_bias) return fail(DDP_E_INVAL, "%s: grad_weight is grad_bias", fn);
        if (!workspace) return fail(DDP_E_INVAL, "%s: workspace is NULL", fn);
        if (reinterpret_cast<uintptr_t>(workspace) & 255)
            return fail(DDP_E_INVAL, "%s: workspace is not 256-byte aligned", fn);
        const int64_t need = 8 * dim * most_parts(ntokens, dim);
        if (workspace_bytes < need)
            return fail(DDP_E_INVAL, "%s: workspace of %lld bytes, needs %lld", fn, static_cast<long long>(workspace_bytes),
                        static_cast<long long>(need));
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int parts = 0, packs = 1;
    if (ntokens > 0) {
        if ((st = check_rows(fn, "grad_out", grad_out, grad_stride, ntokens, dim)) != DDP_OK) return st;
        if ((st = check_rows(fn, "x", x, x_stride, ntokens, dim)) != DDP_OK) return st;
        if ((st = check_rows(fn, "grad_x", grad_x, grad_x_stride, ntokens, dim)) != DDP_OK) return st;
        if (grad_sum && (st = check_rows(fn, "grad_sum", grad_sum, grad_sum_stride, ntokens, dim)) != DDP_OK) return st;
        if (!weight) return fail(DDP_E_INVAL, "%s: weight is NULL", fn);
        if (!mean || !rstd) return fail(DDP_E_INVAL, "%s: mean or rstd is NULL", fn);
        if (ntokens == 1) grad_stride = x_stride = grad_x_stride = grad_sum_stride = 0;
        const bool vectors = dim % (16 / elem_size(dtype)) == 0 && row_vectors(grad_out, grad_stride, dtype) &&
                             row_vectors(x, x_stride, dtype) && row_vectors(grad_x, grad_x_stride, dtype) &&
                             (!grad_sum || row_vectors(grad_sum, grad_sum_stride, dtype));
        const BwdArgs a{grad_out, x, grad_sum, columns_of(weight, w_dtype), mean, rstd, grad_x, columns ? static_cast<float*>(workspace) : nullptr,
                        grad_stride, x_stride, grad_sum_stride, grad_x_stride, static_cast<int32_t>(ntokens),
                        static_cast<int32_t>(dim), 0, 1.f / static_cast<float>(dim)};
        const cudaError_t e = DDP_FOR_TYPE(dtype, backward)(a, vectors, &parts, &packs, s);
        if (e != cudaSuccess) return launched(fn, e);
    }
    if (!columns || (parts == 0 && accumulate)) return ddp::ok();
    const JoinArgs j{static_cast<const float*>(workspace), {grad_weight, grad_bias}, parts, static_cast<int32_t>(dim), packs, accumulate};
    const dim3 grid(static_cast<unsigned>((dim + 31) / 32), 2);
    const auto join = gw_dtype == DDP_F32 ? join_columns_kernel<DDP_F32> : gw_dtype == DDP_BF16 ? join_columns_kernel<DDP_BF16> : join_columns_kernel<DDP_F16>;
    return launched(fn, launch_chained(join, grid, 1024, 0, s, j));
}
