// Token embedding: lookup with a scale, and the table's gradient by sorted tokens.
//
//   out[t] = s * W[id_t]                      dW[v] = s * sum over t with id_t = v of dY[t]
//
// The gradient is a segmented sum.  Tokens are sorted by id (equal ids in token
// order) and each row of dW is the fp32 sum of its run, taken in that order: no
// atomics, the same bits every time.  HBM-bound: dY is read once, dW written once.
//
// Sort: one launch in which each of N CTAs owns the ids that leave its number as the
// remainder by N, reads all the tokens and keeps those of its ids.  A token's place is
// (tokens with smaller remainders) + (tokens with its remainder and smaller ids) +
// (earlier tokens with its id): no CTA needs a result of another.  The order that comes
// out keeps equal ids together, which is all the sums need, and the frequent ids, which
// are often neighbours, are dealt out over the CTAs (with ranges of neighbouring ids the
// owner of the most frequent ones took 84 us where even ids took 31, at 65521 tokens).
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
// HBM-bound: a row read and a row written for each token, 16 bytes a thread where the
// tensors allow it.  8192 rows of 768 fp32: 10 us with cold caches (50 MB, 5.0 TB/s); one
// row is a launch and three dependent reads, 3.6 us.
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
constexpr uint16_t kNone = 0xffff;
// Tokens are counted in 32 bits, up to a step of the loops beyond the last one (512, and 2048 in the stretches' lengths).
constexpr int64_t kMaxSortTokens = (int64_t{1} << 31) - 4096;
constexpr int kMaxRange = 1024;  // ids a sorting CTA owns at most (its counters: 4 bytes an id and warp)
constexpr int kMinSortCtas = 128;  // a power of two, one wave
constexpr int kIdBatch = 8;      // loads of ids a thread keeps in flight
constexpr int kSortSmem = 220 * 1024;  // counters, and the tokens' places in the range where they fit

struct SortArgs {
    const void* ids;
    int32_t id_bytes;
    int32_t ntokens;
    int64_t vocab, padding_idx;
    int32_t range;   // ids per CTA at most
    int32_t shift;   // 2^shift CTAs
    int32_t* order;  // [ntokens] sorted tokens
    int32_t* key;    // [ntokens] their ids
    int2* run;       // [vocab] first place of each id in `order` and the one after its last
    int32_t* total;  // tokens in `order`
    int* status;
    int32_t cached;  // the second pass reads what the first one left in shared memory
    // rows of ids that do not occur (nullptr: left alone)
    uint8_t* clear;
    int64_t clear_stride, clear_bytes;
};

// Bound by every CTA's look at every token, from L2: 8 bytes and a dozen instructions.  9 us
// for 8192 tokens, 39 us for 65521 (a first pass of 18 us, the owner of the most frequent
// ids 17 us in the second; the rows to clear are written meanwhile).
__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortArgs a)
{
    extern __shared__ int32_t sh[];  // [warp][range] counters, then places
    __shared__ int32_t less_w[kSortWarps], part[kSortWarps];
    __shared__ uint8_t seen[kMaxRange];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* cnt = sh + warp * a.range;
    uint16_t* place = reinterpret_cast<uint16_t*>(sh + kSortWarps * a.range);  // [ntokens], where it fits
    // the CTA's ids: own + (r << shift), r < nr
    const uint32_t own = blockIdx.x, mask = (1u << a.shift) - 1u, vocab32 = static_cast<uint32_t>(a.vocab);
    const uint32_t pad32 = a.padding_idx >= 0 && a.padding_idx < a.vocab ? static_cast<uint32_t>(a.padding_idx) : 0xffffffffu;
    const int nr = own < vocab32 ? static_cast<int>((vocab32 - own - 1) >> a.shift) + 1 : 0;
    for (int i = tid; i < kSortWarps * a.range; i += kSortThreads) sh[i] = 0;
    __syncthreads();
    wait_for_previous();
    // each warp counts a contiguous stretch of tokens (a multiple of 64 of them)
    const int per = (a.ntokens + 64 * kSortWarps - 1) / (64 * kSortWarps) * 64;
    const int t0 = min(warp * per, a.ntokens), t1 = min(t0 + per, a.ntokens);
    int32_t less = 0;
    bool bad = false;
    // The remainder of a token's id, or one that no CTA has; ids of 2^31 and more are out of
    // any vocabulary.  (Few instructions: every CTA looks at every token.)
    auto remainder = [&](int64_t id) {
        const uint32_t x = static_cast<uint32_t>(id);
        const bool known = static_cast<uint32_t>(static_cast<uint64_t>(id) >> 32) == 0 && x < vocab32;
        if (blockIdx.x == 0) bad |= !known;
        return known && x != pad32 ? x & mask : 0xffffffffu;
    };
    auto row_of = [&](uint32_t rem, int64_t id) { return rem == own ? static_cast<uint32_t>(id) >> a.shift : uint32_t{kNone}; };
    // pairs of ids in 16-byte (8-byte) loads where the list starts on such a boundary
    const bool pairs = (reinterpret_cast<uintptr_t>(a.ids) & (2 * a.id_bytes - 1)) == 0;
    const int whole = pairs ? t0 + (t1 - t0) / 2 * 2 : t0;
    for (int t = t0 + 2 * lane; t < whole; t += 64 * kIdBatch) {
        int64_t id[kIdBatch][2];
#pragma unroll
        for (int j = 0; j < kIdBatch; ++j) {
            const int u = t + 64 * j;
            if (u >= whole) continue;
            if (a.id_bytes == 8) {
                const longlong2 v = __ldg(reinterpret_cast<const longlong2*>(static_cast<const long long*>(a.ids) + u));
                id[j][0] = v.x; id[j][1] = v.y;
            } else {
                const int2 v = __ldg(reinterpret_cast<const int2*>(static_cast<const int*>(a.ids) + u));
                id[j][0] = v.x; id[j][1] = v.y;
            }
        }
#pragma unroll
        for (int j = 0; j < kIdBatch; ++j) {
            if (t + 64 * j >= whole) continue;
            const uint32_t p = remainder(id[j][0]), q = remainder(id[j][1]);
            less += (p < own) + (q < own);
            uint32_t rows = 0xffffffffu;
            if (p == own || q == own) {
                rows = row_of(p, id[j][0]) | (row_of(q, id[j][1]) << 16);
                if (p == own) atomicAdd(&cnt[rows & 0xffffu], 1);
                if (q == own) atomicAdd(&cnt[rows >> 16], 1);
            }
            if (a.cached) *reinterpret_cast<uint32_t*>(place + t + 64 * j) = rows;  // t is even
        }
    }
    for (int t = whole + lane; t < t1; t += 32) {
        const int64_t id = load_id(a.ids, a.id_bytes, t);
        const uint32_t p = remainder(id), r = row_of(p, id);
        less += p < own;
        if (r != kNone) atomicAdd(&cnt[r], 1);
        if (a.cached) place[t] = static_cast<uint16_t>(r);
    }
    if (bad) atomicOr(a.status, kErrId);
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
    // the last CTA's tokens are the last
    if (blockIdx.x + 1 == gridDim.x && tid == kSortThreads - 1) *a.total = before + inc;
    if (tid < nr) {
        int32_t at = before + inc - total;
        seen[tid] = total > 0;
        a.run[own + (static_cast<uint32_t>(tid) << a.shift)] = make_int2(at, at + total);
        // the counters become the first places of the id's tokens from each warp's stretch
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = sh[w * a.range + tid];
            sh[w * a.range + tid] = at;
            at += c;
        }
    }
    __syncthreads();
    // 64 tokens at a time, two a lane: most groups have none of the CTA's ids
    for (int t = t0; t < t1; t += 64 * kIdBatch) {
        uint32_t rows[kIdBatch];
#pragma unroll
        for (int j = 0; j < kIdBatch; ++j) {
            const int u = t + 64 * j + 2 * lane;
            rows[j] = 0xffffffffu;
            if (u >= t1) continue;
            if (a.cached) {
                rows[j] = *reinterpret_cast<const uint32_t*>(place + u);
                if (u + 1 >= t1) rows[j] |= 0xffff0000u;
            } else {
                const int64_t p = load_id(a.ids, a.id_bytes, u), q = u + 1 < t1 ? load_id(a.ids, a.id_bytes, u + 1) : -1;
                rows[j] = row_of(remainder(p), p) | (row_of(remainder(q), q) << 16);
            }
        }
#pragma unroll
        for (int j = 0; j < kIdBatch; ++j) {
            if (!__any_sync(0xffffffffu, rows[j] != 0xffffffffu)) continue;
            // the first 32 tokens of the group, then the others: lane i takes token i of the half
            for (int half = 0; half < 2; ++half) {
                const uint32_t pair = __shfl_sync(0xffffffffu, rows[j], half * 16 + (lane >> 1));
                const int r = static_cast<int>((lane & 1) ? pair >> 16 : pair & 0xffffu);
                const bool mine = r != kNone;
                const uint32_t any = __ballot_sync(0xffffffffu, mine);
                if (mine) {
                    const uint32_t same = __match_any_sync(any, r);
                    const int at = cnt[r] + __popc(same & ((1u << lane) - 1u));
                    a.order[at] = t + 64 * j + 32 * half + lane;
                    a.key[at] = static_cast<int32_t>(own + (static_cast<uint32_t>(r) << a.shift));
                    __syncwarp(same);
                    if (lane == __ffs(same) - 1) cnt[r] += __popc(same);
                }
                __syncwarp();
            }
        }
    }
    // the rows of the CTA's ids that do not occur: nothing to wait for
    if (a.clear) {
        for (int r = warp; r < nr; r += kSortWarps) {
            if (seen[r]) continue;
            uint8_t* row = a.clear + (own + (static_cast<int64_t>(r) << a.shift)) * a.clear_stride;
            const int64_t head = min(a.clear_bytes, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15));
            const int64_t body = head + (a.clear_bytes - head) / 16 * 16;
            if (lane * 2 < head) *reinterpret_cast<uint16_t*>(row + lane * 2) = 0;
            for (int64_t c = head + lane * 16; c < body; c += 512) *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
            if (body + lane * 2 < a.clear_bytes) *reinterpret_cast<uint16_t*>(row + body + lane * 2) = 0;
        }
    }
}

// Runs of equal ids are cut into chunks of the sorted order, so that a frequent word's
// run is summed by many warps.  A warp sums one chunk in one slab of columns; a CTA's
// eight warps take eight chunks in a row, a block.  A run inside a chunk goes to the
// table at once; a run's part that reaches over the chunk's edge stays in shared memory
// until the block's parts are added, and what reaches over the block's edge goes to the
// workspace: `head`, the part of a run that began before the block (chunk), and `tail`,
// the part of one that begins in it and goes on.
struct GradArgs {
    const void* g;
    int64_t gs;
    const int32_t* order;
    const int32_t* key;
    const int2* run;
    const int32_t* total;
    int64_t ntokens, dim;
    int32_t chunk;
    float* edge;  // [blocks][head, tail][dim]
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
    // A row's columns into a warp's slot of kSlotBytes; past the row's end, zeros.  VEC: an
    // asynchronous copy, complete after batch_done().
    static constexpr int kSlotBytes = 32 * N * static_cast<int>(sizeof(typename Elem<DT>::T));
    __device__ __forceinline__ static void fetch(uint8_t* slot, const void* g, int64_t row, int64_t dim, int64_t slab, int lane)
    {
        using T = typename Elem<DT>::T;
        const T* p = static_cast<const T*>(g) + row;
        if (VEC) {
            const bool in = at(slab, lane, 0) < dim;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             static_cast<uint32_t>(__cvta_generic_to_shared(slot + lane * 16))),
                         "l"(in ? p + at(slab, lane, 0) : p), "r"(in ? 16 : 0)
                         : "memory");
        } else {
            T v[N];
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = at(slab, lane, j) < dim ? p[at(slab, lane, j)] : Elem<DT>::from_f(0.f);
#pragma unroll
            for (int j = 0; j < N; ++j) reinterpret_cast<T*>(slot)[lane + 32 * j] = v[j];
        }
    }
    __device__ __forceinline__ static void batch_end()
    {
        if (VEC) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // all batches but the newest are there
    __device__ __forceinline__ static void batch_done()
    {
        if (VEC) asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
    }
    __device__ __forceinline__ static void add(const uint8_t* slot, int lane, float (&acc)[N])
    {
        using T = typename Elem<DT>::T;
        if (VEC) {
            const Vec<DT> v = *reinterpret_cast<const Vec<DT>*>(slot + lane * 16);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += Elem<DT>::to_f(v.v[VEC ? j : 0]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += Elem<DT>::to_f(reinterpret_cast<const T*>(slot)[lane + 32 * j]);
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

// Bound by HBM where there are many tokens, by four dependent reads where there are few.  A
// warp has 16 rows of 512 bytes on their way in shared memory, not in registers: unrolled
// over them the code outgrew the instruction cache (25 us where it now takes 9, at 8192
// tokens x 768 bf16).  65521 tokens x 1024 fp16, a third of them padding: 28 us, 115 MB.
constexpr int kSumWarps = 8;  // chunks of a block
constexpr int kRows = 8;      // rows of a batch; a warp has two on their way
template <int DT, bool VEC> constexpr int sum_smem() { return kSumWarps * 2 * kRows * Columns<DT, VEC>::kSlotBytes; }

template <int DT, int WT, bool VEC> __global__ void __launch_bounds__(32 * kSumWarps) chunk_kernel(GradArgs a)
{
    using C = Columns<DT, VEC>;
    extern __shared__ __align__(16) uint8_t slots[];
    __shared__ float edges[kSumWarps][2][C::N][32];  // head, tail
    __shared__ bool starts[kSumWarps], goes_on[kSumWarps], through[kSumWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t slabs = (a.dim + C::kSlab - 1) / C::kSlab;
    const int64_t block = blockIdx.x / slabs, slab = blockIdx.x - block * slabs;
    const int64_t c0 = (block * kSumWarps + warp) * a.chunk;
    uint8_t* mine = slots + warp * 2 * kRows * C::kSlotBytes;
    wait_for_previous();
    allow_next();
    // the chunk's tokens and ids, the id before it and the one after it, and how many tokens
    // there are, in one go (what lies past the last token is left over from before)
    const bool in = lane < a.chunk && c0 + lane < a.ntokens;
    int32_t tok = in ? a.order[c0 + lane] : 0, key = in ? a.key[c0 + lane] : -1;
    int32_t prior = c0 > 0 && c0 < a.ntokens ? a.key[c0 - 1] : -1, after = c0 + a.chunk < a.ntokens ? a.key[c0 + a.chunk] : -1;
    const int64_t n = *a.total;
    const int count = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(a.chunk), n - c0)));
    if (lane >= count) tok = 0, key = -1;
    if (c0 + a.chunk >= n) after = -1;
    float acc[C::N];
#pragma unroll
    for (int k = 0; k < C::N; ++k) acc[k] = 0.f;
    int32_t now = __shfl_sync(0xffffffffu, key, 0);
    const bool began_before = count > 0 && prior == now;
    bool first = true;
    // two buffers of kRows rows: one is on its way while the other is summed
    auto fetch = [&](int i) {
        uint8_t* to = mine + (i / kRows & 1) * kRows * C::kSlotBytes;
        const int rows = min(kRows, count - i);
#pragma unroll 4
        for (int j = 0; j < rows; ++j)
            C::fetch(to + j * C::kSlotBytes, a.g, static_cast<int64_t>(__shfl_sync(0xffffffffu, tok, i + j)) * a.gs, a.dim, slab, lane);
        C::batch_end();
    };
    fetch(0);
    for (int i = 0; i < count; i += kRows) {
        const int rows = min(kRows, count - i);
        const uint8_t* from = mine + (i / kRows & 1) * kRows * C::kSlotBytes;
        fetch(i + kRows);
        C::batch_done();
#pragma unroll 1
        for (int j = 0; j < rows; ++j) {
            const bool at_end = i + j + 1 == count;
            const int32_t in_chunk = __shfl_sync(0xffffffffu, key, (i + j + 1) & 31);
            const int32_t next = at_end ? after : in_chunk;
            C::add(from + j * C::kSlotBytes, lane, acc);
            if (next == now && !at_end) continue;
            const bool head = first && began_before;
            if (head || next == now) {
#pragma unroll
                for (int k = 0; k < C::N; ++k) edges[warp][head ? 0 : 1][k][lane] = acc[k];
                if (at_end && lane == 0) through[warp] = head && next == now;
            } else {
                C::template store<WT>(a, now, slab, lane, acc);
                if (at_end && lane == 0) through[warp] = false;
            }
            if (at_end && lane == 0) goes_on[warp] = next == now;
#pragma unroll
            for (int k = 0; k < C::N; ++k) acc[k] = 0.f;
            first = false;
            now = next;
        }
        __syncwarp();
    }
    if (lane == 0) {
        starts[warp] = began_before;
        if (count == 0) goes_on[warp] = through[warp] = false;
    }
    __syncthreads();
    // The parts of runs over the chunks' edges: the run that came into the block by warp 0,
    // the one that begins in a warp's chunk and goes on by that warp.
    for (int side = warp == 0 ? 0 : 1; side < 2; ++side) {
        if (side == 0 ? !starts[0] : !(goes_on[warp] && !through[warp])) continue;
#pragma unroll
        for (int k = 0; k < C::N; ++k) acc[k] = edges[warp][side][k][lane];
        bool open = side == 0 ? through[0] : true;
        int u = warp + 1;
        for (; open && u < kSumWarps; ++u) {
#pragma unroll
            for (int k = 0; k < C::N; ++k) acc[k] += edges[u][0][k][lane];
            open = through[u];
        }
        if (side == 0 || open) {
            C::store_edge(a.edge + (block * 2 + side) * a.dim, a.dim, slab, lane, acc);
        } else {
            C::template store<WT>(a, a.key[c0 + a.chunk - 1], slab, lane, acc);
        }
    }
}

// Runs that reach over blocks' edges: the tail where a run begins, then the heads of the
// blocks that it goes on in.  A warp sums one run in one slab of columns.
constexpr int kJoinWarps = 4;
template <int DT, int WT, bool VEC> __global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(GradArgs a, int64_t blocks)
{
    using C = Columns<DT, VEC>;
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
    const int64_t slab = unit / blocks, block = unit - slab * blocks;
    const int64_t span = static_cast<int64_t>(a.chunk) * kSumWarps, end = (block + 1) * span;
    wait_for_previous();
    if (slab * C::kSlab >= a.dim || end >= *a.total) return;
    const int32_t v = a.key[end - 1];
    const int64_t s0 = a.run[v].x, s1 = a.run[v].y;
    if (s1 <= end || s0 < end - span) return;  // it ends here, or began before this block
    const int parts = static_cast<int>((s1 - 1) / span - block + 1);
    const float* edge = a.edge + block * 2 * a.dim;
    float acc[C::N];
    C::load_edge(edge + a.dim, a.dim, slab, lane, acc);
    for (int p = 1; p < parts; p += 4) {
        float x[4][C::N];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (p + j < parts) C::load_edge(edge + (p + j) * 2 * a.dim, a.dim, slab, lane, x[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (p + j < parts)
#pragma unroll
                for (int k = 0; k < C::N; ++k) acc[k] += x[j][k];
    }
    C::template store<WT>(a, v, slab, lane, acc);
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Tokens a warp sums: short chunks spread few tokens over the SMs, longer ones have fewer edges.
int32_t chunk_for(int64_t ntokens) { return ntokens <= 16384 ? 16 : 32; }

struct EmbeddingSpace {
    int64_t order, key, run, count, edge, total;  // byte offsets
};
EmbeddingSpace space_for(int64_t ntokens, int64_t vocab, int64_t dim)
{
    EmbeddingSpace e{};
    const int64_t chunk = chunk_for(ntokens);
    e.order = 0;
    e.key = e.order + round_up(4 * ntokens, 256);
    e.run = e.key + round_up(4 * ntokens, 256);
    e.count = e.run + round_up(8 * vocab, 256);
    e.edge = e.count + 256;
    const int64_t span = chunk * kSumWarps;
    e.total = e.edge + round_up((ntokens + span - 1) / span * 8 * dim, 256);
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
    if (dim < 1 || dim >= (int64_t{1} << 28)) return fail(DDP_E_INVAL, "%s: dim = %lld outside [1, 2^28)", fn, static_cast<long long>(dim));
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
    const int64_t span = static_cast<int64_t>(g.chunk) * kSumWarps, blocks = (ntokens + span - 1) / span;
    constexpr int smem = sum_smem<DT, VEC>();
    static std::atomic<bool> ready[ddp::kMaxDevices] = {};
    const int dev = ddp::current_device();
    cudaError_t e;
    if (dev < 0 || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(chunk_kernel<DT, WT, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0) ready[dev].store(true, std::memory_order_relaxed);
    }
    e = launch_chained(chunk_kernel<DT, WT, VEC>, dim3(static_cast<unsigned>(blocks * slabs)), 32 * kSumWarps, smem, s, g);
    if (e != cudaSuccess || blocks == 1) return e;
    return launch_chained(join_kernel<DT, WT, VEC>, dim3(static_cast<unsigned>((blocks * slabs + kJoinWarps - 1) / kJoinWarps)),
                          32 * kJoinWarps, 0, s, g, blocks);
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
    if (ntokens < 0 || ntokens >= kMaxSortTokens || vocab < 1 || vocab >= (int64_t{1} << 31) || dim < 1 || dim >= (int64_t{1} << 28))
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
    if (ntokens >= kMaxSortTokens) return fail(DDP_E_INVAL, "%s: ntokens = %lld is 2^31 - 4096 or more", fn, static_cast<long long>(ntokens));
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
    a.run = reinterpret_cast<int2*>(w + sp.run);
    a.total = reinterpret_cast<int32_t*>(w + sp.count);
    a.status = status;
    if (!accumulate) {
        a.clear = static_cast<uint8_t*>(grad_weight);
        a.clear_stride = gw_stride * es;
        a.clear_bytes = dim * es;
    }
    int64_t ctas = kMinSortCtas;
    while ((vocab + ctas - 1) / ctas > kMaxRange) ctas *= 2;
    while ((int64_t{1} << a.shift) < ctas) ++a.shift;
    a.range = static_cast<int32_t>((vocab + ctas - 1) / ctas);
    static std::atomic<bool> ready[ddp::kMaxDevices] = {};
    const int dev = ddp::current_device();
    cudaError_t err = cudaSuccess;
    if (dev < 0 || !ready[dev].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
        if (err != cudaSuccess) return fail(DDP_E_CUDA, "%s: shared memory: %s", fn, cudaGetErrorString(err));
        if (dev >= 0) ready[dev].store(true, std::memory_order_relaxed);
    }
    const int64_t counters = kSortWarps * a.range * 4;
    a.cached = counters + 2 * ntokens + 4 <= kSortSmem;
    err = launch_chained(sort_kernel, dim3(static_cast<unsigned>(ctas)), kSortThreads,
                         static_cast<int>(counters + (a.cached ? 2 * ntokens + 4 : 0)), s, a);
    if (err == cudaSuccess && ntokens > 0) {
        const GradArgs g{grad_out, grad_stride, a.order, a.key, a.run, a.total, ntokens, dim, chunk_for(ntokens),
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
