// Softmax cross entropy of hidden states against a vocabulary projection, and its
// gradients, without storing the logits.
//
//   z = H W^T          lse[t] = log sum_v exp z[t][v]          loss[t] = lse[t] - z[t][y_t]
//   G[t][v] = dl[t] (exp(z[t][v] - lse[t]) - [v = y_t])        dH = G W        dW = G^T H
//
// Forward: each tile of z is reduced to one maximum and one sum of exponentials a
// row before it is dropped; a second kernel joins the tiles' pairs.  Backward: z is
// computed again, one piece of the vocabulary at a time, and G of that piece is
// written in 16 bits for the two gradient products.
//
// Tokens without a target are left out first: the hidden states of the others are
// gathered into consecutive rows, so masked-word training pays for the masked
// words only and nothing an ignored row holds can reach a result.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "lm_common.cuh"
#include "umma.cuh"

namespace ddplm {
namespace {

constexpr int kRowTile = 256;   // rows of the gathered arrays are padded to this
constexpr int kPrepThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// G's scale in fp16: its largest magnitude, 1 after the division by the largest
// |grad_loss|, is moved to 2^14, so that probabilities down to 2^-28 stay normal
// numbers.  bf16 has fp32's exponents and needs none.
template <int DT> constexpr float g_scale() { return DT == DDP_F16 ? 16384.f : 1.f; }

struct Space {
    int64_t count, gmax, rows, target, ratio, lse, hidden, part, ztarget, grad, acc, weight, total;
    int64_t piece, ntiles, tpad, dpad;
};

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

Space space_for(bool backward, int64_t T, int64_t V, int64_t D, int64_t piece, bool copy_weight)
{
    Space s{};
    s.tpad = round_up(std::max<int64_t>(T, 1), kRowTile);
    s.dpad = round_up(D, 8);
    s.ntiles = (V + 127) / 128;  // one pair of statistics a row for each 128 words
    const int64_t vpad = round_up(V, 256);
    if (piece <= 0) piece = std::max<int64_t>(1024, (int64_t{1} << 27) / s.tpad);
    s.piece = std::min(vpad, round_up(piece, 256));
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t p = at;
        at += round_up(bytes, 256);
        return p;
    };
    s.count = take(4);
    s.gmax = take(4);
    s.rows = take(4 * s.tpad);
    s.target = take(4 * s.tpad);
    s.hidden = take(2 * s.tpad * s.dpad);
    if (backward) {
        s.ratio = take(4 * s.tpad);
        s.lse = take(4 * s.tpad);
        s.grad = take(2 * s.tpad * s.piece);
        s.acc = take(s.piece < vpad ? 4 * s.tpad * s.dpad : 0);
    } else {
        s.part = take(8 * s.tpad * s.ntiles);
        s.ztarget = take(4 * s.tpad);
    }
    if (copy_weight) s.weight = take(2 * V * s.dpad);
    s.total = at;
    return s;
}

// ---------------------------------------------------------------------------
// gather: tokens that have a target, in consecutive rows
// ---------------------------------------------------------------------------
struct PrepArgs {
    const void* hidden;
    int64_t hs;
    const void* targets;
    int32_t id_bytes;
    int64_t ignore;
    int32_t T;
    int64_t vocab, dim, dpad;
    int32_t slab;         // tokens a CTA gathers
    int32_t* count;
    int32_t* rows;        // gathered row -> token
    int32_t* target;      // gathered row -> target
    uint16_t* out;        // [tpad][dpad]
    int* status;
    // forward: results of tokens without a target
    float* loss;
    float* lse_out;
    // backward
    const float* lse_in;
    const float* gl;
    int32_t gl_stride;
    float* lse;           // gathered
    float* ratio;         // gathered: grad_loss / gmax * g_scale
    float* gmax;          // largest finite |grad_loss| of the gathered rows (1 if that is 0)
    uint16_t* gh;         // rows to clear
    int64_t ghs;
    float g_scale;
};

__device__ __forceinline__ bool token_target(const PrepArgs& a, int t, int64_t* y)
{
    *y = load_id(a.targets, a.id_bytes, t);
    if (*y == a.ignore) return false;
    if (*y < 0 || *y >= a.vocab) {
        atomicOr(a.status, kErrId);
        return false;
    }
    return true;
}

__device__ __forceinline__ int block_sum(int v, int* sh)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    int r = 0;
    for (int w = 0; w < kPrepThreads / 32; ++w) r += sh[w];
    __syncthreads();
    return r;
}

// Every CTA counts the tokens with a target before its own slab, and all of them, itself.
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(PrepArgs a)
{
    __shared__ int sh[kPrepThreads / 32];
    __shared__ float shf[kPrepThreads / 32];
    __shared__ int place[kPrepThreads];  // of the slab's tokens: gathered row or -1
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * a.slab, t1 = min(a.T, t0 + a.slab);
    int before = 0, all = 0;
    float gm = 0.f;
    for (int t = tid; t < a.T; t += kPrepThreads) {
        int64_t y;
        if (!token_target(a, t, &y)) continue;
        ++all;
        before += t < t0;
        if (a.gl) {
            const float g = fabsf(a.gl[static_cast<int64_t>(t) * a.gl_stride]);
            if (g > gm && g <= 3.4028234663852886e38f) gm = g;
        }
    }
    before = block_sum(before, sh);
    all = block_sum(all, sh);
    for (int o = 16; o; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
    if (lane == 0) shf[warp] = gm;
    __syncthreads();
    for (int w = 0; w < kPrepThreads / 32; ++w) gm = fmaxf(gm, shf[w]);
    if (gm == 0.f) gm = 1.f;
    if (blockIdx.x == 0 && tid == 0) {
        *a.count = all;
        if (a.gmax) *a.gmax = gm;
    }
    // places of the slab's tokens (slab <= kPrepThreads), in token order
    {
        const int t = t0 + tid;
        int64_t y = 0;
        const bool has = t < t1 && token_target(a, t, &y);
        const uint32_t m = __ballot_sync(0xffffffffu, has);
        if (lane == 0) sh[warp] = __popc(m);
        __syncthreads();
        int at = before + __popc(m & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) at += sh[w];
        place[tid] = has ? at : -1;
        if (has) {
            a.rows[at] = t;
            a.target[at] = static_cast<int32_t>(y);
            if (a.gl) {
                a.lse[at] = a.lse_in[t];
                a.ratio[at] = a.gl[static_cast<int64_t>(t) * a.gl_stride] / gm * a.g_scale;
            }
        } else if (t < t1 && a.loss) {
            a.loss[t] = 0.f;
            a.lse_out[t] = 0.f;
        }
    }
    __syncthreads();
    for (int i = warp; i < t1 - t0; i += kPrepThreads / 32) {
        const int at = place[i];
        const uint16_t* src = static_cast<const uint16_t*>(a.hidden) + static_cast<int64_t>(t0 + i) * a.hs;
        if (at >= 0) {
            uint16_t* dst = a.out + static_cast<int64_t>(at) * a.dpad;
            for (int64_t c = lane; c < a.dpad; c += 32) dst[c] = c < a.dim ? src[c] : 0;
        } else if (a.gh) {
            uint16_t* dst = a.gh + static_cast<int64_t>(t0 + i) * a.ghs;
            for (int64_t c = lane; c < a.dim; c += 32) dst[c] = 0;
        }
    }
    // rows up to the tile's end are zeros (past the T-th the copies supply them): they are terms of dW's sums
    const int end = min(a.T, (all + kRowTile - 1) / kRowTile * kRowTile);
    for (int r = all + blockIdx.x; r < end; r += gridDim.x)
        for (int64_t c = tid; c < a.dpad; c += kPrepThreads) a.out[static_cast<int64_t>(r) * a.dpad + c] = 0;
}

__global__ void __launch_bounds__(256)
copy_weight_kernel(const uint16_t* w, int64_t ws, int64_t vocab, int64_t dim, uint16_t* out, int64_t dpad)
{
    for (int64_t v = blockIdx.x; v < vocab; v += gridDim.x)
        for (int64_t c = threadIdx.x; c < dpad; c += blockDim.x) out[v * dpad + c] = c < dim ? w[v * ws + c] : 0;
}

// ---------------------------------------------------------------------------
// products: C[m][n] = sum_k A[m][k] B[n][k], and what is done with C
// ---------------------------------------------------------------------------
// Two CTAs on a pair of SMs share one 256 x 256 tile of C: each holds 128 rows of
// A and 128 of B in shared memory and 128 rows of C in tensor memory, and one
// thread of the first CTA issues the products of both.  Per CTA:
//   warp 8     copies 128 x 64 boxes of A and B into a ring of stages;
//   warp 9     (first CTA) issues four k = 16 products a stage;
//   warps 0-7  take finished tiles out of tensor memory, which holds two, so that
//              a tile's epilogue runs under the next tile's products.
// The grid is one pair of CTAs for each pair of SMs; a pair takes every npairs-th tile.
enum Use { USE_STATS, USE_GRAD, USE_DH, USE_DW };

constexpr int kTile = 256;               // rows and columns of a pair's tile
constexpr int kHalf = 128;               // rows of A, of B and of C that one CTA holds
constexpr int kBlockK = 64;              // one 128-byte row of 16-bit values
constexpr int kStages = 6;
constexpr int kOperandBytes = kHalf * kBlockK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpiWarps = 8;
constexpr int kStagingBytes = 4096;      // per epilogue warp: 32 rows of 128 bytes
constexpr int kProductThreads = 32 * (kEpiWarps + 2);
constexpr int kProductSmem = kStages * kStageBytes + kEpiWarps * kStagingBytes + 1024;

struct Product {
    CUtensorMap ta, tb;
    int64_t M, N, K;
    const int32_t* count; // gathered rows: bounds M (STATS, GRAD, DH) or K (DW)
    int64_t rows_cap;     // rows of the gathered arrays that exist
    int64_t v0;           // first word of the piece
    const int32_t* target;
    int* status;
    // STATS
    float2* part;
    int64_t tpad;
    float* ztarget;
    // GRAD
    const float* lse;
    const float* ratio;
    void* g;
    int64_t gld;
    // DH, DW
    const float* gmax;
    float inv_scale;
    float* acc;           // fp32 sums over the pieces (nullptr: one piece)
    int32_t first, last;
    const int32_t* rows;
    void* out;
    int64_t os;
    int32_t out_f32, accumulate, vec;
};

template <int USE> struct Majors {
    static constexpr bool a_mn = USE == USE_DW;
    static constexpr bool b_mn = USE == USE_DH || USE == USE_DW;
};

// one CTA's 128 rows of an operand, 64 of k: one box, or two where m (n) is contiguous
template <bool MN>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, int row, int k, uint32_t bar)
{
    if (MN) {
        tensor_load(dst, map, row, k, bar);
        tensor_load(dst + kOperandBytes / 2, map, row + 64, k, bar);
    } else {
        tensor_load(dst, map, k, row, bar);
    }
}
// descriptor of k = 16 values at step j of a stage
template <bool MN> __device__ __forceinline__ uint64_t step_desc(uint32_t base, int j)
{
    return MN ? operand_desc(base + j * 2048, kOperandBytes / 2, 1024) : operand_desc(base + j * 32, 16, 1024);
}

__device__ __forceinline__ void tile_values(uint32_t taddr, bool empty, float (&c)[32])
{
    uint32_t v[32];
    if (empty) {
#pragma unroll
        for (int j = 0; j < 32; ++j) c[j] = 0.f;
        return;
    }
    tmem_load32(taddr, v);
#pragma unroll
    for (int j = 0; j < 32; ++j) c[j] = __uint_as_float(v[j]);
}

// 16-byte chunk `ch` (of 8) of row r in a warp's staging area, spread over the banks
__device__ __forceinline__ uint32_t staged(uint32_t base, int r, int ch) { return base + r * 128 + ((ch ^ (r & 7)) << 4); }
__device__ __forceinline__ void sts16(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

template <int DT> __device__ __forceinline__ uint32_t pack2(float a, float b)
{
    typename Elem<DT>::T x[2] = {Elem<DT>::from_f(a), Elem<DT>::from_f(b)};
    return *reinterpret_cast<uint32_t*>(x);
}

template <int DT, int USE>
__device__ __forceinline__ void epilogue(const Product& p, uint32_t taddr, bool empty, int64_t m0, int64_t n0, int64_t M,
                                         uint32_t staging, int half, int lane)
{
    using T = typename Elem<DT>::T;
    const int64_t m = m0 + lane;  // this thread's row; n0: the warp's first of 128 columns
    float c[32];
    if (USE == USE_STATS) {
        float mx = -INFINITY, s = 0.f;
        const bool in = m < M;
        const int64_t y = in ? p.target[m] : -1;
        for (int q = 0; q < 4; ++q) {
            tile_values(taddr + q * 32, empty, c);
            const int64_t n = n0 + q * 32;
            if (n >= p.N) break;
            if (n + 32 > p.N) {
#pragma unroll
                for (int j = 0; j < 32; ++j) c[j] = n + j < p.N ? c[j] : -INFINITY;
            }
            if (y >= n && y < n + 32) {
                float z = 0.f;
#pragma unroll
                for (int j = 0; j < 32; ++j) z = y - n == j ? c[j] : z;
                p.ztarget[m] = z;
            }
            float cm = c[0];
#pragma unroll
            for (int j = 1; j < 32; ++j) cm = fmaxf(cm, c[j]);
            const float top = fmaxf(mx, cm);
            if (top != -INFINITY) {  // all of them minus infinity: they add nothing
                const float shift = top * kLog2e;
                s *= mx == -INFINITY ? 0.f : exp2f(mx * kLog2e - shift);
                float a0 = 0.f, a1 = 0.f;
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    a0 += exp2f(fmaf(c[j], kLog2e, -shift));
                    a1 += exp2f(fmaf(c[j + 1], kLog2e, -shift));
                }
                s += a0 + a1;
                mx = top;
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) s += c[j] != c[j] ? c[j] : 0.f;  // a NaN among them stays
            }
        }
        if (in && n0 < p.N) p.part[(n0 >> 7) * p.tpad + m] = make_float2(mx, s);
    } else if (USE == USE_GRAD) {
        const bool in = m < M;
        const float shift = in ? p.lse[m] * kLog2e : 0.f;
        const float ratio = in ? p.ratio[m] : 0.f;
        const int64_t y = in ? p.target[m] - p.v0 : -1;
        for (int q = 0; q < 2; ++q) {
            for (int h = 0; h < 2; ++h) {
                const int64_t n = n0 + q * 64 + h * 32;
                tile_values(taddr + q * 64 + h * 32, empty, c);
#pragma unroll
                for (int j = 0; j < 32; ++j) c[j] = exp2f(fmaf(c[j], kLog2e, -shift));
                if (y >= n && y < n + 32) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) c[j] -= y - n == j ? 1.f : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) c[j] = ratio == 0.f ? 0.f : c[j] * ratio;
                if (n + 32 > p.N) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) c[j] = n + j < p.N ? c[j] : 0.f;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sts16(staged(staging, lane, h * 4 + k),
                          make_uint4(pack2<DT>(c[8 * k], c[8 * k + 1]), pack2<DT>(c[8 * k + 2], c[8 * k + 3]),
                                     pack2<DT>(c[8 * k + 4], c[8 * k + 5]), pack2<DT>(c[8 * k + 6], c[8 * k + 7])));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3), ch = lane & 7;
                if (m0 + r < p.rows_cap)
                    *reinterpret_cast<uint4*>(static_cast<T*>(p.g) + (m0 + r) * p.gld + n0 + q * 64 + ch * 8) =
                        lds16(staged(staging, r, ch));
            }
            __syncwarp();
        }
    } else {
        const float alpha = *p.gmax * p.inv_scale;
        for (int q = 0; q < 4; ++q) {
            tile_values(taddr + q * 32, empty, c);
            if (n0 + q * 32 >= p.N) break;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sts16(staged(staging, lane, k), make_uint4(__float_as_uint(c[4 * k]), __float_as_uint(c[4 * k + 1]),
                                                           __float_as_uint(c[4 * k + 2]), __float_as_uint(c[4 * k + 3])));
            __syncwarp();
            const int64_t n = n0 + q * 32 + (lane & 7) * 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3);
                const uint4 raw = lds16(staged(staging, r, lane & 7));
                float x[4] = {__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z), __uint_as_float(raw.w)};
                const int64_t row = m0 + r;
                if (row >= M || n >= p.N) continue;
                const int width = static_cast<int>(min(static_cast<int64_t>(4), p.N - n));
                if (USE == USE_DH && p.acc) {
                    float* a = p.acc + row * p.tpad + n;  // tpad: the sums' row stride, a multiple of 4
                    if (!p.first) {
                        const float4 o = *reinterpret_cast<const float4*>(a);
                        x[0] += o.x; x[1] += o.y; x[2] += o.z; x[3] += o.w;
                    }
                    if (!p.last) {
                        *reinterpret_cast<float4*>(a) = make_float4(x[0], x[1], x[2], x[3]);
                        continue;
                    }
                }
                const int64_t at = (USE == USE_DH ? p.rows[row] : p.v0 + row) * p.os + n;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] *= alpha;
                if (USE == USE_DW && p.out_f32) {
                    float* o = static_cast<float*>(p.out) + at;
                    if (p.vec && width == 4) {
                        if (p.accumulate) {
                            const float4 v = *reinterpret_cast<const float4*>(o);
                            x[0] += v.x; x[1] += v.y; x[2] += v.z; x[3] += v.w;
                        }
                        *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
                    } else {
                        for (int j = 0; j < width; ++j) o[j] = x[j] + (p.accumulate ? o[j] : 0.f);
                    }
                } else {
                    T* o = static_cast<T*>(p.out) + at;
                    if (p.vec && width == 4) {
                        if (USE == USE_DW && p.accumulate) {
                            const uint2 v = *reinterpret_cast<const uint2*>(o);
                            const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[j] += Elem<DT>::to_f(t[j]);
                        }
                        *reinterpret_cast<uint2*>(o) = make_uint2(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]));
                    } else {
                        for (int j = 0; j < width; ++j)
                            o[j] = Elem<DT>::from_f(x[j] + (USE == USE_DW && p.accumulate ? Elem<DT>::to_f(o[j]) : 0.f));
                    }
                }
            }
            __syncwarp();
        }
    }
}

template <int DT, int USE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1) product_kernel(const __grid_constant__ Product p)
{
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
    __shared__ uint32_t tmem_base;
    __shared__ volatile int dead;
    const uint32_t base = (smem_addr(dyn) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_addr(bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto tfull = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
    auto tempty = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };

    if (threadIdx.x == 0) {
        dead = 0;
        for (int s = 0; s < kStages; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(tfull(b), 1);
            bar_init(tempty(b), 2 * kEpiWarps);
        }
        bar_init_fence();
        tensor_map_prefetch(&p.ta);
        tensor_map_prefetch(&p.tb);
    }
    if (warp == 9) tmem_alloc(smem_addr(&tmem_base), 512);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = tmem_base;

    const int64_t count = *p.count;
    const int64_t M = USE == USE_DW ? p.M : min(p.M, count);
    const int64_t K = USE == USE_DW ? min(p.K, count) : p.K;
    const int mt = static_cast<int>((M + kTile - 1) / kTile), nt = static_cast<int>((p.N + kTile - 1) / kTile);
    const int nkb = static_cast<int>((K + kBlockK - 1) / kBlockK);
    const int64_t tiles = static_cast<int64_t>(mt) * nt;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (warp == 8) {
        if (lane == 0 && nkb > 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int64_t t = pair; ok && t < tiles; t += npairs) {
                const int m = static_cast<int>(t % mt) * kTile + static_cast<int>(rank) * kHalf;
                const int n = static_cast<int>(t / mt) * kTile + static_cast<int>(rank) * kHalf;
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!(ok = bar_wait(empty(s), ((it / kStages) & 1) ^ 1, &dead))) break;
                    // both CTAs' bytes are counted on the first CTA's barrier
                    if (rank == 0) bar_expect(full(s), 2 * kStageBytes);
                    const uint32_t bar = cluster_addr(full(s), 0);
                    const uint32_t a = base + s * kStageBytes;
                    load_operand<Majors<USE>::a_mn>(a, &p.ta, m, kb * kBlockK, bar);
                    load_operand<Majors<USE>::b_mn>(a + kOperandBytes, &p.tb, n, kb * kBlockK, bar);
                }
            }
            // the last arrivals on this CTA's barriers come before it may leave
            for (int i = 0; ok && i < kStages; ++i, ++it) ok = bar_wait(empty(it % kStages), ((it / kStages) & 1) ^ 1, &dead);
        }
    } else if (warp == 9) {
        if (rank == 0 && lane == 0 && nkb > 0) {
            constexpr uint32_t desc = product_desc(DT == DDP_BF16, Majors<USE>::a_mn, Majors<USE>::b_mn, kTile, kTile);
            uint32_t it = 0, j = 0;
            bool ok = true;
            for (int64_t t = pair; ok && t < tiles; t += npairs, ++j) {
                const int b = j & 1;
                if (!(ok = bar_wait(tempty(b), ((j >> 1) & 1) ^ 1, &dead))) break;
                tmem_fence_after();
                const uint32_t d = tmem + b * kTile;
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!(ok = bar_wait(full(s), (it / kStages) & 1, &dead))) break;
                    tmem_fence_after();
                    const uint32_t a = base + s * kStageBytes;
#pragma unroll
                    for (int k = 0; k < kBlockK / 16; ++k)
                        product_pair(d, step_desc<Majors<USE>::a_mn>(a, k), step_desc<Majors<USE>::b_mn>(a + kOperandBytes, k),
                                     desc, kb > 0 || k > 0);
                    product_commit(empty(s));
                }
                if (ok) product_commit(tfull(b));
            }
        }
    } else {
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t staging = base + kStages * kStageBytes + warp * kStagingBytes;
        uint32_t j = 0;
        for (int64_t t = pair; t < tiles; t += npairs, ++j) {
            const int b = j & 1;
            if (nkb > 0) {
                if (!__all_sync(0xffffffffu, bar_wait(tfull(b), (j >> 1) & 1, &dead))) break;
                tmem_fence_after();
            }
            const int64_t m0 = (t % mt) * kTile + rank * kHalf + quarter * 32;
            const int64_t n0 = (t / mt) * kTile + half * kHalf;
            __syncwarp();
            epilogue<DT, USE>(p, tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * kTile + half * kHalf, nkb == 0, m0,
                              n0, M, staging, half, lane);
            tmem_fence_before();
            __syncwarp();
            if (lane == 0 && nkb > 0) bar_arrive_cluster(cluster_addr(tempty(b), 0));
        }
    }
    __syncthreads();
    if (dead) {
        // a wait gave up: report it, and let copies and products in flight end before the memory is given back
        if (threadIdx.x == 0) {
            atomicOr(p.status, kErrWait);
            const uint64_t t0 = clock_ns();
            for (uint32_t i = 0; i < (1u << 24) && clock_ns() - t0 < 20000000ull; ++i) {}
        }
        __syncthreads();
    }
    tmem_fence_before();
    cluster_sync();
    tmem_fence_after();
    if (warp == 9) tmem_free(tmem, 512);
}

// A matrix of 16-bit values, `inner` contiguous values a row, cut in boxes of 64 values by `box_rows` rows.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static std::atomic<void*> cached{nullptr};
    void* f = cached.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        cached.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeFn>(f);
}

bool make_map(CUtensorMap* map, int dtype, const void* ptr, int64_t inner, int64_t rows, int64_t stride, int box_rows)
{
    const EncodeFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {kBlockK, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t unit[2] = {1, 1};
    return f(map, dtype == DDP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
             const_cast<void*>(ptr), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the operands' maps: A is [M x K] and B [N x K] seen as stored, `*_stride` between stored rows
template <int DT, int USE>
cudaError_t launch_product(Product& p, const void* a, int64_t a_stride, const void* b, int64_t b_stride, cudaStream_t s)
{
    static std::atomic<int> cached[ddp::kMaxDevices] = {};
    if (Majors<USE>::a_mn ? !make_map(&p.ta, DT, a, p.M, p.K, a_stride, kBlockK) : !make_map(&p.ta, DT, a, p.K, p.M, a_stride, kHalf))
        return cudaErrorInvalidValue;
    if (Majors<USE>::b_mn ? !make_map(&p.tb, DT, b, p.N, p.K, b_stride, kBlockK) : !make_map(&p.tb, DT, b, p.K, p.N, b_stride, kHalf))
        return cudaErrorInvalidValue;
    const int dev = ddp::current_device();
    int pairs = dev >= 0 ? cached[dev].load(std::memory_order_relaxed) : 0;
    if (!pairs) {
        cudaError_t e = cudaFuncSetAttribute(product_kernel<DT, USE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kProductSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kProductThreads);
        cfg.dynamicSmemBytes = kProductSmem;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 2;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&pairs, product_kernel<DT, USE>, &cfg);
        if (e != cudaSuccess) return e;
        pairs = std::max(1, std::min(pairs, ddp::device_sm_count() / 2));
        if (dev >= 0) cached[dev].store(pairs, std::memory_order_relaxed);
    }
    const int64_t tiles = ((p.M + kTile - 1) / kTile) * ((p.N + kTile - 1) / kTile);
    const int grid = 2 * static_cast<int>(std::min<int64_t>(tiles, pairs));
    product_kernel<DT, USE><<<grid, kProductThreads, kProductSmem, s>>>(p);
    return cudaGetLastError();
}

// joins the (maximum, sum) pairs of each gathered row: 32 threads a row, in a fixed order
constexpr int kJoinRows = 8;
__device__ __forceinline__ float2 join_pairs(float2 a, float2 b)
{
    const float m = fmaxf(a.x, b.x);
    // a side whose words are all minus infinity brings 0 (or a NaN, which stays)
    const float sa = a.x == -INFINITY ? a.y : a.y * exp2f((a.x - m) * kLog2e);
    const float sb = b.x == -INFINITY ? b.y : b.y * exp2f((b.x - m) * kLog2e);
    return make_float2(m, sa + sb);
}
// The target's logit is computed again with fp32 multiply-adds: the tensor cores cut
// off low bits at each step of k, and a loss is a small difference of two logits.
// Both places it enters by take the better value: loss = lse - z_y, and lse itself,
// moved by p_y (z_y - what the tile had).
template <int DT>
__global__ void __launch_bounds__(32 * kJoinRows)
combine_kernel(const int32_t* count, const int32_t* rows, const float2* part, int64_t tpad, int ntiles,
               const float* ztarget, const void* hidden, int64_t dpad, const void* weight, int64_t ws, int64_t dim,
               const int32_t* target, float* loss, float* lse)
{
    using T = typename Elem<DT>::T;
    __shared__ float2 sh[32][kJoinRows];
    __shared__ float dot[32][kJoinRows];
    const int r = threadIdx.x % kJoinRows, g = threadIdx.x / kJoinRows;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * kJoinRows + r;
    const bool in = m < *count;
    float2 q = make_float2(-INFINITY, 0.f);
    float d = 0.f;
    if (in) {
        const T* h = static_cast<const T*>(hidden) + m * dpad;
        const T* w = static_cast<const T*>(weight) + target[m] * ws;
        const int64_t whole = dim / 8 * 8;
#pragma unroll 4
        for (int64_t c = g * 8; c < whole; c += 256) {
            const Vec<DT> x = *reinterpret_cast<const Vec<DT>*>(h + c), y = *reinterpret_cast<const Vec<DT>*>(w + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) d = fmaf(Elem<DT>::to_f(x.v[j]), Elem<DT>::to_f(y.v[j]), d);
        }
        if (whole + g < dim) d = fmaf(Elem<DT>::to_f(h[whole + g]), Elem<DT>::to_f(w[whole + g]), d);
#pragma unroll 4
        for (int j = g; j < ntiles; j += 32) q = join_pairs(q, part[j * tpad + m]);
    }
    sh[g][r] = q;
    dot[g][r] = d;
    for (int o = 16; o; o >>= 1) {
        __syncthreads();
        if (g < o) {
            sh[g][r] = join_pairs(sh[g][r], sh[g + o][r]);
            dot[g][r] += dot[g + o][r];
        }
    }
    if (g == 0 && in) {
        float l = sh[0][r].x + logf(sh[0][r].y), z = ztarget[m];
        const float delta = dot[0][r] - z;
        if (fabsf(delta) < 1.f) {  // not where a logit is infinite or NaN
            l += exp2f((z - l) * kLog2e) * delta;
            z = dot[0][r];
        }
        lse[rows[m]] = l;
        loss[rows[m]] = l - z;
    }
}

struct Call {
    const void* hidden;
    int64_t hs;
    const void* weight;
    int64_t ws;
    int32_t dtype;
    int64_t T, V, D;
    const void* targets;
    int32_t id_bytes;
    int64_t ignore;
};

ddp_status check(const char* fn, const Call& c, const void* workspace, int64_t workspace_bytes, int64_t need)
{
    using ddp::fail;
    if (c.T < 0) return fail(DDP_E_INVAL, "%s: ntokens = %lld < 0", fn, static_cast<long long>(c.T));
    if (c.T >= (int64_t{1} << 31) - 512) return fail(DDP_E_INVAL, "%s: ntokens = %lld is too large", fn, static_cast<long long>(c.T));
    if (c.V < 1 || c.V >= (int64_t{1} << 31) - 512) return fail(DDP_E_INVAL, "%s: vocab = %lld out of range", fn, static_cast<long long>(c.V));
    if (c.D < 1 || c.D >= (int64_t{1} << 24)) return fail(DDP_E_INVAL, "%s: dim = %lld out of range", fn, static_cast<long long>(c.D));
    if (c.dtype != DDP_BF16 && c.dtype != DDP_F16) return fail(DDP_E_INVAL, "%s: dtype %d is neither DDP_BF16 nor DDP_F16", fn, c.dtype);
    if (c.id_bytes != 4 && c.id_bytes != 8) return fail(DDP_E_INVAL, "%s: id_bytes = %d is neither 4 nor 8", fn, c.id_bytes);
    if (c.hs < c.D) return fail(DDP_E_INVAL, "%s: hidden's stride %lld < dim = %lld", fn, static_cast<long long>(c.hs), static_cast<long long>(c.D));
    if (c.ws < c.D) return fail(DDP_E_INVAL, "%s: weight's stride %lld < dim = %lld", fn, static_cast<long long>(c.ws), static_cast<long long>(c.D));
    if (!c.weight) return fail(DDP_E_INVAL, "%s: weight is NULL", fn);
    if (c.T > 0 && (!c.hidden || !c.targets)) return fail(DDP_E_INVAL, "%s: hidden or targets is NULL", fn);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need)
        return fail(DDP_E_INVAL, "%s: workspace of %lld bytes (16-byte aligned), needs %lld", fn,
                    static_cast<long long>(workspace ? workspace_bytes : 0), static_cast<long long>(need));
    return DDP_OK;
}

bool needs_copy(const Call& c) { return !aligned16(c.weight) || c.ws % 8 != 0; }

// gathers, and the weight's aligned copy where it needs one
void launch_prep(PrepArgs& a, const Call& c, const Space& sp, char* w, int* status, cudaStream_t s, const void** weight, int64_t* ws)
{
    a.hidden = c.hidden;
    a.hs = c.hs;
    a.targets = c.targets;
    a.id_bytes = c.id_bytes;
    a.ignore = c.ignore;
    a.T = static_cast<int32_t>(c.T);
    a.vocab = c.V;
    a.dim = c.D;
    a.dpad = sp.dpad;
    a.slab = static_cast<int32_t>(std::min<int64_t>(kPrepThreads, std::max<int64_t>(32, c.T / 1024)));
    a.count = reinterpret_cast<int32_t*>(w + sp.count);
    a.rows = reinterpret_cast<int32_t*>(w + sp.rows);
    a.target = reinterpret_cast<int32_t*>(w + sp.target);
    a.out = reinterpret_cast<uint16_t*>(w + sp.hidden);
    a.status = status;
    prep_kernel<<<static_cast<unsigned>((c.T + a.slab - 1) / a.slab), kPrepThreads, 0, s>>>(a);
    *weight = c.weight;
    *ws = c.ws;
    if (needs_copy(c)) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(w + sp.weight);
        copy_weight_kernel<<<static_cast<unsigned>(std::min<int64_t>(c.V, 1 << 20)), 256, 0, s>>>(
            static_cast<const uint16_t*>(c.weight), c.ws, c.V, c.D, dst, sp.dpad);
        *weight = dst;
        *ws = sp.dpad;
    }
}

template <int DT> cudaError_t run_forward(const Call& c, const Space& sp, char* w, int* status, float* loss, float* lse, cudaStream_t s)
{
    PrepArgs a{};
    a.loss = loss;
    a.lse_out = lse;
    const void* weight;
    int64_t ws;
    launch_prep(a, c, sp, w, status, s, &weight, &ws);
    Product p{};
    p.M = c.T; p.N = c.V; p.K = c.D;
    p.count = a.count;
    p.target = a.target;
    p.status = status;
    p.part = reinterpret_cast<float2*>(w + sp.part);
    p.tpad = sp.tpad;
    p.ztarget = reinterpret_cast<float*>(w + sp.ztarget);
    const cudaError_t e = launch_product<DT, USE_STATS>(p, a.out, sp.dpad, weight, ws, s);
    if (e != cudaSuccess) return e;
    combine_kernel<DT><<<static_cast<unsigned>((c.T + kJoinRows - 1) / kJoinRows), 32 * kJoinRows, 0, s>>>(
        a.count, a.rows, p.part, sp.tpad, static_cast<int>(sp.ntiles), p.ztarget, a.out, sp.dpad, weight, ws, c.D, a.target,
        loss, lse);
    return cudaGetLastError();
}

template <int DT>
cudaError_t run_backward(const Call& c, const Space& sp, char* w, int* status, const float* lse, const float* gl, int gl_stride,
                  void* gh, int64_t ghs, void* gw, int64_t gws, int gw_f32, int accumulate, cudaStream_t s)
{
    PrepArgs a{};
    a.lse_in = lse;
    a.gl = gl;
    a.gl_stride = gl_stride;
    a.lse = reinterpret_cast<float*>(w + sp.lse);
    a.ratio = reinterpret_cast<float*>(w + sp.ratio);
    a.gmax = reinterpret_cast<float*>(w + sp.gmax);
    a.gh = static_cast<uint16_t*>(gh);
    a.ghs = ghs;
    a.g_scale = g_scale<DT>();
    const void* weight;
    int64_t ws;
    launch_prep(a, c, sp, w, status, s, &weight, &ws);
    for (int64_t v0 = 0; v0 < c.V; v0 += sp.piece) {
        const int64_t words = std::min(sp.piece, c.V - v0);
        const char* wp = static_cast<const char*>(weight) + 2 * v0 * ws;
        Product p{};
        p.count = a.count;
        p.rows_cap = c.T;
        p.status = status;
        p.v0 = v0;
        p.target = a.target;
        p.lse = a.lse;
        p.ratio = a.ratio;
        p.g = w + sp.grad;
        p.gld = sp.piece;
        p.gmax = a.gmax;
        p.inv_scale = 1.f / g_scale<DT>();
        p.rows = a.rows;
        p.tpad = sp.dpad;
        Product q = p;
        q.M = c.T; q.N = words; q.K = c.D;
        cudaError_t e = launch_product<DT, USE_GRAD>(q, a.out, sp.dpad, wp, ws, s);
        if (e == cudaSuccess && gh) {
            q = p;
            q.M = c.T; q.N = c.D; q.K = words;
            q.first = v0 == 0;
            q.last = v0 + words == c.V;
            q.acc = q.first && q.last ? nullptr : reinterpret_cast<float*>(w + sp.acc);
            q.out = gh; q.os = ghs;
            q.vec = aligned16(gh) && ghs % 4 == 0;
            e = launch_product<DT, USE_DH>(q, p.g, p.gld, wp, ws, s);
        }
        if (e == cudaSuccess && gw) {
            q = p;
            q.M = words; q.N = c.D; q.K = c.T;
            q.out = gw; q.os = gws; q.out_f32 = gw_f32; q.accumulate = accumulate;
            q.vec = aligned16(gw) && gws % 4 == 0;
            e = launch_product<DT, USE_DW>(q, p.g, p.gld, a.out, sp.dpad, s);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

}  // namespace
}  // namespace ddplm

using namespace ddplm;

extern "C" ddp_status ddp_vocab_loss_workspace(int64_t ntokens, int64_t vocab, int64_t dim, int64_t piece,
                                               int32_t weight_aligned, int64_t* forward_bytes, int64_t* backward_bytes)
{
    const char* fn = "ddp_vocab_loss_workspace";
    if (!forward_bytes || !backward_bytes) return ddp::fail(DDP_E_INVAL, "%s: an output is NULL", fn);
    if (ntokens < 0 || ntokens >= (int64_t{1} << 31) - 512 || vocab < 1 || vocab >= (int64_t{1} << 31) - 512 || dim < 1 ||
        dim >= (int64_t{1} << 24) || piece < 0)
        return ddp::fail(DDP_E_INVAL, "%s: ntokens = %lld, vocab = %lld, dim = %lld, piece = %lld out of range", fn,
                         static_cast<long long>(ntokens), static_cast<long long>(vocab), static_cast<long long>(dim),
                         static_cast<long long>(piece));
    *forward_bytes = space_for(false, ntokens, vocab, dim, piece, !weight_aligned).total;
    *backward_bytes = space_for(true, ntokens, vocab, dim, piece, !weight_aligned).total;
    return ddp::ok();
}

extern "C" ddp_status ddp_vocab_loss_forward(const void* hidden, int64_t hidden_stride, const void* weight,
                                             int64_t weight_stride, int32_t dtype, int64_t ntokens, int64_t vocab,
                                             int64_t dim, const void* targets, int32_t id_bytes, int64_t ignore_index,
                                             float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                                             void* stream)
{
    const char* fn = "ddp_vocab_loss_forward";
    const Call c{hidden, hidden_stride, weight, weight_stride, dtype, ntokens, vocab, dim, targets, id_bytes, ignore_index};
    Space sp{};
    if (ntokens >= 0 && vocab >= 1 && dim >= 1 && dim < (int64_t{1} << 24)) sp = space_for(false, ntokens, vocab, dim, 0, needs_copy(c));
    const ddp_status st = check(fn, c, workspace, workspace_bytes, sp.total);
    if (st != DDP_OK) return st;
    if (ntokens == 0) return ddp::ok();
    if (!loss || !lse) return ddp::fail(DDP_E_INVAL, "%s: loss or lse is NULL", fn);
    int* status = lm_status_word();
    if (!status) return ddp::fail(DDP_E_CUDA, "%s: the status word is unavailable", fn);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* w = static_cast<char*>(workspace);
    const cudaError_t err = dtype == DDP_BF16 ? run_forward<DDP_BF16>(c, sp, w, status, loss, lse, s)
                                              : run_forward<DDP_F16>(c, sp, w, status, loss, lse, s);
    if (err != cudaSuccess) return ddp::fail(DDP_E_CUDA, "%s: kernel launch failed: %s", fn, cudaGetErrorString(err));
    return ddp::ok();
}

extern "C" ddp_status ddp_vocab_loss_backward(const void* hidden, int64_t hidden_stride, const void* weight,
                                              int64_t weight_stride, int32_t dtype, int64_t ntokens, int64_t vocab,
                                              int64_t dim, const void* targets, int32_t id_bytes, int64_t ignore_index,
                                              const float* lse, const float* grad_loss, int32_t grad_loss_stride,
                                              void* grad_hidden, int64_t gh_stride, void* grad_weight,
                                              int64_t gw_stride, int32_t gw_dtype, int32_t accumulate, int64_t piece,
                                              void* workspace, int64_t workspace_bytes, void* stream)
{
    using ddp::fail;
    const char* fn = "ddp_vocab_loss_backward";
    const Call c{hidden, hidden_stride, weight, weight_stride, dtype, ntokens, vocab, dim, targets, id_bytes, ignore_index};
    if (piece < 0) return fail(DDP_E_INVAL, "%s: piece = %lld < 0", fn, static_cast<long long>(piece));
    Space sp{};
    if (ntokens >= 0 && vocab >= 1 && dim >= 1 && dim < (int64_t{1} << 24)) sp = space_for(true, ntokens, vocab, dim, piece, needs_copy(c));
    const ddp_status st = check(fn, c, workspace, workspace_bytes, sp.total);
    if (st != DDP_OK) return st;
    if (!grad_hidden && !grad_weight) return fail(DDP_E_INVAL, "%s: both outputs are NULL", fn);
    if (grad_hidden && gh_stride < dim)
        return fail(DDP_E_INVAL, "%s: grad_hidden's stride %lld < dim = %lld", fn, static_cast<long long>(gh_stride), static_cast<long long>(dim));
    if (grad_weight && gw_stride < dim)
        return fail(DDP_E_INVAL, "%s: grad_weight's stride %lld < dim = %lld", fn, static_cast<long long>(gw_stride), static_cast<long long>(dim));
    if (grad_weight && gw_dtype != dtype && gw_dtype != DDP_F32)
        return fail(DDP_E_INVAL, "%s: gw_dtype %d is neither dtype nor DDP_F32", fn, gw_dtype);
    if (grad_loss_stride != 0 && grad_loss_stride != 1) return fail(DDP_E_INVAL, "%s: grad_loss_stride = %d is neither 0 nor 1", fn, grad_loss_stride);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ntokens == 0) {
        if (grad_weight && !accumulate) {
            const int64_t es = gw_dtype == DDP_F32 ? 4 : 2;
            const cudaError_t e = cudaMemset2DAsync(grad_weight, gw_stride * es, 0, dim * es, vocab, s);
            if (e != cudaSuccess) return fail(DDP_E_CUDA, "%s: clearing grad_weight: %s", fn, cudaGetErrorString(e));
        }
        return ddp::ok();
    }
    if (!lse || !grad_loss) return fail(DDP_E_INVAL, "%s: lse or grad_loss is NULL", fn);
    int* status = lm_status_word();
    if (!status) return fail(DDP_E_CUDA, "%s: the status word is unavailable", fn);
    char* w = static_cast<char*>(workspace);
    const int f32 = gw_dtype == DDP_F32;
    const cudaError_t err =
        dtype == DDP_BF16 ? run_backward<DDP_BF16>(c, sp, w, status, lse, grad_loss, grad_loss_stride, grad_hidden, gh_stride,
                                                   grad_weight, gw_stride, f32, accumulate != 0, s)
                          : run_backward<DDP_F16>(c, sp, w, status, lse, grad_loss, grad_loss_stride, grad_hidden, gh_stride,
                                                  grad_weight, gw_stride, f32, accumulate != 0, s);
    if (err != cudaSuccess) return fail(DDP_E_CUDA, "%s: kernel launch failed: %s", fn, cudaGetErrorString(err));
    return ddp::ok();
}
