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
#include <cmath>

#include "lm_common.cuh"

namespace ddplm {
namespace {

constexpr int kRowTile = 256;   // rows of the gathered arrays are padded to this
constexpr int kTileM = 64, kTileN = 64, kTileK = 16;
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
    s.ntiles = (V + kTileN - 1) / kTileN;
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
        s.acc = take(s.piece < vpad ? 4 * s.tpad * D : 0);
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
    // rows up to the tile's end are zeros: they are terms of dW's sums
    const int end = (all + kRowTile - 1) / kRowTile * kRowTile;
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
enum Use { USE_STATS, USE_GRAD, USE_DH, USE_DW };

struct Product {
    const void* a;
    int64_t am, ak;       // strides of A in elements
    const void* b;
    int64_t bn, bk;
    int64_t M, N, K;
    const int32_t* count; // gathered rows: bounds M (STATS, GRAD, DH) or K (DW)
    int64_t v0;           // first word of the piece
    int64_t vocab;
    const int32_t* target;
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
    int32_t out_f32, accumulate;
};

template <int DT, int USE> __global__ void __launch_bounds__(256) product_kernel(Product p)
{
    using T = typename Elem<DT>::T;
    __shared__ float sa[kTileK][kTileM + 1], sb[kTileK][kTileN + 1];
    __shared__ float2 red[kTileM][17];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t count = *p.count;
    const int64_t M = USE == USE_DW ? p.M : min(p.M, count);
    const int64_t K = USE == USE_DW ? min(p.K, count) : p.K;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTileM, n0 = static_cast<int64_t>(blockIdx.x) * kTileN;
    const int64_t mend = USE == USE_GRAD ? (count + kRowTile - 1) / kRowTile * kRowTile : M;
    if (m0 >= mend) return;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += kTileK) {
        for (int i = tid; i < kTileM * kTileK; i += 256) {
            const int m = p.ak == 1 ? i / kTileK : i % kTileM, k = p.ak == 1 ? i % kTileK : i / kTileM;
            sa[k][m] = (m0 + m < M && k0 + k < K) ? Elem<DT>::to_f(static_cast<const T*>(p.a)[(m0 + m) * p.am + (k0 + k) * p.ak]) : 0.f;
        }
        for (int i = tid; i < kTileN * kTileK; i += 256) {
            const int n = p.bk == 1 ? i / kTileK : i % kTileN, k = p.bk == 1 ? i % kTileK : i / kTileN;
            sb[k][n] = (n0 + n < p.N && k0 + k < K) ? Elem<DT>::to_f(static_cast<const T*>(p.b)[(n0 + n) * p.bn + (k0 + k) * p.bk]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTileK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    if (USE == USE_STATS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + ty * 4 + i;
            float mx = -INFINITY, s = 0.f;
            for (int j = 0; j < 4; ++j)
                if (n0 + tx * 4 + j < p.N) mx = fmaxf(mx, acc[i][j]);
            for (int j = 0; j < 4; ++j)
                if (n0 + tx * 4 + j < p.N) {
                    s += mx == -INFINITY ? 0.f : exp2f((acc[i][j] - mx) * kLog2e);
                    if (m < M && p.target[m] == n0 + tx * 4 + j) p.ztarget[m] = acc[i][j];
                }
            red[ty * 4 + i][tx] = make_float2(mx, s);
        }
        __syncthreads();
        if (tid < kTileM && m0 + tid < M) {
            float mx = -INFINITY, s = 0.f;
            for (int j = 0; j < 16; ++j) mx = fmaxf(mx, red[tid][j].x);
            for (int j = 0; j < 16; ++j)
                if (red[tid][j].x != -INFINITY) s += red[tid][j].y * exp2f((red[tid][j].x - mx) * kLog2e);
            p.part[blockIdx.x * p.tpad + m0 + tid] = make_float2(mx, s);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            const float c = acc[i][j];
            if (USE == USE_GRAD) {
                float g = 0.f;  // rows and words beyond the end are zeros
                if (m < M && n < p.N) {
                    g = exp2f((c - p.lse[m]) * kLog2e) - (p.target[m] == p.v0 + n ? 1.f : 0.f);
                    g = p.ratio[m] == 0.f ? 0.f : g * p.ratio[m];
                }
                if (n < p.gld) static_cast<T*>(p.g)[m * p.gld + n] = Elem<DT>::from_f(g);
            } else if (m < M && n < p.N) {
                const float alpha = *p.gmax * p.inv_scale;
                if (USE == USE_DH) {
                    float s = c;
                    if (p.acc) {
                        if (!p.first) s += p.acc[m * p.N + n];
                        if (!p.last) p.acc[m * p.N + n] = s;
                    }
                    if (p.last) static_cast<T*>(p.out)[p.rows[m] * p.os + n] = Elem<DT>::from_f(s * alpha);
                } else if (p.out_f32) {
                    float* o = static_cast<float*>(p.out) + (p.v0 + m) * p.os + n;
                    *o = c * alpha + (p.accumulate ? *o : 0.f);
                } else {
                    T* o = static_cast<T*>(p.out) + (p.v0 + m) * p.os + n;
                    *o = Elem<DT>::from_f(c * alpha + (p.accumulate ? Elem<DT>::to_f(*o) : 0.f));
                }
            }
        }
}

template <int DT, int USE> void launch_product(const Product& p, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>((p.N + kTileN - 1) / kTileN), static_cast<unsigned>((p.M + kTileM - 1) / kTileM));
    product_kernel<DT, USE><<<grid, 256, 0, s>>>(p);
}

// join the tiles' (maximum, sum) pairs of each gathered row
__global__ void __launch_bounds__(256)
combine_kernel(const int32_t* count, const int32_t* rows, const float2* part, int64_t tpad, int64_t ntiles,
               const float* ztarget, float* loss, float* lse)
{
    const int64_t m = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (m >= *count) return;
    float mx = -INFINITY, s = 0.f;
    for (int64_t j = 0; j < ntiles; ++j) mx = fmaxf(mx, part[j * tpad + m].x);
    for (int64_t j = 0; j < ntiles; ++j) {
        const float2 q = part[j * tpad + m];
        if (q.x != -INFINITY) s += q.y * exp2f((q.x - mx) * kLog2e);
    }
    const float l = mx + logf(s);
    lse[rows[m]] = l;
    loss[rows[m]] = l - ztarget[m];
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

template <int DT> void run_forward(const Call& c, const Space& sp, char* w, int* status, float* loss, float* lse, cudaStream_t s)
{
    PrepArgs a{};
    a.loss = loss;
    a.lse_out = lse;
    const void* weight;
    int64_t ws;
    launch_prep(a, c, sp, w, status, s, &weight, &ws);
    Product p{};
    p.a = a.out; p.am = sp.dpad; p.ak = 1;
    p.b = weight; p.bn = ws; p.bk = 1;
    p.M = c.T; p.N = c.V; p.K = c.D;
    p.count = a.count;
    p.vocab = c.V;
    p.target = a.target;
    p.part = reinterpret_cast<float2*>(w + sp.part);
    p.tpad = sp.tpad;
    p.ztarget = reinterpret_cast<float*>(w + sp.ztarget);
    launch_product<DT, USE_STATS>(p, s);
    combine_kernel<<<static_cast<unsigned>((c.T + 255) / 256), 256, 0, s>>>(a.count, a.rows, p.part, sp.tpad, sp.ntiles, p.ztarget, loss, lse);
}

template <int DT>
void run_backward(const Call& c, const Space& sp, char* w, int* status, const float* lse, const float* gl, int gl_stride,
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
        p.vocab = c.V;
        p.v0 = v0;
        p.target = a.target;
        p.lse = a.lse;
        p.ratio = a.ratio;
        p.g = w + sp.grad;
        p.gld = sp.piece;
        p.gmax = a.gmax;
        p.inv_scale = 1.f / g_scale<DT>();
        p.rows = a.rows;
        Product q = p;
        q.a = a.out; q.am = sp.dpad; q.ak = 1;
        q.b = wp; q.bn = ws; q.bk = 1;
        q.M = sp.tpad; q.N = words; q.K = c.D;
        launch_product<DT, USE_GRAD>(q, s);
        if (gh) {
            q = p;
            q.a = p.g; q.am = p.gld; q.ak = 1;
            q.b = wp; q.bn = 1; q.bk = ws;
            q.M = c.T; q.N = c.D; q.K = words;
            q.first = v0 == 0;
            q.last = v0 + words == c.V;
            q.acc = q.first && q.last ? nullptr : reinterpret_cast<float*>(w + sp.acc);
            q.out = gh; q.os = ghs;
            launch_product<DT, USE_DH>(q, s);
        }
        if (gw) {
            q = p;
            q.a = p.g; q.am = 1; q.ak = p.gld;
            q.b = a.out; q.bn = 1; q.bk = sp.dpad;
            q.M = words; q.N = c.D; q.K = sp.tpad;
            q.out = gw; q.os = gws; q.out_f32 = gw_f32; q.accumulate = accumulate;
            launch_product<DT, USE_DW>(q, s);
        }
    }
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
    if (dtype == DDP_BF16) run_forward<DDP_BF16>(c, sp, w, status, loss, lse, s);
    else run_forward<DDP_F16>(c, sp, w, status, loss, lse, s);
    const cudaError_t err = cudaGetLastError();
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
    if (dtype == DDP_BF16)
        run_backward<DDP_BF16>(c, sp, w, status, lse, grad_loss, grad_loss_stride, grad_hidden, gh_stride, grad_weight, gw_stride, f32, accumulate != 0, s);
    else
        run_backward<DDP_F16>(c, sp, w, status, lse, grad_loss, grad_loss_stride, grad_hidden, gh_stride, grad_weight, gw_stride, f32, accumulate != 0, s);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return fail(DDP_E_CUDA, "%s: kernel launch failed: %s", fn, cudaGetErrorString(err));
    return ddp::ok();
}
