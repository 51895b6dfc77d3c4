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
//
// Bound by the tensor cores: 2 T V D operations forward, 8 T V D for a step (6 without the
// second z).  Measured on a GB300 (2 T V D = 632 GFLOP at 8192 tokens x 50257 words x 768,
// bf16): a step 1.73 to 1.85 ms, 1.46 to 1.37 PFLOP/s, the longer one back to back under the
// power limit.  At 4096 x 131072 x 4096 the step, seconds long, runs at what that limit
// leaves (10.6 ms, 1.63 PFLOP/s; cuBLAS for seconds: 1.74).
//
// Rounded to 16 bits on the way: G, the one rounding that a form in fp32 does not have.  The
// tensor cores take 16-bit operands; G in two parts would double both gradient products.
// It leaves the gradients about 1.2 times as far from the exact ones as one rounding of
// the result alone (1.96e-3 beside 1.66e-3 in bf16, 2.55e-4 beside 2.07e-4 in fp16).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "lm_common.cuh"
#include "umma.cuh"

namespace ddplm {
namespace {

constexpr int kRowTile = 256;   // rows of the gathered arrays are padded to this
constexpr int kPrepThreads = 256;
// Tokens are counted in 32 bits, up to a step of the gather's loop (2048) beyond the last one; words up to a tile's.
constexpr int64_t kMaxTokens = (int64_t{1} << 31) - 4096;
constexpr int64_t kMaxVocab = (int64_t{1} << 31) - 512;
constexpr int kFewTokens = 2;      // up to so many the forward pass goes without matrix products
constexpr int kMaxFewCtas = 1024;
// Elements of G that are held at a time: 537 MB.  More pieces are more launches, which cost
// about 8 us each at their ends (with cold caches the masked step at 30522 x 1024 takes 400 us
// with half of it, 352 so; 8192 tokens x 50257 x 768 1.765 ms and 1.75).
constexpr int64_t kPieceElements = int64_t{1} << 28;
constexpr float kLog2e = 1.4426950408889634f;

// G's scale in fp16: its largest magnitude, 1 after the division by the largest
// |grad_loss|, is moved to 2^14, so that probabilities down to 2^-28 stay normal
// numbers.  bf16 has fp32's exponents and needs none.
template <int DT> constexpr float g_scale() { return DT == DDP_F16 ? 16384.f : 1.f; }

// A token whose |grad_loss| is below kMinRatio of the largest would leave too few of fp16's
// bits to its probabilities.  Its row of G is held times 2^k, back up to kMinRatio or just
// above (probabilities down to 2^-18 normal, the smallest step 2^-28); dH's row is multiplied by
// 2^-k in fp32, and dW takes its hidden state times 2^-k in fp16, exactly but for what
// falls below fp16's smallest normal number.  Other rows are not touched by this (k = 0).
constexpr float kMinRatio = 0x1p-10f;

// dH's tiles are split along the vocabulary while there are fewer than this many
// of them, about one for each pair of SMs (by a constant, so that the order of its sums
// does not depend on the device).
constexpr int kSplitTiles = 76;
__host__ __device__ __forceinline__ int dh_splits(int mt, int nt, int nkb)
{
    const int want = (kSplitTiles + mt * nt - 1) / (mt * nt), most = (nkb + 7) / 8;
    return want < most ? want : most;
}

struct Space {
    int64_t count, gmax, rows, target, ratio, back, lse, hidden, hidden_w, part, ztarget, grad, acc, weight, total;
    int64_t piece, pieces, ntiles, tpad, dpad, grad_bytes;
};

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

Space space_for(bool backward, int64_t T, int64_t V, int64_t D, int64_t piece, bool copy_weight)
{
    Space s{};
    s.tpad = round_up(std::max<int64_t>(T, 1), kRowTile);
    s.dpad = round_up(D, 8);
    s.ntiles = (V + 127) / 128;  // one pair of statistics a row for each 128 words
    const int64_t vpad = round_up(V, 256);
    // G in two buffers of half the words asked for, one filled while the other is read
    if (piece <= 0) piece = std::max<int64_t>(2048, kPieceElements / s.tpad);
    const int64_t most = piece >= vpad ? vpad : std::min(vpad, round_up(piece, 512) / 2);
    // equal pieces: the last one is a launch of its own, which a few words would leave idle
    s.pieces = (V + most - 1) / most;
    s.piece = std::min(most, round_up((V + s.pieces - 1) / s.pieces, 256));
    s.pieces = backward ? (V + s.piece - 1) / s.piece : 0;
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
        // (fp16's; bf16 has no use for these two)
        s.back = take(4 * s.tpad);
        s.hidden_w = take(2 * s.tpad * s.dpad);
        s.lse = take(4 * s.tpad);
        s.grad_bytes = round_up(2 * s.tpad * most, 256);
        s.grad = take(s.grad_bytes * std::min<int64_t>(s.pieces, 2));
        // splits x rows: at most (kSplitTiles / nt + mt) tiles of rows
        const int64_t nt = (D + 255) / 256;
        s.acc = take(4 * s.dpad * (s.tpad + kRowTile * ((kSplitTiles + nt - 1) / nt)));
    } else {
        // (for a few tokens: a pair for each token and CTA)
        s.part = take(std::max<int64_t>(8 * s.tpad * s.ntiles, 8 * kFewTokens * kMaxFewCtas));
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
    float* ratio;         // gathered: grad_loss / gmax * g_scale (fp16: and * 2^k)
    float* back;          // fp16, gathered: 2^-k
    uint16_t* out_w;      // fp16, [tpad][dpad]: gathered rows times 2^-k (nullptr: no weight gradient)
    float* gmax;          // largest finite |grad_loss| of the gathered rows (1 if that is 0)
    uint16_t* gh;         // rows to clear
    int64_t ghs;
    float g_scale;
    int32_t vec;          // hidden (and gh) in 16-byte vectors
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

// Values [c, c + 8) of a row that may start anywhere, zeros past its end.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t c, int64_t dim)
{
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < dim ? __ldg(row + c + j) : 0;
    return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

// eight fp16 values times f
__device__ __forceinline__ uint4 times8(uint4 v, float f)
{
    __half* h = reinterpret_cast<__half*>(&v);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = __float2half_rn(__half2float(h[j]) * f);
    return v;
}

// Every CTA counts the tokens with a target before its own slab, and all of them, itself:
// no launch of its own for the places, and 8 bytes a token and CTA from L2.  Bound by the
// latency of four dependent reads; 13 us for 8192 rows of 768 (25 MB) with cold caches.
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(PrepArgs a)
{
    __shared__ int sh[kPrepThreads / 32];
    __shared__ float shf[kPrepThreads / 32];
    __shared__ int place[kPrepThreads];  // of the slab's tokens: gathered row or -1
    __shared__ float backs[kPrepThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * a.slab, t1 = min(a.T, t0 + a.slab);
    wait_for_previous();
    int before = 0, all = 0;
    float gm = 0.f;
    // eight tokens a thread at a time, their loads in flight together
    for (int t = tid; t < a.T; t += 8 * kPrepThreads) {
        int64_t y[8];
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int u = t + j * kPrepThreads;
            y[j] = u < a.T ? load_id(a.targets, a.id_bytes, u) : a.ignore;
            g[j] = a.gl && u < a.T ? a.gl[static_cast<int64_t>(u) * a.gl_stride] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (y[j] == a.ignore || y[j] < 0 || y[j] >= a.vocab) continue;
            ++all;
            before += t + j * kPrepThreads < t0;
            const float x = fabsf(g[j]);
            if (x > gm && x <= 3.4028234663852886e38f) gm = x;
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
                float r = a.gl[static_cast<int64_t>(t) * a.gl_stride] / gm, back = 1.f;
                if (a.back) {
                    const float size = fabsf(r);
                    if (size > 0.f && size < kMinRatio) {
                        const int k = ilogbf(kMinRatio) - ilogbf(size);
                        r = ldexpf(r, k);
                        back = ldexpf(1.f, -k);
                    }
                    a.back[at] = back;
                }
                backs[tid] = back;
                a.ratio[at] = r * a.g_scale;
            }
        } else if (t < t1 && a.loss) {
            a.loss[t] = 0.f;
            a.lse_out[t] = 0.f;
        }
    }
    __syncthreads();
    // rows in 16-byte vectors where the tensors allow it
    const int64_t vecs = a.vec ? a.dpad / 8 : 0;
    const int rows = t1 - t0;
    for (int64_t i = tid; i < vecs * rows; i += 4 * kPrepThreads) {
        uint4 v[4];
        uint16_t *to[4], *to_w[4];
        float back[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t k = i + j * kPrepThreads;
            to[j] = to_w[j] = nullptr;
            if (k >= vecs * rows) continue;
            const int r = static_cast<int>(static_cast<uint32_t>(k) / static_cast<uint32_t>(vecs));
            const int64_t c = (k - r * vecs) * 8;
            v[j] = make_uint4(0, 0, 0, 0);
            if (place[r] >= 0) {
                to[j] = a.out + static_cast<int64_t>(place[r]) * a.dpad + c;
                if (a.out_w) to_w[j] = a.out_w + static_cast<int64_t>(place[r]) * a.dpad + c, back[j] = backs[r];
                v[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.hidden) + static_cast<int64_t>(t0 + r) * a.hs + c);
            } else if (a.gh) {
                to[j] = a.gh + static_cast<int64_t>(t0 + r) * a.ghs + c;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (to[j]) *reinterpret_cast<uint4*>(to[j]) = v[j];
            if (to_w[j]) *reinterpret_cast<uint4*>(to_w[j]) = back[j] == 1.f ? v[j] : times8(v[j], back[j]);
        }
    }
    if (!a.vec) {
        const int64_t all_vecs = a.dpad / 8;
        for (int64_t i = tid; i < all_vecs * rows; i += kPrepThreads) {
            const int r = static_cast<int>(i / all_vecs);
            const int64_t c = (i - r * all_vecs) * 8;
            if (place[r] >= 0) {
                const uint4 v = load8(static_cast<const uint16_t*>(a.hidden) + static_cast<int64_t>(t0 + r) * a.hs, c, a.dim);
                const int64_t at = static_cast<int64_t>(place[r]) * a.dpad + c;
                *reinterpret_cast<uint4*>(a.out + at) = v;
                if (a.out_w) *reinterpret_cast<uint4*>(a.out_w + at) = backs[r] == 1.f ? v : times8(v, backs[r]);
            } else if (a.gh)
                for (int64_t k = c; k < min(c + 8, a.dim); ++k) a.gh[static_cast<int64_t>(t0 + r) * a.ghs + k] = 0;
        }
    }
    // rows up to the tile's end are zeros (past the T-th the copies supply them): they are terms of dW's sums
    const int end = min(a.T, (all + kRowTile - 1) / kRowTile * kRowTile);
    for (int64_t r = static_cast<int64_t>(all) + blockIdx.x; r < end; r += gridDim.x)
        for (int64_t c = tid * 8; c < a.dpad; c += kPrepThreads * 8) {
            *reinterpret_cast<uint4*>(a.out + r * a.dpad + c) = make_uint4(0, 0, 0, 0);
            if (a.out_w) *reinterpret_cast<uint4*>(a.out_w + r * a.dpad + c) = make_uint4(0, 0, 0, 0);
        }
}

// An aligned copy of rows that start anywhere: a thread gathers 8 values at a time, the
// cache line stays in L1 for the eight loads.
__global__ void __launch_bounds__(256)
copy_weight_kernel(const uint16_t* w, int64_t ws, int64_t vocab, int64_t dim, uint16_t* out, int64_t dpad)
{
    wait_for_previous();
    const int64_t vecs = dpad / 8, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < vocab * vecs; i += 2 * step) {
        uint4 x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t k = i + j * step, v = k / vecs;
            if (k < vocab * vecs) x[j] = load8(w + v * ws, (k - v * vecs) * 8, dim);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (i + j * step < vocab * vecs) *reinterpret_cast<uint4*>(out + (i + j * step) * 8) = x[j];
    }
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
// A launch runs one or several products, one a use at most, their tiles one after the other, longest
// first: with dH and dW of one piece of the vocabulary comes G of the next, whose
// short tiles fill what the long ones leave idle at the end.  A pair takes every
// npairs-th tile; its warps work the tiles out for themselves and exchange nothing but
// the barriers' counts.
//
// Why so: a CTA's 128 x 256 share of a tile needs 32 KB of operands for 512 cycles of
// products; alone, without the pair, it would need 48 KB, more than an SM gets from L2 in
// that time.  Six stages are 192 KB; four to six made no difference.  What did: the code
// written out for each use (466 -> 443 us forward at 8192 x 50257 x 768, when it came; 356
// now) and reading ahead what dH and dW add to (masked step 480 -> 402 then, 298 now).
// Where k is short the epilogue is the bound: 2.1 us a tile at 128 values of k, twice what
// its exponentials take.  146 registers, one CTA an SM.  At 4096 x 16384 x 768 the tensor
// pipe is active 68% of the time in the statistics, 59% in G, 83% in dH and dW.
// what becomes of C, in the order in which a launch runs them
enum Use { USE_DH, USE_DW, USE_GRAD, USE_STATS, kUses };

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
constexpr int kGroup = 32;               // tiles along the fast side before the slow side moves on

struct Maps {
    CUtensorMap a, b;
};
struct Product {
    int64_t M, N, K;      // all zero: this use is not in the launch
    int64_t rows_cap;     // rows of the gathered arrays that exist
    int64_t v0;           // first word of the piece
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
    const float* back;    // DH, fp16: a factor for each row
    float* acc;           // dH: fp32 sums over pieces and splits, [split][row][ald]
    int64_t ald;
    int32_t first, last;
    const int32_t* rows;
    void* out;
    int64_t os;
    int32_t out_f32, accumulate, vec;
};
// The kernel's code is written out for each use, so that a product's arguments have
// fixed places in the parameters: with an index that a tile brings along, a forward pass
// at 4096 x 131072 x 4096 took 2.50 ms, with fixed places 2.22.
struct Batch {
    Maps map[kUses];
    Product job[kUses];
    const int32_t* count; // gathered rows: bounds M (STATS, GRAD, DH) or K (DW)
    int* status;
};

// What a launch's warps know of a product: its tiles, and how many there are.
struct Shape {
    int32_t mt, nt, nkb, splits;
    int64_t M, tiles;
};
__device__ __forceinline__ Shape shape_of(const Product& p, int use, int64_t count)
{
    Shape s;
    const int64_t K = use == USE_DW ? min(p.K, count) : p.K;
    s.M = use == USE_DW ? p.M : min(p.M, count);
    s.mt = static_cast<int>((s.M + kTile - 1) / kTile);
    s.nt = static_cast<int>((p.N + kTile - 1) / kTile);
    s.nkb = static_cast<int>((K + kBlockK - 1) / kBlockK);
    // (the splits follow from the whole product's length, not this piece's: the sums' layout is the same for every piece)
    s.splits = use == USE_DH && s.mt > 0 && s.nt > 0 ? dh_splits(s.mt, s.nt, static_cast<int>((p.gld + kBlockK - 1) / kBlockK)) : 1;
    s.tiles = static_cast<int64_t>(s.mt) * s.nt * s.splits;
    return s;
}
struct Tile {
    int32_t use, m, n, split, kb0, kb1;
};
// Tile t of a launch.  Tiles that run at the same time share operands: up to kGroup
// along the side whose operand is the smaller one (the hidden states), then a
// step along the other, so that the larger one is read from HBM once.
// (32-bit arithmetic: the copies and the products stand still while their threads think.)
__device__ __forceinline__ Tile tile_at(uint32_t t, const Shape* shapes)
{
    Tile r{};
    while (r.use + 1 < kUses && t >= static_cast<uint32_t>(shapes[r.use].tiles)) t -= static_cast<uint32_t>(shapes[r.use++].tiles);
    const Shape& s = shapes[r.use];
    const uint32_t mn = static_cast<uint32_t>(s.mt) * s.nt;
    r.split = static_cast<int>(t / mn);
    t -= r.split * mn;
    const bool n_fast = r.use == USE_DW;
    const uint32_t fast = n_fast ? s.nt : s.mt, slow = n_fast ? s.mt : s.nt;
    const uint32_t group = t / (kGroup * slow), in = t - group * kGroup * slow;
    const uint32_t width = min(static_cast<uint32_t>(kGroup), fast - group * kGroup), o = in / width;
    const uint32_t i = group * kGroup + (in - o * width);
    r.m = static_cast<int>(n_fast ? o : i);
    r.n = static_cast<int>(n_fast ? i : o);
    const int per = (s.nkb + s.splits - 1) / s.splits;
    r.kb0 = min(s.nkb, r.split * per);
    r.kb1 = min(s.nkb, r.kb0 + per);
    return r;
}

// operands whose rows (not k) are contiguous in memory
template <int USE> struct Majors {
    static constexpr bool a_mn = USE == USE_DW;
    static constexpr bool b_mn = USE == USE_DH || USE == USE_DW;
};

// one CTA's 128 rows of an operand, 64 of k: one box, or two where the rows are contiguous
template <bool MN> __device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, int row, int k, uint32_t bar)
{
    if (MN) {
        tensor_load(dst, map, row, k, bar);
        tensor_load(dst + kOperandBytes / 2, map, row + 64, k, bar);
    } else {
        tensor_load(dst, map, k, row, bar);
    }
}

// 2^x; results below 2^-126 are zero: no probability that small adds to a sum of 1
__device__ __forceinline__ float pow2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
__device__ __forceinline__ void epilogue(const Product& p, const Shape& shape, const Tile& tile, uint32_t taddr, bool empty,
                                         int64_t m0, int64_t n0, uint32_t staging, int lane)
{
    using T = typename Elem<DT>::T;
    const int64_t M = shape.M;
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
            // (four chains: with little k the epilogue is what a tile takes)
            float cm[4] = {c[0], c[1], c[2], c[3]};
#pragma unroll
            for (int j = 4; j < 32; ++j) cm[j & 3] = fmaxf(cm[j & 3], c[j]);
            const float top = fmaxf(fmaxf(mx, fmaxf(cm[0], cm[1])), fmaxf(cm[2], cm[3]));
            if (top != -INFINITY) {  // all of them minus infinity: they add nothing
                const float shift = top * kLog2e;
                s *= mx == -INFINITY ? 0.f : pow2(mx * kLog2e - shift);
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 32; ++j) part[j & 3] += pow2(fmaf(c[j], kLog2e, -shift));
                s += (part[0] + part[1]) + (part[2] + part[3]);
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
                for (int j = 0; j < 32; ++j) c[j] = pow2(fmaf(c[j], kLog2e, -shift));
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
        // dH of one piece without splits needs no sums in memory
        const bool sums = USE == USE_DH && !(p.first && p.last && shape.splits == 1);
        const bool result = USE != USE_DH || (p.last && shape.splits == 1);
        float* acc = p.acc + static_cast<int64_t>(tile.split) * shape.mt * kTile * p.ald;
        const bool adds = sums ? !p.first : USE == USE_DW && p.accumulate;
        const bool f32 = USE == USE_DW && p.out_f32;
        const int32_t token = USE == USE_DH && result && m < M ? p.rows[m] : 0;
        constexpr bool kRowFactors = USE == USE_DH && DT == DDP_F16;
        const float row_alpha = kRowFactors && result && m < M ? alpha * p.back[m] : alpha;
        for (int q = 0; q < 4; ++q) {
            const int64_t n = n0 + q * 32 + (lane & 7) * 4;
            if (n0 + q * 32 >= p.N) break;
            const int width = static_cast<int>(max(int64_t{0}, min(int64_t{4}, p.N - n)));
            const bool wide = p.vec && width == 4;
            // what is added to, all of it on its way before the first value is needed
            float old[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t row = m0 + i * 4 + (lane >> 3);
#pragma unroll
                for (int j = 0; j < 4; ++j) old[i][j] = 0.f;
                if (!adds || row >= M || width == 0) continue;
                if (sums) {
                    *reinterpret_cast<float4*>(old[i]) = *reinterpret_cast<const float4*>(acc + row * p.ald + n);  // ald: a multiple of 8
                } else if (f32) {
                    const float* o = static_cast<const float*>(p.out) + (p.v0 + row) * p.os + n;
                    if (wide) *reinterpret_cast<float4*>(old[i]) = *reinterpret_cast<const float4*>(o);
                    else
                        for (int j = 0; j < 4; ++j) old[i][j] = j < width ? o[j] : 0.f;
                } else {
                    const T* o = static_cast<const T*>(p.out) + (p.v0 + row) * p.os + n;
                    if (wide) {
                        const uint2 v = *reinterpret_cast<const uint2*>(o);
                        const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
                        for (int j = 0; j < 4; ++j) old[i][j] = Elem<DT>::to_f(t[j]);
                    } else {
                        for (int j = 0; j < 4; ++j) old[i][j] = j < width ? Elem<DT>::to_f(o[j]) : 0.f;
                    }
                }
            }
            tile_values(taddr + q * 32, empty, c);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sts16(staged(staging, lane, k), make_uint4(__float_as_uint(c[4 * k]), __float_as_uint(c[4 * k + 1]),
                                                           __float_as_uint(c[4 * k + 2]), __float_as_uint(c[4 * k + 3])));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3);
                const int32_t to = USE == USE_DH ? __shfl_sync(0xffffffffu, token, r) : 0;
                const float factor = kRowFactors ? __shfl_sync(0xffffffffu, row_alpha, r) : alpha;
                const uint4 raw = lds16(staged(staging, r, lane & 7));
                float x[4] = {__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z), __uint_as_float(raw.w)};
                const int64_t row = m0 + r;
                if (row >= M || width == 0) continue;
                if (sums) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] += old[i][j];
                    if (!result) {
                        *reinterpret_cast<float4*>(acc + row * p.ald + n) = make_float4(x[0], x[1], x[2], x[3]);
                        continue;
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = x[j] * factor + (USE == USE_DW ? old[i][j] : 0.f);
                const int64_t at = (USE == USE_DH ? to : p.v0 + row) * p.os + n;
                if (f32) {
                    float* o = static_cast<float*>(p.out) + at;
                    if (wide) *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
                    else
                        for (int j = 0; j < width; ++j) o[j] = x[j];
                } else {
                    T* o = static_cast<T*>(p.out) + at;
                    if (wide) *reinterpret_cast<uint2*>(o) = make_uint2(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]));
                    else
                        for (int j = 0; j < width; ++j) o[j] = Elem<DT>::from_f(x[j]);
                }
            }
            __syncwarp();
        }
    }
}

// One thread copies a tile's operands, `it` stages into the ring.
template <int USE>
__device__ __forceinline__ bool copy_operands(const Batch& batch, int m, int n, const Tile& x, uint32_t it, uint32_t rank,
                                              uint32_t base, uint32_t bar0, volatile int* dead)
{
    const uint32_t lead = cluster_addr(bar0, 0);
    uint32_t s = it % kStages, parity = ((it / kStages) & 1) ^ 1;
    for (int kb = x.kb0; kb < x.kb1; ++kb) {
        if (!bar_wait(bar0 + 8u * (kStages + s), parity, dead)) return false;
        // both CTAs' bytes are counted on the first CTA's barrier
        if (rank == 0) bar_expect(bar0 + 8u * s, 2 * kStageBytes);
        const uint32_t a = base + s * kStageBytes;
        load_operand<Majors<USE>::a_mn>(a, &batch.map[USE].a, m, kb * kBlockK, lead + 8u * s);
        load_operand<Majors<USE>::b_mn>(a + kOperandBytes, &batch.map[USE].b, n, kb * kBlockK, lead + 8u * s);
        if (++s == kStages) {
            s = 0;
            parity ^= 1;
        }
    }
    return true;
}

// One thread issues a tile's products, `it` stages into the ring.  It has the time of
// four products (about 500 cycles) for each stage, so nothing but additions of
// constants is left in the loop.
template <int DT, int USE>
__device__ __forceinline__ bool issue_products(uint32_t d, int blocks, uint32_t it, uint32_t base, uint32_t bar0, volatile int* dead)
{
    constexpr bool A_MN = Majors<USE>::a_mn, B_MN = Majors<USE>::b_mn;
    constexpr uint32_t desc = product_desc(DT == DDP_BF16, A_MN, B_MN, kTile, kTile);
    // rows contiguous: 8 k (1024 bytes) after 8 k, blocks of 64 rows apart; k contiguous: 16 k are 32 bytes
    constexpr uint64_t a_step = (A_MN ? 2048 : 32) >> 4, b_step = (B_MN ? 2048 : 32) >> 4;
    const uint64_t a0 = operand_desc(base, A_MN ? kOperandBytes / 2 : 16, 1024);
    const uint64_t b0 = operand_desc(base + kOperandBytes, B_MN ? kOperandBytes / 2 : 16, 1024);
    uint32_t s = it % kStages, parity = (it / kStages) & 1;
    for (int kb = 0; kb < blocks; ++kb) {
        if (!bar_wait(bar0 + 8u * s, parity, dead)) return false;
        tmem_fence_after();
        const uint64_t a = a0 + s * (kStageBytes >> 4), b = b0 + s * (kStageBytes >> 4);
#pragma unroll
        for (int k = 0; k < kBlockK / 16; ++k) product_pair(d, a + k * a_step, b + k * b_step, desc, kb > 0 || k > 0);
        product_commit(bar0 + 8u * (kStages + s));
        if (++s == kStages) {
            s = 0;
            parity ^= 1;
        }
    }
    return true;
}

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1) product_kernel(const __grid_constant__ Batch batch)
{
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
    __shared__ Shape shapes[kUses];
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
#pragma unroll
        for (int i = 0; i < kUses; ++i) {
            if (batch.job[i].M == 0) continue;
            tensor_map_prefetch(&batch.map[i].a);
            tensor_map_prefetch(&batch.map[i].b);
        }
    }
    if (warp == 9) tmem_alloc(smem_addr(&tmem_base), 512);
    wait_for_previous();
#pragma unroll
    for (int i = 0; i < kUses; ++i)
        if (threadIdx.x == 32 * i) shapes[i] = shape_of(batch.job[i], i, *batch.count);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = tmem_base;

    uint32_t total = 0;
#pragma unroll
    for (int i = 0; i < kUses; ++i) total += static_cast<uint32_t>(shapes[i].tiles);
    const uint32_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (warp == 8) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t t = pair; ok && t < total; t += npairs) {
                const Tile x = tile_at(t, shapes);
                const int m = x.m * kTile + static_cast<int>(rank) * kHalf, n = x.n * kTile + static_cast<int>(rank) * kHalf;
                if (x.use == USE_DH) ok = copy_operands<USE_DH>(batch, m, n, x, it, rank, base, bar0, &dead);
                else if (x.use == USE_DW) ok = copy_operands<USE_DW>(batch, m, n, x, it, rank, base, bar0, &dead);
                else if (x.use == USE_GRAD) ok = copy_operands<USE_GRAD>(batch, m, n, x, it, rank, base, bar0, &dead);
                else ok = copy_operands<USE_STATS>(batch, m, n, x, it, rank, base, bar0, &dead);
                it += x.kb1 - x.kb0;
            }
            // the last arrivals on this CTA's barriers come before it may leave
            for (int i = 0; ok && i < kStages; ++i, ++it) ok = bar_wait(empty(it % kStages), ((it / kStages) & 1) ^ 1, &dead);
        }
    } else if (warp == 9) {
        if (rank == 0 && lane == 0) {
            uint32_t it = 0, j = 0;
            bool ok = true;
            for (uint32_t t = pair; ok && t < total; t += npairs) {
                const Tile x = tile_at(t, shapes);
                if (x.kb0 == x.kb1) continue;
                const int b = j & 1;
                if (!(ok = bar_wait<true>(tempty(b), ((j >> 1) & 1) ^ 1, &dead))) break;
                tmem_fence_after();
                const uint32_t d = tmem + b * kTile;
                const int blocks = x.kb1 - x.kb0;
                if (x.use == USE_DH) ok = issue_products<DT, USE_DH>(d, blocks, it, base, bar0, &dead);
                else if (x.use == USE_DW) ok = issue_products<DT, USE_DW>(d, blocks, it, base, bar0, &dead);
                else ok = issue_products<DT, USE_GRAD>(d, blocks, it, base, bar0, &dead);  // and USE_STATS
                it += blocks;
                if (ok) product_commit(tfull(b));
                ++j;
            }
        }
    } else {
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t staging = base + kStages * kStageBytes + warp * kStagingBytes;
        uint32_t j = 0;
        for (uint32_t t = pair; t < total; t += npairs) {
            const Tile x = tile_at(t, shapes);
            const bool none = x.kb0 == x.kb1;
            const int b = j & 1;
            if (!none) {
                if (!__all_sync(0xffffffffu, bar_wait(tfull(b), (j >> 1) & 1, &dead))) break;
                tmem_fence_after();
                ++j;
            }
            const int64_t m0 = static_cast<int64_t>(x.m) * kTile + rank * kHalf + quarter * 32;
            const int64_t n0 = static_cast<int64_t>(x.n) * kTile + half * kHalf;
            const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * kTile + half * kHalf;
            const Shape& sh = shapes[x.use];
            if (x.use == USE_DH) epilogue<DT, USE_DH>(batch.job[USE_DH], sh, x, taddr, none, m0, n0, staging, lane);
            else if (x.use == USE_DW) epilogue<DT, USE_DW>(batch.job[USE_DW], sh, x, taddr, none, m0, n0, staging, lane);
            else if (x.use == USE_GRAD) epilogue<DT, USE_GRAD>(batch.job[USE_GRAD], sh, x, taddr, none, m0, n0, staging, lane);
            else epilogue<DT, USE_STATS>(batch.job[USE_STATS], sh, x, taddr, none, m0, n0, staging, lane);
            tmem_fence_before();
            __syncwarp();
            if (lane == 0 && !none) bar_arrive_cluster(cluster_addr(tempty(b), 0));
        }
    }
    __syncthreads();
    if (dead) {
        // a wait gave up: report it, and let copies and products in flight end before the memory is given back
        if (threadIdx.x == 0) {
            atomicOr(batch.status, kErrWait);
            const uint64_t t0 = clock_ns();
            for (uint32_t i = 0; i < (1u << 24) && clock_ns() - t0 < 20000000ull; ++i) {}
        }
        __syncthreads();
    }
    // Arrivals on the other CTA's barriers that nobody waits for have landed before either CTA
    // leaves: its shared memory is another kernel's then.
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    tmem_fence_before();
    cluster_sync();
    tmem_fence_after();
    if (warp == 9) tmem_free(tmem, 512);
}

// dH where its tiles were split along the vocabulary: the splits' sums, in order.  HBM-bound;
// it returns at once where there were no splits.
template <int DT>
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ Product p, const int32_t* count)
{
    using T = typename Elem<DT>::T;
    wait_for_previous();
    const Shape sh = shape_of(p, USE_DH, *count);
    if (sh.splits == 1) return;
    const float scale = *p.gmax * p.inv_scale;
    const int64_t quads = p.ald / 4, size = static_cast<int64_t>(sh.mt) * kTile * p.ald;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < sh.M * quads; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = i / quads, n = (i - row * quads) * 4;
        const float alpha = DT == DDP_F16 ? scale * p.back[row] : scale;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int s = 0; s < sh.splits; ++s) {
            const float4 v = *reinterpret_cast<const float4*>(p.acc + s * size + row * p.ald + n);
            x[0] += v.x; x[1] += v.y; x[2] += v.z; x[3] += v.w;
        }
        T* o = static_cast<T*>(p.out) + p.rows[row] * p.os + n;
        if (p.vec && n + 4 <= p.N) {
            *reinterpret_cast<uint2*>(o) = make_uint2(pack2<DT>(x[0] * alpha, x[1] * alpha), pack2<DT>(x[2] * alpha, x[3] * alpha));
        } else {
            for (int j = 0; j < 4; ++j)
                if (n + j < p.N) o[j] = Elem<DT>::from_f(x[j] * alpha);
        }
    }
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
bool set_product(Batch& batch, const Product& p, const void* a, int64_t a_stride, const void* b, int64_t b_stride)
{
    batch.job[USE] = p;
    Maps& m = batch.map[USE];
    return (Majors<USE>::a_mn ? make_map(&m.a, DT, a, p.M, p.K, a_stride, kBlockK) : make_map(&m.a, DT, a, p.K, p.M, a_stride, kHalf)) &&
           (Majors<USE>::b_mn ? make_map(&m.b, DT, b, p.N, p.K, b_stride, kBlockK) : make_map(&m.b, DT, b, p.K, p.N, b_stride, kHalf));
}

template <int DT> cudaError_t launch_products(const Batch& batch, cudaStream_t s)
{
    static std::atomic<int> cached[ddp::kMaxDevices] = {};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = kProductSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const int dev = ddp::current_device();
    int pairs = dev >= 0 ? cached[dev].load(std::memory_order_relaxed) : 0;
    if (!pairs) {
        cudaError_t e = cudaFuncSetAttribute(product_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kProductSmem);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveClusters(&pairs, product_kernel<DT>, &cfg);
        if (e != cudaSuccess) return e;
        pairs = std::max(1, std::min(pairs, ddp::device_sm_count() / 2));
        if (dev >= 0) cached[dev].store(pairs, std::memory_order_relaxed);
    }
    int64_t tiles = 0;
    for (int i = 0; i < kUses; ++i) {
        const Product& p = batch.job[i];
        const int64_t mt = (p.M + kTile - 1) / kTile, nt = (p.N + kTile - 1) / kTile;
        tiles += mt * nt;
        if (i == USE_DH && p.M) tiles += kSplitTiles;  // fewer rows on the device may mean more splits
    }
    cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(tiles, pairs)));
    // (the cluster's size is the kernel's own.)  Neither this kernel nor the one after it is
    // launched to start while the kernel before it ends: no CTA takes over shared memory
    // whose last owner's pair still runs.
    cfg.numAttrs = 0;
    return cudaLaunchKernelEx(&cfg, product_kernel<DT>, batch);
}

// Joins the (maximum, sum) pairs of each gathered row, m = max m_i and s = sum s_i 2^((m_i - m) log2 e):
// 32 threads a row and eight rows a CTA, so that 64 bytes of neighbouring rows' pairs are
// read together and one row alone is still read by 32 threads.  In a fixed order.
constexpr int kJoinRows = 8;
__device__ __forceinline__ float2 join_pairs(float2 a, float2 b)
{
    const float m = fmaxf(a.x, b.x);
    // a side whose words are all minus infinity brings 0 (or a NaN, which stays)
    const float sa = a.x == -INFINITY ? a.y : a.y * pow2((a.x - m) * kLog2e);
    const float sb = b.x == -INFINITY ? b.y : b.y * pow2((b.x - m) * kLog2e);
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
    wait_for_previous();
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

// ---------------------------------------------------------------------------
// forward for a few tokens
// ---------------------------------------------------------------------------
// HBM-bound: the weight is read once, a warp takes four of its rows at a time and
// multiplies them with every token's hidden state, which shared memory holds.  One CTA an
// SM, with 128 KB of the weight on its way all the time.  At 50257 x
// 768 one token takes 27 us with cold caches (50 on the tensor cores; this kernel alone 17.5
// us, 4.4 TB/s), 22 back to back, and two 30 (cold); four took 66 (52) with registers
// instead of the ring.
constexpr int kFewElements = 32768;  // of hidden states in shared memory
constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 4;        // (the reduction over the lanes is written for four)
constexpr int kFewStages = 8;      // parts on their way to a warp: four rows' 256 values, 2 KB
constexpr int kFewStageBytes = kFewRows * 512;

struct FewArgs {
    const void* hidden;
    int64_t hs;
    const void* weight;
    int64_t ws, V, D;
    const void* targets;
    int32_t id_bytes, T;
    int64_t ignore;
    float2* part;   // [token][CTA]
    float* ztarget;
    float* loss;
    float* lse;
    int32_t ctas;
    int* status;
};

template <int DT, int NT, bool VEC> __global__ void __launch_bounds__(kFewThreads) few_kernel(FewArgs a)
{
    using T = typename Elem<DT>::T;
    extern __shared__ __align__(16) uint8_t few_smem[];
    __shared__ float2 joined[kFewWarps][NT];
    uint8_t* ring = few_smem + (threadIdx.x >> 5) * kFewStages * kFewStageBytes;
    T* h = reinterpret_cast<T*>(few_smem + (VEC ? kFewWarps * kFewStages * kFewStageBytes : 0));  // [NT][dpad], zeros past the row's end
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t dpad = (a.D + 7) / 8 * 8;
    wait_for_previous();
    int64_t y[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) y[t] = t < a.T ? load_id(a.targets, a.id_bytes, t) : a.ignore;
    for (int64_t i = tid; i < NT * dpad; i += kFewThreads) {
        const int64_t t = i / dpad, c = i - t * dpad;
        h[i] = t < a.T && c < a.D ? static_cast<const T*>(a.hidden)[t * a.hs + c] : Elem<DT>::from_f(0.f);
    }
    __syncthreads();
    float2 st[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) st[t] = make_float2(-INFINITY, 0.f);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kFewWarps, w0 = static_cast<int64_t>(blockIdx.x) * kFewWarps + warp;
    // Part i of this warp: rows [v, v + 4) with v = 4 (w0 + warps (i / parts)), values [256 (i % parts), ...).
    // A row's part goes straight to shared memory, several parts ahead, zeros past the row's end;
    // each lane reads back only what it copied itself.
    const int parts = static_cast<int>((a.D + 255) / 256);
    int64_t ahead_v = w0 * kFewRows;
    int ahead_c = 0, ahead_s = 0;
    auto copy_part = [&]() {
        if (ahead_v < a.V) {
            const int64_t c = ahead_c * 256 + lane * 8;
            const int bytes = static_cast<int>(max(int64_t{0}, min(int64_t{16}, (a.D - c) * 2)));
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                // rows past the last word copy the last word's
                const T* src = static_cast<const T*>(a.weight) + min(ahead_v + r, a.V - 1) * a.ws + (bytes ? c : 0);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(ring + ahead_s * kFewStageBytes + r * 512 + lane * 16)),
                             "l"(src), "r"(bytes)
                             : "memory");
            }
            if (++ahead_c == parts) {
                ahead_c = 0;
                ahead_v += warps * kFewRows;
            }
            ahead_s = ahead_s + 1 == kFewStages ? 0 : ahead_s + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (VEC)
        for (int i = 0; i < kFewStages - 1; ++i) copy_part();
    int stage = 0;
    for (int64_t v0 = w0 * kFewRows; v0 < a.V; v0 += warps * kFewRows) {
        float z[kFewRows][NT] = {};
        if (VEC) {
            for (int p = 0; p < parts; ++p) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kFewStages - 2) : "memory");
                Vec<DT> x[kFewRows];
#pragma unroll
                for (int r = 0; r < kFewRows; ++r)
                    x[r] = *reinterpret_cast<const Vec<DT>*>(ring + stage * kFewStageBytes + r * 512 + lane * 16);
                stage = stage + 1 == kFewStages ? 0 : stage + 1;
                copy_part();
                const int64_t c = p * 256 + lane * 8;
                if (c >= a.D) continue;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const Vec<DT> q = *reinterpret_cast<const Vec<DT>*>(h + t * dpad + c);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int r = 0; r < kFewRows; ++r) z[r][t] = fmaf(Elem<DT>::to_f(x[r].v[j]), Elem<DT>::to_f(q.v[j]), z[r][t]);
                }
            }
        } else {
            const T* w[kFewRows];
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) w[r] = static_cast<const T*>(a.weight) + min(v0 + r, a.V - 1) * a.ws;
#pragma unroll 4
            for (int64_t c = lane; c < a.D; c += 32)
#pragma unroll
                for (int r = 0; r < kFewRows; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t) z[r][t] = fmaf(Elem<DT>::to_f(w[r][c]), Elem<DT>::to_f(h[t * dpad + c]), z[r][t]);
        }
        // The four rows' sums over the lanes, the rows dealt out on the way: lanes 8r to 8r + 7 end with
        // row r, and keep the statistics of the rows they have had.
        const bool up = lane & 16, right = lane & 8;
        const int64_t v = v0 + (lane >> 3);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float a0 = up ? z[2][t] : z[0][t], a1 = up ? z[3][t] : z[1][t];
            const float b0 = a0 + __shfl_xor_sync(0xffffffffu, up ? z[0][t] : z[2][t], 16);
            const float b1 = a1 + __shfl_xor_sync(0xffffffffu, up ? z[1][t] : z[3][t], 16);
            float x = (right ? b1 : b0) + __shfl_xor_sync(0xffffffffu, right ? b0 : b1, 8);
#pragma unroll
            for (int o = 4; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (v < a.V) {
                if (y[t] == v && (lane & 7) == 0) a.ztarget[t] = x;
                st[t] = join_pairs(st[t], x == -INFINITY ? make_float2(-INFINITY, 0.f) : make_float2(x, 1.f));
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int o = 8; o <= 16; o *= 2)
            st[t] = join_pairs(st[t], make_float2(__shfl_xor_sync(0xffffffffu, st[t].x, o), __shfl_xor_sync(0xffffffffu, st[t].y, o)));
#pragma unroll
    for (int t = 0; t < NT; ++t)
        if (lane == 0) joined[warp][t] = st[t];
    __syncthreads();
    if (tid < NT && tid < a.T) {
        float2 q = joined[0][tid];
        for (int w = 1; w < kFewWarps; ++w) q = join_pairs(q, joined[w][tid]);
        a.part[static_cast<int64_t>(tid) * gridDim.x + blockIdx.x] = q;
    }
}

__global__ void __launch_bounds__(256) few_join_kernel(FewArgs a)
{
    __shared__ float2 sh[256];
    const int t = blockIdx.x, tid = threadIdx.x;
    wait_for_previous();
    const int64_t y = load_id(a.targets, a.id_bytes, t);
    if (y < 0 || y >= a.V || y == a.ignore) {
        if (tid == 0) {
            if (y != a.ignore) atomicOr(a.status, kErrId);
            a.loss[t] = 0.f;
            a.lse[t] = 0.f;
        }
        return;
    }
    float2 q = make_float2(-INFINITY, 0.f);
    for (int i = tid; i < a.ctas; i += 256) q = join_pairs(q, a.part[static_cast<int64_t>(t) * a.ctas + i]);
    sh[tid] = q;
    for (int o = 128; o; o >>= 1) {
        __syncthreads();
        if (tid < o) sh[tid] = join_pairs(sh[tid], sh[tid + o]);
    }
    if (tid == 0) {
        const float l = sh[0].x + logf(sh[0].y);
        a.lse[t] = l;
        a.loss[t] = l - a.ztarget[t];
    }
}

bool few_tokens(int64_t T, int64_t D)
{
    return T <= kFewTokens && T * round_up(D, 8) <= kFewElements;
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
    if (c.T >= kMaxTokens) return fail(DDP_E_INVAL, "%s: ntokens = %lld is too large", fn, static_cast<long long>(c.T));
    if (c.V < 1 || c.V >= kMaxVocab) return fail(DDP_E_INVAL, "%s: vocab = %lld out of range", fn, static_cast<long long>(c.V));
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

template <int DT, int NT> cudaError_t launch_few_as(const FewArgs& a, bool vec, cudaStream_t s)
{
    constexpr int kRing = kFewWarps * kFewStages * kFewStageBytes;
    const int smem = NT * static_cast<int>(round_up(a.D, 8)) * 2 + (vec ? kRing : 0);
    static std::atomic<bool> ready[ddp::kMaxDevices] = {};
    const int dev = ddp::current_device();
    if (dev < 0 || !ready[dev].load(std::memory_order_relaxed)) {
        for (auto k : {few_kernel<DT, NT, true>, few_kernel<DT, NT, false>}) {
            const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kFewElements + kRing);
            if (e != cudaSuccess) return e;
        }
        if (dev >= 0) ready[dev].store(true, std::memory_order_relaxed);
    }
    const cudaError_t e = launch_chained(vec ? few_kernel<DT, NT, true> : few_kernel<DT, NT, false>,
                                         dim3(static_cast<unsigned>(a.ctas)), kFewThreads, smem, s, a);
    return e != cudaSuccess ? e : launch_chained(few_join_kernel, dim3(static_cast<unsigned>(a.T)), 256, 0, s, a);
}
template <int DT> cudaError_t launch_few(const FewArgs& a, bool vec, cudaStream_t s)
{
    return a.T == 1 ? launch_few_as<DT, 1>(a, vec, s) : launch_few_as<DT, kFewTokens>(a, vec, s);
}

bool needs_copy(const Call& c) { return !aligned16(c.weight) || c.ws % 8 != 0; }

// gathers, and the weight's aligned copy where it needs one
cudaError_t launch_prep(PrepArgs& a, const Call& c, const Space& sp, char* w, int* status, cudaStream_t s, const void** weight, int64_t* ws)
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
    a.vec = c.D % 8 == 0 && c.hs % 8 == 0 && aligned16(c.hidden) && (!a.gh || (aligned16(a.gh) && a.ghs % 8 == 0));
    cudaError_t e = launch_chained(prep_kernel, dim3(static_cast<unsigned>((c.T + a.slab - 1) / a.slab)), kPrepThreads, 0, s, a);
    if (e != cudaSuccess) return e;
    *weight = c.weight;
    *ws = c.ws;
    if (needs_copy(c)) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(w + sp.weight);
        e = launch_chained(copy_weight_kernel, dim3(static_cast<unsigned>(8 * ddp::device_sm_count())), 256, 0, s,
                           static_cast<const uint16_t*>(c.weight), c.ws, c.V, c.D, dst, sp.dpad);
        *weight = dst;
        *ws = sp.dpad;
    }
    return e;
}

template <int DT> cudaError_t run_forward(const Call& c, const Space& sp, char* w, int* status, float* loss, float* lse, cudaStream_t s)
{
    if (few_tokens(c.T, c.D)) {
        FewArgs f{c.hidden, c.hs, c.weight, c.ws, c.V, c.D, c.targets, c.id_bytes, static_cast<int32_t>(c.T), c.ignore,
                  reinterpret_cast<float2*>(w + sp.part), reinterpret_cast<float*>(w + sp.ztarget), loss, lse, 0, status};
        const int64_t want = (c.V + kFewRows * kFewWarps - 1) / (kFewRows * kFewWarps);
        f.ctas = static_cast<int32_t>(std::min<int64_t>({want, ddp::device_sm_count(), kMaxFewCtas}));
        return launch_few<DT>(f, aligned16(c.weight) && c.ws % 8 == 0, s);
    }
    PrepArgs a{};
    a.loss = loss;
    a.lse_out = lse;
    const void* weight;
    int64_t ws;
    cudaError_t e = launch_prep(a, c, sp, w, status, s, &weight, &ws);
    if (e != cudaSuccess) return e;
    Batch batch{};
    batch.count = a.count;
    batch.status = status;
    Product p{};
    p.M = c.T; p.N = c.V; p.K = c.D;
    p.target = a.target;
    p.part = reinterpret_cast<float2*>(w + sp.part);
    p.tpad = sp.tpad;
    p.ztarget = reinterpret_cast<float*>(w + sp.ztarget);
    if (!set_product<DT, USE_STATS>(batch, p, a.out, sp.dpad, weight, ws)) return cudaErrorInvalidValue;
    e = launch_products<DT>(batch, s);
    if (e != cudaSuccess) return e;
    return launch_plain(combine_kernel<DT>, dim3(static_cast<unsigned>((c.T + kJoinRows - 1) / kJoinRows)), 32 * kJoinRows, s,
                        static_cast<const int32_t*>(a.count), static_cast<const int32_t*>(a.rows),
                          static_cast<const float2*>(p.part), sp.tpad, static_cast<int>(sp.ntiles),
                          static_cast<const float*>(p.ztarget), static_cast<const void*>(a.out), sp.dpad, weight, ws, c.D,
                          static_cast<const int32_t*>(a.target), loss, lse);
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
    if (DT == DDP_F16) {
        a.back = reinterpret_cast<float*>(w + sp.back);
        if (gw) a.out_w = reinterpret_cast<uint16_t*>(w + sp.hidden_w);
    }
    const void* weight;
    int64_t ws;
    cudaError_t e = launch_prep(a, c, sp, w, status, s, &weight, &ws);
    if (e != cudaSuccess) return e;
    // step i: dH and dW of piece i - 1, G of piece i
    for (int64_t i = 0; i <= sp.pieces; ++i) {
        Batch batch{};
        batch.count = a.count;
        batch.status = status;
        for (int64_t piece = i - 1; piece <= i; ++piece) {
            if (piece < 0 || piece >= sp.pieces) continue;
            const int64_t v0 = piece * sp.piece, words = std::min(sp.piece, c.V - v0);
            const char* wp = static_cast<const char*>(weight) + 2 * v0 * ws;
            Product p{};
            p.rows_cap = c.T;
            p.v0 = v0;
            p.target = a.target;
            p.lse = a.lse;
            p.ratio = a.ratio;
            p.g = w + sp.grad + (piece & 1) * sp.grad_bytes;
            p.gld = sp.piece;
            p.gmax = a.gmax;
            p.back = a.back;
            p.inv_scale = 1.f / g_scale<DT>();
            p.rows = a.rows;
            p.acc = reinterpret_cast<float*>(w + sp.acc);
            p.ald = sp.dpad;
            if (piece == i) {
                p.M = c.T; p.N = words; p.K = c.D;
                if (!set_product<DT, USE_GRAD>(batch, p, a.out, sp.dpad, wp, ws)) return cudaErrorInvalidValue;
                continue;
            }
            if (gh) {
                Product q = p;
                q.M = c.T; q.N = c.D; q.K = words;
                q.first = piece == 0;
                q.last = piece + 1 == sp.pieces;
                q.out = gh; q.os = ghs;
                q.vec = aligned16(gh) && ghs % 4 == 0;
                if (!set_product<DT, USE_DH>(batch, q, p.g, p.gld, wp, ws)) return cudaErrorInvalidValue;
            }
            if (gw) {
                Product q = p;
                q.M = words; q.N = c.D; q.K = c.T;
                q.out = gw; q.os = gws; q.out_f32 = gw_f32; q.accumulate = accumulate;
                q.vec = aligned16(gw) && gws % 4 == 0;
                if (!set_product<DT, USE_DW>(batch, q, p.g, p.gld, DT == DDP_F16 ? a.out_w : a.out, sp.dpad)) return cudaErrorInvalidValue;
            }
        }
        e = launch_products<DT>(batch, s);
        if (e == cudaSuccess && gh && i == sp.pieces) {
            const int64_t quads = c.T * (sp.dpad / 4);
            e = launch_plain(finish_kernel<DT>, dim3(static_cast<unsigned>(std::min<int64_t>((quads + 255) / 256, 4 * ddp::device_sm_count()))),
                             256, s, batch.job[USE_DH], static_cast<const int32_t*>(a.count));
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace ddplm

using namespace ddplm;

extern "C" ddp_status ddp_vocab_loss_workspace(int64_t ntokens, int64_t vocab, int64_t dim, int64_t piece,
                                               int32_t weight_aligned, int64_t* forward_bytes, int64_t* backward_bytes)
{
    const char* fn = "ddp_vocab_loss_workspace";
    if (!forward_bytes || !backward_bytes) return ddp::fail(DDP_E_INVAL, "%s: an output is NULL", fn);
    if (ntokens < 0 || ntokens >= kMaxTokens || vocab < 1 || vocab >= kMaxVocab || dim < 1 ||
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
