// One AdamW step over many tensors, with moments in 32 or in 8 bits.
//
//   c = min(1, max_norm / (norm / S + 1e-6)) / S,   g' = c g
//   m <- b1 m + (1 - b1) g',   v <- b2 v + (1 - b2) g'^2
//   p <- p - (lr wd p + lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)),   copy <- round(p)
//
// Moments in 8 bits: 256 values of a tensor share a scale s and are e4m3 multiples of it, m itself
// and, for v, its square root (whose range in a block is half as many binades); s puts the largest
// at 448.  Both are rounded up or down by chance, with the probabilities that keep the mean: an
// e4m3 step is 6 to 12% of a value, a second moment moves by 0.1% at a time, and to the nearest it
// would stay where it is for good (a simulation whose gradients change their sizes after 3000 steps
// has sqrt(v) off by a factor of 2.9 (rms) 3000 steps later, by 1.5 in this form and in fp32).  The
// bits of chance are a counter's, mixed by splitmix64 (Steele, Lea and Flood, 2014): the same seed
// and step give the same ones.  A second moment that is not zero is never held as zero.
//
// A warp takes 256 values at a time, a lane eight in a row, so that the maximum behind a scale
// needs no barrier; nothing is read twice, and the clip costs no pass.  Two CTAs share an SM: with
// three the registers spill.
//
// Measured on a GB300 (graph replays).  32 bits, HBM-bound: 334M fp32 parameters with bf16 copies
// 1.56 ms (10.0 GB, 6.4 TB/s, 0.94 of the copy; three CTAs an SM 1.64, a ring as in 8 bits 1.69);
// 124M bf16 parameters and gradients 427 us (6.4 TB/s); 292M fp32 off boundaries 1.26 ms (6.5 TB/s, as
// on them), with bf16 copies 1.39; 0.3M in 17 tensors 6.2 us.  8 bits, bound by instructions (590 a lane and block of 256 before the
// roots and quotients were rounded exactly: 123 for the codes, 91 for conversions, 76 for the step,
// 66 for chances and scales, the rest the ring's): 124M fp32 parameters with bf16 copies 420 us
// (5.3 TB/s; three slots 508), bf16 ones without copies 396 us (3.1 TB/s; 312 with the hardware's
// roots and a product for each quotient, whose codes differ for a few values in a million), 14M bf16
// off boundaries 58 us (49).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cuda_fp8.h>

#include "lm_common.cuh"

namespace ddplm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerSm = 2;   // CTAs on an SM
constexpr int kBlock = DDP_ADAMW_BLOCK;
constexpr int kEach = kBlock / 32;   // values of a lane
static_assert(kEach == 8, "a lane's values are two vectors of fp32");

constexpr float kE4m3Max = 448.f;

struct StepArgs {
    const ddp_adamw_tensor* tensors;
    const int64_t* first_block;
    int32_t ntensors;
    int64_t nblocks;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t* state;   // the steps taken; CTAs of this step that are done
    const float *lr_at, *norm;
    float lr, b1, b2, one_b1, one_b2, log_b1, log_b2, eps, inv_scale, max_norm;
    uint64_t seed;
    float one;   // 1, which the compiler does not know
};

// What every value's step takes from the call: the same in all threads.
struct Common {
    float g;         // times a gradient
    float lr;
    float step;      // lr / (1 - b1^t)
    float root;      // 1 / sqrt(1 - b2^t)
    int64_t t;
    bool skip;
};
__device__ __forceinline__ Common common_of(const StepArgs& a)
{
    Common c;
    c.t = a.state[0] + 1;
    c.lr = a.lr_at ? *a.lr_at : a.lr;
    c.g = a.inv_scale;
    c.skip = false;
    if (a.norm) {
        // (operations of their own: codes in 8 bits depend on each rounding)
        const float norm = __fmul_rn(*a.norm, a.inv_scale);
        c.skip = !(fabsf(norm) < INFINITY);
        const float ratio = __fdiv_rn(a.max_norm, __fadd_rn(norm, 1e-6f));
        c.g *= ratio > 1.f ? 1.f : ratio;
    }
    // 1 - b^t without the cancellation at small t
    const float t = static_cast<float>(c.t);
    c.step = c.lr / -expm1f(t * a.log_b1);
    c.root = 1.f / sqrtf(-expm1f(t * a.log_b2));
    return c;
}

// Off by a unit in the last place.
__device__ __forceinline__ float root_of(float x)
{
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Off by two units in the last place; 0 for what is below 2^-126 and for a divisor above 2^126.
__device__ __forceinline__ float quotient(float x, float y)
{
    float r;
    asm("div.approx.ftz.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// ---------------------------------------------------------------------------
// eight values a lane
// ---------------------------------------------------------------------------
// A lane works on values 8 lane to 8 lane + 7 of a block.  How the warp gets them from memory and puts them back follows
// from where the block lies:
//   WHOLE    256 values on a 16-byte boundary: vectors;
//   SHIFTED  256 values off a boundary (tensors packed tight), others of the tensor before and behind them: the vectors
//            that cover them, whose words the lanes pass on to their neighbours.  The covering vectors hold up to 14
//            bytes of the values beside the block as well, which other warps may be stepping; they are not used;
//   STRIDED  a tensor's first block off a boundary, its last block: single values, lane + 32 j, exchanged through 1 KB of
//            shared memory of the warp.
enum Mode { WHOLE, SHIFTED, STRIDED };

// skip: bytes of the block's first value behind a boundary, the same for all of a tensor's blocks
__device__ __forceinline__ Mode mode_of(int skip, bool whole, bool inside)
{
    return skip == 0 ? (whole ? WHOLE : STRIDED) : inside ? SHIFTED : STRIDED;
}

// Values as they lie in memory.
struct Raw {
    uint32_t r[8];      // WHOLE, SHIFTED: two vectors of fp32, or one of 16 bits; STRIDED: a value each
    uint32_t more[4];   // SHIFTED, lane 31: the vector behind
};

template <typename T> __device__ __forceinline__ void load_strided(Raw& x, const T* p, int n, int lane)
{
#pragma unroll
    for (int j = 0; j < kEach; ++j) x.r[j] = lane + 32 * j < n ? p[lane + 32 * j] : T(0);
}

// Copies the vectors that hold a block, asynchronously, all lanes together.
__device__ __forceinline__ void fetch_block(uint32_t to, const char* p, bool wide, Mode mode, int lane)
{
    if (mode == STRIDED) return;   // (loaded where it is used: the ends of tensors)
    const char* q = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t{15}) + 16 * lane;
    copy16(to + 16 * lane, q);
    if (wide) copy16(to + 512 + 16 * lane, q + 512);
    if (mode == SHIFTED && lane == 31) copy16(to + (wide ? 1024 : 512), q + (wide ? 528 : 16));
}
__device__ __forceinline__ const void* vectors_of(const void* p) { return reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t{15}); }
// p: the block's first value in memory; vectors: those that hold the block, there or in the ring; n: its values
__device__ __forceinline__ void load_raw(Raw& x, const void* vectors, const void* p, bool wide, Mode mode, int n, int lane)
{
    if (mode == STRIDED) {
        if (wide) load_strided(x, static_cast<const uint32_t*>(p), n, lane);
        else load_strided(x, static_cast<const uint16_t*>(p), n, lane);
        return;
    }
    const uint4* q = static_cast<const uint4*>(vectors);
    if (wide) {
        const uint4 a = q[2 * lane], b = q[2 * lane + 1];
        x.r[0] = a.x, x.r[1] = a.y, x.r[2] = a.z, x.r[3] = a.w, x.r[4] = b.x, x.r[5] = b.y, x.r[6] = b.z, x.r[7] = b.w;
    } else {
        const uint4 a = q[lane];
        x.r[0] = a.x, x.r[1] = a.y, x.r[2] = a.z, x.r[3] = a.w;
    }
    if (mode == SHIFTED && lane == 31) {
        const uint4 c = q[wide ? 64 : 32];
        x.more[0] = c.x, x.more[1] = c.y, x.more[2] = c.z, x.more[3] = c.w;
    }
}

// The words of a SHIFTED block's lane: from `words` of them, word A on, and the next lane's.
template <int A, int WORDS> __device__ __forceinline__ void words_from(uint32_t (&to)[WORDS + 1], const Raw& x, int lane)
{
    uint32_t w[WORDS + 4];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = x.r[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[WORDS + i] = i <= A ? __shfl_down_sync(0xffffffffu, x.r[i], 1) : 0u;
        if (lane == 31) w[WORDS + i] = x.more[i];
    }
#pragma unroll
    for (int i = 0; i <= WORDS; ++i) to[i] = w[min(i + A, WORDS + 3)];
}
template <int WORDS> __device__ __forceinline__ void shifted_words(uint32_t (&to)[WORDS + 1], const Raw& x, int skip_words, int lane)
{
    switch (skip_words) {
        case 0: words_from<0, WORDS>(to, x, lane); break;
        case 1: words_from<1, WORDS>(to, x, lane); break;
        case 2: words_from<2, WORDS>(to, x, lane); break;
        default: words_from<3, WORDS>(to, x, lane); break;
    }
}

__device__ __forceinline__ float low_as_float(uint32_t r, int dtype)
{
    return dtype == DDP_BF16 ? __uint_as_float(r << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(r)));
}
__device__ __forceinline__ void pairs_to_floats(float (&f)[kEach], const uint32_t* r, int dtype)
{
    if (dtype == DDP_BF16) {
#pragma unroll
        for (int j = 0; j < kEach / 2; ++j) {
            f[2 * j] = __uint_as_float(r[j] << 16);
            f[2 * j + 1] = __uint_as_float(r[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kEach / 2; ++j) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&r[j]));
            f[2 * j] = x.x;
            f[2 * j + 1] = x.y;
        }
    }
}

// A lane's eight values.  skip: bytes of the block's first value behind a boundary.
__device__ __forceinline__ void to_floats(float (&f)[kEach], const Raw& x, int dtype, Mode mode, int skip, float* room, int lane)
{
    if (mode == STRIDED) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kEach; ++j) room[lane + 32 * j] = dtype == DDP_F32 ? __uint_as_float(x.r[j]) : low_as_float(x.r[j], dtype);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kEach; j += 4) {
            const float4 q = reinterpret_cast<const float4*>(room)[2 * lane + j / 4];
            f[j] = q.x, f[j + 1] = q.y, f[j + 2] = q.z, f[j + 3] = q.w;
        }
    } else if (dtype == DDP_F32) {
        if (mode == SHIFTED) {
            uint32_t w[9];
            shifted_words<8>(w, x, skip >> 2, lane);
#pragma unroll
            for (int j = 0; j < kEach; ++j) f[j] = __uint_as_float(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kEach; ++j) f[j] = __uint_as_float(x.r[j]);
        }
    } else if (mode == SHIFTED) {
        uint32_t w[5];
        shifted_words<4>(w, x, skip >> 2, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 8 * (skip & 2));
        pairs_to_floats(f, w, dtype);
    } else {
        pairs_to_floats(f, x.r, dtype);
    }
}

__device__ __forceinline__ uint32_t low_of_float(float f, int dtype)
{
    return dtype == DDP_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f)) : __half_as_ushort(__float2half_rn(f));
}
__device__ __forceinline__ uint32_t pair_of_floats(float a, float b, int dtype)
{
    if (dtype == DDP_BF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&x);
    }
    const __half2 x = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
}

// The other way: the words of a lane's covering vectors, from its own and the lane before's.  w[0] is the last word of
// those before word -A (for halves of words).
template <int A, int WORDS> __device__ __forceinline__ void words_to(uint32_t (&to)[WORDS + 1], const uint32_t (&own)[WORDS], int lane)
{
    uint32_t w[WORDS + 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = i >= 3 - A ? __shfl_up_sync(0xffffffffu, own[WORDS - 4 + i], 1) : 0u;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[4 + i] = own[i];
#pragma unroll
    for (int i = 0; i <= WORDS; ++i) to[i] = w[3 - A + i];
}
template <int WORDS> __device__ __forceinline__ void covering_words(uint32_t (&to)[WORDS + 1], const uint32_t (&own)[WORDS], int skip_words, int lane)
{
    switch (skip_words) {
        case 0: words_to<0, WORDS>(to, own, lane); break;
        case 1: words_to<1, WORDS>(to, own, lane); break;
        case 2: words_to<2, WORDS>(to, own, lane); break;
        default: words_to<3, WORDS>(to, own, lane); break;
    }
}

__device__ __forceinline__ void store(void* p, int dtype, Mode mode, int n, const float (&f)[kEach], float* room, int lane)
{
    if (mode == STRIDED) {
        __syncwarp();
        reinterpret_cast<float4*>(room)[2 * lane] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(room)[2 * lane + 1] = make_float4(f[4], f[5], f[6], f[7]);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = lane + 32 * j;
            if (i >= n) continue;
            if (dtype == DDP_F32) static_cast<float*>(p)[i] = room[i];
            else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(low_of_float(room[i], dtype));
        }
        return;
    }
    uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t{15});
    const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    if (dtype == DDP_F32) {
        uint32_t own[8], w[9];
#pragma unroll
        for (int j = 0; j < kEach; ++j) own[j] = __float_as_uint(f[j]);
        if (mode == WHOLE) {
            q[2 * lane] = make_uint4(own[0], own[1], own[2], own[3]);
            q[2 * lane + 1] = make_uint4(own[4], own[5], own[6], own[7]);
            return;
        }
        const int a = skip >> 2;   // 1 to 3
        covering_words<8>(w, own, a, lane);
        if (lane) q[2 * lane] = make_uint4(w[1], w[2], w[3], w[4]);
        q[2 * lane + 1] = make_uint4(w[5], w[6], w[7], w[8]);
        // the block's ends, in vectors that are not its own alone
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            if (lane == 0 && j < 4 - a) static_cast<uint32_t*>(p)[j] = own[j];
            if (lane == 31 && j < a) static_cast<uint32_t*>(p)[kBlock - 1 - j] = own[7 - j];
        }
    } else {
        uint32_t own[4], w[5];
#pragma unroll
        for (int j = 0; j < 4; ++j) own[j] = pair_of_floats(f[2 * j], f[2 * j + 1], dtype);
        if (mode == WHOLE) {
            q[lane] = make_uint4(own[0], own[1], own[2], own[3]);
            return;
        }
        const int h = skip >> 1;   // values before the block in its first vector, 1 to 7
        covering_words<4>(w, own, skip >> 2, lane);
        if (skip & 2) {
#pragma unroll
            for (int j = 3; j >= 0; --j) w[j + 1] = __funnelshift_r(w[j], w[j + 1], 16);
        }
        if (lane) q[lane] = make_uint4(w[1], w[2], w[3], w[4]);
#pragma unroll
        for (int j = 0; j < 7; ++j) {
            if (lane == 0 && j < 8 - h) static_cast<uint16_t*>(p)[j] = static_cast<uint16_t>(own[j / 2] >> (16 * (j & 1)));
            if (lane == 31 && j < h) static_cast<uint16_t*>(p)[kBlock - 1 - j] = static_cast<uint16_t>(own[(7 - j) / 2] >> (16 * ((7 - j) & 1)));
        }
    }
}

// ---------------------------------------------------------------------------
// moments in 8 bits
// ---------------------------------------------------------------------------
// Two values in one instruction.
struct Two {
    uint64_t v;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit Two(float a) : Two(a, a) {}
    __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Two operator*(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two operator+(Two a, Two b)
{
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The square roots of v = (v0, v1), from the hardware's reciprocal one and its remainder (Markstein, 1990): rounded once from
// 2^-102 on, where the remainder is exact (compared for every normal number), off by an ulp or two in some below.
__device__ __forceinline__ Two roots_of(Two v, float v0, float v1)
{
    float y0, y1;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y0) : "f"(v0));
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y1) : "f"(v1));
    // (0, infinity and NaN stand for themselves)
    const Two y(v0 > 0.f && v0 < INFINITY ? y0 : 1.f, v1 > 0.f && v1 < INFINITY ? y1 : 1.f);
    const Two g = v * y;
    const Two e = fma2(g, g * Two(-1.f), v);
    float e0, e1;
    e.get(e0, e1);
    return fma2(Two(v0 < INFINITY ? e0 : 0.f, v1 < INFINITY ? e1 : 0.f), y * Two(0.5f), g);
}

__host__ __device__ __forceinline__ uint64_t mixed(uint64_t z)
{
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;

__device__ __forceinline__ float2 of_codes(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    return __half22float2(__half2(h));
}

__device__ __forceinline__ void from_codes(Two (&f)[kEach / 2], uint2 q, float scale)
{
#pragma unroll
    for (int j = 0; j < kEach / 2; ++j) {
        const float2 x = of_codes((j < 2 ? q.x : q.y) >> (16 * (j & 1)) & 0xffffu);
        f[j] = Two(x.x, x.y) * Two(scale);
    }
}

// The larger magnitude, where a NaN beats everything.
__device__ __forceinline__ float larger(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}
// The scale of a block, from each lane's values: a NaN or an infinity among them becomes the scale.
__device__ __forceinline__ float scale_of(const float (&f)[kEach])
{
    float top = larger(larger(larger(f[0], f[1]), larger(f[2], f[3])), larger(larger(f[4], f[5]), larger(f[6], f[7])));
    // (as whole numbers magnitudes are in the same order, NaN last)
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    const float s = top * (1.f / kE4m3Max);   // (a product by the rounded reciprocal is the format's own rule)
    return s < 0x1p-126f ? 0.f : s;   // (its reciprocal is finite; a block below that is held as zeros)
}

// Four values' 16 bits of chance each, with a half of the last behind them, 8 bits up: what is added below.
__device__ __forceinline__ void chances_of(uint32_t* to, uint64_t z)
{
    const uint32_t lo = static_cast<uint32_t>(z), hi = static_cast<uint32_t>(z >> 32);
    to[0] = __byte_perm(lo, 0x80u, 0x7104);
    to[1] = __byte_perm(lo, 0x80u, 0x7324);
    to[2] = __byte_perm(hi, 0x80u, 0x7104);
    to[3] = __byte_perm(hi, 0x80u, 0x7324);
}

// Codes of a lane's values, rounded by chance.  Times 2^-120 a multiple of the scale has its e4m3 exponent as its own,
// with e4m3's smallest numbers among fp32's subnormal ones, so that the code is bits 20 to 26 and the 20 bits below are the
// fraction of a step to which the chance is added; all of it is moved up by 4 to put the code into a byte.
// The largest, 14 steps of its binade, is off by 2 2^-24 of itself at most, and the largest chance is 2^-17 short of a step,
// so that no finite value gets past 448.
// All that decides a code is rounded to fp32 operation by operation, in the order that the declaration gives, so that the codes
// are those of any other program that does the same: an ulp would be a step of 6 to 12% for a few values in a million.
// FLOOR: what is not zero is held as the smallest code at least.
template <bool FLOOR> __device__ __forceinline__ uint2 to_codes(const float (&f)[kEach], float scale, const uint32_t (&chance)[kEach])
{
    const float inv = scale == 0.f ? 0.f : __frcp_rn(scale);
    float x[kEach];
#pragma unroll
    for (int j = 0; j < kEach; j += 2) {
        // the quotient, rounded once: a product with the reciprocal and its remainder (Markstein, 1990), which is exact for
        // values from 2^-101 on
        const Two y(f[j], f[j + 1]), q = y * Two(inv);
        (fma2(fma2(q, Two(-scale), y), Two(inv), q) * Two(0x1p-120f)).get(x[j], x[j + 1]);
    }
    uint32_t q[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        q[j] = __float_as_uint(x[j]) * 16u + chance[FLOOR ? j : j ^ 1];   // (a sign moves out at the top)
        if (FLOOR) q[j] = max(q[j], min(__float_as_uint(f[j]), 0x01000000u));   // (a root is above 2^-75, or zero)
        else q[j] |= __float_as_uint(f[j]) & 0x80000000u;
    }
    uint32_t r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        r[h] = __byte_perm(__byte_perm(q[4 * h], q[4 * h + 1], 0x0073), __byte_perm(q[4 * h + 2], q[4 * h + 3], 0x0073), 0x5410);
    return make_uint2(r[0], r[1]);
}

// ---------------------------------------------------------------------------
// the step
// ---------------------------------------------------------------------------
// The last tensor whose first block is `block` or before it.
__device__ __forceinline__ int tensor_of(const StepArgs& a, int64_t block)
{
    int lo = 0, hi = a.ntensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.first_block[mid] <= block) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The step is counted when every CTA has read the count.
__device__ __forceinline__ void count_step(const StepArgs& a, const Common& c)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const unsigned before = atomicInc(reinterpret_cast<unsigned*>(a.state + 1), gridDim.x - 1);
        if (before == gridDim.x - 1 && !c.skip) a.state[0] = c.t;
    }
}

// Moments in 32 bits.
__global__ void __launch_bounds__(kThreads, kPerSm) adamw_kernel(const __grid_constant__ StepArgs a)
{
    __shared__ __align__(16) float rooms[kWarps][kBlock];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* room = rooms[warp];
    wait_for_previous();
    allow_next();
    const Common c = common_of(a);
    // a contiguous slice for each CTA, whose warps take every eighth block of it
    const int64_t per = a.nblocks / gridDim.x, more = a.nblocks % gridDim.x;
    const int64_t b0 = per * blockIdx.x + min(static_cast<int64_t>(blockIdx.x), more), b1 = b0 + per + (blockIdx.x < more);
    if (!c.skip && b0 + warp < b1) {
        int k = tensor_of(a, b0 + warp);
        int64_t next = -1, left = 0;   // the tensor's last block and one; its values from the block on
        bool start = false;            // the tensor's first block
        const char* gp = nullptr;
        char *pp = nullptr, *cp = nullptr;
        int gd = 0, pd = 0, cd = 0;
        float decay = 0.f;
        for (int64_t block = b0 + warp; block < b1; block += kWarps) {
            if (block >= next) {
                while (a.first_block[k + 1] <= block) ++k;
                const ddp_adamw_tensor t = a.tensors[k];
                next = a.first_block[k + 1];
                const int64_t at = (block - a.first_block[k]) * kBlock;
                start = at == 0;
                left = t.grad ? t.numel - at : 0;
                gd = t.grad_dtype, pd = t.param_dtype, cd = t.copy_dtype;
                gp = static_cast<const char*>(t.grad) + at * (gd == DDP_F32 ? 4 : 2);
                pp = static_cast<char*>(t.param) + at * (pd == DDP_F32 ? 4 : 2);
                cp = t.copy ? static_cast<char*>(t.copy) + at * (cd == DDP_F32 ? 4 : 2) : nullptr;
                decay = c.lr * t.weight_decay;
            }
            if (left <= 0) continue;
            const bool whole = left >= kBlock, inside = !start && left >= kBlock + 8;
            const int n = whole ? kBlock : static_cast<int>(left);
            const int gskip = static_cast<int>(reinterpret_cast<uintptr_t>(gp) & 15), pskip = static_cast<int>(reinterpret_cast<uintptr_t>(pp) & 15);
            const Mode gm = mode_of(gskip, whole, inside), pm = mode_of(pskip, whole, inside);
            Raw graw, praw;
            load_raw(graw, vectors_of(gp), gp, gd == DDP_F32, gm, n, lane);
            load_raw(praw, vectors_of(pp), pp, pd == DDP_F32, pm, n, lane);
            float m[kEach], v[kEach], p[kEach], g[kEach];
            const float4* mp = static_cast<const float4*>(a.m) + block * (kBlock / 4) + 2 * lane;
            const float4* vp = static_cast<const float4*>(a.v) + block * (kBlock / 4) + 2 * lane;
#pragma unroll
            for (int j = 0; j < kEach; j += 4) {
                const float4 x = mp[j / 4], y = vp[j / 4];
                m[j] = x.x, m[j + 1] = x.y, m[j + 2] = x.z, m[j + 3] = x.w;
                v[j] = y.x, v[j + 1] = y.y, v[j + 2] = y.z, v[j + 3] = y.w;
            }
            to_floats(g, graw, gd, gm, gskip, room, lane);
            to_floats(p, praw, pd, pm, pskip, room, lane);
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const float x = g[j] * c.g;
                m[j] = fmaf(a.b1, m[j], a.one_b1 * x);
                v[j] = fmaf(a.b2, v[j], a.one_b2 * (x * x));
                // (one rounding at the parameter's size)
                p[j] -= fmaf(decay, p[j], quotient(c.step * m[j], fmaf(root_of(v[j]), c.root, a.eps)));
            }
            store(pp, pd, pm, n, p, room, lane);
            if (cp) store(cp, cd, mode_of(static_cast<int>(reinterpret_cast<uintptr_t>(cp) & 15), whole, inside), n, p, room, lane);
            float4* mo = static_cast<float4*>(a.m) + block * (kBlock / 4) + 2 * lane;
            float4* vo = static_cast<float4*>(a.v) + block * (kBlock / 4) + 2 * lane;
#pragma unroll
            for (int j = 0; j < kEach; j += 4) {
                mo[j / 4] = make_float4(m[j], m[j + 1], m[j + 2], m[j + 3]);
                vo[j / 4] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            }
            left -= kWarps * kBlock;
            start = false;
            gp += kWarps * kBlock * (gd == DDP_F32 ? 4 : 2);
            pp += kWarps * kBlock * (pd == DDP_F32 ? 4 : 2);
            if (cp) cp += kWarps * kBlock * (cd == DDP_F32 ? 4 : 2);
        }
    }
    count_step(a, c);
}

// Moments in 8 bits.  So few bytes a value leave too little on the way while a warp works on a block, so the blocks to come
// are copied into a ring of the warp's in shared memory, with what has to be known of them.
struct __align__(16) Slot {
    char g[1056], p[1056];   // 66 vectors: of fp32, off a boundary, 65
    char m[kBlock], v[kBlock];
    const char* gp;
    char *pp, *cp;
    float decay;
    uint32_t kinds;   // values (0: nothing to do) | gd << 9 | pd << 11 | cd << 13 | gm << 15 | pm << 17 | cm << 19
    float m_scale, v_scale;
};
constexpr int kSlots = 4;
struct WarpRoom {
    Slot slot[kSlots];
    float room[kBlock];
};

__global__ void __launch_bounds__(kThreads, kPerSm) adamw8_kernel(const __grid_constant__ StepArgs a)
{
    extern __shared__ __align__(16) char shared[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    WarpRoom& mine = reinterpret_cast<WarpRoom*>(shared)[warp];
    wait_for_previous();
    allow_next();
    const Common c = common_of(a);
    const int64_t per = a.nblocks / gridDim.x, more = a.nblocks % gridDim.x;
    const int64_t b0 = per * blockIdx.x + min(static_cast<int64_t>(blockIdx.x), more), b1 = b0 + per + (blockIdx.x < more);
    if (!c.skip && b0 + warp < b1) {
        // the block that is fetched next, and its tensor
        int64_t ahead = b0 + warp, next = -1, left = 0;   // next: the block behind the tensor's last; left: its values from here on
        int k = tensor_of(a, ahead);
        bool start = false;   // the tensor's first block
        const char* gp = nullptr;
        char *pp = nullptr, *cp = nullptr;
        uint32_t types = 0, gstep = 0, pstep = 0, cstep = 0;   // bytes from a block to the warp's next
        float decay = 0.f;
        const char* from = static_cast<const char*>(lane < 16 ? a.m : a.v) + ahead * kBlock + 16 * (lane & 15);
        auto fetch = [&](int at) {
            if (ahead < b1) {
                Slot& to = mine.slot[at];
                if (ahead >= next) {
                    while (a.first_block[k + 1] <= ahead) ++k;
                    const ddp_adamw_tensor t = a.tensors[k];
                    next = a.first_block[k + 1];
                    const int64_t skip = (ahead - a.first_block[k]) * kBlock;
                    start = skip == 0;
                    left = t.grad ? t.numel - skip : 0;
                    const int gs = t.grad_dtype == DDP_F32 ? 4 : 2, ps = t.param_dtype == DDP_F32 ? 4 : 2, cs = t.copy_dtype == DDP_F32 ? 4 : 2;
                    types = t.grad_dtype << 9 | t.param_dtype << 11 | t.copy_dtype << 13;
                    gp = static_cast<const char*>(t.grad) + skip * gs;
                    pp = static_cast<char*>(t.param) + skip * ps;
                    cp = t.copy ? static_cast<char*>(t.copy) + skip * cs : nullptr;
                    gstep = kWarps * kBlock * gs, pstep = kWarps * kBlock * ps, cstep = t.copy ? kWarps * kBlock * cs : 0;
                    decay = c.lr * t.weight_decay;
                }
                const bool whole = left >= kBlock, inside = !start && left >= kBlock + 8;
                const int n = whole ? kBlock : max(static_cast<int>(left), 0);
                const Mode gm = mode_of(reinterpret_cast<uintptr_t>(gp) & 15, whole, inside);
                const Mode pm = mode_of(reinterpret_cast<uintptr_t>(pp) & 15, whole, inside);
                const Mode cm = mode_of(reinterpret_cast<uintptr_t>(cp) & 15, whole, inside);
                if (lane == 0) {
                    to.gp = gp, to.pp = pp, to.cp = cp;
                    to.decay = decay;
                    to.kinds = n | types | gm << 15 | pm << 17 | cm << 19;
                }
                if (n > 0) {
                    fetch_block(smem_address(to.g), gp, (types >> 9 & 3) == DDP_F32, gm, lane);
                    fetch_block(smem_address(to.p), pp, (types >> 11 & 3) == DDP_F32, pm, lane);
                    copy16(smem_address(to.m) + 16 * lane, from);   // (m's 256 bytes, then v's)
                    if (lane < 2) copy4(smem_address(&to.m_scale) + 4 * lane, (lane ? a.v_scale : a.m_scale) + ahead);
                }
                ahead += kWarps;
                left -= kWarps * kBlock;
                start = false;
                gp += gstep;
                pp += pstep;
                cp += cstep;
                from += kWarps * kBlock;
            }
            copies_commit();
        };
#pragma unroll
        for (int i = 0; i < kSlots - 1; ++i) fetch(i);
        uint64_t counter = mixed(a.seed + static_cast<uint64_t>(c.t + 1) * kGolden) +
                           static_cast<uint64_t>((b0 + warp) * (kBlock / 4) + 2 * lane + 1) * kGolden;
        const Two b1s(a.b1), b2s(a.b2), one_b1(a.one_b1), one_b2(a.one_b2), coef(c.g), step(c.step), bias(c.root), eps(a.eps), one(a.one);
        int at = 0;
        for (int64_t block = b0 + warp; block < b1; block += kWarps, counter += kWarps * (kBlock / 4) * kGolden) {
            copies_wait<kSlots - 2>();
            __syncwarp();   // every lane's copies are there, and the slot before has been read
            fetch(at == 0 ? kSlots - 1 : at - 1);
            const Slot& now = mine.slot[at];
            at = at == kSlots - 1 ? 0 : at + 1;
            const uint32_t kinds = now.kinds;
            const int n = kinds & 511;
            if (n == 0) continue;
            const int gd = kinds >> 9 & 3, pd = kinds >> 11 & 3, cd = kinds >> 13 & 3;
            const Mode gm = static_cast<Mode>(kinds >> 15 & 3), pm = static_cast<Mode>(kinds >> 17 & 3), cm = static_cast<Mode>(kinds >> 19 & 3);
            float g[kEach], p[kEach], m[kEach], root[kEach];
            {
                Raw raw;
                load_raw(raw, now.g, now.gp, gd == DDP_F32, gm, n, lane);
                to_floats(g, raw, gd, gm, static_cast<int>(reinterpret_cast<uintptr_t>(now.gp) & 15), mine.room, lane);
                load_raw(raw, now.p, now.pp, pd == DDP_F32, pm, n, lane);
                to_floats(p, raw, pd, pm, static_cast<int>(reinterpret_cast<uintptr_t>(now.pp) & 15), mine.room, lane);
            }
            Two ms[kEach / 2], vs[kEach / 2];
            from_codes(ms, reinterpret_cast<const uint2*>(now.m)[lane], now.m_scale);
            from_codes(vs, reinterpret_cast<const uint2*>(now.v)[lane], now.v_scale);
            const Two decay2(-now.decay);
#pragma unroll
            for (int j = 0; j < kEach; j += 2) {
                const Two x = Two(g[j], g[j + 1]) * coef;
                // (times one: nvcc 13.0 makes a product and a sum of pairs one operation, their roundings given or not)
                const Two mn = fma2(b1s * ms[j / 2], one, one_b1 * x), vo = vs[j / 2];
                const Two vn = fma2(b2s * (vo * vo), one, one_b2 * (x * x));
                float v0, v1, d0, d1, s0, s1;
                mn.get(m[j], m[j + 1]);
                vn.get(v0, v1);
                roots_of(vn, v0, v1).get(root[j], root[j + 1]);
                fma2(Two(root[j], root[j + 1]), bias, eps).get(d0, d1);
                (step * mn).get(s0, s1);
                // (one rounding at the parameter's size)
                const Two was(p[j], p[j + 1]);
                (was + fma2(decay2, was, Two(-quotient(s0, d0), -quotient(s1, d1)))).get(p[j], p[j + 1]);
            }
            store(now.pp, pd, pm, n, p, mine.room, lane);
            if (now.cp) store(now.cp, cd, cm, n, p, mine.room, lane);
            uint32_t chance[kEach];
#pragma unroll
            for (int j = 0; j < kEach; j += 4) chances_of(chance + j, mixed(counter + (j / 4) * kGolden));
            const float sm = scale_of(m), sv = scale_of(root);
            static_cast<uint2*>(a.m)[block * (kBlock / 8) + lane] = to_codes<false>(m, sm, chance);
            static_cast<uint2*>(a.v)[block * (kBlock / 8) + lane] = to_codes<true>(root, sv, chance);
            if (lane < 2) (lane ? a.v_scale : a.m_scale)[block] = lane ? sv : sm;
        }
        copies_wait<0>();
    }
    count_step(a, c);
}

cudaError_t launch(const StepArgs& a, bool bits8, cudaStream_t s)
{
    constexpr int smem = kWarps * sizeof(WarpRoom);
    static std::atomic<bool> ready[ddp::kMaxDevices] = {};
    const int64_t most = static_cast<int64_t>(ddp::device_sm_count()) * kPerSm;
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((a.nblocks + kWarps - 1) / kWarps, most)));
    if (bits8) return launch_with_room(adamw8_kernel, ready, grid, kThreads, smem, smem, a, s);
    return launch_chained(adamw_kernel, dim3(grid), kThreads, 0, s, a);
}

}  // namespace
}  // namespace ddplm

extern "C" ddp_status ddp_adamw_step(const ddp_adamw_tensor* tensors, const int64_t* first_block, int32_t ntensors,
                                     int64_t nblocks, void* exp_avg, void* exp_avg_sq, float* exp_avg_scale,
                                     float* exp_avg_sq_scale, int32_t state_bits, int64_t* state, double lr,
                                     const float* lr_at, double beta1, double beta2, double eps, uint64_t seed,
                                     double grad_scale, const float* norm, double max_norm, void* stream)
{
    using namespace ddplm;
    using ddp::fail;
    const char* fn = "ddp_adamw_step";
    if (ntensors < 0) return fail(DDP_E_INVAL, "%s: ntensors = %d < 0", fn, ntensors);
    if (nblocks < 0) return fail(DDP_E_INVAL, "%s: nblocks = %lld < 0", fn, static_cast<long long>(nblocks));
    if (ntensors == 0 && nblocks > 0) return fail(DDP_E_INVAL, "%s: blocks without tensors", fn);
    if (state_bits != 8 && state_bits != 32) return fail(DDP_E_INVAL, "%s: state_bits %d is neither 8 nor 32", fn, state_bits);
    if (!state) return fail(DDP_E_INVAL, "%s: state is NULL", fn);
    if (nblocks > 0) {
        if (!tensors || !first_block) return fail(DDP_E_INVAL, "%s: a table is NULL", fn);
        if (!exp_avg || !exp_avg_sq) return fail(DDP_E_INVAL, "%s: a moment is NULL", fn);
        if (!aligned16(exp_avg) || !aligned16(exp_avg_sq)) return fail(DDP_E_INVAL, "%s: a moment is not 16-byte aligned", fn);
        if (state_bits == 8 && (!exp_avg_scale || !exp_avg_sq_scale)) return fail(DDP_E_INVAL, "%s: a scale is NULL", fn);
    }
    if (!lr_at && !(lr >= 0. && lr <= 3e38)) return fail(DDP_E_INVAL, "%s: lr = %g", fn, lr);
    if (!(beta1 >= 0. && beta1 < 1.)) return fail(DDP_E_INVAL, "%s: beta1 = %g is not in [0, 1)", fn, beta1);
    if (!(beta2 >= 0. && beta2 < 1.)) return fail(DDP_E_INVAL, "%s: beta2 = %g is not in [0, 1)", fn, beta2);
    // (a divisor below 2^-126 would be taken for 0)
    if (!(eps == 0. || (eps >= 0x1p-126 && eps <= 3e38))) return fail(DDP_E_INVAL, "%s: eps = %g", fn, eps);
    // (neither it nor its reciprocal overflows)
    if (!(grad_scale >= 1. / 3e38 && grad_scale <= 3e38)) return fail(DDP_E_INVAL, "%s: grad_scale = %g", fn, grad_scale);
    if (norm && !(max_norm >= 0.)) return fail(DDP_E_INVAL, "%s: max_norm = %g is negative or NaN", fn, max_norm);
    const StepArgs a{tensors, first_block, ntensors, nblocks, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, state,
                     lr_at, norm, static_cast<float>(lr), static_cast<float>(beta1), static_cast<float>(beta2),
                     static_cast<float>(1. - beta1), static_cast<float>(1. - beta2), static_cast<float>(std::log(beta1)),
                     static_cast<float>(std::log(beta2)), static_cast<float>(eps), static_cast<float>(1. / grad_scale),
                     max_norm > 3e38 ? INFINITY : static_cast<float>(max_norm), seed, 1.f};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch(a, state_bits == 8, s);
    if (e != cudaSuccess) return fail(DDP_E_CUDA, "%s: kernel launch failed: %s", fn, cudaGetErrorString(e));
    return ddp::ok();
}
