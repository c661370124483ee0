// The weights' update: norm of all gradients with its clipping factor, and an
// AdamW step over many tensors in one launch.
//
//   g' = scale g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p  = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// One pass: every element's parameter, gradient and moments are read once and
// written once, with nothing kept in between, so HBM bounds it.  The tensors'
// addresses travel with the launch (kernel parameters), so a captured graph
// keeps them and no table has to be copied to the GPU.  A warp takes 256
// elements, which is also what shares a scale of 8-bit moments.
//
// Moments in 8 bits: m = s_m c |c| with c in -127 .. 127, sqrt(v) = s_v c^2 with
// c in 0 .. 255, s from the block's largest.  The square law spends the codes
// where moments of a block lie: steps of 1.6% (0.8% of sqrt(v)) at the largest,
// 16% at a hundredth of it, down to 6e-5 (1.5e-5) of it.  Codes are rounded up or
// down at random (16 bits of a counter-based mix of seed, step, tensor and
// element): v moves by less than a code a step, and rounding to nearest would
// never let it move.  A positive v never gets code 0, so no division by eps alone
// comes from the coding.
// Up with the code's own fraction f (ROUND_CODES), the value's expectation is too
// large by s f (1 - f) a step, which is nothing for large codes; a steady m or
// sqrt(v) of 1e-3 of its block's largest is kept 0.2% and 0.6% too large, of 1e-4
// 24% and 20%, m of 1e-5 4.6 times.  With the value's place between the values of
// the two codes (ROUND_VALUES) the expectations of m and v are exact, but for v
// below code 1.  134 M elements, BF16 with masters: 368 us and 438.
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include <type_traits>

#include "ap_common.cuh"

namespace ap {
namespace {

constexpr int kUpThreads = 256;
constexpr int kUpWarps = kUpThreads / kWarp;
constexpr int kBlock = AP_ADAMW_BLOCK; // elements of a warp and of a scale
constexpr int kEach = kBlock / kWarp;  // 8 elements of a lane: 4 at 4 lane, 4 at 128 + 4 lane
static_assert(kEach == 8, "two vectors of four");
using bf16_t = __nv_bfloat16;

// The tensors of one launch: `first` is the number of blocks before each.
struct UpTensor {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
};
template <int CAP> struct UpTable {
    int count, base; // base: number of the first tensor
    uint32_t vec;    // all addresses allow vectors
    uint32_t first[CAP + 1];
    UpTensor t[CAP];
};
constexpr int kFew = 56, kMany = 440; // 4 and 32 KB of parameters

struct UpStep {
    float lr, one_b1, b1, one_b2, b2, eps, decay;
    float ln_b1[2], ln_b2[2]; // ln b as the sum of two
    uint32_t seed;
    const float *d_lr, *d_scale;
    const uint32_t *d_skip;
    int32_t *d_step;
    bool last; // of the step's launches
};

__device__ __forceinline__ void load4(const float *p, float (&x)[4])
{
    const float4 v = __ldcs(reinterpret_cast<const float4 *>(p));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load4(const bf16_t *p, float (&x)[4])
{
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float *p, const float (&x)[4])
{
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
}
__device__ __forceinline__ void store4(bf16_t *p, const float (&x)[4])
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    uint2 v;
    memcpy(&v.x, &a, 4);
    memcpy(&v.y, &b, 4);
    __stcs(reinterpret_cast<uint2 *>(p), v);
}
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16_t v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t *p, float v) { *p = __float2bfloat16_rn(v); }

// A lane's 8 elements of the block at `at` (n elements in all; vec: whole block, aligned).
template <typename E> __device__ __forceinline__ void load8(const E *p, int64_t at, int64_t n, bool vec, float (&x)[8])
{
    const int lane = (int)lane_id();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = at + h * (kBlock / 2) + lane * 4;
        if (vec) {
            float y[4];
            load4(p + i, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[h * 4 + j] = y[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[h * 4 + j] = i + j < n ? to_f(p[i + j]) : 0.f;
        }
    }
}
template <typename E> __device__ __forceinline__ void store8(E *p, int64_t at, int64_t n, bool vec, const float (&x)[8])
{
    const int lane = (int)lane_id();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = at + h * (kBlock / 2) + lane * 4;
        if (vec) {
            const float y[4] = {x[h * 4], x[h * 4 + 1], x[h * 4 + 2], x[h * 4 + 3]};
            store4(p + i, y);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < n) put(p + i + j, x[h * 4 + j]);
        }
    }
}

// The codes of the lane's 8 elements, four to a word.  Blocks begin at
// multiples of 256 codes and are padded to them, so words are aligned and whole.
__device__ __forceinline__ void load_codes(const void *p, int64_t at, uint32_t (&c)[2])
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(static_cast<const char *>(p) + at) + lane_id();
    c[0] = __ldcs(w);
    c[1] = __ldcs(w + kBlock / 8);
}
__device__ __forceinline__ void store_codes(void *p, int64_t at, const uint32_t (&c)[2])
{
    uint32_t *w = reinterpret_cast<uint32_t *>(static_cast<char *>(p) + at) + lane_id();
    __stcs(w, c[0]);
    __stcs(w + kBlock / 8, c[1]);
}
// Integers below 2^23 sit in the last bits of 2^23 plus them, so bytes become
// numbers, and numbers their integer parts, without the conversion unit (which
// six conversions an element keep as busy as HBM).
constexpr float kBig = 8388608.f; // 2^23
constexpr uint32_t kBigBits = 0x4b000000u;
__device__ __forceinline__ float byte_of(uint32_t w, int j) // byte j, not signed
{
    return __uint_as_float(__byte_perm(w, kBigBits, 0x7440 | j)) - kBig;
}
__device__ __forceinline__ float code_m(uint32_t w, int j) // c |c| of byte j (the caller flips the sign bits: c + 128)
{
    const float c = __uint_as_float(__byte_perm(w, kBigBits, 0x7440 | j)) - (kBig + 128.f);
    return c * fabsf(c);
}
__device__ __forceinline__ float code_v(uint32_t w, int j) // c^2
{
    const float c = byte_of(w, j);
    return c * c;
}
constexpr uint32_t kSigns = 0x80808080u;
// floor(x - 1) in the last bits
__device__ __forceinline__ uint32_t floor_bits(float x) { return __float_as_uint(__fadd_rd(x, kBig - 1.f)); }
// 1 and the low or high 16 bits as a fraction
__device__ __forceinline__ float low_fraction(uint32_t u) { return __uint_as_float((u << 7 & 0x7fff80u) | 0x3f800000u); }
__device__ __forceinline__ float high_fraction(uint32_t u) { return __uint_as_float((u >> 9 & 0x7fff80u) | 0x3f800000u); }
__device__ __forceinline__ uint32_t four_bytes(const uint32_t (&c)[8], int h)
{
    return __byte_perm(__byte_perm(c[4 * h], c[4 * h + 1], 0x0040), __byte_perm(c[4 * h + 2], c[4 * h + 3], 0x0040), 0x5410);
}

// The finalizer of MurmurHash3 (Appleby), a mixing of 32 bits.
__device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x85EBCA6Bu;
    x ^= x >> 13;
    x *= 0xC2B2AE35u;
    return x ^ x >> 16;
}
constexpr uint32_t kGolden = 0x9E3779B9u;

// Single instructions, within 2^-22 of the values.  The root takes numbers below
// the normal ones as they are: v is the gradients' square, so that v and sqrt(v)
// are positive together, eps = 0 included (134 M elements in 8 bits 367 us for 360
// with those as 0; a branch to that form where all are normal numbers: 366).  What
// divides (b, or a block's scale) is a normal number or counts as 0.
__device__ __forceinline__ float sqrt_fast(float x)
{
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sqrt_code(float x) // of codes: below 2^-126 it is 0
{
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float div_fast(float a, float b)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(b));
    return a * y;
}

// The code of x in units of its square (last byte; x <= the largest code's square), up from the root's floor where the
// fraction, 1 + that and half a place, is below the place of value(x) between those of the two squares.  The root may be off
// by a rounding: a code that is one too small for it goes up always, one too large never.
template <typename Fn> __device__ __forceinline__ uint32_t between_codes(float x, float fraction, Fn value)
{
    const float at = __fadd_rd(sqrt_code(x), kBig), c = at - kBig, low = c * c, high = low + (2.f * c + 1.f);
    const float place = fraction - (1.f - 0.5f / 65536.f);
    return __float_as_uint(at) + (place * (value(high) - value(low)) < value(x) - value(low));
}

// 1 - b^t from ln b: expm1 keeps its precision for few steps.
__device__ __forceinline__ float correction(const float (&ln_b)[2], float t)
{
    return -expm1f(fmaf(ln_b[0], t, ln_b[1] * t));
}

// The block's largest value from the lanes' (not negative); NaN and infinity are larger than all numbers.
__device__ __forceinline__ float block_max(float v)
{
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

template <int CAP> __device__ __forceinline__ int tensor_of(const UpTable<CAP> &tab, uint32_t b)
{
    int lo = 0, hi = tab.count - 1; // the last tensor whose first block is not after b, with blocks of its own
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (tab.first[mid] <= b)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// A lane's 8 elements of a block as they lie in memory.
template <typename E> struct Raw;
template <> struct Raw<float> {
    float4 w[2];
    __device__ __forceinline__ float at(int j) const
    {
        const float4 &x = w[j / 4];
        return j % 4 == 0 ? x.x : j % 4 == 1 ? x.y : j % 4 == 2 ? x.z : x.w;
    }
};
template <> struct Raw<bf16_t> {
    uint2 w[2];
    __device__ __forceinline__ float at(int j) const
    {
        const uint32_t x = j % 4 < 2 ? w[j / 4].x : w[j / 4].y;
        return __uint_as_float(j & 1 ? x & 0xffff0000u : x << 16);
    }
};
template <typename E> __device__ __forceinline__ void load_raw(const E *p, int64_t at, int64_t n, bool vec, Raw<E> &x)
{
    using Vec = decltype(x.w[0]);
    const int lane = (int)lane_id();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = at + h * (kBlock / 2) + lane * 4;
        if (vec) {
            x.w[h] = __ldcs(reinterpret_cast<std::remove_reference_t<Vec> *>(const_cast<E *>(p + i)));
        } else {
            E y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                put(y + j, 0.f);
                if (i + j < n) y[j] = p[i + j];
            }
            memcpy(&x.w[h], y, sizeof(y));
        }
    }
}
// What a kernel is made for: moments of 32 bits, or of 8 with either rounding.
enum Moments { k32, kCodes, kValues };
template <int BITS> constexpr bool kAheadOf = BITS != k32;
template <int BITS> constexpr int kUpBlocksOf = BITS == k32 ? 1 : 3;
// What a lane has of a block: parameters, gradients and moments.
template <typename P, typename G, int BITS> struct UpBlock {
    Raw<P> p;
    Raw<G> g;
    Raw<float> m, v;
    uint32_t cm[2], cv[2];
    float sm, sv;
    int i; // the tensor
    int64_t at;
    bool vec;
};

// The work word while a call runs: blocks that are done, and what the first block to ask found, which all blocks of all
// launches go by, since the word that skips a step may change at any time.
constexpr int kGoes = 1 << 30, kSkips = 1 << 29;

template <int CAP, typename P, typename G, bool MASTER, int BITS>
__global__ void __launch_bounds__(kUpThreads, kUpBlocksOf<BITS>) k_adamw(const __grid_constant__ UpTable<CAP> tab, const UpStep s)
{
    pdl_begin();
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    const int32_t taken = *s.d_step;
    const float scale = s.d_scale ? *s.d_scale : 1.f, lr = s.d_lr ? *s.d_lr : s.lr;
    const uint32_t blocks = tab.first[tab.count];
    using Q = std::conditional_t<MASTER, float, P>;
    using Block = UpBlock<Q, G, BITS>;
    uint32_t b = blockIdx.x * kUpWarps + wid;
    int i = tensor_of(tab, b);
    const auto load = [&](Block &x) { // block b
        while (b >= tab.first[i + 1]) ++i;
        const UpTensor &q = tab.t[i];
        x.i = i;
        x.at = (int64_t)(b - tab.first[i]) * kBlock;
        x.vec = tab.vec && x.at + kBlock <= q.n;
        load_raw(MASTER ? reinterpret_cast<const Q *>(q.master) : static_cast<const Q *>(q.param), x.at, q.n, x.vec, x.p);
        load_raw(static_cast<const G *>(q.grad), x.at, q.n, x.vec, x.g);
        if constexpr (BITS != k32) {
            load_codes(q.m, x.at, x.cm);
            load_codes(q.v, x.at, x.cv);
            x.sm = q.m_scale[x.at / kBlock];
            x.sv = q.v_scale[x.at / kBlock];
        } else {
            load_raw(static_cast<const float *>(q.m), x.at, q.n, x.vec, x.m);
            load_raw(static_cast<const float *>(q.v), x.at, q.n, x.vec, x.v);
        }
    };
    constexpr bool kAhead = kAheadOf<BITS>; // the next block is on its way while one is worked on
    Block next;
    if (b < blocks) load(next); // (on its way while the step's constants are formed)
    const int t = taken + 1;
    const float less = -(lr * s.decay); // (1 - lr decay as a factor would round the decay to multiples of 2^-24)
    const float rate = __fdiv_rn(lr, correction(s.ln_b1, (float)t));
    const float root = __frsqrt_rn(correction(s.ln_b2, (float)t));
    const uint32_t seeded = mix(s.seed + kGolden * (uint32_t)t);
    bool skips = !(fabsf(scale) < INFINITY);
    if (s.d_skip) { // (the same for all blocks)
        __shared__ int s_skips;
        if (threadIdx.x == 0) {
            const int mine = skips || *reinterpret_cast<const volatile uint32_t *>(s.d_skip) ? kSkips : kGoes;
            const int first = atomicCAS(s.d_step + 1, 0, mine);
            s_skips = (first ? first : mine) & kSkips;
        }
        __syncthreads();
        skips = s_skips != 0;
    }
    if (skips) b = blocks;
    while (b < blocks) {
        const Block x = next;
        b += gridDim.x * kUpWarps;
        if (kAhead && b < blocks) load(next);
        const UpTensor &q = tab.t[x.i];
        const int64_t n = q.n, at = x.at;
        const bool vec = x.vec;
        float p[8], m[8], v[8], r[8];
        if constexpr (BITS != k32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m[j] = code_m(x.cm[j / 4] ^ kSigns, j % 4) * x.sm;
                const float y = code_v(x.cv[j / 4], j % 4) * x.sv;
                v[j] = y * y;
            }
            if (at + kBlock > n) // what the codes behind the last element hold is of no account
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at + (j / 4) * (kBlock / 2) + lane * 4 + j % 4 >= n) m[j] = v[j] = 0.f;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m[j] = x.m.at(j);
                v[j] = x.v.at(j);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float g = x.g.at(j) * scale;
            m[j] = fmaf(s.b1, m[j], s.one_b1 * g);
            v[j] = fmaf(s.b2, v[j], s.one_b2 * g * g);
            r[j] = sqrt_fast(v[j]);
            const float at_p = x.p.at(j);
            p[j] = at_p + fmaf(less, at_p, -rate * div_fast(m[j], fmaf(r[j], root, s.eps)));
        }
        if constexpr (MASTER) store8(q.master, at, n, vec, p);
        store8(static_cast<P *>(q.param), at, n, vec, p);
        if constexpr (BITS == k32) {
            store8(static_cast<float *>(q.m), at, n, vec, m);
            store8(static_cast<float *>(q.v), at, n, vec, v);
        } else {
            float top_m = 0.f, top_r = 0.f; // (elements beyond n are 0; max that keeps NaN)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                top_m = __uint_as_float(max(__float_as_uint(top_m), __float_as_uint(fabsf(m[j]))));
                top_r = __uint_as_float(max(__float_as_uint(top_r), __float_as_uint(r[j])));
            }
            top_m = block_max(top_m);
            top_r = block_max(top_r);
            // a block with a value that is no number becomes NaN whole
            const float sm = top_m < INFINITY ? top_m * (1.f / (127.f * 127.f)) : NAN;
            const float sv = top_r < INFINITY ? top_r * (1.f / (255.f * 255.f)) : NAN;
            // (scales below the normal numbers, of moments below 2^-112, give codes of 0)
            const float im = sm >= FLT_MIN ? div_fast(1.f, sm) : 0.f, iv = sv >= FLT_MIN ? div_fast(1.f, sv) : 0.f;
            const uint32_t key = mix((uint32_t)(tab.base + x.i) + seeded);
            uint32_t cm[8], cv[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t e = (uint32_t)at + (j / 4) * (kBlock / 2) + lane * 4 + j % 4;
                const uint32_t u = mix(e * kGolden + key);
                const float xm = fabsf(m[j]) * im, xv = r[j] * iv;
                uint32_t c, d;
                if constexpr (BITS == kCodes) {
                    c = floor_bits(fminf(sqrt_code(xm) + low_fraction(u), 128.f));
                    d = floor_bits(fmaxf(fminf(sqrt_code(xv) + high_fraction(u), 256.f), 2.f));
                } else {
                    c = between_codes(fminf(xm, 127.f * 127.f), low_fraction(u), [](float q) { return q; });
                    d = between_codes(fminf(xv, 255.f * 255.f), high_fraction(u), [](float q) { return q * q; });
                    d = max(d & 255u, 1u);
                }
                cm[j] = m[j] < 0.f ? 0u - c : c; // (last byte)
                cv[j] = r[j] > 0.f ? d : 0u;
            }
            const uint32_t wm[2] = {four_bytes(cm, 0), four_bytes(cm, 1)}, wv[2] = {four_bytes(cv, 0), four_bytes(cv, 1)};
            store_codes(q.m, at, wm);
            store_codes(q.v, at, wv);
            if (lane == 0) {
                q.m_scale[at / kBlock] = sm;
                q.v_scale[at / kBlock] = sv;
            }
        }
        if (!kAhead && b < blocks) load(next);
    }
    // the last block of the last launch moves the step on; the work word is 0 again then
    if (s.last) {
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            if ((atomicAdd(s.d_step + 1, 1) & (kSkips - 1)) == (int)gridDim.x - 1) {
                if (!skips) s.d_step[0] = t;
                s.d_step[1] = 0;
            }
        }
    }
}

// Sums of squares as pairs of FP32: the sum, and what its additions rounded away.
struct Pair {
    float sum, rest;
};
__device__ __forceinline__ void add_to(Pair &a, float x)
{
    const float to = __fadd_rn(a.sum, x), back = __fsub_rn(to, a.sum);
    a.rest += __fadd_rn(__fsub_rn(a.sum, __fsub_rn(to, back)), __fsub_rn(x, back));
    a.sum = to;
}
__device__ __forceinline__ void add_lanes(Pair &a)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float s = __shfl_xor_sync(0xffffffffu, a.sum, off), r = __shfl_xor_sync(0xffffffffu, a.rest, off);
        add_to(a, s);
        a.rest += r;
    }
}
template <int WARPS> __device__ __forceinline__ void add_block(Pair &a) // (warp 0 receives it)
{
    __shared__ Pair s_sum[WARPS];
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    add_lanes(a);
    if (lane == 0) s_sum[wid] = a;
    __syncthreads();
    if (wid == 0) {
        a = lane < WARPS ? s_sum[lane] : Pair{0.f, 0.f};
        add_lanes(a);
    }
}

// The gradients' squares: four blocks of elements at a time, 8 of each a lane.
constexpr int kNormBlocks4 = 4;
template <int CAP, typename G>
__global__ void __launch_bounds__(kUpThreads) k_norm(const __grid_constant__ UpTable<CAP> tab, Pair *part)
{
    pdl_begin();
    const uint32_t blocks = tab.first[tab.count];
    uint32_t b = blockIdx.x * kUpWarps + threadIdx.x / kWarp;
    int i = tensor_of(tab, b);
    Pair a = {0.f, 0.f};
    for (; b < blocks; b += gridDim.x * kUpWarps) {
        while (b >= tab.first[i + 1]) ++i;
        const UpTensor &x = tab.t[i];
        const int64_t at = (int64_t)(b - tab.first[i]) * (kNormBlocks4 * kBlock), n = x.n;
        float g[kNormBlocks4][8];
        if (tab.vec && at + kNormBlocks4 * kBlock <= n) {
#pragma unroll
            for (int q = 0; q < kNormBlocks4; ++q) load8(static_cast<const G *>(x.grad), at + q * kBlock, n, true, g[q]);
        } else {
#pragma unroll
            for (int q = 0; q < kNormBlocks4; ++q) load8(static_cast<const G *>(x.grad), at + q * kBlock, n, false, g[q]);
        }
#pragma unroll
        for (int q = 0; q < kNormBlocks4; ++q) {
            float y = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) y = fmaf(g[q][j], g[q][j], y);
            add_to(a, y);
        }
    }
    add_block<kUpWarps>(a);
    if (threadIdx.x == 0) part[blockIdx.x] = a;
}

constexpr int kNormThreads = 1024;
__global__ void __launch_bounds__(kNormThreads) k_norm_finish(const Pair *part, int n, float max_norm, float *out)
{
    pdl_begin();
    Pair a = {0.f, 0.f};
    for (int i = threadIdx.x; i < n; i += kNormThreads) {
        const Pair p = part[i];
        add_to(a, p.sum);
        a.rest += p.rest;
    }
    add_block<kNormThreads / kWarp>(a);
    if (threadIdx.x == 0) {
        const float norm = __fsqrt_rn(a.sum < INFINITY ? a.sum + a.rest : a.sum);
        out[0] = norm;
        out[1] = !(norm < INFINITY) ? NAN : max_norm > 0.f && norm > max_norm ? __fdiv_rn(max_norm, norm) : 1.f;
    }
}

// The moments that 8-bit codes stand for.
template <typename O>
__global__ void __launch_bounds__(kUpThreads) k_moments(const void *m, const void *v, const float *m_scale, const float *v_scale,
                                                        int64_t blocks, O *m_out, O *v_out)
{
    pdl_begin();
    const int64_t step = (int64_t)gridDim.x * kUpWarps;
    for (int64_t b = (int64_t)blockIdx.x * kUpWarps + threadIdx.x / kWarp; b < blocks; b += step) {
        uint32_t cm[2], cv[2];
        load_codes(m, b * kBlock, cm);
        load_codes(v, b * kBlock, cv);
        const float sm = m_scale[b], sv = v_scale[b];
        float x[8], y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = code_m(cm[j / 4] ^ kSigns, j % 4) * sm;
            y[j] = code_v(cv[j / 4], j % 4) * sv;
            y[j] *= y[j];
        }
        store8(m_out, b * kBlock, blocks * kBlock, true, x);
        store8(v_out, b * kBlock, blocks * kBlock, true, y);
    }
}

// ---- host ------------------------------------------------------------------------

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool float_type(int32_t d) { return d == AP_DTYPE_BF16 || d == AP_DTYPE_F32; }
unsigned size_of(int32_t d) { return d == AP_DTYPE_BF16 ? 2 : 4; }
int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// Calls go(table) for tables of at most CAP tensors: tensors from `from` on.
template <int CAP> void fill(UpTable<CAP> &tab, const ap_adamw_tensor *t, int from, int to, unsigned psize, unsigned gsize,
                             bool grads_only)
{
    const int unit = grads_only ? kNormBlocks4 : 1; // blocks of elements that a warp takes at a time
    tab.count = to - from;
    tab.base = from;
    tab.vec = 1;
    uint32_t at = 0;
    for (int i = from; i < to; ++i) {
        const ap_adamw_tensor &x = t[i];
        tab.first[i - from] = at;
        at += (uint32_t)((blocks_of(x.n) + unit - 1) / unit);
        tab.t[i - from] = {x.param, x.grad, (float *)x.master, x.m, x.v, x.m_scale, x.v_scale, x.n};
        if (!x.n) continue;
        bool ok = aligned(x.grad, 4 * gsize);
        if (!grads_only) ok = ok && aligned(x.param, 4 * psize) && aligned(x.master, 16) && aligned(x.m, 16) && aligned(x.v, 16);
        if (!ok) tab.vec = 0;
    }
    tab.first[to - from] = at;
}

// The end of the launch that begins at tensor `from`: at most CAP tensors, and
// fewer than 2^31 blocks of elements.
int launch_end(const ap_adamw_tensor *t, int n, int from, int cap)
{
    int64_t at = 0;
    int i = from;
    for (; i < n && i - from < cap; ++i) {
        at += blocks_of(t[i].n);
        if (at > INT32_MAX - 65536 && i > from) break;
    }
    return i;
}

ap_status tensors_ok(const char *who, const ap_adamw_tensor *t, int32_t n)
{
    if (n < 0 || (n > 0 && !t)) return fail(AP_EINVAL, "%s: bad list of %d tensors", who, n);
    for (int i = 0; i < n; ++i) {
        if (t[i].n < 0 || t[i].n > (int64_t(1) << 38)) return fail(AP_EINVAL, "%s: tensor %d of %lld elements", who, i, (long long)t[i].n);
        if (t[i].n && !t[i].grad) return fail(AP_EINVAL, "%s: NULL pointer in tensor %d", who, i);
    }
    return AP_OK;
}

template <int CAP, typename P, typename G, bool MASTER, int BITS>
ap_status launch_adamw(const UpTable<CAP> &tab, const UpStep &s, cudaStream_t st)
{
    const auto kernel = k_adamw<CAP, P, G, MASTER, BITS>;
    static const int resident = resident_grid((const void *)kernel, kUpThreads);
    const int64_t want = ((int64_t)tab.first[tab.count] + kUpWarps - 1) / kUpWarps;
    launch(kernel, (int)(want < 1 ? 1 : want < resident ? want : resident), kUpThreads, 0, st, tab, s);
    AP_CHECK_LAUNCH("adamw_step launch");
    return AP_OK;
}

template <int CAP> ap_status adamw_launches(const ap_adamw_tensor *t, int32_t n, const ap_adamw_config &c, UpStep s, cudaStream_t st)
{
    int from = 0;
    do {
        const int to = launch_end(t, n, from, CAP);
        UpTable<CAP> tab;
        fill(tab, t, from, to, size_of(c.param_dtype), size_of(c.grad_dtype), false);
        s.last = to == n;
        ap_status r;
#define AP_ADAMW(P, G, M) \
    r = c.state_bits == 32 ? launch_adamw<CAP, P, G, M, k32>(tab, s, st)                  \
        : c.rounding == AP_ADAMW_ROUND_CODES ? launch_adamw<CAP, P, G, M, kCodes>(tab, s, st) \
                                             : launch_adamw<CAP, P, G, M, kValues>(tab, s, st)
        const bool g16 = c.grad_dtype == AP_DTYPE_BF16;
        if (c.param_dtype == AP_DTYPE_F32) {
            if (g16)
                AP_ADAMW(float, bf16_t, false);
            else
                AP_ADAMW(float, float, false);
        } else if (c.master) {
            if (g16)
                AP_ADAMW(bf16_t, bf16_t, true);
            else
                AP_ADAMW(bf16_t, float, true);
        } else if (g16)
            AP_ADAMW(bf16_t, bf16_t, false);
        else
            AP_ADAMW(bf16_t, float, false);
#undef AP_ADAMW
        if (r != AP_OK) return r;
        from = to;
    } while (from < n);
    return AP_OK;
}

constexpr int kNormBlocks = 1216; // of a launch, at most
int norm_launches(const ap_adamw_tensor *t, int32_t n)
{
    const int cap = n <= kFew ? kFew : kMany;
    int count = 0;
    for (int from = 0; from < n; ++count) from = launch_end(t, n, from, cap);
    return count > 0 ? count : 1;
}

template <int CAP>
ap_status norm_launch_all(const ap_adamw_tensor *t, int32_t n, int32_t dtype, float max_norm, float *out, Pair *part,
                          cudaStream_t st)
{
    int from = 0, parts = 0;
    do {
        const int to = launch_end(t, n, from, CAP);
        UpTable<CAP> tab;
        fill(tab, t, from, to, 4, size_of(dtype), true);
        const int64_t want = ((int64_t)tab.first[tab.count] + kUpWarps - 1) / kUpWarps;
        const int grid = (int)(want < 1 ? 1 : want < kNormBlocks ? want : kNormBlocks);
        if (dtype == AP_DTYPE_BF16)
            launch(k_norm<CAP, bf16_t>, grid, kUpThreads, 0, st, tab, part + parts);
        else
            launch(k_norm<CAP, float>, grid, kUpThreads, 0, st, tab, part + parts);
        AP_CHECK_LAUNCH("grad_norm launch");
        parts += grid;
        from = to;
    } while (from < n);
    launch(k_norm_finish, 1, kNormThreads, 0, st, part, parts, max_norm, out);
    AP_CHECK_LAUNCH("grad_norm finish launch");
    return AP_OK;
}

} // namespace
} // namespace ap

extern "C" ap_status ap_grad_norm_scratch_bytes(const ap_adamw_tensor *tensors, int32_t n, int64_t *bytes)
{
    using namespace ap;
    if (!bytes) return fail(AP_EINVAL, "grad_norm_scratch_bytes: NULL pointer");
    if (const ap_status s = tensors_ok("grad_norm_scratch_bytes", tensors, n); s != AP_OK) return s;
    *bytes = (int64_t)norm_launches(tensors, n) * kNormBlocks * 8;
    return AP_OK;
}

extern "C" ap_status ap_grad_norm(const ap_adamw_tensor *tensors, int32_t n, int32_t grad_dtype, float max_norm, float *out,
                                  void *scratch, int64_t scratch_bytes, void *stream)
{
    AP_NVTX_RANGE("ap_grad_norm");
    using namespace ap;
    if (const ap_status s = tensors_ok("grad_norm", tensors, n); s != AP_OK) return s;
    if (!float_type(grad_dtype)) return fail(AP_EINVAL, "grad_norm: type %d", grad_dtype);
    if (!out || !scratch) return fail(AP_EINVAL, "grad_norm: NULL pointer");
    if (!aligned(scratch, 16)) return fail(AP_EINVAL, "grad_norm: scratch not 16-byte aligned");
    const int64_t need = (int64_t)norm_launches(tensors, n) * kNormBlocks * 8;
    if (scratch_bytes < need)
        return fail(AP_EINVAL, "grad_norm: scratch of %lld bytes, %lld needed", (long long)scratch_bytes, (long long)need);
    for (int i = 0; i < n; ++i)
        if (!aligned(tensors[i].grad, size_of(grad_dtype))) return fail(AP_EINVAL, "grad_norm: tensor %d not aligned", i);
    Pair *part = static_cast<Pair *>(scratch);
    cudaStream_t st = (cudaStream_t)stream;
    return n <= kFew ? norm_launch_all<kFew>(tensors, n, grad_dtype, max_norm, out, part, st)
                     : norm_launch_all<kMany>(tensors, n, grad_dtype, max_norm, out, part, st);
}

extern "C" ap_status ap_adamw_step(const ap_adamw_tensor *tensors, int32_t n, const ap_adamw_config *cfg, void *stream)
{
    AP_NVTX_RANGE("ap_adamw_step");
    using namespace ap;
    if (!cfg) return fail(AP_EINVAL, "adamw_step: NULL config");
    const ap_adamw_config &c = *cfg;
    if (const ap_status s = tensors_ok("adamw_step", tensors, n); s != AP_OK) return s;
    if (!float_type(c.param_dtype) || !float_type(c.grad_dtype))
        return fail(AP_EINVAL, "adamw_step: types %d, %d", c.param_dtype, c.grad_dtype);
    if (c.state_bits != 8 && c.state_bits != 32) return fail(AP_EINVAL, "adamw_step: state_bits=%d", c.state_bits);
    if (c.rounding != AP_ADAMW_ROUND_CODES && c.rounding != AP_ADAMW_ROUND_VALUES)
        return fail(AP_EINVAL, "adamw_step: rounding=%u", c.rounding);
    if (c.master != 0 && (c.master != 1 || c.param_dtype != AP_DTYPE_BF16))
        return fail(AP_EINVAL, "adamw_step: master=%d with parameters of type %d", c.master, c.param_dtype);
    if (!(c.beta1 >= 0.0 && c.beta1 < 1.0 && c.beta2 >= 0.0 && c.beta2 < 1.0 && c.eps >= 0.0))
        return fail(AP_EINVAL, "adamw_step: beta1=%g beta2=%g eps=%g", c.beta1, c.beta2, c.eps);
    if (!c.d_step || !aligned(c.d_step, 4)) return fail(AP_EINVAL, "adamw_step: bad step words");
    for (int i = 0; i < n; ++i) {
        const ap_adamw_tensor &x = tensors[i];
        if (!x.n) continue;
        if (!x.param || !x.m || !x.v || (c.master && !x.master) || (c.state_bits == 8 && (!x.m_scale || !x.v_scale)))
            return fail(AP_EINVAL, "adamw_step: NULL pointer in tensor %d", i);
        if (!aligned(x.param, size_of(c.param_dtype)) || !aligned(x.grad, size_of(c.grad_dtype)) || !aligned(x.master, 4) ||
            !aligned(x.m, 4) || !aligned(x.v, 4) || !aligned(x.m_scale, 4) || !aligned(x.v_scale, 4))
            return fail(AP_EINVAL, "adamw_step: tensor %d not aligned", i);
    }
    UpStep s = {};
    s.lr = (float)c.lr;
    s.b1 = (float)c.beta1;
    s.b2 = (float)c.beta2;
    s.one_b1 = (float)(1.0 - c.beta1);
    s.one_b2 = (float)(1.0 - c.beta2);
    s.eps = (float)c.eps;
    s.decay = (float)c.weight_decay;
    for (int q = 0; q < 2; ++q) {
        const double ln = log(q ? c.beta2 : c.beta1); // -infinity at 0: the correction is 1
        float *to = q ? s.ln_b2 : s.ln_b1;
        to[0] = (float)ln;
        to[1] = ln > -INFINITY ? (float)(ln - (double)to[0]) : 0.f;
    }
    s.seed = c.seed;
    s.d_lr = c.d_lr;
    s.d_scale = c.d_scale;
    s.d_skip = c.d_skip;
    s.d_step = c.d_step;
    cudaStream_t st = (cudaStream_t)stream;
    return n <= kFew ? adamw_launches<kFew>(tensors, n, c, s, st) : adamw_launches<kMany>(tensors, n, c, s, st);
}

extern "C" ap_status ap_adamw_moments(const void *m, const void *v, const float *m_scale, const float *v_scale, int64_t n,
                                      int32_t out_dtype, void *m_out, void *v_out, void *stream)
{
    AP_NVTX_RANGE("ap_adamw_moments");
    using namespace ap;
    if (n < 0 || n % kBlock) return fail(AP_EINVAL, "adamw_moments: n=%lld", (long long)n);
    if (!float_type(out_dtype)) return fail(AP_EINVAL, "adamw_moments: type %d", out_dtype);
    if (n == 0) return AP_OK;
    if (!m || !v || !m_scale || !v_scale || !m_out || !v_out) return fail(AP_EINVAL, "adamw_moments: NULL pointer");
    if (!aligned(m, 4) || !aligned(v, 4) || !aligned(m_scale, 4) || !aligned(v_scale, 4) || !aligned(m_out, 4 * size_of(out_dtype)) ||
        !aligned(v_out, 4 * size_of(out_dtype)))
        return fail(AP_EINVAL, "adamw_moments: not aligned");
    const int64_t blocks = n / kBlock, want = (blocks + kUpWarps - 1) / kUpWarps, most = (int64_t)sm_count() * 8;
    const int grid = (int)(want < most ? want : most);
    cudaStream_t st = (cudaStream_t)stream;
    if (out_dtype == AP_DTYPE_BF16)
        launch(k_moments<bf16_t>, grid, kUpThreads, 0, st, m, v, m_scale, v_scale, blocks, (bf16_t *)m_out, (bf16_t *)v_out);
    else
        launch(k_moments<float>, grid, kUpThreads, 0, st, m, v, m_scale, v_scale, blocks, (float *)m_out, (float *)v_out);
    AP_CHECK_LAUNCH("adamw_moments launch");
    return AP_OK;
}
