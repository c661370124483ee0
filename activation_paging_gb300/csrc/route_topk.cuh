// Top-k routing of one token by one warp, shared by the router and the fused
// route + count/rank kernel.
//
// Top-k routing over the experts (Megatron-LM pull 7342, "Validation and
// performance": top-k 8).  Selection compares the raw logits (an equal logit
// goes to the lower expert id) in k rounds of a warp arg-max built from two
// redux.sync reductions; lane j keeps the j-th winner.  Because the softmax
// denominator cancels in the renormalisation,
// w_j = exp(l_j - m) / sum_sel exp(l_i - m), with m the row maximum (= the
// first winner), so only k exponentials are evaluated.
#pragma once

#include <float.h>
#include <math.h>

#include "ap_common.cuh"

namespace ap {
namespace {

// Order-preserving map of a finite float to uint32 (larger float -> larger
// key); -0 is first turned into +0 so that the two compare equal, as floats do.
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// (ka, ea) before (kb, eb): larger key first, then the lower expert id.
__device__ __forceinline__ bool before(uint32_t ka, int ea, uint32_t kb, int eb)
{
    return ka > kb || (ka == kb && ea < eb);
}

// Each lane sorts its NV candidates (odd-even transposition, constant
// indices), then k rounds each take the warp-wide best head with two
// redux.sync reductions (max key, then min id among equal keys); the winning
// lane shifts its list.  All 32 lanes call it with their candidates (a lane
// without one holds key 0 and id kNoExpert); lane j < k receives the j-th
// winner's key and id.
constexpr int kNoExpert = 0x7fffffff;

template <int NV>
__device__ __forceinline__ void choose_rounds(uint32_t (&key)[NV], int (&ex)[NV], int k, int lane, uint32_t *my_key,
                                              int *my_e)
{
#pragma unroll
    for (int r = 0; r < NV; ++r) {
#pragma unroll
        for (int i = r & 1; i + 1 < NV; i += 2) {
            if (before(key[i + 1], ex[i + 1], key[i], ex[i])) {
                const uint32_t tk = key[i];
                key[i] = key[i + 1];
                key[i + 1] = tk;
                const int te = ex[i];
                ex[i] = ex[i + 1];
                ex[i + 1] = te;
            }
        }
    }
    *my_key = 0;
    *my_e = 0;
    for (int j = 0; j < k; ++j) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, key[0]);
        const int emin = __reduce_min_sync(0xffffffffu, key[0] == m ? ex[0] : kNoExpert);
        if (key[0] == m && ex[0] == emin) {
#pragma unroll
            for (int i = 0; i + 1 < NV; ++i) {
                key[i] = key[i + 1];
                ex[i] = ex[i + 1];
            }
            key[NV - 1] = 0u;
            ex[NV - 1] = kNoExpert;
        }
        if (lane == j) {
            *my_key = m;
            *my_e = emin;
        }
    }
}

// The softmax over the chosen logits (lane j < k holds the j-th, top is the
// largest of all).
__device__ __forceinline__ float chosen_weight(float logit, float top, int k, int lane)
{
    const float z = (lane < k) ? expf(logit - top) : 0.f;
    float s = z;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return __fdiv_rn(z, s);
}

// choose_rounds, with lane j's renormalised weight in *wt and the largest logit
// in every lane's *top.
template <int NV>
__device__ __forceinline__ void select_token(uint32_t (&key)[NV], int (&ex)[NV], int k, int lane, int *e, float *wt,
                                             float *top)
{
    uint32_t my_key;
    choose_rounds<NV>(key, ex, k, lane, &my_key, e);
    *top = key_value(__shfl_sync(0xffffffffu, my_key, 0));
    *wt = chosen_weight(key_value(my_key), *top, k, lane);
}

// The largest of the lanes' values (NaN aside).
__device__ __forceinline__ float reduce_max(float v)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// Shared memory of one warp for select_token_slots: (logit, id) pairs.
struct TopkSlots {
    float2 cand[kWarp + 2];
    float2 sel[kWarp];
};

// The choice of choose_rounds in about half the instructions for rows of 128 and more
// experts, with a little shared memory.  The k-th largest of the lanes' maxima
// bounds the k-th largest logit from below, so only logits that reach it can
// be chosen: little more than k of them as a rule.  They are moved to one lane
// each, ranked by counting, and put in rank order.  Where more than 32 reach
// it (ties, or many large logits in one lane) or fewer than k do (NaN,
// -infinity), the rounds above run instead.  Results are the rounds', bit
// for bit, for rows of numbers (infinities among them); of a row that holds NaN
// other experts may be chosen.  v[i][c]: the logit of expert (lane + 32 i) * VEC + c, -infinity
// beyond E.
// Lane j < k receives the j-th value and its id, every lane the
// largest value in *top.  The slots are free again after a __syncwarp().
template <int VEC, int N>
__device__ __forceinline__ void choose_token_slots(const float (&v)[N][VEC], int E, int k, int lane, TopkSlots &s,
                                                   int *e, float *value, float *top)
{
    float cur = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c) cur = fmaxf(cur, v[i][c]);
    const float first = reduce_max(cur);
    float least = first;
#pragma unroll 4
    for (int j = 1; j < k; ++j) {
        cur = cur == least ? -INFINITY : cur;
        least = reduce_max(cur);
    }
    int own = 0; // of this lane, then with those of the lanes below
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c) own += v[i][c] >= least;
    int upto = own;
#pragma unroll
    for (int off = 1; off < kWarp; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += o;
    }
    const int n = __shfl_sync(0xffffffffu, upto, kWarp - 1);
    if (least == -INFINITY || n < k || n > kWarp) { // warp-uniform
        uint32_t key[N * VEC];
        int ex[N * VEC];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const int id = (lane + kWarp * i) * VEC + c;
                key[i * VEC + c] = id < E ? order_key(v[i][c]) : 0u;
                ex[i * VEC + c] = id < E ? id : kNoExpert;
            }
        uint32_t my_key;
        choose_rounds<N * VEC>(key, ex, k, lane, &my_key, e);
        *value = key_value(my_key);
        *top = __shfl_sync(0xffffffffu, *value, 0);
        return;
    }
    float2 *at = s.cand + (upto - own);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c)
            if (v[i][c] >= least) *at++ = make_float2(v[i][c], __int_as_float((lane + kWarp * i) * VEC + c));
    if (lane == 0) s.cand[n] = make_float2(-INFINITY, 0.f);
    __syncwarp();
    const float2 mine = s.cand[lane];
    int rank = -1; // itself counts once
    for (int c = 0; c < n; c += 2) {
        const float4 o = *reinterpret_cast<const float4 *>(&s.cand[c]);
        rank += (o.x >= mine.x) + (o.z >= mine.x);
    }
    if (__reduce_add_sync(0xffffffffu, lane < n ? (unsigned)rank : 0u) != (unsigned)(n * (n - 1) / 2)) { // ties
        rank = 0;
        for (int c = 0; c < n; ++c) {
            const float2 o = s.cand[c];
            rank += o.x > mine.x || (o.x == mine.x && __float_as_int(o.y) < __float_as_int(mine.y));
        }
    }
    if (lane < n && rank < k) s.sel[rank] = mine;
    __syncwarp();
    const float2 chosen = s.sel[lane < k ? lane : 0];
    *e = __float_as_int(chosen.y);
    *value = chosen.x;
    *top = first;
}

// choose_token_slots, with lane j's renormalised weight.
template <int VEC, int N>
__device__ __forceinline__ void select_token_slots(const float (&v)[N][VEC], int E, int k, int lane, TopkSlots &s,
                                                   int *e, float *wt, float *top)
{
    float value;
    choose_token_slots<VEC, N>(v, E, k, lane, s, e, &value, top);
    *wt = chosen_weight(value, *top, k, lane);
    __syncwarp(); // the slots are free for the next token
}

// Loads one token's row and selects from it.
template <int NV>
__device__ __forceinline__ void route_token(const float *__restrict__ row, int E, int k, int lane, int *e, float *wt)
{
    uint32_t key[NV];
    int ex[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int ei = lane + kWarp * i;
        const bool ok = ei < E;
        key[i] = ok ? order_key(__ldcs(row + ei)) : 0u; // 0 sorts below every finite logit
        ex[i] = ok ? ei : kNoExpert;
    }
    float top;
    select_token<NV>(key, ex, k, lane, e, wt, &top);
}

} // namespace
} // namespace ap
