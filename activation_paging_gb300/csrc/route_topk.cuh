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
// expert in *e and its renormalised weight in *wt, every lane the largest
// logit in *top.
constexpr int kNoExpert = 0x7fffffff;

template <int NV>
__device__ __forceinline__ void select_token(uint32_t (&key)[NV], int (&ex)[NV], int k, int lane, int *e, float *wt,
                                             float *top)
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
    uint32_t my_key = 0;
    int my_e = 0;
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
            my_key = m;
            my_e = emin;
        }
    }
    const float mv = key_value(__shfl_sync(0xffffffffu, my_key, 0)); // the largest logit
    const float z = (lane < k) ? expf(key_value(my_key) - mv) : 0.f;
    float s = z;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    *e = my_e;
    *wt = __fdiv_rn(z, s);
    *top = mv;
}

// The largest of the lanes' values (NaN aside).
__device__ __forceinline__ float reduce_max(float v)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// Shared memory of one warp for select_token_slots.
struct TopkSlots {
    float val[kWarp + 4];
    int id[kWarp];
    float sel_val[kWarp];
    int sel_id[kWarp];
};

// The same selection in about half the instructions for rows of 128 and more
// experts, with a little shared memory.  The k-th largest of the lanes' maxima
// bounds the k-th largest logit from below, so only logits that reach it can
// be chosen: little more than k of them as a rule.  They are moved to one lane
// each, ranked by counting, and put in rank order.  Where more than 32 reach
// it (ties, or many large logits in one lane) or fewer than k do (NaN,
// -infinity), the rounds above run instead.  Results are select_token's, bit
// for bit.  v[i][c]: the logit of expert (lane + 32 i) * VEC + c, -infinity
// beyond E.
template <int VEC, int N>
__device__ __forceinline__ void select_token_slots(const float (&v)[N][VEC], int E, int k, int lane, TopkSlots &s,
                                                   int *e, float *wt, float *top)
{
    float cur = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c) cur = fmaxf(cur, v[i][c]);
    const float first = reduce_max(cur);
    float least = first;
    for (int j = 1; j < k; ++j) {
        cur = cur == least ? -INFINITY : cur;
        least = reduce_max(cur);
    }
    uint32_t has[N][VEC];
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            has[i][c] = __ballot_sync(0xffffffffu, v[i][c] >= least);
            n += __popc(has[i][c]);
        }
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
        select_token<N * VEC>(key, ex, k, lane, e, wt, top);
        return;
    }
    int at = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            if (v[i][c] >= least) {
                const int to = at + __popc(has[i][c] & lanemask_lt());
                s.val[to] = v[i][c];
                s.id[to] = (lane + kWarp * i) * VEC + c;
            }
            at += __popc(has[i][c]);
        }
    if (lane < 4) s.val[n + lane] = -INFINITY;
    __syncwarp();
    const float mine = s.val[lane];
    const int my_id = s.id[lane];
    int rank = -1; // itself counts once
    for (int c = 0; c < n; c += 4) {
        const float4 o = *reinterpret_cast<const float4 *>(&s.val[c]);
        rank += (o.x >= mine) + (o.y >= mine) + (o.z >= mine) + (o.w >= mine);
    }
    if (__reduce_add_sync(0xffffffffu, lane < n ? (unsigned)rank : 0u) != (unsigned)(n * (n - 1) / 2)) { // ties
        rank = 0;
        for (int c = 0; c < n; ++c) rank += s.val[c] > mine || (s.val[c] == mine && s.id[c] < my_id);
    }
    if (lane < n && rank < k) {
        s.sel_val[rank] = mine;
        s.sel_id[rank] = my_id;
    }
    __syncwarp();
    const float z = (lane < k) ? expf(s.sel_val[lane] - first) : 0.f;
    float sum = z;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    *e = s.sel_id[lane < k ? lane : 0];
    *wt = __fdiv_rn(z, sum);
    *top = first;
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
