// Routing with its balance loss, and the gradient of the router's logits.
//
// Forward.  For a group g of tokens with n counting tokens, softmax rows p and
// chosen pairs counted in c:
//   loss = coef / G * sum_g E * sum_e c[g,e] / (n k) * (sum_t p[t,e] / n).
// The counts are constants of the loss, so d loss / d p[t,e] = slope[g,e] =
// coef * E * c[g,e] / (G k n^2) is one number per group and expert, and all
// that the backward pass needs.
// One pass over the logits (k_route_balance): a warp routes a token (as
// k_route_topk does, with fewer instructions), and adds its softmax row to
// sums that stay in registers; a block adds its warps up and writes one row of
// sums and counts.  A second kernel (k_balance_finish) adds the blocks' rows in
// block order and forms prob, slope and the loss.  Few tokens take one launch
// of one cluster (k_balance_cluster).  Every order is fixed by the sizes, so
// equal inputs give equal bits.
// Bound by instruction issue, not by HBM: the selection takes about 400
// instructions of a warp per token at 128 experts and top 8 (32768 tokens: 18
// us of the 21.8; reading the logits is 2.5).
//
// Backward.  With q = p * (slope - <p, slope>) and the selected softmax w:
//   dlogits = dloss * q + scatter(w * (dw - <w, dw>)).
// One pass: a warp holds a token's row in registers, recomputes its softmax,
// and adds the k selected terms through shared memory.  Bound by HBM: 70 MB in
// 13.3 us at 32768 x 256.
#include "route_topk.cuh"

namespace ap {
namespace {

constexpr int kBalThreads = 256; // of the backward kernel
constexpr int kBalWarps = kBalThreads / kWarp;
constexpr int kBalBlocks = 304;  // row-sum blocks of all groups together, at most (one group per block beyond)
constexpr int kFinThreads = 1024;
constexpr int kFinWarps = kFinThreads / kWarp;
constexpr int kFinCols = 8; // experts of a block: 64 bytes of a row of sums and counts

// Warps of a row-sum block: 16 while a lane's logits and sums fit 64 registers, else 8.
constexpr int bal_warps(int E) { return E <= 256 ? 16 : 8; }

struct BalancePlan {
    int64_t S, G, blocks; // tokens per group, groups, blocks per group
    int64_t off_n, off_lp, off_p, bytes;
};

template <int VEC> struct Floats;
template <> struct Floats<4> { using T = float4; };
template <> struct Floats<1> { using T = float; };

// exp(x) for x <= 0 as 2^(x log2 e): relative error (2.2 |x| + 4) 2^-24, where
// expf takes twice the instructions for (|x| + 4) 2^-24.
__device__ __forceinline__ float exp_neg(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
    return y;
}

// Routes the tokens t, t + step, ... below t_end of one group and adds the
// softmax rows of those that count to acc, their pairs to s_cnt; returns how
// many counted.  Lane l holds the vectors l, l + 32, ... of VEC experts each
// (N of them).
template <int VEC, int N>
__device__ __forceinline__ int route_tokens(const float *logits, int64_t t, int64_t t_end, int64_t step, int E, int k,
                                            const uint8_t *mask, int32_t *__restrict__ idx, float *__restrict__ w,
                                            TopkSlots &slots, int *s_cnt, float (&acc)[N][VEC])
{
    using Vec = typename Floats<VEC>::T;
    const int lane = (int)lane_id();
    const int nvec = E / VEC;
    int n = 0;
    const float *next = logits + t * E;
    idx += t * k + lane;
    w += t * k + lane;
    for (; t < t_end; t += step, next += step * E, idx += step * k, w += step * k) {
        const Vec *row = reinterpret_cast<const Vec *>(next);
        float v[N][VEC];
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) v[i][c] = -INFINITY;
            if (lane + kWarp * i < nvec) {
                const Vec x = __ldcs(row + lane + kWarp * i);
                memcpy(v[i], &x, sizeof(Vec));
            }
        }
        const bool counts = !mask || mask[t];
        int e;
        float wt, top;
        select_token_slots<VEC, N>(v, E, k, lane, slots, &e, &wt, &top);
        const bool some = top != -INFINITY; // warp-uniform
        if (lane < k) {
            *idx = e;
            *w = some ? wt : 0.f;
        }
        if (some && counts) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    v[i][c] = exp_neg(v[i][c] - top); // -infinity (no such expert, or one masked out) gives 0
                    sum += v[i][c];
                }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const float inv = __frcp_rn(sum);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) acc[i][c] += v[i][c] * inv;
            if (lane < k) atomicAdd(&s_cnt[e], 1);
            ++n;
        }
    }
    return n;
}

// Zero sums, counts and token count; then, after the tokens, the warp's sums
// into its row of s_sum.
template <int VEC, int N> __device__ __forceinline__ void zero_sums(float (&acc)[N][VEC])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[i][c] = 0.f;
}
template <int VEC, int N>
__device__ __forceinline__ void store_sums(float *row, const float (&acc)[N][VEC], int E)
{
    using Vec = typename Floats<VEC>::T;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if ((int)lane_id() + kWarp * i < E / VEC) {
            Vec x;
            memcpy(&x, acc[i], sizeof(Vec));
            reinterpret_cast<Vec *>(row)[lane_id() + kWarp * i] = x;
        }
}

template <int VEC, int N, int W>
__global__ void __launch_bounds__(W *kWarp)
    k_route_balance(const float *logits, int64_t T, int E, int k, int64_t S, int blocks,
                    const uint8_t *mask, int32_t *__restrict__ idx, float *__restrict__ w,
                    int32_t *__restrict__ part_n, float2 *__restrict__ part, uint32_t *done)
{
    pdl_begin();
    extern __shared__ __align__(16) float s_mem[];
    float *s_sum = s_mem;                                // [W][E]
    int *s_cnt = reinterpret_cast<int *>(s_mem + W * E); // [E]
    __shared__ __align__(16) TopkSlots s_slots[W];
    __shared__ int s_n;
    const int wid = threadIdx.x / kWarp;
    if (blockIdx.x == 0 && threadIdx.x == 0) *done = 0;
    if (threadIdx.x == 0) s_n = 0;
    for (int e = threadIdx.x; e < E; e += W * kWarp) s_cnt[e] = 0;
    __syncthreads();

    const int64_t g = blockIdx.x / blocks;
    const int b = (int)(blockIdx.x - g * blocks);
    const int64_t t_end = (g + 1) * S < T ? (g + 1) * S : T;
    float acc[N][VEC];
    zero_sums(acc);
    const int n = route_tokens<VEC, N>(logits, g * S + (int64_t)b * W + wid, t_end, (int64_t)blocks * W, E, k, mask, idx,
                                       w, s_slots[wid], s_cnt, acc);
    store_sums(s_sum + wid * E, acc, E);
    if (lane_id() == 0 && n) atomicAdd(&s_n, n);
    __syncthreads();
    const int64_t at = (int64_t)blockIdx.x * E;
    for (int e = threadIdx.x; e < E; e += W * kWarp) {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < W; ++q) sum += s_sum[q * E + e];
        part[at + e] = make_float2(sum, __int_as_float(s_cnt[e]));
    }
    if (threadIdx.x == 0) part_n[blockIdx.x] = s_n;
}

// What one expert of a group comes to: its row entries, and its loss term.
__device__ __forceinline__ float balance_entry(float sum, int cnt, int n, int E, int k, int64_t G, float coef,
                                               int32_t *counts, float *prob, float *slope)
{
    const float nf = (float)(n > 0 ? n : 1);
    const float sl = coef * (float)E / ((float)G * (float)k) * (float)cnt / (nf * nf);
    *counts = cnt;
    *prob = __fdiv_rn(sum, nf);
    *slope = sl;
    return sl * sum;
}

// Few tokens: one launch, no work space.  One cluster takes all groups: with
// at most as many groups as blocks, a group has `per` blocks, whose sums go to
// its first block's shared memory; with more, a block takes every gridDim-th
// group.  Loss terms are added in expert, group and block order.
constexpr int kClusterBlocks = 8; // the largest portable cluster
// 256 tokens of 8 experts take 5.6 us either way, 1000 of 128 on 8 SMs 15 us
// and on all of them 8, but the second launch and the work space cost 5 us of
// host time, which is above 20 us; 800 tokens of 1000 experts took 37 us.
constexpr int64_t kClusterTokens = 1024, kClusterLogits = 1 << 18;
bool one_cluster(int64_t T, int32_t E) { return T <= kClusterTokens && T * E <= kClusterLogits; }
template <int VEC, int N, int W>
__global__ void __launch_bounds__(W *kWarp)
    k_balance_cluster(const float *logits, int T, int E, int k, int S, int G, int per,
                      const uint8_t *mask, float coef, int32_t *__restrict__ idx, float *__restrict__ w,
                      int32_t *__restrict__ counts, float *__restrict__ prob, float *__restrict__ slope,
                      float *__restrict__ loss)
{
    cluster_arrive();
    pdl_begin();
    extern __shared__ __align__(16) float s_mem[];
    float *s_sum = s_mem;                                                            // [W][E]
    int *s_cnt = reinterpret_cast<int *>(s_mem + W * E);                             // [E]
    float2 *s_part = reinterpret_cast<float2 *>(s_mem + (W + 1) * E + ((W + 1) * E & 1)); // [per][E] of the group's blocks
    __shared__ __align__(16) TopkSlots s_slots[W];
    __shared__ int s_n, s_ns[kClusterBlocks];
    __shared__ float s_term[W], s_loss[kClusterBlocks];
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    const int me = blockIdx.x, first = me / per * per; // the grid is one cluster
    float block_loss = 0.f;                            // (of thread 0)
    auto finish = [&](int g, int parts) { // the group's entries from the sums of its blocks, all in s_part
        int n = 0;
        for (int r = 0; r < parts; ++r) n += s_ns[r];
        float term = 0.f;
        for (int e = threadIdx.x; e < E; e += W * kWarp) {
            float sum = 0.f;
            int cnt = 0;
            for (int r = 0; r < parts; ++r) {
                sum += s_part[r * E + e].x;
                cnt += __float_as_int(s_part[r * E + e].y);
            }
            const int64_t at = (int64_t)g * E + e;
            term += balance_entry(sum, cnt, n, E, k, G, coef, counts + at, prob + at, slope + at);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) term += __shfl_xor_sync(0xffffffffu, term, off);
        if (lane == 0) s_term[wid] = term;
        __syncthreads();
        if (threadIdx.x == 0)
            for (int q = 0; q < W; ++q) block_loss += s_term[q];
    };
    cluster_wait(); // all blocks have started: their shared memory may be written
    for (int g = me / per; g < G; g += gridDim.x / per) {
        if (threadIdx.x == 0) s_n = 0;
        for (int e = threadIdx.x; e < E; e += W * kWarp) s_cnt[e] = 0;
        __syncthreads();
        const int64_t t_end = (int64_t)(g + 1) * S < T ? (int64_t)(g + 1) * S : T;
        float acc[N][VEC];
        zero_sums(acc);
        const int n = route_tokens<VEC, N>(logits, (int64_t)g * S + (me - first) * W + wid, t_end, (int64_t)per * W, E, k,
                                           mask, idx, w, s_slots[wid], s_cnt, acc);
        store_sums(s_sum + wid * E, acc, E);
        if (lane == 0 && n) atomicAdd(&s_n, n);
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += W * kWarp) {
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < W; ++q) sum += s_sum[q * E + e];
            cluster_store(cluster_addr(smem_addr(&s_part[(me - first) * E + e]), first),
                          make_uint2(__float_as_uint(sum), (uint32_t)s_cnt[e]));
        }
        if (threadIdx.x == 0) cluster_store(cluster_addr(smem_addr(&s_ns[me - first]), first), (uint32_t)s_n);
        if (per == 1) {
            __syncthreads();
            finish(g, 1);
            __syncthreads();
        }
    }
    if (per > 1) {
        cluster_sync();
        if (me == first && me / per < G) finish(me / per, per);
    }
    if (threadIdx.x == 0)
        cluster_store(cluster_addr(smem_addr(&s_loss[me]), 0), __float_as_uint(block_loss));
    cluster_sync(); // (no block's shared memory is touched after this)
    if (me == 0 && threadIdx.x == 0) {
        float total = 0.f;
        for (unsigned r = 0; r < gridDim.x; ++r) total += s_loss[r];
        *loss = total;
    }
}

// The split and the layout of the work space: one row of E sums and counts and
// one token count per block, one loss term per kFinCols experts of a group, and the
// counter of finished blocks of the second kernel.
BalancePlan balance_plan(int64_t T, int32_t E, int64_t group_tokens)
{
    BalancePlan p = {};
    p.S = group_tokens > 0 && group_tokens < T ? group_tokens : (T > 0 ? T : 1);
    p.G = (T + p.S - 1) / p.S;
    p.blocks = 1;
    if (p.G > 0) {
        const int64_t warps = bal_warps(E);
        const int64_t most = (p.S + warps - 1) / warps;
        p.blocks = kBalBlocks / p.G;
        if (p.blocks > most) p.blocks = most;
        if (p.blocks < 1) p.blocks = 1;
    }
    if (one_cluster(T, E)) return p; // no work space
    auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    const int64_t rows = p.G * p.blocks;
    p.off_n = 256;
    p.off_lp = p.off_n + up(rows * 4);
    p.off_p = p.off_lp + up(p.G * ((E + kFinCols - 1) / kFinCols) * 4);
    p.bytes = p.off_p + up(rows * E * 8);
    return p;
}

// One block per group and kFinCols experts.  Thread (r, c) adds rows r, r + 128,
// ... of its group's blocks in column c; the 128 sums of a column are added in
// a fixed tree; the last block to finish adds the loss terms up in block order.
__global__ void __launch_bounds__(kFinThreads)
    k_balance_finish(int E, int k, int64_t G, int blocks, float coef, const int32_t *part_n,
                     const float2 *part, float *loss_part, int32_t *__restrict__ counts,
                     float *__restrict__ prob, float *__restrict__ slope, float *__restrict__ loss, uint32_t *done)
{
    pdl_begin();
    constexpr int kRows = kFinThreads / kFinCols;
    __shared__ float2 s_part[kFinCols][kFinWarps];
    __shared__ int s_n;
    __shared__ float s_term[kFinCols], s_tot[kFinWarps];
    __shared__ bool s_last;
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    const int pieces = (E + kFinCols - 1) / kFinCols;
    const int64_t g = blockIdx.x / pieces;
    const int col0 = (int)(blockIdx.x - g * pieces) * kFinCols;
    const int c = lane % kFinCols, e = col0 + c, r0 = threadIdx.x / kFinCols;
    float sum = 0.f;
    int cnt = 0;
    if (wid == kFinWarps - 1) {
        int n = 0;
#pragma unroll 10
        for (int b = lane; b < blocks; b += kWarp) n += part_n[g * blocks + b];
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) s_n = n;
    }
    constexpr int U = 3; // all of 304 blocks in flight
    for (int b0 = r0; b0 < blocks; b0 += U * kRows) {
        float2 r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * kRows;
            r[u] = e < E && b < blocks ? part[(g * blocks + b) * E + e] : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sum += r[u].x;
            cnt += __float_as_int(r[u].y);
        }
    }
#pragma unroll
    for (int off = kFinCols; off < kWarp; off <<= 1) { // the lanes of the same column
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
        cnt += __shfl_xor_sync(0xffffffffu, cnt, off);
    }
    if (lane < kFinCols) s_part[c][wid] = make_float2(sum, __int_as_float(cnt));
    __syncthreads();
    if (wid < kFinCols) { // warp q finishes column q
        const float2 x = s_part[wid][lane];
        sum = x.x;
        cnt = __reduce_add_sync(0xffffffffu, __float_as_int(x.y));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) {
            const int64_t at = g * E + col0 + wid;
            s_term[wid] = col0 + wid < E
                              ? balance_entry(sum, cnt, s_n, E, k, G, coef, counts + at, prob + at, slope + at)
                              : 0.f;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float term = 0.f;
#pragma unroll
        for (int q = 0; q < kFinCols; ++q) term += s_term[q];
        loss_part[blockIdx.x] = term;
        __threadfence();
        s_last = atomicAdd(done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float total = 0.f;
    for (int64_t i = threadIdx.x; i < gridDim.x; i += kFinThreads) total += __ldcg(loss_part + i);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    if (lane == 0) s_tot[wid] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        total = 0.f;
#pragma unroll
        for (int q = 0; q < kFinWarps; ++q) total += s_tot[q];
        *loss = total;
    }
}

__global__ void k_zero_word(float *p)
{
    pdl_begin();
    *p = 0.f;
}

// A warp per token; lane l holds the vectors l, l + 32, ... of VEC experts
// each (N of them).  The selected terms are added through a row of shared
// memory per warp, zero between tokens.  Up to 8 logits a lane, the next
// token's reads go out before this one is worked on (32768 x 256: 17.6 us
// without).
template <int VEC, int N>
__global__ void __launch_bounds__(kBalThreads)
    k_route_backward(const float *logits, int64_t T, int E, int k, const int32_t *idx, const float *w, const float *dw,
                     const float *slope, const float *dloss, int64_t S, const uint8_t *mask, float *dlogits,
                     uint32_t *d_status)
{
    pdl_begin();
    using V = typename Floats<VEC>::T;
    extern __shared__ __align__(16) float s_mem[];
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    float *s_add = s_mem + wid * ((E + 3) & ~3);
    for (int e = lane; e < E; e += kWarp) s_add[e] = 0.f;
    __syncwarp();
    const float gl = slope ? (dloss ? *dloss : 1.0f) : 0.f;
    const int nvec = E / VEC;
    const int64_t warps = (int64_t)gridDim.x * kBalWarps;
    struct Token {
        float x[N][VEC]; // logits, -infinity where there are none
        int e;           // the lane's pair
        float w, dw;
        bool on; // has the second term (warp-uniform)
    };
    auto read = [&](Token &tok, int64_t t) {
        tok.on = slope && (!mask || mask[t]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int s = lane + kWarp * i;
#pragma unroll
            for (int c = 0; c < VEC; ++c) tok.x[i][c] = -INFINITY;
            if (tok.on && s < nvec) {
                const V v = reinterpret_cast<const V *>(logits + t * E)[s];
                memcpy(tok.x[i], &v, sizeof(V));
            }
        }
        tok.e = -1;
        tok.w = tok.dw = 0.f;
        if (dw && lane < k) {
            tok.e = idx[t * k + lane];
            tok.w = w[t * k + lane];
            tok.dw = dw[t * k + lane];
        }
    };
    constexpr bool kAhead = N * VEC <= 8;
    int64_t t = (int64_t)blockIdx.x * kBalWarps + wid;
    if (t >= T) return;
    Token next;
    if (kAhead) read(next, t);
    for (; t < T; t += warps) {
        Token tok;
        if constexpr (kAhead) {
            tok = next;
            if (t + warps < T) read(next, t + warps);
        } else {
            read(tok, t);
        }
        float (&d)[N][VEC] = tok.x;
        if (tok.on) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) top = fmaxf(top, d[i][c]);
            top = reduce_max(top);
            const bool some = top != -INFINITY;
            if (!some) top = 0.f; // (every exponential is 0 then)
            const V *srow = reinterpret_cast<const V *>(slope + (S < T ? (uint32_t)t / (uint32_t)S : 0u) * (int64_t)E);
            float sl[N][VEC], sum = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int s = lane + kWarp * i;
#pragma unroll
                for (int c = 0; c < VEC; ++c) sl[i][c] = 0.f;
                if (s < nvec) {
                    const V v = srow[s];
                    memcpy(sl[i], &v, sizeof(V));
                }
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    d[i][c] = exp_neg(d[i][c] - top);
                    sum += d[i][c];
                    dot += d[i][c] * sl[i][c];
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, off);
                dot += __shfl_xor_sync(0xffffffffu, dot, off);
            }
            const float inv = some ? __frcp_rn(sum) : 0.f;
            const float mean = dot * inv;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) d[i][c] = gl * (d[i][c] * inv) * (sl[i][c] - mean);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) d[i][c] = 0.f;
        }
        const bool valid = tok.e >= 0 && tok.e < E;
        if (dw) {
            if (lane < k && !valid && d_status) atomicOr(d_status, AP_FLAG_BAD_INDEX);
            float dot = tok.w * tok.dw;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            if (valid) s_add[tok.e] = tok.w * (tok.dw - dot);
            __syncwarp();
        }
        V *out = reinterpret_cast<V *>(dlogits + t * E);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int s = lane + kWarp * i;
            if (s < nvec) {
                float a[VEC];
                const V v = reinterpret_cast<const V *>(s_add)[s];
                memcpy(a, &v, sizeof(V));
#pragma unroll
                for (int c = 0; c < VEC; ++c) a[c] += d[i][c];
                V o;
                memcpy(&o, a, sizeof(V));
                out[s] = o;
            }
        }
        if (dw) {
            __syncwarp();
            if (valid) s_add[tok.e] = 0.f;
            __syncwarp();
        }
    }
}

// (On an SM partition that takes no cluster of 8 the cluster is smaller, and sums add up in another order.)
template <int VEC, int N, int W>
ap_status launch_balance_cluster(const float *logits, int T, int E, int k, int S, int G, const uint8_t *mask, float coef,
                                 int32_t *idx, float *w, int32_t *counts, float *prob, float *slope, float *loss,
                                 cudaStream_t st)
{
    const auto kernel = k_balance_cluster<VEC, N, W>;
    constexpr int kMaxE = VEC * N * kWarp;
    constexpr auto smem_of = [](int e, int per) { return (size_t)((W + 1) * e + 1 + 2 * per * e) * 4; };
    static const cudaError_t attr = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                         (int)smem_of(kMaxE, kClusterBlocks));
    if (attr != cudaSuccess) return cuda_fail(attr, "route_balance");
    const int most = cluster_fit((const void *)kernel, W * kWarp, smem_of(E, kClusterBlocks), kClusterBlocks, st);
    // one token a warp, in blocks of one cluster, while the groups and the warps want them
    int blocks = 1;
    while (blocks < most && (blocks * W < T || blocks < G)) blocks *= 2;
    const int per = G <= blocks ? blocks / G : 1;
    launch_cluster(kernel, blocks, W * kWarp, smem_of(E, per), blocks, st, logits, T, E, k, S, G, per, mask, coef, idx,
                   w, counts, prob, slope, loss);
    AP_CHECK_LAUNCH("route_balance launch");
    return AP_OK;
}

template <int VEC, int N>
void launch_route_backward(const float *logits, int64_t T, int E, int k, const int32_t *idx, const float *w,
                           const float *dw, const float *slope, const float *dloss, int64_t S, const uint8_t *mask,
                           float *dlogits, uint32_t *d_status, cudaStream_t st)
{
    const size_t smem = (size_t)kBalWarps * ((E + 3) & ~3) * 4;
    const int64_t want = (T + kBalWarps - 1) / kBalWarps;
    // one wave: 13.4 us at 32768 x 256, where 16 blocks an SM take 16.9
    static const int resident = resident_grid((const void *)k_route_backward<VEC, N>, kBalThreads,
                                              (size_t)kBalWarps * VEC * N * kWarp * 4);
    launch(k_route_backward<VEC, N>, (int)(want < resident ? want : resident), kBalThreads, smem, st, logits, T, E, k, idx, w,
           dw, slope, dloss, S, mask, dlogits, d_status);
}

bool balance_sizes_ok(int64_t T, int32_t E, int32_t k, int64_t group_tokens)
{
    return T >= 0 && T < (int64_t(1) << 31) && E >= 1 && E <= 1024 && k >= 1 && k <= E && k <= 32 && group_tokens >= 0;
}

} // namespace
} // namespace ap

extern "C" ap_status ap_route_balance_scratch_bytes(int64_t T, int32_t E, int64_t group_tokens, int64_t *bytes)
{
    using namespace ap;
    if (!bytes || !balance_sizes_ok(T, E, 1, group_tokens))
        return fail(AP_EINVAL, "route_balance_scratch_bytes: bad sizes T=%lld E=%d group_tokens=%lld", (long long)T, E,
                    (long long)group_tokens);
    *bytes = balance_plan(T, E, group_tokens).bytes;
    return AP_OK;
}

extern "C" ap_status ap_route_balance(const float *logits, int64_t T, int32_t E, int32_t k, int64_t group_tokens,
                                      const uint8_t *mask, float coef, int32_t *idx, float *w, int32_t *counts,
                                      float *prob, float *slope, float *loss, void *scratch, int64_t scratch_bytes,
                                      void *stream)
{
    AP_NVTX_RANGE("ap_route_balance");
    using namespace ap;
    if (!balance_sizes_ok(T, E, k, group_tokens))
        return fail(AP_EINVAL, "route_balance: bad sizes T=%lld E=%d k=%d group_tokens=%lld", (long long)T, E, k,
                    (long long)group_tokens);
    if (!loss) return fail(AP_EINVAL, "route_balance: NULL pointer");
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {
        launch(k_zero_word, 1, 1, 0, st, loss);
        AP_CHECK_LAUNCH("route_balance launch");
        return AP_OK;
    }
    const BalancePlan p = balance_plan(T, E, group_tokens);
    if (!logits || !idx || !w || !counts || !prob || !slope || (p.bytes > 0 && !scratch))
        return fail(AP_EINVAL, "route_balance: NULL pointer");
    if (reinterpret_cast<uintptr_t>(scratch) & 15) return fail(AP_EINVAL, "route_balance: scratch not 16-byte aligned");
    if (scratch_bytes < p.bytes)
        return fail(AP_EINVAL, "route_balance: scratch of %lld bytes, %lld needed", (long long)scratch_bytes,
                    (long long)p.bytes);
    // vectors where every lane gets one (fewer lanes with experts leave no bound from the lanes' maxima): 23.8 us at
    // 32768 x 256, single loads 24.6
    const bool vec = E >= 128 && E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
    if (one_cluster(T, E)) {
#define AP_BALANCE(VEC, N, W)                                                                                         \
    launch_balance_cluster<VEC, N, W>(logits, (int)T, E, k, (int)p.S, (int)p.G, mask, coef, idx, w, counts, prob, slope, \
                                      loss, st)
        if (vec) {
            if (E <= 128) return AP_BALANCE(4, 1, 16);
            if (E <= 256) return AP_BALANCE(4, 2, 16);
            if (E <= 512) return AP_BALANCE(4, 4, 8);
            return AP_BALANCE(4, 8, 8);
        }
        if (E <= 32) return AP_BALANCE(1, 1, 16);
        if (E <= 64) return AP_BALANCE(1, 2, 16);
        if (E <= 128) return AP_BALANCE(1, 4, 16);
        if (E <= 256) return AP_BALANCE(1, 8, 16);
        if (E <= 512) return AP_BALANCE(1, 16, 8);
        return AP_BALANCE(1, 32, 8);
#undef AP_BALANCE
    }
    const int64_t pieces = (E + kFinCols - 1) / kFinCols;
    if (p.G * p.blocks > INT32_MAX || p.G * pieces > INT32_MAX)
        return fail(AP_EINVAL, "route_balance: %lld groups of %d experts are more than one launch takes",
                    (long long)p.G, E);
    char *sc = static_cast<char *>(scratch);
    uint32_t *done = reinterpret_cast<uint32_t *>(sc);
    int32_t *part_n = reinterpret_cast<int32_t *>(sc + p.off_n);
    float *loss_part = reinterpret_cast<float *>(sc + p.off_lp);
    float2 *part = reinterpret_cast<float2 *>(sc + p.off_p);
    const int grid = (int)(p.G * p.blocks);
    const int warps = bal_warps(E);
    const size_t smem = (size_t)(warps + 1) * E * 4;
    auto go = [&](auto *kernel) {
        launch(kernel, grid, warps * kWarp, smem, st, logits, T, E, k, p.S, (int)p.blocks, mask, idx, w, part_n, part,
               done);
    };
    if (vec) {
        if (E <= 128)
            go(k_route_balance<4, 1, 16>);
        else if (E <= 256)
            go(k_route_balance<4, 2, 16>);
        else if (E <= 512)
            go(k_route_balance<4, 4, 8>);
        else
            go(k_route_balance<4, 8, 8>);
    } else if (E <= 32)
        go(k_route_balance<1, 1, 16>);
    else if (E <= 64)
        go(k_route_balance<1, 2, 16>);
    else if (E <= 128)
        go(k_route_balance<1, 4, 16>);
    else if (E <= 256)
        go(k_route_balance<1, 8, 16>);
    else if (E <= 512)
        go(k_route_balance<1, 16, 8>);
    else
        go(k_route_balance<1, 32, 8>);
    AP_CHECK_LAUNCH("route_balance launch");
    launch(k_balance_finish, (int)(p.G * pieces), kFinThreads, 0, st, E, k, p.G, (int)p.blocks, coef, part_n, part,
           loss_part, counts, prob, slope, loss, done);
    AP_CHECK_LAUNCH("route_balance finish launch");
    return AP_OK;
}

extern "C" ap_status ap_route_backward(const float *logits, int64_t T, int32_t E, int32_t k, const int32_t *idx,
                                       const float *w, const float *dw, const float *slope, const float *dloss,
                                       int64_t group_tokens, const uint8_t *mask, float *dlogits, uint32_t *d_status,
                                       void *stream)
{
    AP_NVTX_RANGE("ap_route_backward");
    using namespace ap;
    if (!balance_sizes_ok(T, E, k, group_tokens))
        return fail(AP_EINVAL, "route_backward: bad sizes T=%lld E=%d k=%d group_tokens=%lld", (long long)T, E, k,
                    (long long)group_tokens);
    if (T == 0) return AP_OK;
    if (!dlogits || (slope && !logits) || (dw && (!idx || !w)))
        return fail(AP_EINVAL, "route_backward: NULL pointer");
    const int64_t S = group_tokens > 0 && group_tokens < T ? group_tokens : T;
    cudaStream_t st = (cudaStream_t)stream;
    const uintptr_t al = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(slope) |
                         reinterpret_cast<uintptr_t>(dlogits);
    const bool vec = E % 4 == 0 && (al & 15) == 0; // 13.3 us at 32768 x 256, single loads 15.1 (255 experts)
#define AP_ROUTE_BWD(VEC, N) \
    launch_route_backward<VEC, N>(logits, T, E, k, idx, w, dw, slope, dloss, S, mask, dlogits, d_status, st)
    if (vec) {
        if (E <= 128)
            AP_ROUTE_BWD(4, 1);
        else if (E <= 256)
            AP_ROUTE_BWD(4, 2);
        else if (E <= 512)
            AP_ROUTE_BWD(4, 4);
        else
            AP_ROUTE_BWD(4, 8);
    } else {
        if (E <= 32)
            AP_ROUTE_BWD(1, 1);
        else if (E <= 64)
            AP_ROUTE_BWD(1, 2);
        else if (E <= 128)
            AP_ROUTE_BWD(1, 4);
        else if (E <= 256)
            AP_ROUTE_BWD(1, 8);
        else if (E <= 512)
            AP_ROUTE_BWD(1, 16);
        else
            AP_ROUTE_BWD(1, 32);
    }
#undef AP_ROUTE_BWD
    AP_CHECK_LAUNCH("route_backward launch");
    return AP_OK;
}
