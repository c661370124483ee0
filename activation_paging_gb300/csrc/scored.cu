// Routing by scores, with a bias that balances the experts and with groups of
// experts, the gradient of its logits, and the step of the bias.
//
// Forward.  Scores s = softmax(l) or sigmoid(l); the choice goes by c = s + bias:
// of the groups of E / groups consecutive experts the top_groups with the
// largest sum of their one or two best c, in them the k largest c.  The weights
// are the scores themselves, without the bias: scale * s_j [/ sum_sel s].
// One warp per token, one pass: the row stays in registers, its choices go
// through shared memory for the groups' sums, and the selection is the one of
// the other routers (route_topk.cuh).
// Choices that are near one another in single precision are not settled there:
// where the order of two that matter (neighbours among the k, the border behind
// them, the border between groups) lies within the error bounds below, the
// few experts in question are compared in double precision, for about one token
// in a thousand.  So ids do not depend on how single precision rounds.  Without
// a bias, and with groups that go by their best expert, the logits themselves
// have the scores' order and nothing is near.  (All of a row's choices in double
// precision, 8 exponentials a lane one after the other, made the slowest warp
// take 25 us longer.)
//
// Backward.  With q the chosen scores and u_j = dw_j - sum_i w_i dw_i / scale:
//   sigmoid, renormalised   dl_j = scale q_j / S (1 - sigma_j) u_j
//   sigmoid                 dl_j = scale sigma_j (1 - sigma_j) dw_j
//   softmax, renormalised   dl_j = scale q_j / S u_j
//   softmax                 dl_e = p_e (scale dw_e - sum_j p_j scale dw_j), all experts
// The first three touch k logits of a row and write zeros beside.  Experts that
// were chosen for want of others (w = 0 forwards) are no part of the sums; which
// these are the logits do not say, so the weights are read for it.
#include "route_topk.cuh"

namespace ap {
namespace {

constexpr int kScWarps = 8;
constexpr int kScThreads = kScWarps * kWarp;
constexpr float kUlp = 5.9604645e-8f; // 2^-24

struct ScoredArgs {
    const float *logits, *bias;
    const uint8_t *mask;
    int32_t *idx;
    float *w;
    int32_t *counts;
    int64_t T;
    int E, k;
    int groups, size, top_groups, best; // size: experts of a group
    int shift;                          // groups of 4 << shift experts, as long as a warp's lanes hold one; else -1
    uint32_t inv_size;                  // ceil(2^20 / size): e / size = e * inv_size >> 20 for e < 1024
    float scale;
    bool sigmoid, renorm;
};

template <int VEC> struct ScVec;
template <> struct ScVec<4> { using T = float4; };
template <> struct ScVec<1> { using T = float; };

// 2^(x log2 e): relative error (1.5 |x| + 4) 2^-24.
__device__ __forceinline__ float exp_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
    return y;
}
// The same without the growth in |x|, for x <= 0: what the product rounds away,
// and the constant's rest, as a first-order correction.  6 2^-24.
__device__ __forceinline__ float exp_near(float x)
{
    x = x < -200.f ? -200.f : x; // (the power is 0 there already; -infinity has no rest)
    constexpr float kLog2e = 1.44269504f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;
    const float y = x * kLog2e, rest = fmaf(x, kRest, fmaf(x, kLog2e, -y));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    return fmaf(e, rest * kLn2, e);
}
__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Single errors of a choice, with which two of them are near: a sigmoid by
// exp_fast, an addition and a reciprocal has at most s (1 - s) (1.5 |x| + 4) u
// + 3 u s <= 4.4 u, a softmax value at most (2.2 d + 17 + E / 32) u of itself,
// d e^-d <= 1 / e of the largest: 50 u of that one.  Adding the bias rounds by
// u |c|.  near() bounds the two of a pair.
__device__ __forceinline__ float near_of(bool sigmoid, float p_top, float c)
{
    return (sigmoid ? 16.f * kUlp : 128.f * kUlp * p_top) + 4.f * kUlp * fabsf(c);
}

// The two largest of a group's values, over the lanes that share the group.
template <typename F> struct Best2 {
    F first, second;
    __device__ __forceinline__ void take(F v)
    {
        const F low = v > first ? first : v;
        second = low > second ? low : second;
        first = v > first ? v : first;
    }
};

// The choice in double precision of an expert with logit x and bias b.  Without
// a bias softmax values keep their order undivided by the row's sum.
__device__ __noinline__ double exact_choice(bool sigmoid, bool biased, float x, float b, float top, double sum)
{
    double c = sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top);
    if (biased) c = (sigmoid ? c : c / sum) + (double)b;
    return c == c && x > -INFINITY ? c : -INFINITY;
}
__device__ __noinline__ double exact_sum(const float *logits, int E, float top)
{
    double sum = 0.0;
    for (int i = (int)lane_id(); i < E; i += kWarp) sum += exp((double)logits[i] - (double)top);
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    return sum;
}
// What exact comparisons of a token need.
struct Exact {
    const ScoredArgs &a;
    const float *logits;
    float top;
    double sum;
    __device__ __forceinline__ Exact(const ScoredArgs &args, int64_t t, float row_top)
        : a(args), logits(args.logits + t * args.E), top(row_top), sum(1.0)
    {
        if (!a.sigmoid && a.bias) sum = exact_sum(logits, a.E, top);
    }
    __device__ __forceinline__ double of(int e) const
    {
        return exact_choice(a.sigmoid, a.bias != nullptr, logits[e], a.bias ? a.bias[e] : 0.f, top, sum);
    }
};

// The score of a group by its best experts, and how far single precision may be off.
struct GroupScore {
    float score, err;
};
__device__ __forceinline__ GroupScore group_score(const ScoredArgs &a, const Best2<float> &b, float p_top)
{
    GroupScore g;
    g.score = a.best == 2 ? b.first + b.second : b.first;
    if (!(g.score == g.score)) g.score = -INFINITY;
    g.err = near_of(a.sigmoid, p_top, b.first) + (a.best == 2 ? near_of(a.sigmoid, p_top, b.second) : 0.f);
    if (!(g.err < INFINITY)) g.err = 0.f; // of -infinity: nothing rounds
    return g;
}
__device__ __forceinline__ void best_of_lanes(Best2<float> &b, int from, int to) // over lanes that differ in these bits
{
    for (int off = from; off < to; off <<= 1) {
        const float o1 = __shfl_xor_sync(0xffffffffu, b.first, off), o2 = __shfl_xor_sync(0xffffffffu, b.second, off);
        b.second = fmaxf(fminf(b.first, o1), fmaxf(b.second, o2));
        b.first = fmaxf(b.first, o1);
    }
}

// Lane g's score of group g from the warp's choices in shared memory; every
// group has `lanes` lanes (a power of two).
__device__ __forceinline__ GroupScore scan_groups(const float *row, const ScoredArgs &a, int lane, int lanes, float p_top)
{
    const int g = lane / lanes, sub = lane - g * lanes;
    Best2<float> b = {-INFINITY, -INFINITY};
    if (g < a.groups) {
        // the groups begin at different places of theirs, so that groups of 32 experts meet different banks
        const int n = (a.size - sub + lanes - 1) / lanes;
        int i = g < n ? g : 0;
        for (int c = 0; c < n; ++c) {
            b.take(row[g * a.size + sub + i * lanes]);
            if (++i == n) i = 0;
        }
    }
    best_of_lanes(b, 1, lanes);
    GroupScore s = group_score(a, b, p_top);
    const int from = lane < a.groups ? lane * lanes : 0;
    s.score = __shfl_sync(0xffffffffu, s.score, from);
    s.err = __shfl_sync(0xffffffffu, s.err, from);
    return s;
}

// The exact scores of the groups `opens`, lane g of group g: by those experts
// that may be among their best.
__device__ __noinline__ double exact_groups(const ScoredArgs &a, int64_t t, const float *row, float top, float p_top, uint32_t opens)
{
    const int lane = (int)lane_id();
    const Exact x(a, t, top);
    double mine = -INFINITY;
    for (uint32_t left = opens; left; left &= left - 1) {
        const int h = __ffs(left) - 1;
        Best2<float> b = {-INFINITY, -INFINITY};
        for (int i = lane; i < a.size; i += kWarp) b.take(row[h * a.size + i]);
        best_of_lanes(b, 1, kWarp);
        float low = a.best == 2 ? b.second : b.first;
        low -= near_of(a.sigmoid, p_top, low); // (-infinity: all)
        Best2<double> d = {-INFINITY, -INFINITY};
        for (int i = lane; i < a.size; i += kWarp) {
            const float v = row[h * a.size + i];
            if (v > -INFINITY && !(v < low)) d.take(x.of(h * a.size + i));
        }
        for (int off = 1; off < kWarp; off <<= 1) {
            const double o1 = __shfl_xor_sync(0xffffffffu, d.first, off), o2 = __shfl_xor_sync(0xffffffffu, d.second, off);
            d.take(o1);
            d.take(o2);
        }
        if (lane == h) mine = a.best == 2 ? d.first + d.second : d.first;
    }
    return mine;
}

// The choice among the experts that `row` (the warp's choices) puts at or above
// `low`, in double precision: n <= 32 of them, a lane each.
__device__ __noinline__ void choose_few(const ScoredArgs &a, int64_t t, float top, const float *row, float low, int n, int *list, int *e)
{
    const int lane = (int)lane_id();
    int at = 0;
    for (int i0 = 0; i0 < a.E; i0 += kWarp) {
        const bool on = i0 + lane < a.E && row[i0 + lane] >= low;
        const uint32_t who = __ballot_sync(0xffffffffu, on);
        if (on) list[at + __popc(who & lanemask_lt())] = i0 + lane;
        at += __popc(who);
    }
    __syncwarp();
    const Exact x(a, t, top);
    const int mine = lane < n ? list[lane] : -1;
    const double c = lane < n ? x.of(mine) : -INFINITY;
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const double o = __shfl_sync(0xffffffffu, c, j);
        rank += o > c || (o == c && j < lane); // (the list rises)
    }
    __syncwarp();
    if (lane < n) list[rank] = mine;
    __syncwarp();
    if (lane < a.k) *e = list[lane];
}

// The same where more are at the border: the row's choices anew in double
// precision, k rounds over them.  Lane j < k receives the j-th id.
__device__ __noinline__ void choose_many(const ScoredArgs &a, int64_t t, float top, double *wide, const float *row, int *e)
{
    const int lane = (int)lane_id();
    const Exact x(a, t, top);
    // from the end, as the row lies in the same memory
    for (int i0 = (a.E - 1) / kWarp * kWarp; i0 >= 0; i0 -= kWarp) {
        const int i = i0 + lane;
        const float v = i < a.E ? row[i] : -INFINITY;
        const double c = v > -INFINITY ? x.of(i) : -INFINITY;
        __syncwarp();
        if (i < a.E) wide[i] = c;
        __syncwarp();
    }
    for (int j = 0; j < a.k; ++j) {
        double best = -INFINITY;
        int at = kNoExpert; // a chosen expert's place holds NaN
        for (int i = lane; i < a.E; i += kWarp)
            if (wide[i] > best || (wide[i] == best && i < at)) {
                best = wide[i];
                at = i;
            }
        for (int off = 16; off > 0; off >>= 1) {
            const double o = __shfl_xor_sync(0xffffffffu, best, off);
            const int oa = __shfl_xor_sync(0xffffffffu, at, off);
            if (oa != kNoExpert && (at == kNoExpert || o > best || (o == best && oa < at))) {
                best = o;
                at = oa;
            }
        }
        if (lane == j) *e = at;
        __syncwarp();
        if (at % kWarp == lane) wide[at] = NAN;
        __syncwarp();
    }
}

// The chosen scores up to a factor that all of them share: of the softmax
// relative to the largest chosen, of the sigmoid times e^-min(0, largest), so
// that scores near 0 keep their ratios: e^(l - shift) / (1 + e^l) below 0.  The
// relative error is (d + 18) u with d = |l - shift|, which its difference rounds
// by; without a shift 18 u.
__device__ __forceinline__ float score_of(bool sigmoid, float l, float shift)
{
    const float e = exp_near(sigmoid && l > 0.f ? -l : l - shift);
    if (!sigmoid) return e;
    const float below = shift == 0.f ? e : exp_near(l); // (l > 0 only with shift = 0)
    return (l > 0.f ? 1.f : e) * rcp_fast(1.f + below);
}

// Lane l holds the vectors l, l + 32, ... of VEC experts each (N of them).
template <int VEC, int N, bool GROUPS>
__global__ void __launch_bounds__(kScThreads, VEC * N <= 8 ? 4 : VEC * N <= 16 ? 2 : 1)
    k_route_scored(const __grid_constant__ ScoredArgs a)
{
    pdl_begin();
    using Vec = typename ScVec<VEC>::T;
    extern __shared__ __align__(16) double s_rows[]; // [warps][E], then the counts [E]
    __shared__ __align__(16) TopkSlots s_slots[kScWarps];
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    const int E = a.E, k = a.k, nvec = E / VEC;
    double *row64 = s_rows + (size_t)wid * E;
    float *row = reinterpret_cast<float *>(row64);
    int *s_cnt = reinterpret_cast<int *>(s_rows + (size_t)kScWarps * E);
    if (a.counts) {
        for (int e = threadIdx.x; e < E; e += kScThreads) s_cnt[e] = 0;
        __syncthreads();
    }
    // the logits' order is the choices' order
    const bool direct = !a.bias && (!GROUPS || a.best == 1);
    int lanes = kWarp; // of a group
    while (lanes * a.groups > kWarp) lanes >>= 1;
    const int64_t step = (int64_t)gridDim.x * kScWarps;
    for (int64_t t = (int64_t)blockIdx.x * kScWarps + wid; t < a.T; t += step) {
        const Vec *src = reinterpret_cast<const Vec *>(a.logits + t * E);
        float v[N][VEC];
        float top = -INFINITY;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) v[i][c] = -INFINITY;
            if (lane + kWarp * i < nvec) {
                const Vec x = __ldcs(src + lane + kWarp * i);
                memcpy(v[i], &x, sizeof(Vec));
            }
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                odd |= !(v[i][c] == v[i][c]);
                top = fmaxf(top, v[i][c]);
            }
        }
        top = reduce_max(top);
        odd = __any_sync(0xffffffffu, odd) || (!a.sigmoid && top == INFINITY);
        const bool some = top > -INFINITY;
        float sum = 1.f;
        if (!a.sigmoid && (!direct || !a.renorm)) {
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) sum += exp_fast(v[i][c] - top);
            sum = warp_sum(sum);
        }
        const float inv = __fdiv_rn(1.f, sum);
        if (!direct) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = lane + kWarp * i;
                float b[VEC], y[VEC];
#pragma unroll
                for (int c = 0; c < VEC; ++c) b[c] = 0.f;
                if (a.bias && at < nvec) {
                    const Vec x = reinterpret_cast<const Vec *>(a.bias)[at];
                    memcpy(b, &x, sizeof(Vec));
                }
                if (a.sigmoid) {
#pragma unroll
                    for (int c = 0; c < VEC; ++c) y[c] = rcp_fast(1.f + exp_fast(-v[i][c]));
                } else {
#pragma unroll
                    for (int c = 0; c < VEC; ++c) y[c] = exp_fast(v[i][c] - top) * inv;
                }
#pragma unroll
                for (int c = 0; c < VEC; ++c) // (the larger of NaN and -infinity is -infinity)
                    v[i][c] = v[i][c] > -INFINITY ? fmaxf(y[c] + b[c], -INFINITY) : -INFINITY;
            }
        }
        if (odd) { // (warp-uniform) a row that holds NaN has no order: the first k experts
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) v[i][c] = -INFINITY;
        }
        const auto row_store = [&] {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (lane + kWarp * i < nvec) {
                    Vec x;
                    memcpy(&x, v[i], sizeof(Vec));
                    reinterpret_cast<Vec *>(row)[lane + kWarp * i] = x;
                }
            __syncwarp();
        };
        if constexpr (GROUPS) {
            // lane g: group g's score
            GroupScore mine = {-INFINITY, 0.f};
            if (VEC == 4 && a.shift >= 0) { // (warp-uniform) groups of 4 << shift experts: whole lanes, a power of two of them
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    Best2<float> b = {fmaxf(v[i][0], v[i][VEC > 1]), fminf(v[i][0], v[i][VEC > 1])};
#pragma unroll
                    for (int c = 2; c < VEC; ++c) {
                        b.second = fmaxf(b.second, fminf(b.first, v[i][c]));
                        b.first = fmaxf(b.first, v[i][c]);
                    }
                    best_of_lanes(b, 1, 1 << a.shift);
                    const GroupScore g = group_score(a, b, inv);
                    const int at = lane << a.shift; // group `lane` begins with this vector
                    const float s = __shfl_sync(0xffffffffu, g.score, at & 31), r = __shfl_sync(0xffffffffu, g.err, at & 31);
                    if (at >> 5 == i) mine = {s, r};
                }
            } else {
                row_store();
                mine = scan_groups(row, a, lane, lanes, inv);
            }
            const bool is = lane < a.groups;
            if (!is) mine = {-INFINITY, 0.f};
            int rank = 0;
            for (int h = 0; h < a.groups; ++h) {
                const float o = __shfl_sync(0xffffffffu, mine.score, h);
                rank += o > mine.score || (o == mine.score && h < lane);
            }
            bool in_group = is && rank < a.top_groups;
            if (!direct) {
                const float least = -reduce_max(in_group ? mine.err - mine.score : -INFINITY);
                const float most = reduce_max(is && !in_group ? mine.score + mine.err : -INFINITY);
                if (most >= least && most > -INFINITY) { // (warp-uniform) the groups at the border
                    const bool open = is && (in_group ? mine.score - mine.err <= most : mine.score + mine.err >= least);
                    const uint32_t opens = __ballot_sync(0xffffffffu, open);
                    row_store();
                    const double exact = exact_groups(a, t, row, top, inv, opens);
                    int place = 0;
                    for (uint32_t left = opens; left; left &= left - 1) {
                        const int h = __ffs(left) - 1;
                        const double o = __shfl_sync(0xffffffffu, exact, h);
                        place += o > exact || (o == exact && h < lane);
                    }
                    const int room = a.top_groups - __popc(__ballot_sync(0xffffffffu, in_group && !open));
                    if (open) in_group = place < room;
                }
            }
            const uint32_t keep = __ballot_sync(0xffffffffu, in_group);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (VEC == 4 && a.shift >= 0) {
                    if (!(keep >> ((lane + kWarp * i >> a.shift) & 31) & 1))
#pragma unroll
                        for (int c = 0; c < VEC; ++c) v[i][c] = -INFINITY;
                } else {
#pragma unroll
                    for (int c = 0; c < VEC; ++c) {
                        const uint32_t e = (lane + kWarp * i) * VEC + c;
                        if (e < (uint32_t)E && !(keep >> (e * a.inv_size >> 20) & 1)) v[i][c] = -INFINITY;
                    }
                }
            __syncwarp();
        }
        int e;
        float value, first;
        choose_token_slots<VEC, N>(v, E, k, lane, s_slots[wid], &e, &value, &first);
        const float last = __shfl_sync(0xffffffffu, value, k - 1);
        // (chosen with a choice of -infinity: none of those that may be chosen)
        const bool in = lane < k && value > -INFINITY;
        if (!direct) {
            // neighbours among the chosen, and what lies at the last one's border
            const float before = __shfl_up_sync(0xffffffffu, value, 1);
            bool close = lane > 0 && in && before - value <= near_of(a.sigmoid, inv, value);
            // (fewer than k that may be chosen: there is no border behind them)
            const float low = last > -INFINITY ? last - near_of(a.sigmoid, inv, last) : -FLT_MAX;
            int upto = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) upto += v[i][c] >= low;
            upto = __reduce_add_sync(0xffffffffu, upto);
            const bool border = upto > k;
            if (__any_sync(0xffffffffu, close) || border) {
                // equal logits with equal biases have equal choices, whatever the rounding: the lower id is first
                const float *l = a.logits + t * E;
                const float mine = lane < k ? l[e] : 0.f, own = a.bias && lane < k ? a.bias[e] : 0.f;
                const float l1 = __shfl_up_sync(0xffffffffu, mine, 1), b1 = __shfl_up_sync(0xffffffffu, own, 1);
                close &= !(l1 == mine && b1 == own);
                const float ll = __shfl_sync(0xffffffffu, mine, k - 1), bl = __shfl_sync(0xffffffffu, own, k - 1);
                if (border) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
#pragma unroll
                        for (int c = 0; c < VEC; ++c) {
                            const int x = (lane + kWarp * i) * VEC + c;
                            if (v[i][c] >= low && v[i][c] <= last + (last - low))
                                close |= !(l[x] == ll && (!a.bias || a.bias[x] == bl));
                        }
                }
                if (__any_sync(0xffffffffu, close)) { // (warp-uniform)
                    __syncwarp();
                    row_store();
                    // those that may be chosen keep their places in front of those that may not
                    int again = e;
                    if (upto <= kWarp)
                        choose_few(a, t, top, row, low, upto, reinterpret_cast<int *>(&s_slots[wid]), &again);
                    else
                        choose_many(a, t, top, row64, row, &again);
                    if (in) e = again;
                }
            }
        }
        __syncwarp(); // the row and the slots are free
        // weights
        const float l = lane < k ? a.logits[t * E + e] : -INFINITY;
        float wt = 0.f;
        if (odd) {
            wt = NAN;
        } else if (some) { // (warp-uniform)
            const float most = reduce_max(in ? l : -INFINITY);
            if (a.renorm) {
                const float shift = a.sigmoid ? fminf(most, 0.f) : most;
                const float q = in ? score_of(a.sigmoid, l, shift) : 0.f;
                const float all = warp_sum(q);
                wt = all > 0.f ? q * (rcp_fast(all) * a.scale) : 0.f;
            } else if (in) {
                wt = (a.sigmoid ? score_of(true, l, 0.f) : exp_near(l - top) * inv) * a.scale;
            }
        }
        if (lane < k) {
            a.idx[t * k + lane] = e;
            a.w[t * k + lane] = wt;
            if (a.counts && (odd || some) && (!a.mask || a.mask[t])) atomicAdd(&s_cnt[e], 1);
        }
        __syncwarp();
    }
    if (a.counts) {
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += kScThreads)
            if (s_cnt[e]) atomicAdd(&a.counts[e], s_cnt[e]);
    }
}

// A warp per token: the row's zeros (or its dense term) and the k chosen terms,
// which go through a row of shared memory per warp, zero between tokens.
template <int VEC, int N, bool DENSE>
__global__ void __launch_bounds__(kScThreads)
    k_route_scored_backward(const float *logits, int64_t T, int E, int k, const int32_t *idx, const float *dw, const float *w,
                            bool sigmoid, bool renorm, float scale, float *dlogits, uint32_t *d_status)
{
    pdl_begin();
    using Vec = typename ScVec<VEC>::T;
    extern __shared__ __align__(16) float s_mem[];
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp, nvec = E / VEC;
    float *s_add = s_mem + wid * ((E + 3) & ~3);
    for (int e = lane; e < E; e += kWarp) s_add[e] = 0.f;
    __syncwarp();
    const int64_t step = (int64_t)gridDim.x * kScWarps;
    for (int64_t t = (int64_t)blockIdx.x * kScWarps + wid; t < T; t += step) {
        int e = lane < k ? idx[t * k + lane] : 0;
        float g = lane < k ? dw[t * k + lane] * scale : 0.f;
        bool in = lane < k && e >= 0 && e < E;
        if (lane < k && !in && d_status) atomicOr(d_status, AP_FLAG_BAD_INDEX);
        if (w) { // chosen for want of others: w = 0, whatever the logits
            const float was = lane < k ? w[t * k + lane] : 0.f;
            in = in && was != 0.f;
            g = !in ? 0.f : was == was ? g : NAN;
        }
        float v[N][VEC];
        float add = 0.f, dot = 0.f;
        if constexpr (DENSE) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
#pragma unroll
                for (int c = 0; c < VEC; ++c) v[i][c] = -INFINITY;
                if (lane + kWarp * i < nvec) {
                    const Vec x = reinterpret_cast<const Vec *>(logits + t * E)[lane + kWarp * i];
                    memcpy(v[i], &x, sizeof(Vec));
                }
#pragma unroll
                for (int c = 0; c < VEC; ++c) top = fmaxf(top, v[i][c]);
            }
            const float l = in ? logits[t * E + e] : -INFINITY;
            top = reduce_max(top);
            const bool some = top > -INFINITY;
            if (!some) top = 0.f; // (every exponential is 0 then)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    v[i][c] = exp_fast(v[i][c] - top);
                    sum += v[i][c];
                }
            sum = warp_sum(sum);
            const float inv = some ? __fdiv_rn(1.f, sum) : 0.f;
            const float p = in ? exp_fast(l - top) * inv : 0.f;
            dot = warp_sum(p * g);
            add = p * g;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) v[i][c] *= -inv * dot;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) v[i][c] = 0.f;
            const float l = in ? logits[t * E + e] : -INFINITY;
            const float less = sigmoid ? __fdiv_rn(1.f, 1.f + expf(l)) : 1.f; // 1 - sigma
            if (renorm) {
                const float most = reduce_max(l);
                const float q = l > -INFINITY ? score_of(sigmoid, l, sigmoid ? fminf(most, 0.f) : most) : 0.f;
                const float all = warp_sum(q);
                const float w = all > 0.f ? __fdiv_rn(q, all) : all == 0.f ? 0.f : NAN;
                dot = warp_sum(w * g);
                add = w * less * (g - dot);
            } else {
                add = l > -INFINITY ? score_of(true, l, 0.f) * less * g : l == l ? 0.f : NAN;
            }
        }
        if (in) s_add[e] = add;
        __syncwarp();
        Vec *out = reinterpret_cast<Vec *>(dlogits + t * E);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + kWarp * i < nvec) {
                const Vec x = reinterpret_cast<const Vec *>(s_add)[lane + kWarp * i];
                float y[VEC];
                memcpy(y, &x, sizeof(Vec));
#pragma unroll
                for (int c = 0; c < VEC; ++c) y[c] += v[i][c];
                Vec o;
                memcpy(&o, y, sizeof(Vec));
                out[lane + kWarp * i] = o;
            }
        __syncwarp();
        if (in) s_add[e] = 0.f;
        __syncwarp();
    }
}

// bias[e] += rate where expert e had fewer than its share of the pairs, -= rate
// where more.  One block: the share is that of all counts.
__global__ void __launch_bounds__(1024) k_route_bias_step(float *bias, int32_t *counts, int E, float rate, bool reset)
{
    pdl_begin();
    __shared__ long long s_sum[kWarp];
    __shared__ long long s_all;
    const int lane = (int)lane_id(), e = threadIdx.x;
    const long long n = e < E ? counts[e] : 0;
    long long sum = n;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) s_sum[e / kWarp] = sum;
    __syncthreads();
    if (e < kWarp) {
        sum = e < (int)blockDim.x / kWarp ? s_sum[e] : 0;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (e == 0) s_all = sum;
    }
    __syncthreads();
    if (e < E) {
        const long long d = s_all - (long long)E * n;
        if (d) bias[e] += d > 0 ? rate : -rate;
        if (reset) counts[e] = 0;
    }
}

ap_status scored_sizes(const char *who, int64_t T, int32_t E, int32_t k, int32_t score)
{
    if (T < 0 || T >= (int64_t(1) << 31) || E < 1 || E > 1024 || k < 1 || k > E || k > 32)
        return fail(AP_EINVAL, "%s: bad sizes T=%lld E=%d k=%d", who, (long long)T, E, k);
    if (score != AP_SCORE_SOFTMAX && score != AP_SCORE_SIGMOID) return fail(AP_EINVAL, "%s: unknown score %d", who, score);
    return AP_OK;
}

template <int VEC, int N, bool GROUPS> ap_status launch_scored_form(const ScoredArgs &a, cudaStream_t st)
{
    const auto kernel = k_route_scored<VEC, N, GROUPS>;
    constexpr int kMaxE = VEC * N * kWarp;
    static const cudaError_t attr = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                         (kScWarps * 8 + 4) * kMaxE);
    if (attr != cudaSuccess) return cuda_fail(attr, "route_scored");
    static const int resident = resident_grid((const void *)kernel, kScThreads, (kScWarps * 8 + 4) * kMaxE);
    const int64_t want = (a.T + kScWarps - 1) / kScWarps;
    launch(kernel, (int)(want < resident ? want : resident), kScThreads, (size_t)(kScWarps * 8 + 4) * a.E, st, a);
    AP_CHECK_LAUNCH("route_scored launch");
    return AP_OK;
}

template <int VEC, int N> ap_status launch_scored(const ScoredArgs &a, cudaStream_t st)
{
    return a.groups > 1 ? launch_scored_form<VEC, N, true>(a, st) : launch_scored_form<VEC, N, false>(a, st);
}

template <int VEC, int N>
ap_status launch_scored_backward(bool dense, const float *logits, int64_t T, int E, int k, const int32_t *idx, const float *dw,
                                 const float *w, bool sigmoid, bool renorm, float scale, float *dlogits, uint32_t *d_status, cudaStream_t st)
{
    const size_t smem = (size_t)kScWarps * ((E + 3) & ~3) * 4;
    const int64_t want = (T + kScWarps - 1) / kScWarps;
    auto go = [&](auto *kernel) {
        static const int resident = resident_grid((const void *)kernel, kScThreads, (size_t)kScWarps * VEC * N * kWarp * 4);
        launch(kernel, (int)(want < resident ? want : resident), kScThreads, smem, st, logits, T, E, k, idx, dw, w, sigmoid,
               renorm, scale, dlogits, d_status);
    };
    if (dense)
        go(k_route_scored_backward<VEC, N, true>);
    else
        go(k_route_scored_backward<VEC, N, false>);
    AP_CHECK_LAUNCH("route_scored_backward launch");
    return AP_OK;
}

} // namespace
} // namespace ap

extern "C" ap_status ap_route_scored(const float *logits, int64_t T, int32_t E, int32_t k, int32_t score, const float *bias,
                                     int32_t groups, int32_t top_groups, int32_t group_best, int32_t renorm, float scale,
                                     const uint8_t *mask, int32_t *idx, float *w, int32_t *counts, void *stream)
{
    AP_NVTX_RANGE("ap_route_scored");
    using namespace ap;
    if (const ap_status s = scored_sizes("route_scored", T, E, k, score); s != AP_OK) return s;
    if (groups < 1 || groups > 32 || E % groups || top_groups < 1 || top_groups > groups ||
        (int64_t)top_groups * (E / groups) < k)
        return fail(AP_EINVAL, "route_scored: bad groups: %d of %d for E=%d k=%d", top_groups, groups, E, k);
    if (group_best < 1 || group_best > 2 || (groups > 1 && group_best > E / groups))
        return fail(AP_EINVAL, "route_scored: bad group_best=%d", group_best);
    if (T == 0) return AP_OK;
    if (!logits || !idx || !w) return fail(AP_EINVAL, "route_scored: NULL pointer");
    const int size = E / groups;
    int shift = -1;
    for (int q = 0; q <= 5; ++q)
        if (size == 4 << q) shift = q;
    const ScoredArgs a = {logits, bias, mask, idx,  w,          counts,     T,
                          E,      k,    groups, size, top_groups, group_best, shift, (uint32_t)(((1 << 20) + size - 1) / size),
                          scale,  score == AP_SCORE_SIGMOID, renorm != 0};
    cudaStream_t st = (cudaStream_t)stream;
    const uintptr_t al = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(bias);
    if (E >= 128 && E % 4 == 0 && (al & 15) == 0) {
        if (E <= 128) return launch_scored<4, 1>(a, st);
        if (E <= 256) return launch_scored<4, 2>(a, st);
        if (E <= 512) return launch_scored<4, 4>(a, st);
        return launch_scored<4, 8>(a, st);
    }
    if (E <= 32) return launch_scored<1, 1>(a, st);
    if (E <= 64) return launch_scored<1, 2>(a, st);
    if (E <= 128) return launch_scored<1, 4>(a, st);
    if (E <= 256) return launch_scored<1, 8>(a, st);
    if (E <= 512) return launch_scored<1, 16>(a, st);
    return launch_scored<1, 32>(a, st);
}

extern "C" ap_status ap_route_scored_backward(const float *logits, int64_t T, int32_t E, int32_t k, const int32_t *idx,
                                              const float *dw, int32_t score, int32_t renorm, float scale, float *dlogits,
                                              uint32_t *d_status, void *stream)
{
    return ap_route_scored_backward_weighted(logits, T, E, k, idx, dw, nullptr, score, renorm, scale, dlogits, d_status, stream);
}

extern "C" ap_status ap_route_scored_backward_weighted(const float *logits, int64_t T, int32_t E, int32_t k, const int32_t *idx,
                                                       const float *dw, const float *w, int32_t score, int32_t renorm,
                                                       float scale, float *dlogits, uint32_t *d_status, void *stream)
{
    AP_NVTX_RANGE("ap_route_scored_backward");
    using namespace ap;
    if (const ap_status s = scored_sizes("route_scored_backward", T, E, k, score); s != AP_OK) return s;
    if (T == 0) return AP_OK;
    if (!logits || !idx || !dw || !dlogits) return fail(AP_EINVAL, "route_scored_backward: NULL pointer");
    const bool sigmoid = score == AP_SCORE_SIGMOID, dense = !sigmoid && !renorm;
    cudaStream_t st = (cudaStream_t)stream;
    const uintptr_t al = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits);
#define AP_SCORED_BWD(VEC, N) \
    return launch_scored_backward<VEC, N>(dense, logits, T, E, k, idx, dw, w, sigmoid, renorm != 0, scale, dlogits, d_status, st)
    if (E % 4 == 0 && (al & 15) == 0) {
        if (E <= 128) AP_SCORED_BWD(4, 1);
        if (E <= 256) AP_SCORED_BWD(4, 2);
        if (E <= 512) AP_SCORED_BWD(4, 4);
        AP_SCORED_BWD(4, 8);
    }
    if (E <= 32) AP_SCORED_BWD(1, 1);
    if (E <= 64) AP_SCORED_BWD(1, 2);
    if (E <= 128) AP_SCORED_BWD(1, 4);
    if (E <= 256) AP_SCORED_BWD(1, 8);
    if (E <= 512) AP_SCORED_BWD(1, 16);
    AP_SCORED_BWD(1, 32);
#undef AP_SCORED_BWD
}

extern "C" ap_status ap_route_bias_step(float *bias, int32_t *counts, int32_t E, float rate, int32_t reset, void *stream)
{
    AP_NVTX_RANGE("ap_route_bias_step");
    using namespace ap;
    if (E < 1 || E > 1024) return fail(AP_EINVAL, "route_bias_step: bad E=%d", E);
    if (!bias || !counts) return fail(AP_EINVAL, "route_bias_step: NULL pointer");
    launch(k_route_bias_step, 1, (E + kWarp - 1) / kWarp * kWarp, 0, (cudaStream_t)stream, bias, counts, E, rate, reset != 0);
    AP_CHECK_LAUNCH("route_bias_step launch");
    return AP_OK;
}
