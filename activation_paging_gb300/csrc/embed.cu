// Embedding lookup with a scale, and the gradient of the table.
//
// Lookup: out[t] = round(scale * table[ids[t]]), one warp per piece of a row;
// bound by HBM (16384 x 2048 BF16 rows of a 151936-row table: 95 MB in 18 us).
//
// Gradient: dtable[v] (+)= scale * sum over the tokens with id v of dout[t].
// Up to 1024 tokens take one launch (k_embed_small), more take three (beyond
// what one cluster sorts, 131072 tokens as a rule, the sort takes three for
// each of its one to four digits):
//   1. The tokens are sorted by id (stable radix sort, least significant digit
//      first; ids that do not count sort last), so an id's tokens are one run
//      in token order.
//   2. k_embed_sum: a block takes a tile of 8 * rows sorted tokens and a slice
//      of the columns, each warp `rows` tokens of it.  Rows add up in single
//      precision; a run inside one warp goes straight to dtable, the warps'
//      partial rows of a run that spans warps are joined in shared memory,
//      and a run that spans tiles leaves one partial row per tile: `head`
//      where it began in an earlier tile, `tail` where it begins and goes on.
//   3. k_embed_join adds the partial rows of each such run in tile order, and
//      zeros the rows that no id names where the gradient is written whole.
// No floating-point atomics: every sum has one order, fixed by ids and sizes.
// Each row of dout is read once, each row of dtable that an id names read and
// written once, beside the partial rows (at most 2 of single precision for
// every tile, 256 rows where there are many and 32 at the least).  Sums are
// bound by HBM where there is much to add (32768 x 7168, 30% padding: 154 us,
// 828 MB); at 8192 x 2048 the sort takes 8 us of the 25, the sums 14 (of which
// 4 to start and to join), the join 3.
#include <cuda_bf16.h>

#include "ap_common.cuh"
#include "embed_ring.cuh"

namespace ap {
namespace {

// ---- rows of either type -------------------------------------------------------
// VE consecutive elements, as the widest loads that VE elements of the type
// allow (at most 16 bytes each).
template <typename E, int VE> struct alignas(sizeof(E) * VE < 16 ? sizeof(E) * VE : 16) Pack {
    E v[VE];
};
using bf16_t = __nv_bfloat16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16_t v) { return __bfloat162float(v); }
template <typename E> __device__ __forceinline__ E from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16_t from_f<bf16_t>(float v) { return __float2bfloat16_rn(v); }

// Loads a pack now, if `on`: the compiler keeps the load where it stands
// (it would move one whose value is used under a condition down to that use,
// and a batch of loads would wait for memory one after the other).
template <typename P> __device__ __forceinline__ void load_now(P &v, const P *p, bool on)
{
    if constexpr (sizeof(P) == 16) {
        uint4 r = {0, 0, 0, 0};
        asm volatile("{ .reg .pred q; setp.ne.u32 q, %5, 0; @q ld.global.v4.u32 {%0, %1, %2, %3}, [%4]; }"
                     : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
                     : "l"(p), "r"((uint32_t)on));
        memcpy(&v, &r, 16);
    } else if constexpr (sizeof(P) == 8) {
        uint2 r = {0, 0};
        asm volatile("{ .reg .pred q; setp.ne.u32 q, %3, 0; @q ld.global.v2.u32 {%0, %1}, [%2]; }"
                     : "+r"(r.x), "+r"(r.y)
                     : "l"(p), "r"((uint32_t)on));
        memcpy(&v, &r, 8);
    } else if constexpr (sizeof(P) == 4) {
        uint32_t r = 0;
        asm volatile("{ .reg .pred q; setp.ne.u32 q, %2, 0; @q ld.global.u32 %0, [%1]; }"
                     : "+r"(r)
                     : "l"(p), "r"((uint32_t)on));
        memcpy(&v, &r, 4);
    } else if constexpr (sizeof(P) == 2) {
        uint16_t r = 0;
        asm volatile("{ .reg .pred q; setp.ne.u32 q, %2, 0; @q ld.global.u16 %0, [%1]; }"
                     : "+h"(r)
                     : "l"(p), "r"((uint32_t)on));
        memcpy(&v, &r, 2);
    } else {
        static_assert(sizeof(P) == 32, "pack size");
        struct Half {
            uint4 r;
        };
        Half h[2];
        load_now(h[0], reinterpret_cast<const Half *>(p), on);
        load_now(h[1], reinterpret_cast<const Half *>(p) + 1, on);
        memcpy(&v, h, 32);
    }
}

__device__ __forceinline__ int64_t load_id(const void *ids, bool wide, int64_t t)
{
    return wide ? static_cast<const int64_t *>(ids)[t] : (int64_t) static_cast<const int32_t *>(ids)[t];
}

// A lane's sums, two single-precision values to a register pair, for
// instructions that work on two values at once (each rounded as its own).
// Element e of the lane (group e / VE, place e % VE) is half of pair e / 2.
using f2 = unsigned long long;
template <int VE, int NG> struct Sums {
    static_assert(VE * NG % 2 == 0, "pairs");
    f2 p[VE * NG / 2];
};

__device__ __forceinline__ f2 pack2(uint32_t lo, uint32_t hi)
{
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ float2 unpack2(f2 a)
{
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
    return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Pair q of a lane's elements, in single precision.
template <typename E, int VE, int NG> __device__ __forceinline__ f2 pair_of(const Pack<E, VE> (&v)[NG], int q)
{
    const int e = 2 * q;
    if constexpr (VE == 1) {
        return pack2(__float_as_uint(to_f(v[e].v[0])), __float_as_uint(to_f(v[e + 1].v[0])));
    } else if constexpr (sizeof(E) == 4) {
        f2 d;
        memcpy(&d, &v[e / VE].v[e % VE], 8);
        return d;
    } else { // two BF16 values are the upper halves of two single-precision ones
        uint32_t w;
        memcpy(&w, &v[e / VE].v[e % VE], 4);
        return pack2(w << 16, w & 0xffff0000u);
    }
}

// The elements as packs of type E.
template <typename E, int VE, int NG> __device__ __forceinline__ void unpack(Pack<E, VE> (&o)[NG], const Sums<VE, NG> &a)
{
#pragma unroll
    for (int e = 0; e < VE * NG; e += 2) {
        const float2 x = unpack2(a.p[e / 2]);
        o[e / VE].v[e % VE] = from_f<E>(x.x);
        o[(e + 1) / VE].v[(e + 1) % VE] = from_f<E>(x.y);
    }
}

// Stores a pack that is not read again here: evicted first, so that the rows
// of the table stay in L2.
template <typename P> __device__ __forceinline__ void store_stream(P *p, const P &v)
{
    if constexpr (sizeof(P) == 16) {
        uint4 r;
        memcpy(&r, &v, 16);
        __stcs(reinterpret_cast<uint4 *>(p), r);
    } else if constexpr (sizeof(P) == 8) {
        uint2 r;
        memcpy(&r, &v, 8);
        __stcs(reinterpret_cast<uint2 *>(p), r);
    } else if constexpr (sizeof(P) == 4) {
        uint32_t r;
        memcpy(&r, &v, 4);
        __stcs(reinterpret_cast<uint32_t *>(p), r);
    } else {
        uint16_t r;
        memcpy(&r, &v, 2);
        __stcs(reinterpret_cast<uint16_t *>(p), r);
    }
}

// ---- lookup --------------------------------------------------------------------
// A warp takes a piece of an output row: U vectors a lane.
struct Pieces {
    int64_t t, step_t; // row and piece of the warp; they step by as many pieces as there are warps, divided once
    int piece, step_piece, pieces;
    __device__ explicit Pieces(int n) : pieces(n)
    {
        const int64_t warps = (int64_t)gridDim.x * (blockDim.x / kWarp);
        const int64_t first = (int64_t)blockIdx.x * (blockDim.x / kWarp) + threadIdx.x / kWarp;
        t = first / n;
        piece = (int)(first - t * n);
        step_t = warps / n;
        step_piece = (int)(warps - step_t * n);
    }
    __device__ void next()
    {
        t += step_t;
        piece += step_piece;
        if (piece >= pieces) {
            piece -= pieces;
            ++t;
        }
    }
};

template <typename TO, typename TI, int VE>
__device__ __forceinline__ Pack<TO, VE> scaled(const Pack<TI, VE> &v, float by)
{
    if constexpr (VE == 1) {
        return {from_f<TO>(__fmul_rn(to_f(v.v[0]), by))};
    } else {
        const Pack<TI, VE> in[1] = {v};
        const f2 by2 = pack2(__float_as_uint(by), __float_as_uint(by));
        Pack<TO, VE> to[1];
        Sums<VE, 1> x;
#pragma unroll
        for (int q = 0; q < VE / 2; ++q) x.p[q] = mul2(pair_of<TI, VE, 1>(in, q), by2);
        unpack(to, x);
        return to[0];
    }
}

// Rows on the boundaries of VE elements.
template <typename TI, typename TO, int VE, int U>
__global__ void __launch_bounds__(256)
    k_embed(const TI *table, int64_t V, int64_t ld, const void *ids, bool wide, int64_t T,
            int H, float scale, TO *__restrict__ out, int64_t out_ld, uint32_t *d_status)
{
    pdl_begin();
    using PI = Pack<TI, VE>;
    using PO = Pack<TO, VE>;
    const int nstep = H / VE;
    for (Pieces at((nstep + U * kWarp - 1) / (U * kWarp)); at.t < T; at.next()) {
        const int s0 = at.piece * U * kWarp + (int)lane_id();
        const int64_t id = load_id(ids, wide, at.t);
        const bool ok = id >= 0 && id < V;
        if (!ok && s0 == 0 && d_status) atomicOr(d_status, AP_FLAG_BAD_INDEX);
        const PI *src = reinterpret_cast<const PI *>(table + (ok ? id : 0) * ld);
        PO *dst = reinterpret_cast<PO *>(out + at.t * out_ld);
        PI r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) load_now(r[u], src + s0 + u * kWarp, ok && s0 + u * kWarp < nstep); // (else zeros)
        const float by = ok ? scale : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const PO o = scaled<TO>(r[u], by);
            if (s0 + u * kWarp < nstep) store_stream(dst + s0 + u * kWarp, o);
        }
    }
}

// BF16 rows of odd length, or that start between two pairs on either side:
// stores go by the pairs of the output, and the lone elements before the first
// and after the last pair by the first piece's lanes.  A row of the table that
// lies the other way is loaded by the pairs that it cuts, each lane's second
// half from the next lane; the table's first and last row, whose cut pairs
// reach beyond it, by elements.
template <int U>
__global__ void __launch_bounds__(256)
    k_embed_odd(const bf16_t *table, int64_t V, int64_t ld, const void *ids, bool wide,
                int64_t T, int H, float scale, bf16_t *__restrict__ out, int64_t out_ld, uint32_t *d_status)
{
    pdl_begin();
    using P1 = Pack<bf16_t, 1>;
    using P2 = Pack<bf16_t, 2>;
    const int most = H / 2 > 0 ? H / 2 : 1;
    for (Pieces at((most + U * kWarp - 1) / (U * kWarp)); at.t < T; at.next()) {
        const int lane = (int)lane_id(), s0 = at.piece * U * kWarp + lane;
        const int64_t id = load_id(ids, wide, at.t);
        const bool ok = id >= 0 && id < V;
        if (!ok && s0 == 0 && d_status) atomicOr(d_status, AP_FLAG_BAD_INDEX);
        const P1 *src = reinterpret_cast<const P1 *>(table + (ok ? id : 0) * ld);
        P1 *dst = reinterpret_cast<P1 *>(out + at.t * out_ld);
        const int head = reinterpret_cast<uintptr_t>(dst) & 2 ? 1 : 0;
        const int nstep = (H - head) / 2, rest = H - head - 2 * nstep;
        P2 r[U];
        P1 one;
        const bool cut = reinterpret_cast<uintptr_t>(src + head) & 2;
        if (cut && id > 0 && id < V - 1) {
            const P2 *from = reinterpret_cast<const P2 *>(src + head - 1) + s0;
            P2 a[U + 1];
#pragma unroll
            for (int u = 0; u <= U; ++u) load_now(a[u], from + u * kWarp, s0 + u * kWarp <= nstep && (u < U || lane == 0));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t own, first;
                memcpy(&own, &a[u], 4);
                memcpy(&first, &a[u + 1], 4);
                const uint32_t next = __shfl_sync(0xffffffffu, lane == 0 ? first : own, (lane + 1) & 31);
                const uint32_t both = __byte_perm(own, next, 0x5432);
                memcpy(&r[u], &both, 4);
            }
        } else if (cut) {
            P1 a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = s0 + u * kWarp;
                load_now(a[u], src + head + 2 * s, ok && s < nstep);
                load_now(b[u], src + head + 2 * s + 1, ok && s < nstep);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = {a[u].v[0], b[u].v[0]};
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                load_now(r[u], reinterpret_cast<const P2 *>(src + head) + s0 + u * kWarp, ok && s0 + u * kWarp < nstep);
        }
        const int e = lane < head ? 0 : H - 1;
        const bool edge = at.piece == 0 && lane < head + rest;
        load_now(one, src + e, ok && edge);
        const float by = ok ? scale : 0.f;
        P2 *to = reinterpret_cast<P2 *>(dst + head);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const P2 o = scaled<bf16_t>(r[u], by);
            if (s0 + u * kWarp < nstep) store_stream(to + s0 + u * kWarp, o);
        }
        if (edge) store_stream(dst + e, scaled<bf16_t>(one, by));
    }
}

// ---- sort of the tokens by id ----------------------------------------------------
// Sorted tokens as (id, token); ids that do not count hold V and come last.
constexpr int kMaxDigitBits = 10;

// Sort key of a token: its id, or V for one that does not count.
__device__ __forceinline__ uint32_t sort_key(const void *ids, bool wide, int64_t t, int64_t V, int64_t pad,
                                             uint32_t *d_status)
{
    const int64_t id = load_id(ids, wide, t);
    if (id < 0 || id >= V) { // (pad = -1 is none: an id of -1 is a bad one)
        if (d_status) atomicOr(d_status, AP_FLAG_BAD_INDEX);
        return (uint32_t)V;
    }
    return id == pad ? (uint32_t)V : (uint32_t)id;
}

// Lanes of the warp whose digit equals this lane's (one vote per bit; a lane
// without a token, in = false, gets none).  __match_any_sync takes about 60
// cycles of an SM for each warp: 2000 cycles for one digit of 1024 tokens,
// where the votes take 350.
__device__ __forceinline__ uint32_t same_digit(uint32_t d, bool in, int bits)
{
    uint32_t m = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int b = 0; b < kMaxDigitBits; ++b) {
        if (b < bits) {
            const bool one = d >> b & 1;
            const uint32_t v = __ballot_sync(0xffffffffu, one);
            m &= one ? v : ~v;
        }
    }
    return m;
}

// Ranks the warp's 32 tokens of one step among its tokens of the same digit:
// the count so far plus the equal lanes below.
__device__ __forceinline__ uint32_t warp_rank(uint16_t *cnt, uint32_t d, bool in, int bits)
{
    const uint32_t same = same_digit(d, in, bits);
    uint32_t rank = 0;
    if (in) rank = cnt[d] + __popc(same & lanemask_lt());
    __syncwarp();
    if (in && (same >> lane_id()) == 1u) cnt[d] = (uint16_t)(rank + 1); // the last lane of its digit
    __syncwarp();
    return rank;
}

// Sets the bit of every id that occurs, one lane for each id of the warp.  All lanes call it.
__device__ __forceinline__ void mark_seen(uint32_t *seen, uint32_t key, int64_t V)
{
    const uint32_t same = __match_any_sync(0xffffffffu, key);
    if ((same >> lane_id()) == 1u && key != (uint32_t)V) atomicOr(seen + (key >> 5), 1u << (key & 31));
}

// One cluster sorts up to 16 x 8192 tokens in one launch, in registers and
// (distributed) shared memory.  Block r holds tokens r * per .. r * per + per - 1
// of the current order, warp q of it a run of 32 * ITEMS.  A pass: every warp
// ranks its tokens per digit; the warps' counts are added up per digit; every
// block gives its totals to all blocks; every token goes to its new place in
// the block that holds it, in the last pass to memory.  Bound by the waits of
// its phases on one another (two passes: 8 us at 8192 tokens, 13 us at 16384
// and 32768, 34 us at 131072; a barrier of the cluster takes about 0.7 us);
// three launches per digit, as below, took 35 us at 8192.
constexpr int kClThreads = 1024;
constexpr int kClWarps = kClThreads / kWarp;
constexpr int kClItemsMax = 8;
constexpr int kClBlocksMax = 16; // 8 is the largest portable cluster; fewer are used where 16 do not fit
constexpr int64_t kClBlockTokens = (int64_t)kClThreads * kClItemsMax;

// Dynamic shared memory: the block's tokens, the warps' counts, the blocks' totals.
constexpr size_t cluster_smem(int items, int bits, int blocks)
{
    return (size_t)kClThreads * items * 8 + ((size_t)(kClWarps + blocks) << bits) * 2;
}

// The passes, by one block or (CLUSTER) by all blocks of the cluster that is
// the grid.  smem: the block's tokens, the warps' counts, the blocks' totals
// (cluster_smem bytes).  key_of(t) gives token t's key, out(at, pair, in) takes
// every sorted token (all lanes call it); no block touches another's memory
// after the barrier that precedes it.  CLUSTER: the caller has arrived at the
// cluster's barrier once.
template <int ITEMS, bool CLUSTER, typename Key, typename Out>
__device__ __forceinline__ void sort_passes(int T, int per, int passes, int bits, uint2 *s_pairs, Key key_of, Out out)
{
    // Counts and totals are 16 bits, two digits to a word (bits >= 1, a block holds at most 8192 tokens).
    uint16_t *cnt = reinterpret_cast<uint16_t *>(s_pairs + kClThreads * ITEMS);   // [kClWarps][D]
    __shared__ uint32_t s_base[1 << kMaxDigitBits], s_warp[kClWarps], s_group[kClThreads];
    const int D = 1 << bits, D2 = D / 2;
    uint16_t *tot = cnt + kClWarps * D; // [blocks][D]
    uint32_t *cnt2 = reinterpret_cast<uint32_t *>(cnt), *tot2 = reinterpret_cast<uint32_t *>(tot);
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    const uint32_t me = CLUSTER ? blockIdx.x : 0, blocks = CLUSTER ? gridDim.x : 1;
    const int first = (int)me * per;
    const int n = T - first < per ? T - first : per; // this block's tokens (may be <= 0)
    const int l0 = wid * (ITEMS * kWarp) + lane;
    uint16_t *mine = cnt + wid * D;
    auto sync_all = [&] {
        if (blocks > 1)
            cluster_sync();
        else
            __syncthreads();
    };
    // the warps' counts of a pair of digits are added up by `groups` threads, each over `each` warps
    const int groups = D2 >= kClThreads ? 1 : kClThreads / D2 < kClWarps ? kClThreads / D2 : kClWarps;
    const int each = kClWarps / groups;
    const int pair_of = (int)threadIdx.x & (D2 - 1), group = (int)threadIdx.x / D2;
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * bits;
        uint2 pair[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int l = l0 + i * kWarp;
            if (l < n) {
                if (pass == 0)
                    pair[i] = make_uint2(key_of(first + l), (uint32_t)(first + l));
                else
                    pair[i] = s_pairs[l];
            }
        }
        for (int i = lane; i < D2; i += kWarp) cnt2[wid * D2 + i] = 0; // the warp's own counts
        __syncwarp();
        uint32_t rank[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const bool in = l0 + i * kWarp < n;
            rank[i] = warp_rank(mine, in ? pair[i].x >> shift & (D - 1) : 0u, in, bits);
        }
        __syncthreads();
        uint32_t sum = 0;
        if (group < groups) {
#pragma unroll 8
            for (int q = 0; q < each; ++q) sum += cnt2[(group * each + q) * D2 + pair_of];
            s_group[group * D2 + pair_of] = sum;
        }
        if (CLUSTER && pass == 0) cluster_wait(); // all blocks have started (the caller's arrive)
        __syncthreads();
        if (group < groups) {
            uint32_t base = 0;
#pragma unroll 4
            for (int g = 0; g < group; ++g) base += s_group[g * D2 + pair_of];
#pragma unroll 8
            for (int q = 0; q < each; ++q) {
                uint32_t *c = &cnt2[(group * each + q) * D2 + pair_of];
                const uint32_t v = *c;
                *c = base;
                base += v;
            }
            if (group == groups - 1) { // base is the block's total: to every block
                if (CLUSTER) {
#pragma unroll 4
                    for (uint32_t r = 0; r < blocks; ++r)
                        cluster_store(cluster_addr(smem_addr(&tot2[me * D2 + pair_of]), r), base);
                } else {
                    tot2[pair_of] = base;
                }
            }
        }
        sync_all(); // the totals are there, and no block needs its s_pairs any more
        uint32_t before = 0, all = 0;
        if ((int)threadIdx.x < D) {
#pragma unroll 8
            for (uint32_t r = 0; r < blocks; ++r) {
                const uint32_t c = tot[r * D + threadIdx.x];
                if ((int)r < (int)me) before += c;
                all += c;
            }
        }
        uint32_t x = all; // exclusive sum over the digits
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) s_warp[wid] = x;
        __syncthreads();
        uint32_t lower = lane < wid ? s_warp[lane] : 0u; // the digits of the warps below
        lower = __reduce_add_sync(0xffffffffu, lower);
        if ((int)threadIdx.x < D) s_base[threadIdx.x] = lower + x - all + before;
        __syncthreads();
        const bool last = pass + 1 == passes;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const bool in = l0 + i * kWarp < n;
            const int d = (int)((pair[i].x >> shift) & (D - 1));
            const uint32_t at = in ? s_base[d] + mine[d] + rank[i] : 0u;
            if (last) {
                out(at, pair[i], in);
            } else if (in) {
                const uint32_t to = at / (uint32_t)per;
                if (CLUSTER)
                    cluster_store(cluster_addr(smem_addr(s_pairs + (at - to * per)), to), pair[i]);
                else
                    s_pairs[at] = pair[i];
            }
        }
        // the pairs are in place, and nobody reads the totals any more
        if (!last) sync_all();
    }
}

template <int ITEMS>
__global__ void __launch_bounds__(kClThreads, 1)
    k_sort_cluster(const void *ids, bool wide, int T, int per, int64_t V, int64_t pad, int passes,
                   int bits, uint2 *__restrict__ sorted, uint32_t *__restrict__ seen, uint32_t *d_status)
{
    cluster_arrive();
    pdl_begin_after(); // the sums kernel reads ids and rows ahead of its own wait
    extern __shared__ __align__(16) uint8_t s_mem[];
    if (seen) // cleared before the first barrier of the cluster, set in the last pass
        for (int64_t i = (int64_t)blockIdx.x * kClThreads + threadIdx.x; i < (V + 31) / 32;
             i += (int64_t)gridDim.x * kClThreads)
            seen[i] = 0;
    sort_passes<ITEMS, true>(
        T, per, passes, bits, reinterpret_cast<uint2 *>(s_mem),
        [&](int t) { return sort_key(ids, wide, t, V, pad, d_status); },
        [&](uint32_t at, uint2 pair, bool in) {
            if (seen) mark_seen(seen, in ? pair.x : (uint32_t)V, V);
            if (in) sorted[at] = pair;
        });
}

// Longer inputs: three launches per digit, over tiles of kSortTile tokens.
constexpr int kSortThreads = 256;
constexpr int kSortItems = 8;
constexpr int kSortTile = kSortThreads * kSortItems;

// Digit counts of each tile: hist[d * tiles + tile].  The first pass (in ==
// NULL) reads the ids.
__global__ void __launch_bounds__(kSortThreads)
    k_sort_count(const uint2 *in, const void *ids, bool wide, int64_t T, int64_t V,
                 int64_t pad, int shift, int bits, uint32_t *__restrict__ hist, uint32_t *__restrict__ seen,
                 uint32_t *d_status)
{
    pdl_begin();
    if (seen) // the first pass clears what the last one sets
        for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < (V + 31) / 32;
             i += (int64_t)gridDim.x * kSortThreads)
            seen[i] = 0;
    __shared__ uint32_t s_hist[1 << kMaxDigitBits];
    const int D = 1 << bits;
    for (int d = threadIdx.x; d < D; d += kSortThreads) s_hist[d] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kSortTile;
    for (int i = 0; i < kSortItems; ++i) {
        const int64_t t = t0 + i * kSortThreads + threadIdx.x;
        if (t < T) {
            const uint32_t key = in ? in[t].x : sort_key(ids, wide, t, V, pad, d_status);
            atomicAdd(&s_hist[(key >> shift) & (D - 1)], 1u);
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kSortThreads) hist[(int64_t)d * gridDim.x + blockIdx.x] = s_hist[d];
}

// Exclusive sum of n counts in place, by one cluster: kScanItems counts a
// thread, the blocks' totals exchanged through shared memory.  (One block took
// 1.2 us for every 1024 counts: 300 of 490 us at 500000 tokens.)
constexpr int kScanItems = 16, kScanBlocks = 8, kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads) k_sort_scan(uint32_t *hist, int64_t n)
{
    cluster_arrive();
    pdl_begin();
    __shared__ uint32_t s_warp[32], s_tot[2][kScanBlocks];
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    const uint32_t me = blockIdx.x, blocks = gridDim.x; // the grid is one cluster
    uint32_t carry = 0;
    cluster_wait(); // all blocks have started
    for (int64_t base = 0, turn = 0; base < n; base += (int64_t)blocks * kScanThreads * kScanItems, ++turn) {
        const int64_t i0 = base + ((int64_t)me * kScanThreads + threadIdx.x) * kScanItems;
        uint32_t v[kScanItems], sum = 0;
#pragma unroll
        for (int i = 0; i < kScanItems; ++i) v[i] = i0 + i < n ? hist[i0 + i] : 0u;
#pragma unroll
        for (int i = 0; i < kScanItems; ++i) sum += v[i];
        uint32_t x = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) s_warp[wid] = x;
        __syncthreads();
        const uint32_t lower = __reduce_add_sync(0xffffffffu, lane < wid ? s_warp[lane] : 0u);
        if (threadIdx.x == kScanThreads - 1)
            for (uint32_t r = 0; r < blocks; ++r) cluster_store(cluster_addr(smem_addr(&s_tot[turn & 1][me]), r), lower + x);
        cluster_sync(); // (the totals of the turn before are not written again until the next one)
        uint32_t at = carry + lower + x - sum;
        for (uint32_t r = 0; r < blocks; ++r) {
            const uint32_t t = s_tot[turn & 1][r];
            if ((int)r < (int)me) at += t;
            carry += t;
        }
#pragma unroll
        for (int i = 0; i < kScanItems; ++i) {
            if (i0 + i < n) hist[i0 + i] = at;
            at += v[i];
        }
    }
}

// Moves every token of a tile to its place, keeping the order within a digit:
// warp q ranks its kSortItems * 32 consecutive tokens, 32 at a time.
__global__ void __launch_bounds__(kSortThreads)
    k_sort_scatter(const uint2 *in, const void *ids, bool wide, int64_t T, int64_t V,
                   int64_t pad, int shift, int bits, const uint32_t *hist, uint2 *__restrict__ out,
                   uint32_t *__restrict__ seen)
{
    pdl_begin_after(); // as k_sort_cluster

    constexpr int W = kSortThreads / kWarp;
    __shared__ uint16_t s_cnt[W][1 << kMaxDigitBits];
    const int D = 1 << bits;
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    for (int d = threadIdx.x; d < W * D; d += kSortThreads) s_cnt[d / D][d % D] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kSortTile + wid * (kSortItems * kWarp) + lane;
    uint2 pair[kSortItems];
    uint32_t rank[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const int64_t t = t0 + i * kWarp;
        uint32_t d = 0;
        if (t < T) {
            pair[i] = in ? in[t] : make_uint2(sort_key(ids, wide, t, V, pad, nullptr), (uint32_t)t);
            d = (pair[i].x >> shift) & (D - 1);
        }
        rank[i] = warp_rank(s_cnt[wid], d, t < T, bits);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kSortThreads) {
        uint32_t sum = 0;
#pragma unroll
        for (int q = 0; q < W; ++q) {
            const uint32_t c = s_cnt[q][d];
            s_cnt[q][d] = (uint16_t)sum;
            sum += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const bool in = t0 + i * kWarp < T;
        if (seen) mark_seen(seen, in ? pair[i].x : (uint32_t)V, V);
        if (!in) continue;
        const int d = (int)((pair[i].x >> shift) & (D - 1));
        out[hist[(int64_t)d * gridDim.x + blockIdx.x] + s_cnt[wid][d] + rank[i]] = pair[i];
    }
}

// ---- sums of the runs ------------------------------------------------------------
constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / kWarp;
constexpr int kSumRowsMax = 32;
constexpr int64_t kPrefetchBytes = 64 << 20;
constexpr int64_t kWantItems = 256;

// Where a lane's VE * NG elements of a slice lie: NG groups of VE, 32 lanes apart.
template <int VE, int NG> struct Slice {
    int s0, nstep; // first vector of the lane, vectors in a row
    __device__ bool in(int g) const { return s0 + g * kWarp < nstep; }
    __device__ int at(int g) const { return s0 + g * kWarp; }
};

template <int VE, int NG> __device__ __forceinline__ void zero(Sums<VE, NG> &a)
{
#pragma unroll
    for (int q = 0; q < VE * NG / 2; ++q) a.p[q] = 0;
}

// Not a number, for sums that lack rows.
template <int VE, int NG> __device__ __forceinline__ void spoil(Sums<VE, NG> &a)
{
#pragma unroll
    for (int q = 0; q < VE * NG / 2; ++q) a.p[q] = pack2(0x7fffffffu, 0x7fffffffu);
}

template <typename E, int VE, int NG>
__device__ __forceinline__ void add_row(Sums<VE, NG> &a, const Pack<E, VE> (&v)[NG])
{
#pragma unroll
    for (int q = 0; q < VE * NG / 2; ++q) a.p[q] = add2(a.p[q], pair_of<E, VE, NG>(v, q));
}

template <typename TG, int VE, int NG>
__device__ __forceinline__ void finish_row(TG *row, const Slice<VE, NG> &sl, const Sums<VE, NG> &acc,
                                           const Pack<TG, VE> (&old)[NG], float scale, bool add)
{
    const f2 scale2 = pack2(__float_as_uint(scale), __float_as_uint(scale));
    Sums<VE, NG> x;
#pragma unroll
    for (int q = 0; q < VE * NG / 2; ++q) {
        x.p[q] = mul2(scale2, acc.p[q]);
        if (add) x.p[q] = add2(pair_of<TG, VE, NG>(old, q), x.p[q]);
    }
    Pack<TG, VE> o[NG];
    unpack(o, x);
#pragma unroll
    for (int g = 0; g < NG; ++g)
        if (sl.in(g)) reinterpret_cast<Pack<TG, VE> *>(row)[sl.at(g)] = o[g];
}

template <int VE, int NG>
__device__ __forceinline__ void store_part(float *row, const Slice<VE, NG> &sl, const Sums<VE, NG> &a)
{
    Pack<float, VE> o[NG];
    unpack(o, a);
#pragma unroll
    for (int g = 0; g < NG; ++g)
        if (sl.in(g)) reinterpret_cast<Pack<float, VE> *>(row)[sl.at(g)] = o[g];
}

template <typename E, int VE, int NG>
__device__ __forceinline__ void load_row(Pack<E, VE> (&v)[NG], const E *row, const Slice<VE, NG> &sl, bool on = true)
{
#pragma unroll
    for (int g = 0; g < NG; ++g) load_now(v[g], reinterpret_cast<const Pack<E, VE> *>(row) + sl.at(g), on && sl.in(g));
}

// The same from shared memory.
template <int VE, int NG>
__device__ __forceinline__ void load_part(Pack<float, VE> (&v)[NG], const float *row, const Slice<VE, NG> &sl)
{
#pragma unroll
    for (int g = 0; g < NG; ++g) v[g] = reinterpret_cast<const Pack<float, VE> *>(row)[sl.at(g)];
}

// Asks for `bytes` bytes from p in L2 (a hint; the 16-byte granules that hold them).
__device__ __forceinline__ void prefetch_l2(const void *p, int64_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15;
    const uintptr_t e = (reinterpret_cast<uintptr_t>(p) + bytes + 15) & ~(uintptr_t)15;
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"((uint32_t)(e - a)) : "memory");
}

// While the sort runs on a few SMs, the rows of dout (and, to be added to, the
// rows of dtable that the ids name) start on their way to L2: at most
// kPrefetchBytes, about what the sort's time lets HBM deliver.
template <typename TD, typename TG, bool ADD>
__device__ __forceinline__ void prefetch_inputs(const TD *dout, int64_t dout_ld, const void *ids, bool wide, int64_t T,
                                                int64_t V, int64_t pad, int H, const TG *dtable, int64_t ld)
{
    const int64_t rb = (int64_t)H * sizeof(TD), gb = ADD ? (int64_t)H * sizeof(TG) : 0;
    const int64_t most = kPrefetchBytes / (rb + gb);
    const int64_t n = T < most ? T : most;
    for (int64_t t = (int64_t)threadIdx.x * gridDim.x + blockIdx.x; t < n; t += (int64_t)gridDim.x * blockDim.x) {
        const int64_t id = load_id(ids, wide, t);
        if (id < 0 || id >= V || id == pad) continue;
        prefetch_l2(dout + t * dout_ld, rb);
        if (ADD) prefetch_l2(dtable + id * ld, gb);
    }
}

// How the sums take their rows through a ring in shared memory.
//   kAligned:  every row and slice starts on a 16-byte boundary
//   kAnywhere: rows start anywhere: the 16-byte granules that hold a slice are
//              copied, and read from its first byte on
enum Route { kAligned, kAnywhere };

// A row's stage of the ring: 512 bytes of dout and the same columns of dtable,
// each with room for the granules at its ends, copied kStages rows ahead.
constexpr int kStages = 8;
constexpr int kBatch = 4; // rows taken from the ring at a time
constexpr int kDoutBytes = kWarp * 16;
template <typename TD, Route R> constexpr int kDoutStage = kDoutBytes + (R == kAnywhere ? 16 : 0);
template <typename TD, typename TG, bool ADD, Route R>
constexpr int kStageBytes = kDoutStage<TD, R> +
                            (ADD ? kDoutBytes / (int)sizeof(TD) * (int)sizeof(TG) + (R == kAnywhere ? 16 : 0) : 0);
template <typename TD, typename TG, int VE, int NG, bool ADD, Route R>
constexpr int kSumSmem = kSumWarps * (kStages * kStageBytes<TD, TG, ADD, R> + kWarp * VE * NG * 4);

// A bulk copy of `bytes` bytes (all in 16-byte granules) to shared memory, which completes on the barrier.
__device__ __forceinline__ void copy_bulk(uint32_t to, const void *from, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                 "l"(from), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits for the copies of a phase, at most kWaitLimit tries; false if they did not come.
constexpr int kWaitLimit = 1 << 18;
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity)
{
    for (int i = 0; i < kWaitLimit; ++i) {
        uint32_t done;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(done)
                     : "r"(bar), "r"(parity)
                     : "memory");
        if (done) return true;
    }
    return false;
}

// The granules of [p, p + bytes) inside [lo, hi), the buffer that holds it: a
// buffer's first and last granules may be cut by its ends.
struct Granules {
    uintptr_t first, last; // of the whole granules
    uintptr_t base;        // p's granule, where the stage begins
};
__device__ __forceinline__ Granules granules(uintptr_t p, uint32_t bytes, uintptr_t lo, uintptr_t hi)
{
    Granules g;
    g.base = p & ~(uintptr_t)15;
    g.first = g.base < lo ? g.base + 16 : g.base;
    g.last = (p + bytes + 15) & ~(uintptr_t)15;
    if (g.last > hi) g.last -= 16;
    if (g.last < g.first) g.last = g.first;
    return g;
}

// The elements of [p, p + bytes) that lie in no whole granule, by one lane.
template <typename E>
__device__ __forceinline__ void copy_ends(uint8_t *stage, const Granules &g, uintptr_t p, uint32_t bytes)
{
    if (g.first == g.base && g.last >= p + bytes) return;
    for (uintptr_t q = p; q < p + bytes; q += sizeof(E)) {
        if (q >= g.first && q + sizeof(E) <= g.last) {
            q = g.last - sizeof(E); // on behind the granules
            continue;
        }
        *reinterpret_cast<E *>(stage + (q - g.base)) = *reinterpret_cast<const E *>(q);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); // before a later bulk copy to the same place
}

// A block takes tiles of kSumWarps * rows sorted tokens and slices of the columns.
// Through the ring every warp keeps kStages rows on their way to shared
// memory, over the ends of items, so that the sums do not wait for one row's
// latency.  A lane copies the row of its own token.  Loads into registers left
// 3.3 TB/s at 32768 x 7168 rows, bound by what a warp's registers hold in
// flight.
// Should a batch of copies not arrive in the time that bar_wait gives it, the
// warp sums no staged row any more: every run that it has not ended becomes
// NaN (a part of one makes the whole NaN where it is joined), the flag is set,
// and the warp goes on to the block's barriers as ever.  (156.3 us at 32768 x
// 7168 with a test of the state at every run's begin, 154.4 with spoil_runs.)
template <typename TD, typename TG, int VE, int NG, bool ADD, Route R>
__global__ void __launch_bounds__(kSumThreads, 2)
    k_embed_sum(const TD *dout, int64_t dout_ld, const uint2 *sorted, int64_t T, int64_t V,
                int H, float scale, int rows, uint32_t slices, uint32_t sums, TG *__restrict__ dtable, int64_t ld,
                float *__restrict__ partial, int64_t part_ld, const void *ids, bool wide, int64_t pad,
                uint32_t *d_status)
{
    prefetch_inputs<TD, TG, ADD>(dout, dout_ld, ids, wide, T, V, pad, H, dtable, ld); // (hints: they change no value)
    pdl_begin();
    extern __shared__ __align__(16) uint8_t s_mem[];
    constexpr uint32_t kHead = 1, kThrough = 2, kTail = 4;
    constexpr int kCols = kWarp * VE * NG;
    constexpr int kDout = kDoutStage<TD, R>, kStage = kStageBytes<TD, TG, ADD, R>;
    static_assert(kCols * sizeof(TD) == kDoutBytes, "a slice fills its stage");
    __shared__ uint32_t s_flags[kSumWarps];
    __shared__ uint64_t s_bar[kSumWarps][kStages / kBatch]; // one for each batch of the ring
    const int lane = (int)lane_id(), w = threadIdx.x / kWarp;
    auto s_part = [&](int q) { return reinterpret_cast<float *>(s_mem) + q * kCols; }; // a warp's head
    uint8_t *ring = s_mem + kSumWarps * kCols * 4 + w * (kStages * kStage);
    const uint32_t none = (uint32_t)V;
    const int nstep = H / VE;
    const Slice<VE, NG> mine{lane, kWarp * NG}; // within a slice, for s_part
    [[maybe_unused]] const uintptr_t dout_end = reinterpret_cast<uintptr_t>(dout + (T - 1) * dout_ld + H);
    [[maybe_unused]] const uintptr_t dtable_end = reinterpret_cast<uintptr_t>(dtable + (V - 1) * ld + H);
    // a warp's tokens of an item, with the ids before and after them
    struct Rows {
        uint2 my;
        uint32_t before, ends, direct; // ends: rows that end a run; direct: of those, runs of this warp alone
        int64_t tile;
        int n, live, col0, cols;
        bool began; // the first run began before these rows
        const TD *src; // the lane's token's columns of dout
        TG *dst;       // and of dtable
    };
    auto rows_of = [&](uint32_t it) {
        Rows x;
        x.tile = it / slices;
        x.col0 = (int)(it - (uint32_t)x.tile * slices) * kCols;
        x.cols = H - x.col0 < kCols ? H - x.col0 : kCols;
        const int64_t i0 = (x.tile * kSumWarps + w) * rows;
        x.n = T - i0 >= rows ? rows : T > i0 ? (int)(T - i0) : 0;
        x.my = lane < x.n ? sorted[i0 + lane] : make_uint2(none, 0u);
        x.before = x.n > 0 && i0 > 0 ? sorted[i0 - 1].x : none;
        const uint32_t after = i0 + x.n < T ? sorted[i0 + x.n].x : none;
        uint32_t next = __shfl_down_sync(0xffffffffu, x.my.x, 1);
        if (lane == x.n - 1) next = after;
        x.live = __popc(__ballot_sync(0xffffffffu, x.my.x != none)); // ids that count come first
        x.ends = __ballot_sync(0xffffffffu, x.my.x != none && next != x.my.x);
        x.began = x.live > 0 && x.before == __shfl_sync(0xffffffffu, x.my.x, 0);
        x.direct = x.ends & ~(x.began ? (x.ends & (0u - x.ends)) : 0u);
        x.src = dout + (int64_t)x.my.y * dout_ld + x.col0;
        x.dst = dtable + (int64_t)x.my.x * ld + x.col0;
        return x;
    };
    // the column slice of row r of dtable
    auto dst_of = [&](const Rows &x, int r) {
        return reinterpret_cast<TG *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(x.dst), r));
    };
    RingState state; // (warp-uniform)
    auto wait = [&](int slot, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, bar_wait(smem_addr(&s_bar[w][slot]), parity));
    };
    // kBatch rows of x from r0 on into their stages of the ring: a lane copies its own token's row
    auto fetch = [&](const Rows &x, int r0) {
        const int rows_left = x.live - r0, slot = r0 / kBatch % (kStages / kBatch);
        if (rows_left <= 0 || !state.arm(slot)) return;
        const uint32_t bar = smem_addr(&s_bar[w][slot]);
        const uint32_t db = x.cols * sizeof(TD), gb = x.cols * sizeof(TG);
        const uint32_t mask = (rows_left >= kBatch ? (1u << kBatch) - 1 : (1u << rows_left) - 1) << r0;
        const bool on = mask >> lane & 1, both = ADD && on && (x.direct >> lane & 1);
        uint8_t *stage = ring + lane % kStages * kStage;
        const uint32_t to = smem_addr(stage);
        if constexpr (R == kAligned) {
            if (lane == 0) bar_expect(bar, __popc(mask) * db + (ADD ? __popc(x.direct & mask) * gb : 0u));
            __syncwarp();
            if (on) copy_bulk(to, x.src, db, bar);
            if (both) copy_bulk(to + kDout, x.dst, gb, bar);
        } else {
            const uintptr_t src = reinterpret_cast<uintptr_t>(x.src), dst = reinterpret_cast<uintptr_t>(x.dst);
            Granules s = {}, d = {};
            if (on) s = granules(src, db, reinterpret_cast<uintptr_t>(dout), dout_end);
            if (both) d = granules(dst, gb, reinterpret_cast<uintptr_t>(dtable), dtable_end);
            const uint32_t sn = (uint32_t)(s.last - s.first), dn = (uint32_t)(d.last - d.first);
            const uint32_t all = __reduce_add_sync(0xffffffffu, sn + dn);
            if (lane == 0) bar_expect(bar, all);
            if (on) copy_ends<TD>(stage, s, src, db);
            if (both) copy_ends<TG>(stage + kDout, d, dst, gb);
            __syncwarp();
            if (sn) copy_bulk(to + (uint32_t)(s.first - s.base), reinterpret_cast<const void *>(s.first), sn, bar);
            if (dn) copy_bulk(to + kDout + (uint32_t)(d.first - d.base), reinterpret_cast<const void *>(d.first), dn, bar);
        }
    };
    // where row r's slice begins in its stage
    [[maybe_unused]] auto start_of = [&](const void *p, int r) -> uint32_t {
        if (R != kAnywhere) return 0;
        return __shfl_sync(0xffffffffu, (uint32_t)reinterpret_cast<uintptr_t>(p), r) & 15;
    };
    if (lane < kStages / kBatch) bar_init(smem_addr(&s_bar[w][lane]));
    asm volatile("fence.mbarrier_init.release.cluster;\n\tfence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    Rows ahead;
    if (blockIdx.x < sums) {
        ahead = rows_of(blockIdx.x);
        for (int r = 0; r < kStages; r += kBatch) fetch(ahead, r);
    }
    for (uint32_t it = blockIdx.x; it < sums; it += gridDim.x) {
        const Rows cur = ahead;
        const int64_t tile = cur.tile;
        const int live = cur.live;
        const uint32_t ends = cur.ends, direct = cur.direct;
        const bool began = cur.began;
        const Slice<VE, NG> sl{cur.col0 / VE + lane, nstep};
        const Slice<VE, NG> here{lane, cur.cols / VE}; // the same from the slice's first column
        const bool more = it + gridDim.x < sums;
        if (more) ahead = rows_of(it + gridDim.x);
        Sums<VE, NG> acc;
        zero(acc);
        // once a batch did not arrive: NaN for the runs that end from row r0 on, and left in acc
        auto spoil_runs = [&](int r0) {
            if (lane == 0 && d_status) atomicOr(d_status, AP_FLAG_CORRUPT);
            spoil(acc);
            const Pack<TG, VE> none[NG] = {};
            for (int r = r0; r < live; ++r) {
                if (direct >> r & 1)
                    finish_row(dst_of(cur, r), here, acc, none, scale, false);
                else if (ends >> r & 1)
                    store_part(s_part(w), mine, acc);
            }
        };
        for (int r0 = 0; r0 < live; r0 += kBatch) {
            if (!state.take(r0 / kBatch % (kStages / kBatch), wait)) {
                spoil_runs(r0);
                break;
            }
            const uint8_t *at = ring + r0 % kStages * kStage;
            // the batch's rows, those that end a run, and of them those of this warp alone: in uniform registers,
            // by a reduction, so that the branches on them are uniform
            const uint32_t all = live - r0 >= kBatch ? (1u << kBatch) - 1 : (1u << (live - r0)) - 1;
            const uint32_t bits = __reduce_or_sync(0xffffffffu, (ends >> r0 & all) | (direct >> r0 & all) << 8 | all << 16);
            Pack<TD, VE> v[kBatch][NG];
            Pack<TG, VE> old[kBatch][NG];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint8_t *row = at + u * kStage;
                const uint32_t from = start_of(cur.src, r0 + u);
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    v[u][g] = reinterpret_cast<const Pack<TD, VE> *>(row + from)[mine.at(g)];
                if (ADD && (bits >> (u + 8) & 1)) {
                    const uint32_t from2 = start_of(cur.dst, r0 + u);
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        old[u][g] = reinterpret_cast<const Pack<TG, VE> *>(row + kDout + from2)[mine.at(g)];
                }
            }
            __syncwarp();
            fetch(cur, r0 + kStages);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (bits >> (u + 16) & 1) add_row(acc, v[u]);
                if (bits >> u & 1) { // the sum goes to dtable, or to the warps that join it
                    if (bits >> (u + 8) & 1)
                        finish_row(dst_of(cur, r0 + u), here, acc, old[u], scale, ADD);
                    else
                        store_part(s_part(w), mine, acc);
                    zero(acc);
                }
            }
        }
        // the whole ring is free: the next item's first rows
        if (more)
            for (int r = 0; r < kStages; r += kBatch) fetch(ahead, r);
        uint32_t flags = 0;
        if (began) flags |= kHead;
        if (live > 0 && !(ends >> (live - 1) & 1)) { // the last run goes on
            const bool through = began && ends == 0;
            flags |= through ? kThrough : kTail;
            if (through) store_part(s_part(w), mine, acc); // (a tail stays in the warp's registers)
        }
        if (lane == 0) s_flags[w] = flags;
        __syncthreads();
        // runs that span warps: the warp in which one begins joins it, the last warp joins what entered the tile
        auto join_from = [&](int q) { // adds heads from warp q on; true if the run ends in this tile
            for (; q < kSumWarps; ++q) {
                Pack<float, VE> p[NG];
                load_part(p, s_part(q), mine);
                add_row(acc, p);
                if (!(s_flags[q] & kThrough)) return true;
            }
            return false;
        };
        if (flags & kTail) {
            TG *row = dst_of(cur, live - 1);
            Pack<TG, VE> old[NG];
            if (ADD) load_row(old, row, here); // on its way while the parts are added
            if (join_from(w + 1)) {
                finish_row(row, here, acc, old, scale, ADD);
            } else {
                store_part(partial + (2 * tile + 1) * part_ld, sl, acc);
            }
        }
        if (w == kSumWarps - 1 && (s_flags[0] & kHead)) {
            zero(acc);
            (void)join_from(0);
            store_part(partial + 2 * tile * part_ld, sl, acc);
        }
        __syncthreads();
    }
}

// n zeros from p on, by a warp: 16 bytes a lane between the boundaries, single elements up to the first and from the
// last on.
template <typename TG> __device__ __forceinline__ void zero_span(TG *p, int n)
{
    constexpr int kPer = 16 / (int)sizeof(TG);
    const int lane = (int)lane_id();
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(TG);
    const int to = off ? kPer - off : 0, head = to < n ? to : n;
    const int mid = (n - head) / kPer, rest = n - head - mid * kPer;
    if (lane < head) p[lane] = from_f<TG>(0.f);
    uint4 *q = reinterpret_cast<uint4 *>(p + head);
#pragma unroll 4
    for (int s = lane; s < mid; s += kWarp) q[s] = make_uint4(0, 0, 0, 0);
    if (lane < rest) p[n - rest + lane] = from_f<TG>(0.f);
}

// Zeros the rows of the `items` items that no id names; an item is `rows`
// rows (a power of two, at most 32), taken by one warp of W in a block.  Rows
// without a gap between them are one span: 139243 rows of 481 FP32 values take
// 45 us, 78 row by row in single elements.
// seen_from(r0): bit i says whether row r0 + i is named, for r0 a multiple of `rows`.
template <typename TG, int W, typename Seen>
__device__ __forceinline__ void fill_rows(int64_t items, int rows, int64_t V, int H, TG *__restrict__ dtable,
                                          int64_t ld, Seen seen_from)
{
    const int64_t warps = (int64_t)gridDim.x * W;
    int64_t it = blockIdx.x + (int64_t)gridDim.x * (threadIdx.x / kWarp);
    uint32_t next = it < items ? seen_from(it * rows) : 0u;
    for (; it < items; it += warps) {
        const int64_t r0 = it * rows;
        const uint32_t bits = next;
        if (it + warps < items) next = seen_from((it + warps) * rows); // on its way while these rows are written
        const int n = V - r0 < rows ? (int)(V - r0) : rows;
        for (int r = 0; r < n;) {
            const uint32_t from = bits >> r;
            int e = r + 1;
            if (!(from & 1)) {
                if (ld == H) e = from ? r + __ffs(from) - 1 : n;
                if (e > n) e = n;
                zero_span(dtable + (r0 + r) * ld, (e - r) * H);
            }
            r = e;
        }
    }
}

// Runs that span tiles: the tail of the tile in which one begins and the heads
// of the m tiles it goes on through.  A block takes a tile and a slice (most
// find nothing to do); its warps add up an eighth of the heads each, in tile
// order, and the first one adds their sums to the tail in warp order.
// A gradient that is written whole gets its zeros here.  They need the sort
// alone, but start after this kernel's wait for the sums all the same: nothing
// else makes the sort's `seen` visible to this kernel, and a row that a stale
// word calls unnamed would lose its sum.
template <typename TG, int VE, int NG, bool ADD>
__global__ void __launch_bounds__(kSumThreads)
    k_embed_join(const uint2 *sorted, int64_t T, int64_t V, int H, float scale, int tile_rows,
                 uint32_t slices, uint32_t items, TG *__restrict__ dtable, int64_t ld,
                 const float *partial, int64_t part_ld, const uint32_t *seen,
                 int rows_per_fill)
{
    pdl_begin();
    constexpr int U = 4;
    constexpr int kCols = kWarp * VE * NG;
    __shared__ __align__(16) float s_part[kSumWarps][kCols];
    const int nstep = H / VE;
    const int lane = (int)lane_id(), w = threadIdx.x / kWarp;
    const Slice<VE, NG> mine{lane, kWarp * NG};
    for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) { // (block-uniform)
        const int64_t c = it / slices;
        const int64_t i0 = c * tile_rows, i1 = i0 + tile_rows;
        auto goes_on = [&](int64_t m, uint32_t key) { // does the run reach the m-th tile from i1 on
            return i1 + m * tile_rows < T && sorted[i1 + m * tile_rows].x == key;
        };
        const uint32_t key = sorted[i1 - 1].x;
        const uint32_t before = i0 > 0 ? sorted[i0 - 1].x : (uint32_t)V;
        const uint32_t first = __ballot_sync(0xffffffffu, goes_on(lane, key));
        if (key == (uint32_t)V || !(first & 1) || before == key) continue; // none, or an earlier tile's
        int64_t m = first == 0xffffffffu ? 32 : __ffs(~first) - 1;
        while (m % kWarp == 0) {
            const uint32_t more = __ballot_sync(0xffffffffu, goes_on(m + lane, key));
            if (!more) break;
            m += more == 0xffffffffu ? 32 : __ffs(~more) - 1;
        }
        const Slice<VE, NG> sl{(int)(it - (uint32_t)c * slices) * kWarp * NG + lane, nstep};
        Pack<TG, VE> old[NG];
        Pack<float, VE> tail[NG];
        if (ADD) load_row(old, dtable + (int64_t)key * ld, sl, w == 0);
        load_row(tail, partial + (2 * c + 1) * part_ld, sl, w == 0);
        Sums<VE, NG> acc;
        zero(acc);
        const int64_t q1 = c + 1 + (w + 1) * m / kSumWarps;
        for (int64_t q = c + 1 + w * m / kSumWarps; q < q1; q += U) {
            Pack<float, VE> p[U][NG];
#pragma unroll
            for (int u = 0; u < U; ++u) load_row(p[u], partial + 2 * (q + u) * part_ld, sl, q + u < q1);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (q + u < q1) add_row(acc, p[u]);
        }
        store_part(s_part[w], mine, acc);
        __syncthreads();
        if (w == 0) {
            zero(acc);
            add_row(acc, tail);
#pragma unroll
            for (int q = 0; q < kSumWarps; ++q) {
                Pack<float, VE> p[NG];
                load_part(p, s_part[q], mine);
                add_row(acc, p);
            }
            finish_row(dtable + (int64_t)key * ld, sl, acc, old, scale, ADD);
        }
        __syncthreads();
    }
    if (!ADD) {
        auto seen_from = [&](int64_t r0) {
            struct Word {
                uint32_t bits;
            } word;
            load_now(word, reinterpret_cast<const Word *>(seen) + (r0 >> 5), true); // (stays behind the wait)
            return word.bits >> (r0 & 31);
        };
        fill_rows<TG, kSumWarps>((V + rows_per_fill - 1) / rows_per_fill, rows_per_fill, V, H, dtable, ld, seen_from);
    }
}

// Up to kSmallTokens tokens in one launch, without work space: every block
// sorts all of them for itself in shared memory (up to kRankTokens by counting
// the tokens before each, else by radix passes) and then adds up its share of
// the runs over its slice of the columns: run q belongs to group q % groups.
// A run is cut into pieces of kPiece rows, one warp each; the pieces of a
// longer run meet in shared memory and are added in order.  Without an old
// gradient the rows that no id names are shared out over all blocks.
constexpr int64_t kSmallTokens = kClThreads;
constexpr int kRankTokens = 256; // 6.3 us at 256 x 2048 by counting, 8.4 us by radix passes
constexpr int kPiece = 16;
// pieces of runs longer than one piece: a run of n > 16 has at most 2 n / 17
constexpr int kLongPieces = 2 * (int)kSmallTokens / (kPiece + 1) + 1;
constexpr int kSmallCols = 128;

template <typename TD, typename TG, int VE, bool ADD>
__global__ void __launch_bounds__(kClThreads, 1)
    k_embed_small(const TD *dout, int64_t dout_ld, const void *ids, bool wide, int T,
                  int64_t V, int64_t pad, int H, float scale, int passes, int bits, int slices, int groups,
                  TG *__restrict__ dtable, int64_t ld, int rows_per_fill, uint32_t *d_status)
{
    pdl_begin();
    constexpr int NG = kSmallCols / kWarp / VE;
    extern __shared__ __align__(16) uint8_t s_mem[];
    uint2 *sorted = reinterpret_cast<uint2 *>(s_mem);
    float *s_part = reinterpret_cast<float *>(s_mem + kClThreads * sizeof(uint2)); // after the sort: [kLongPieces][128]
    __shared__ uint32_t s_piece[kSmallTokens], s_count[kClWarps];
    __shared__ int s_head[kClWarps];
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp, tid = threadIdx.x;
    const uint32_t none = (uint32_t)V;
    const uint32_t key =
        tid < T ? sort_key(ids, wide, tid, V, pad, blockIdx.x == 0 ? d_status : nullptr) : none;
    if (key != none && tid % gridDim.x == blockIdx.x) { // its rows start towards L2 while the tokens are sorted
        prefetch_l2(dout + tid * dout_ld, (int64_t)H * sizeof(TD));
        if (ADD) prefetch_l2(dtable + key * ld, (int64_t)H * sizeof(TG));
    }
    if (T <= kRankTokens) {
        uint32_t *s_key = s_piece; // (free until the pieces are listed)
        if (tid < kRankTokens) s_key[tid] = key;
        __syncthreads();
        // four threads count a token's predecessors: smaller keys, and equal ones of lower tokens
        const int t = tid / 4;
        const uint32_t mine = s_key[t];
        uint32_t rank = 0;
        for (int c = tid & 3; c < T; c += 4) {
            const uint32_t other = s_key[c];
            rank += other < mine || (other == mine && c < t);
        }
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        rank += __shfl_xor_sync(0xffffffffu, rank, 2);
        if (t < T && (tid & 3) == 0) sorted[rank] = make_uint2(mine, (uint32_t)t);
    } else {
        sort_passes<1, false>(
            T, T, passes, bits, sorted, [&](int) { return key; }, // (a thread's first token is its own)
            [&](uint32_t at, uint2 pair, bool in) {
                if (in) sorted[at] = pair;
            });
    }
    __syncthreads();
    // the pieces of this block's runs: first token, and for the pieces of longer runs their place in s_part
    const int group = blockIdx.x / slices;
    const uint32_t k = tid < T ? sorted[tid].x : none;
    const bool live = k != none;
    const bool head = live && (tid == 0 || sorted[tid - 1].x != k);
    const uint32_t heads = __ballot_sync(0xffffffffu, head);
    if (lane == 0) {
        s_head[wid] = heads ? wid * kWarp + 31 - __clz(heads) : -1;
        s_count[wid] = __popc(heads);
    }
    __syncthreads();
    int start = __reduce_max_sync(0xffffffffu, lane < wid ? s_head[lane] : -1);
    int run = (int)__reduce_add_sync(0xffffffffu, lane < wid ? s_count[lane] : 0u);
    const uint32_t upto = heads & (lanemask_lt() | 1u << lane);
    if (upto) start = wid * kWarp + 31 - __clz(upto);
    run += __popc(upto) - 1;
    const bool piece = live && (tid - start) % kPiece == 0 && run % groups == group;
    const bool part = piece && (tid != start || (tid + kPiece < T && sorted[tid + kPiece].x == k)); // of a longer run
    const uint32_t pieces = __ballot_sync(0xffffffffu, piece), parts = __ballot_sync(0xffffffffu, part);
    __syncthreads(); // s_count is read
    if (lane == 0) s_count[wid] = __popc(pieces) | __popc(parts) << 16;
    __syncthreads();
    uint32_t at = __reduce_add_sync(0xffffffffu, lane < wid ? s_count[lane] : 0u);
    const int count = (int)(__reduce_add_sync(0xffffffffu, s_count[lane]) & 0xffffu);
    constexpr uint32_t kPart = 1u << 31, kFirst = 1u << 30;
    if (piece)
        s_piece[(at & 0xffffu) + __popc(pieces & lanemask_lt())] =
            (uint32_t)tid | ((at >> 16) + __popc(parts & lanemask_lt())) << 16 | (part ? kPart : 0u) |
            (tid == start ? kFirst : 0u);
    __syncthreads();

    const Slice<VE, NG> mine{lane, kSmallCols / VE};
    if (group < groups) {
        const int slice = blockIdx.x % slices;
        const int col0 = slice * kSmallCols, cols = H - col0 < kSmallCols ? H - col0 : kSmallCols;
        const Slice<VE, NG> here{lane, cols / VE};
        for (int j = wid; j < count; j += kClWarps) {
            const uint32_t info = s_piece[j];
            const int i = (int)(info & 0xffffu);
            const uint2 my = i + lane < T ? sorted[i + lane] : make_uint2(none, 0u);
            const uint32_t id = __shfl_sync(0xffffffffu, my.x, 0);
            const int n = __popc(__ballot_sync(0xffffffffu, lane < kPiece && my.x == id));
            TG *row = dtable + id * ld + col0;
            Pack<TG, VE> old[NG];
            if (ADD) load_row(old, row, here, !(info & kPart));
            Sums<VE, NG> acc;
            zero(acc);
            constexpr int U = 8;
            for (int r0 = 0; r0 < n; r0 += U) {
                Pack<TD, VE> v[U][NG];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint32_t tok = __shfl_sync(0xffffffffu, my.y, r0 + u);
                    load_row(v[u], dout + tok * dout_ld + col0, here, r0 + u < n);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r0 + u < n) add_row(acc, v[u]);
            }
            if (info & kPart)
                store_part(s_part + (info >> 16 & 0x3fff) * kSmallCols, mine, acc);
            else
                finish_row(row, here, acc, old, scale, ADD);
        }
        __syncthreads();
        for (int j = wid; j < count; j += kClWarps) { // longer runs, by the warp of their first piece
            const uint32_t info = s_piece[j];
            if ((info & (kPart | kFirst)) != (kPart | kFirst)) continue;
            TG *row = dtable + sorted[info & 0xffffu].x * ld + col0;
            Pack<TG, VE> old[NG];
            if (ADD) load_row(old, row, here);
            Sums<VE, NG> acc;
            zero(acc);
            for (int q = j; q < count && (q == j || (s_piece[q] & (kPart | kFirst)) == kPart); ++q) {
                Pack<float, VE> p[NG];
                load_part(p, s_part + (s_piece[q] >> 16 & 0x3fff) * kSmallCols, mine);
                add_row(acc, p);
            }
            finish_row(row, here, acc, old, scale, ADD);
        }
    }
    if (ADD) return;
    auto seen_from = [&](int64_t r0) { // a lane looks for one row
        const uint32_t want = (uint32_t)(r0 + lane);
        int lo = 0, hi = T;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sorted[mid].x < want)
                lo = mid + 1;
            else
                hi = mid;
        }
        return __ballot_sync(0xffffffffu, lo < T && sorted[lo].x == want);
    };
    fill_rows<TG, kClWarps>((V + rows_per_fill - 1) / rows_per_fill, rows_per_fill, V, H, dtable, ld, seen_from);
}

// ---- host ------------------------------------------------------------------------
struct EmbedPlan {
    int passes, bits; // radix passes and bits per digit
    int rows;         // sorted tokens per warp of the sums
    int64_t tiles, sum_tiles, part_ld;
    int64_t off_b, off_hist, off_seen, off_part, bytes; // (sorted tokens, one of two buffers, at offset 0)
};

EmbedPlan embed_plan(int64_t T, int64_t V, int32_t H)
{
    EmbedPlan p = {};
    int bits = 1;
    while (bits < 32 && (V >> bits)) ++bits; // keys 0 .. V
    p.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    // (a call's cluster may have fewer blocks than 16: the passes over memory have room from one block's tokens on)
    p.tiles = T > kClBlockTokens ? (T + kSortTile - 1) / kSortTile : 0;
    // the longest tiles that still give kWantItems blocks work (pieces of 256 columns): half as long, they take 169 us
    // for 156 at 32768 x 7168 and 29.2 for 28.3 at 8192 x 2048, since the warps of a block wait for one another per tile
    const int64_t pieces = ((int64_t)H + 255) / 256;
    p.rows = kSumRowsMax;
    while (p.rows > 4 && T * pieces < kWantItems * p.rows * kSumWarps) p.rows /= 2;
    p.sum_tiles = (T + p.rows * kSumWarps - 1) / (p.rows * kSumWarps);
    p.part_ld = ((int64_t)H + 7) / 8 * 8;
    // no work space: one launch, 11.2 us at 1024 x 2048 where three take 13.0, and 7 us of host time for 18
    if (T <= kSmallTokens) return p;
    auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    p.off_b = up(T * 8);
    p.off_hist = p.off_b + (p.tiles ? up(T * 8) : 0);
    p.off_seen = p.off_hist + up((p.tiles << p.bits) * 4);
    p.off_part = p.off_seen + up((V + 31) / 32 * 4);
    p.bytes = p.off_part + up(2 * p.sum_tiles * p.part_ld * 4);
    return p;
}

// Lets k_sort_cluster<ITEMS> have its shared memory and clusters of 16.
template <int ITEMS> cudaError_t sort_attributes()
{
    static const cudaError_t attr = [] {
        const void *k = (const void *)k_sort_cluster<ITEMS>;
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)cluster_smem(ITEMS, kMaxDigitBits, kClBlocksMax));
        return e != cudaSuccess ? e : cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    }();
    return attr;
}

template <int ITEMS>
ap_status sort_cluster(const void *ids, bool wide, int64_t T, int64_t V, int64_t pad, const EmbedPlan &p, int blocks,
                       uint2 *sorted, uint32_t *seen, uint32_t *d_status, cudaStream_t st)
{
    const cudaError_t attr = sort_attributes<ITEMS>();
    if (attr != cudaSuccess) return cuda_fail(attr, "embed_backward sort");
    launch_cluster(k_sort_cluster<ITEMS>, blocks, kClThreads, cluster_smem(ITEMS, p.bits, blocks), blocks, st, ids,
                   wide, (int)T, (int)((T + blocks - 1) / blocks), V, pad, p.passes, p.bits, sorted, seen, d_status);
    AP_CHECK_LAUNCH("embed_backward sort launch");
    return AP_OK;
}

// Sorts the tokens into one of the two buffers at `sc`; *sorted is set to it.
// seen (may be NULL): a bit for every id that occurs.
ap_status sort_tokens(const void *ids, bool wide, int64_t T, int64_t V, int64_t pad, const EmbedPlan &p, char *sc,
                      uint2 **sorted, uint32_t *seen, uint32_t *d_status, cudaStream_t st)
{
    uint2 *buf[2] = {reinterpret_cast<uint2 *>(sc), reinterpret_cast<uint2 *>(sc + p.off_b)};
    *sorted = buf[0];
    const cudaError_t attr = sort_attributes<kClItemsMax>();
    if (attr != cudaSuccess) return cuda_fail(attr, "embed_backward sort");
    const int most = cluster_fit((const void *)k_sort_cluster<kClItemsMax>, kClThreads,
                                 cluster_smem(kClItemsMax, kMaxDigitBits, kClBlocksMax), kClBlocksMax, st);
    if (T <= most * kClBlockTokens) { // 131072 x 512: 87 us in all, with the passes below 137
        int blocks = 1;
        while (blocks < most && (int64_t)blocks * kClThreads < T) blocks *= 2;
        const int64_t each = ((T + blocks - 1) / blocks + kClThreads - 1) / kClThreads; // tokens per thread
        if (each <= 1) return sort_cluster<1>(ids, wide, T, V, pad, p, blocks, buf[0], seen, d_status, st);
        if (each <= 2) return sort_cluster<2>(ids, wide, T, V, pad, p, blocks, buf[0], seen, d_status, st);
        if (each <= 4) return sort_cluster<4>(ids, wide, T, V, pad, p, blocks, buf[0], seen, d_status, st);
        return sort_cluster<8>(ids, wide, T, V, pad, p, blocks, buf[0], seen, d_status, st);
    }
    uint32_t *hist = reinterpret_cast<uint32_t *>(sc + p.off_hist);
    const int scan = cluster_fit((const void *)k_sort_scan, kScanThreads, 0, kScanBlocks, st);
    for (int q = 0; q < p.passes; ++q) {
        const uint2 *in = q ? buf[(q - 1) & 1] : nullptr;
        launch(k_sort_count, (int)p.tiles, kSortThreads, 0, st, in, ids, wide, T, V, pad, q * p.bits, p.bits, hist,
               q == 0 ? seen : nullptr, d_status);
        AP_CHECK_LAUNCH("embed_backward count launch");
        launch_cluster(k_sort_scan, scan, kScanThreads, 0, scan, st, hist, p.tiles << p.bits);
        AP_CHECK_LAUNCH("embed_backward scan launch");
        launch(k_sort_scatter, (int)p.tiles, kSortThreads, 0, st, in, ids, wide, T, V, pad, q * p.bits, p.bits, hist,
               buf[q & 1], q + 1 == p.passes ? seen : nullptr);
        AP_CHECK_LAUNCH("embed_backward scatter launch");
        *sorted = buf[q & 1];
    }
    return AP_OK;
}

bool row_type(int32_t d) { return d == AP_DTYPE_BF16 || d == AP_DTYPE_F32; }
int64_t size_of(int32_t d) { return d == AP_DTYPE_F32 ? 4 : 2; }

// Rows of a buffer can be taken in vectors of VE elements.
bool vec_ok(const void *p, int64_t ld, int32_t dtype, int ve)
{
    const int64_t bytes = ve * size_of(dtype) < 16 ? ve * size_of(dtype) : 16;
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * size_of(dtype) % bytes == 0;
}

int grid_for(int64_t items_per_warp, int resident)
{
    const int64_t want = (items_per_warp + 7) / 8;
    return (int)(want < 1 ? 1 : want < resident ? want : resident);
}

template <typename TI, typename TO>
void embed_typed(const void *table, int64_t V, int64_t ld, int32_t tt, const void *ids, bool wide, int64_t T, int H,
                 float scale, void *out, int64_t out_ld, int32_t ot, uint32_t *d_status, cudaStream_t st)
{
    constexpr bool half = sizeof(TI) == 2 && sizeof(TO) == 2;
    constexpr int VE = half ? 8 : 4;
    const auto go = [&](auto kernel, int per, int resident) {
        const int64_t items = T * ((H + per - 1) / per);
        launch(kernel, grid_for(items, resident), 256, 0, st, static_cast<const TI *>(table), V, ld, ids, wide, T, H,
               scale, static_cast<TO *>(out), out_ld, d_status);
    };
#define AP_EMBED(PER, ...)                                                               \
    do {                                                                                 \
        static const int resident = resident_grid((const void *)__VA_ARGS__, 256);       \
        go(__VA_ARGS__, (PER) * kWarp, resident);                                        \
    } while (0)
    // The widest elements that the rows' alignment allows: 16384 rows of 2048, 2046 and 2047 BF16 take 18.5, 18.7 and
    // 19.6 us (the last by elements: 24.5).  Vectors of a lane in flight: 32768 x 7168 rows 114.3 us (2: 115.3, 8: 114.8).
    if (H % VE == 0 && vec_ok(table, ld, tt, VE) && vec_ok(out, out_ld, ot, VE))
        AP_EMBED(VE * 4, k_embed<TI, TO, VE, 4>);
    else if (H % 2 == 0 && vec_ok(table, ld, tt, 2) && vec_ok(out, out_ld, ot, 2))
        AP_EMBED(2 * 8, k_embed<TI, TO, 2, 8>);
    else if constexpr (half)
        AP_EMBED(2 * 8, k_embed_odd<8>);
    else
        AP_EMBED(16, k_embed<TI, TO, 1, 16>);
#undef AP_EMBED
}

// What the sums kernels take besides their types.
struct SumArgs {
    const void *dout;
    int64_t dout_ld;
    const uint2 *sorted;
    int64_t T, V;
    int H;
    float scale;
    void *dtable;
    int64_t ld;
    float *partial;
    const uint32_t *seen;
    const void *ids;
    bool wide;
    int64_t pad;
    uint32_t *d_status;
};

// Rows of zeros that a warp writes at a time: at most 16 KB, and fewer where that leaves blocks without any (one token,
// 3263 x 108 FP32: 3.8 us, 9.6 with 32 rows a warp and 32 warps a block).
int fill_rows_of(int64_t V, int64_t row_bytes, int64_t blocks)
{
    int rows = 32;
    while (rows > 1 && (rows * row_bytes > (16 << 10) || V < rows * blocks)) rows /= 2;
    return rows;
}

template <typename TD, typename TG, int VE, int NG, bool ADD, Route R>
ap_status embed_sums(const SumArgs &a, const EmbedPlan &p, cudaStream_t st)
{
    TG *dtable = static_cast<TG *>(a.dtable);
    const int slices = (a.H / VE + kWarp * NG - 1) / (kWarp * NG);
    const auto kernel = k_embed_sum<TD, TG, VE, NG, ADD, R>;
    constexpr int smem = kSumSmem<TD, TG, VE, NG, ADD, R>;
    static const cudaError_t attr = cudaFuncSetAttribute((const void *)kernel,
                                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (attr != cudaSuccess) return cuda_fail(attr, "embed_backward sum");
    static const int resident = resident_grid((const void *)kernel, kSumThreads, smem);
    // (more than kSmallTokens tokens: several tiles)
    const int64_t items = p.sum_tiles * slices, joins = (p.sum_tiles - 1) * slices;
    if (items > INT32_MAX)
        return fail(AP_EINVAL, "embed_backward: %lld tokens of %d columns are more than one launch takes", (long long)a.T,
                    a.H);
    launch(kernel, (int)(items < resident ? items : resident), kSumThreads, smem, st, static_cast<const TD *>(a.dout),
           a.dout_ld, a.sorted, a.T, a.V, a.H, a.scale, p.rows, (uint32_t)slices, (uint32_t)items, dtable, a.ld,
           a.partial, p.part_ld, a.ids, a.wide, a.pad, a.d_status);
    AP_CHECK_LAUNCH("embed_backward sum launch");
    static const int resident_j = resident_grid((const void *)k_embed_join<TG, VE, NG, ADD>, kSumThreads);
    const int rows = fill_rows_of(a.V, (int64_t)a.H * sizeof(TG), resident_j);
    const int64_t fills = ADD ? 0 : (a.V + rows - 1) / rows; // blocks the zeros can use
    const int64_t grid = joins > fills ? joins : fills;
    launch(k_embed_join<TG, VE, NG, ADD>, (int)(grid < resident_j ? grid : resident_j), kSumThreads, 0, st, a.sorted, a.T,
           a.V, a.H, a.scale, p.rows * kSumWarps, (uint32_t)slices, (uint32_t)joins, dtable, a.ld, a.partial, p.part_ld,
           a.seen, rows);
    AP_CHECK_LAUNCH("embed_backward join launch");
    return AP_OK;
}

template <typename TD, typename TG, int VE, bool ADD>
ap_status embed_small(const SumArgs &a, const EmbedPlan &p, cudaStream_t st)
{
    const auto kernel = k_embed_small<TD, TG, VE, ADD>;
    constexpr size_t parts = kClThreads * sizeof(uint2) + (size_t)kLongPieces * kSmallCols * 4;
    constexpr size_t most = cluster_smem(1, kMaxDigitBits, 1) > parts ? cluster_smem(1, kMaxDigitBits, 1) : parts;
    static const cudaError_t attr =
        cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (attr != cudaSuccess) return cuda_fail(attr, "embed_backward");
    // as many groups of runs as fill the SMs once, each of some 32 tokens at least
    const int sms = sm_count();
    const int64_t slices = (a.H + kSmallCols - 1) / kSmallCols;
    int64_t groups = a.T > 32 ? (a.T + 31) / 32 : 1;
    if (groups * slices > sms) groups = sms / slices > 0 ? sms / slices : 1;
    const int rows = fill_rows_of(a.V, (int64_t)a.H * sizeof(TG), sms);
    int64_t grid = groups * slices;
    if (!ADD) { // enough blocks for the zeros
        const int64_t fills = (a.V + rows - 1) / rows;
        if (grid < (fills < sms ? fills : sms)) grid = fills < sms ? fills : sms;
    }
    launch(kernel, (int)(grid > 0 ? grid : 1), kClThreads, most, st, static_cast<const TD *>(a.dout), a.dout_ld, a.ids,
           a.wide, (int)a.T, a.V, a.pad, a.H, a.scale, p.passes, p.bits, (int)slices, (int)groups,
           static_cast<TG *>(a.dtable), a.ld, rows, a.d_status);
    AP_CHECK_LAUNCH("embed_backward launch");
    return AP_OK;
}

template <typename TD, typename TG>
ap_status embed_backward_typed(const SumArgs &a, int32_t dt, int32_t gt, bool add, const EmbedPlan &p, cudaStream_t st)
{
    const bool even = a.H % 2 == 0 && vec_ok(a.dout, a.dout_ld, dt, 2) && vec_ok(a.dtable, a.ld, gt, 2);
    if (a.T <= kSmallTokens) {
        if (a.H % 4 == 0 && vec_ok(a.dout, a.dout_ld, dt, 4) && vec_ok(a.dtable, a.ld, gt, 4))
            return add ? embed_small<TD, TG, 4, true>(a, p, st) : embed_small<TD, TG, 4, false>(a, p, st);
        if (even) return add ? embed_small<TD, TG, 2, true>(a, p, st) : embed_small<TD, TG, 2, false>(a, p, st);
        return add ? embed_small<TD, TG, 1, true>(a, p, st) : embed_small<TD, TG, 1, false>(a, p, st);
    }
    // 8192 rows of 1008 (16-byte boundaries), 1002 (pairs) and 1001 columns: 17.8, 19.6 and 20.3 us; element-wise loads
    // through registers took 36.8 us for the last
    constexpr int N = kDoutBytes / kWarp / (int)sizeof(TD); // a lane's columns of a slice
    constexpr int VE = sizeof(TD) == 2 && sizeof(TG) == 2 ? 8 : 4;
    constexpr int V16 = sizeof(TD) == 2 || sizeof(TG) == 2 ? 8 : 4;
    if (a.H % V16 == 0 && vec_ok(a.dout, a.dout_ld, dt, V16) && vec_ok(a.dtable, a.ld, gt, V16))
        return add ? embed_sums<TD, TG, VE, N / VE, true, kAligned>(a, p, st)
                   : embed_sums<TD, TG, VE, N / VE, false, kAligned>(a, p, st);
    if (even)
        return add ? embed_sums<TD, TG, 2, N / 2, true, kAnywhere>(a, p, st)
                   : embed_sums<TD, TG, 2, N / 2, false, kAnywhere>(a, p, st);
    return add ? embed_sums<TD, TG, 1, N, true, kAnywhere>(a, p, st)
               : embed_sums<TD, TG, 1, N, false, kAnywhere>(a, p, st);
}

// (columns: so that an index of a row and the bytes of a row stay well inside 32 bits)
bool embed_sizes_ok(int64_t T, int64_t V, int32_t H)
{
    return T >= 0 && T < (int64_t(1) << 31) && V >= 1 && V < (int64_t(1) << 31) && H >= 1 && H <= 1 << 28;
}

} // namespace
} // namespace ap

extern "C" ap_status ap_embed(const void *table, int64_t V, int64_t table_ld, int32_t table_dtype, const void *ids,
                              int32_t id_bytes, int64_t T, int32_t H, float scale, void *out, int64_t out_ld,
                              int32_t out_dtype, uint32_t *d_status, void *stream)
{
    AP_NVTX_RANGE("ap_embed");
    using namespace ap;
    if (!embed_sizes_ok(T, V, H) || table_ld < H || out_ld < H)
        return fail(AP_EINVAL, "embed: bad sizes T=%lld V=%lld H=%d table_ld=%lld out_ld=%lld", (long long)T,
                    (long long)V, H, (long long)table_ld, (long long)out_ld);
    if (!row_type(table_dtype) || !row_type(out_dtype) || (id_bytes != 4 && id_bytes != 8))
        return fail(AP_EINVAL, "embed: bad types (table %d, out %d, ids of %d bytes)", table_dtype, out_dtype,
                    id_bytes);
    if (T == 0) return AP_OK;
    if (!table || !ids || !out) return fail(AP_EINVAL, "embed: NULL pointer");
    if (reinterpret_cast<uintptr_t>(table) % size_of(table_dtype) || reinterpret_cast<uintptr_t>(ids) % id_bytes ||
        reinterpret_cast<uintptr_t>(out) % size_of(out_dtype))
        return fail(AP_EINVAL, "embed: pointer not aligned to its elements");
    cudaStream_t st = (cudaStream_t)stream;
    const bool wide = id_bytes == 8, fi = table_dtype == AP_DTYPE_F32, fo = out_dtype == AP_DTYPE_F32;
#define AP_EMBED(TI, TO)                                                                                        \
    embed_typed<TI, TO>(table, V, table_ld, table_dtype, ids, wide, T, H, scale, out, out_ld, out_dtype, d_status, \
                        st)
    if (fi && fo)
        AP_EMBED(float, float);
    else if (fi)
        AP_EMBED(float, bf16_t);
    else if (fo)
        AP_EMBED(bf16_t, float);
    else
        AP_EMBED(bf16_t, bf16_t);
#undef AP_EMBED
    AP_CHECK_LAUNCH("embed launch");
    return AP_OK;
}

extern "C" ap_status ap_embed_scratch_bytes(int64_t T, int64_t V, int32_t H, int64_t *bytes)
{
    using namespace ap;
    if (!bytes || !embed_sizes_ok(T, V, H))
        return fail(AP_EINVAL, "embed_scratch_bytes: bad sizes T=%lld V=%lld H=%d", (long long)T, (long long)V, H);
    *bytes = embed_plan(T, V, H).bytes;
    return AP_OK;
}

extern "C" ap_status ap_embed_backward(const void *dout, int64_t dout_ld, int32_t dout_dtype, const void *ids,
                                       int32_t id_bytes, int64_t T, int32_t H, int64_t V, int64_t padding_idx,
                                       float scale, int32_t accumulate, void *dtable, int64_t dtable_ld,
                                       int32_t dtable_dtype, void *scratch, int64_t scratch_bytes, uint32_t *d_status,
                                       void *stream)
{
    AP_NVTX_RANGE("ap_embed_backward");
    using namespace ap;
    if (!embed_sizes_ok(T, V, H) || dout_ld < H || dtable_ld < H || padding_idx < -1 || padding_idx >= V)
        return fail(AP_EINVAL,
                    "embed_backward: bad sizes T=%lld V=%lld H=%d dout_ld=%lld dtable_ld=%lld padding_idx=%lld",
                    (long long)T, (long long)V, H, (long long)dout_ld, (long long)dtable_ld, (long long)padding_idx);
    if (!row_type(dout_dtype) || !row_type(dtable_dtype) || (id_bytes != 4 && id_bytes != 8) || accumulate < 0 ||
        accumulate > 1)
        return fail(AP_EINVAL, "embed_backward: bad types (dout %d, dtable %d, ids of %d bytes, accumulate %d)",
                    dout_dtype, dtable_dtype, id_bytes, accumulate);
    if (T == 0 && accumulate) return AP_OK;
    const EmbedPlan p = embed_plan(T, V, H);
    if (!dtable || (T > 0 && (!dout || !ids)) || (p.bytes > 0 && !scratch))
        return fail(AP_EINVAL, "embed_backward: NULL pointer");
    if (reinterpret_cast<uintptr_t>(dout) % size_of(dout_dtype) || reinterpret_cast<uintptr_t>(ids) % id_bytes ||
        reinterpret_cast<uintptr_t>(dtable) % size_of(dtable_dtype) || (reinterpret_cast<uintptr_t>(scratch) & 15))
        return fail(AP_EINVAL, "embed_backward: pointer not aligned");
    if (scratch_bytes < p.bytes)
        return fail(AP_EINVAL, "embed_backward: scratch of %lld bytes, %lld needed", (long long)scratch_bytes,
                    (long long)p.bytes);
    cudaStream_t st = (cudaStream_t)stream;
    char *sc = static_cast<char *>(scratch);
    SumArgs a = {dout, dout_ld, nullptr, T, V, H, scale, dtable, dtable_ld, nullptr, nullptr, ids, id_bytes == 8,
                 padding_idx, d_status};
    if (T > kSmallTokens) {
        uint32_t *seen = reinterpret_cast<uint32_t *>(sc + p.off_seen);
        uint2 *sorted = nullptr;
        const ap_status ss = sort_tokens(ids, id_bytes == 8, T, V, padding_idx, p, sc, &sorted,
                                         accumulate ? nullptr : seen, d_status, st);
        if (ss != AP_OK) return ss;
        a.sorted = sorted;
        a.partial = reinterpret_cast<float *>(sc + p.off_part);
        a.seen = seen;
    }
    const bool fd = dout_dtype == AP_DTYPE_F32, fg = dtable_dtype == AP_DTYPE_F32, add = accumulate != 0;
    if (fd && fg) return embed_backward_typed<float, float>(a, dout_dtype, dtable_dtype, add, p, st);
    if (fd) return embed_backward_typed<float, bf16_t>(a, dout_dtype, dtable_dtype, add, p, st);
    if (fg) return embed_backward_typed<bf16_t, float>(a, dout_dtype, dtable_dtype, add, p, st);
    return embed_backward_typed<bf16_t, bf16_t>(a, dout_dtype, dtable_dtype, add, p, st);
}
