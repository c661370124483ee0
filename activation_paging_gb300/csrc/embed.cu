// Embedding lookup with a scale, and the gradient of the table.
//
// Lookup: out[t] = round(scale * table[ids[t]]), one warp per piece of a row.
//
// Gradient: dtable[v] (+)= scale * sum over the tokens with id v of dout[t].
//   1. The tokens are sorted by id (stable radix sort, least significant digit
//      first; ids that do not count sort last), so an id's tokens are one run
//      in token order.
//   2. k_embed_sum: a warp takes kChunk sorted tokens and a piece of the
//      columns, adds rows up in single precision, and finishes each run that
//      lies inside its chunk in dtable.  A run that crosses chunks leaves one
//      partial row in each: `head` where it began earlier, `tail` where it
//      begins and goes on.
//   3. k_embed_join adds the partial rows of each such run in chunk order.
// No floating-point atomics: every sum has one order, fixed by ids and sizes.
#include <cuda_bf16.h>

#include "ap_common.cuh"

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

__device__ __forceinline__ int64_t load_id(const void *ids, bool wide, int64_t t)
{
    return wide ? static_cast<const int64_t *>(ids)[t] : (int64_t) static_cast<const int32_t *>(ids)[t];
}

// ---- lookup --------------------------------------------------------------------
template <typename TI, typename TO, int VE, int U>
__global__ void __launch_bounds__(256)
    k_embed(const TI *__restrict__ table, int64_t V, int64_t ld, const void *__restrict__ ids, bool wide, int64_t T,
            int H, float scale, TO *__restrict__ out, int64_t out_ld, uint32_t *d_status)
{
    pdl_begin();
    using PI = Pack<TI, VE>;
    using PO = Pack<TO, VE>;
    const int lane = (int)lane_id();
    const int nstep = H / VE;
    const int pieces = (nstep + U * kWarp - 1) / (U * kWarp);
    const int64_t items = T * pieces;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x / kWarp);
    for (int64_t it = (int64_t)blockIdx.x * (blockDim.x / kWarp) + threadIdx.x / kWarp; it < items; it += warps) {
        const int64_t t = it / pieces;
        const int s0 = (int)(it - t * pieces) * U * kWarp + lane;
        const int64_t id = load_id(ids, wide, t);
        const bool ok = id >= 0 && id < V;
        if (!ok && s0 == 0 && d_status) atomicOr(d_status, AP_FLAG_BAD_INDEX);
        const PI *src = reinterpret_cast<const PI *>(table + (ok ? id : 0) * ld);
        PO *dst = reinterpret_cast<PO *>(out + t * out_ld);
        PI r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (ok && s0 + u * kWarp < nstep) r[u] = src[s0 + u * kWarp];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u * kWarp >= nstep) continue;
            PO o;
#pragma unroll
            for (int i = 0; i < VE; ++i) o.v[i] = from_f<TO>(ok ? __fmul_rn(to_f(r[u].v[i]), scale) : 0.f);
            dst[s0 + u * kWarp] = o;
        }
    }
}

// ---- sort of the tokens by id ----------------------------------------------------
constexpr int kSortThreads = 256;
constexpr int kSortItems = 8;
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kMaxDigitBits = 10;

// Sort key of a token: its id, or V for one that does not count.
__device__ __forceinline__ uint32_t sort_key(const void *ids, bool wide, int64_t t, int64_t V, int64_t pad,
                                             uint32_t *d_status)
{
    const int64_t id = load_id(ids, wide, t);
    if (id == pad) return (uint32_t)V;
    if (id < 0 || id >= V) {
        if (d_status) atomicOr(d_status, AP_FLAG_BAD_INDEX);
        return (uint32_t)V;
    }
    return (uint32_t)id;
}

// Digit counts of each tile: hist[d * tiles + tile].  The first pass (keys ==
// NULL) reads the ids.
__global__ void __launch_bounds__(kSortThreads)
    k_sort_count(const uint32_t *__restrict__ keys, const void *__restrict__ ids, bool wide, int64_t T, int64_t V,
                 int64_t pad, int shift, int bits, uint32_t *__restrict__ hist, uint32_t *d_status)
{
    pdl_begin();
    __shared__ uint32_t s_hist[1 << kMaxDigitBits];
    const int D = 1 << bits;
    for (int d = threadIdx.x; d < D; d += kSortThreads) s_hist[d] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kSortTile;
    for (int i = 0; i < kSortItems; ++i) {
        const int64_t t = t0 + i * kSortThreads + threadIdx.x;
        if (t < T) {
            const uint32_t key = keys ? keys[t] : sort_key(ids, wide, t, V, pad, d_status);
            atomicAdd(&s_hist[(key >> shift) & (D - 1)], 1u);
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kSortThreads) hist[(int64_t)d * gridDim.x + blockIdx.x] = s_hist[d];
}

// Exclusive sum of n counts in place, one block.
__global__ void __launch_bounds__(1024) k_sort_scan(uint32_t *hist, int64_t n)
{
    pdl_begin();
    __shared__ uint32_t s_warp[32];
    __shared__ uint32_t s_carry;
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    if (threadIdx.x == 0) s_carry = 0;
    __syncthreads();
    for (int64_t i0 = 0; i0 < n; i0 += 1024) {
        const int64_t i = i0 + threadIdx.x;
        const uint32_t v = i < n ? hist[i] : 0u;
        uint32_t x = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) s_warp[wid] = x;
        __syncthreads();
        uint32_t base = s_carry;
        for (int q = 0; q < wid; ++q) base += s_warp[q];
        if (i < n) hist[i] = base + x - v;
        __syncthreads();
        if (threadIdx.x == 1023) s_carry = base + x;
        __syncthreads();
    }
}

// Moves every token of a tile to its place, keeping the order within a digit:
// warp q ranks its kSortItems * 32 consecutive tokens, 32 at a time.
__global__ void __launch_bounds__(kSortThreads)
    k_sort_scatter(const uint32_t *__restrict__ keys, const uint32_t *__restrict__ toks, const void *__restrict__ ids,
                   bool wide, int64_t T, int64_t V, int64_t pad, int shift, int bits,
                   const uint32_t *__restrict__ hist, uint32_t *__restrict__ keys_out, uint32_t *__restrict__ toks_out)
{
    pdl_begin();
    constexpr int W = kSortThreads / kWarp;
    __shared__ uint16_t s_cnt[W][1 << kMaxDigitBits];
    const int D = 1 << bits;
    const int lane = (int)lane_id(), wid = threadIdx.x / kWarp;
    for (int d = threadIdx.x; d < W * D; d += kSortThreads) s_cnt[d / D][d % D] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kSortTile + wid * (kSortItems * kWarp) + lane;
    uint32_t key[kSortItems], rank[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const int64_t t = t0 + i * kWarp;
        const bool in = t < T;
        key[i] = in ? (keys ? keys[t] : sort_key(ids, wide, t, V, pad, nullptr)) : 0u;
        // tokens past the end match nobody inside
        const int d = in ? (int)((key[i] >> shift) & (D - 1)) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        if (in) rank[i] = s_cnt[wid][d] + __popc(same & lanemask_lt());
        __syncwarp();
        if (in && (same >> lane) == 1u) s_cnt[wid][d] = (uint16_t)(rank[i] + 1); // the last of its digit
        __syncwarp();
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
        const int64_t t = t0 + i * kWarp;
        if (t >= T) continue;
        const int d = (int)((key[i] >> shift) & (D - 1));
        const uint32_t at = hist[(int64_t)d * gridDim.x + blockIdx.x] + s_cnt[wid][d] + rank[i];
        keys_out[at] = key[i];
        toks_out[at] = toks ? toks[t] : (uint32_t)t;
    }
}

// ---- sums of the runs ------------------------------------------------------------
constexpr int kChunk = 32;

// First position in [0, n) of the sorted keys that is >= key.
__device__ __forceinline__ int64_t lower_bound(const uint32_t *keys, int64_t n, uint32_t key)
{
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < key)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

template <typename TG, int VE>
__device__ __forceinline__ void finish_row(TG *row, int s, const float *acc, float scale, bool accumulate)
{
    using PG = Pack<TG, VE>;
    PG *p = reinterpret_cast<PG *>(row) + s;
    PG o;
    if (accumulate) {
        const PG old = *p;
#pragma unroll
        for (int i = 0; i < VE; ++i) o.v[i] = from_f<TG>(__fadd_rn(to_f(old.v[i]), __fmul_rn(scale, acc[i])));
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) o.v[i] = from_f<TG>(__fmul_rn(scale, acc[i]));
    }
    *p = o;
}

// Rows of ids that do not occur, set to zero: a warp takes kFillRows rows.
constexpr int kFillRows = 8;
template <typename TG, int VE>
__global__ void __launch_bounds__(256)
    k_embed_fill(const uint32_t *__restrict__ keys, int64_t T, int64_t V, int H, TG *__restrict__ dtable, int64_t ld)
{
    pdl_begin();
    using PG = Pack<TG, VE>;
    const int lane = (int)lane_id();
    const int nstep = H / VE;
    PG zero;
#pragma unroll
    for (int i = 0; i < VE; ++i) zero.v[i] = from_f<TG>(0.f);
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x / kWarp);
    for (int64_t r0 = ((int64_t)blockIdx.x * (blockDim.x / kWarp) + threadIdx.x / kWarp) * kFillRows; r0 < V;
         r0 += warps * kFillRows) {
        int64_t at = lower_bound(keys, T, (uint32_t)r0);
        for (int64_t r = r0; r < r0 + kFillRows && r < V; ++r) {
            if (at < T && keys[at] == (uint32_t)r) {
                at = lower_bound(keys, T, (uint32_t)r + 1);
                continue;
            }
            PG *row = reinterpret_cast<PG *>(dtable + r * ld);
            for (int s = lane; s < nstep; s += kWarp) row[s] = zero;
        }
    }
}

template <typename TD, typename TG, int VE, int U>
__global__ void __launch_bounds__(256)
    k_embed_sum(const TD *__restrict__ dout, int64_t dout_ld, const uint32_t *__restrict__ keys,
                const uint32_t *__restrict__ toks, int64_t T, int64_t V, int H, float scale, bool accumulate,
                TG *__restrict__ dtable, int64_t ld, float *__restrict__ partial, int64_t part_ld)
{
    pdl_begin();
    using PD = Pack<TD, VE>;
    using PF = Pack<float, VE>;
    const int lane = (int)lane_id();
    const int nstep = H / VE;
    const int pieces = (nstep + kWarp - 1) / kWarp;
    const int64_t chunks = (T + kChunk - 1) / kChunk;
    const int64_t items = chunks * pieces;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x / kWarp);
    for (int64_t it = (int64_t)blockIdx.x * (blockDim.x / kWarp) + threadIdx.x / kWarp; it < items; it += warps) {
        const int64_t c = it / pieces;
        const int s = (int)(it - c * pieces) * kWarp + lane;
        const int64_t i0 = c * kChunk;
        const int n = (int)(T - i0 < kChunk ? T - i0 : kChunk);
        const uint32_t none = (uint32_t)V;
        const uint32_t my_key = lane < n ? keys[i0 + lane] : none;
        const uint32_t my_tok = lane < n ? toks[i0 + lane] : 0u;
        const uint32_t before = i0 > 0 ? keys[i0 - 1] : none;
        const uint32_t after = i0 + n < T ? keys[i0 + n] : none;
        const int live = __popc(__ballot_sync(0xffffffffu, my_key != none)); // the ids that count come first
        float acc[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) acc[i] = 0.f;
        bool head = true; // still in the chunk's first run
        for (int r0 = 0; r0 < live; r0 += U) {
            PD v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t tok = __shfl_sync(0xffffffffu, my_tok, (r0 + u) & 31);
                if (r0 + u < live && s < nstep)
                    v[u] = reinterpret_cast<const PD *>(dout + (int64_t)tok * dout_ld)[s];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u;
                if (r >= live) break;
                const uint32_t key = __shfl_sync(0xffffffffu, my_key, r);
                const uint32_t next = r + 1 < n ? __shfl_sync(0xffffffffu, my_key, (r + 1) & 31) : after;
                if (s < nstep) {
#pragma unroll
                    for (int i = 0; i < VE; ++i) acc[i] = __fadd_rn(acc[i], to_f(v[u].v[i]));
                }
                const bool goes_on = r + 1 == n && next == key;
                if (r + 1 < n && next == key) continue;
                const bool began_before = head && before == key;
                if (s < nstep) {
                    if (!began_before && !goes_on) {
                        finish_row<TG, VE>(dtable + (int64_t)key * ld, s, acc, scale, accumulate);
                    } else {
                        PF o;
#pragma unroll
                        for (int i = 0; i < VE; ++i) o.v[i] = acc[i];
                        reinterpret_cast<PF *>(partial + (2 * c + (began_before ? 0 : 1)) * part_ld)[s] = o;
                    }
                }
                head = false;
#pragma unroll
                for (int i = 0; i < VE; ++i) acc[i] = 0.f;
            }
        }
    }
}

// Chunk c's tail run, where it goes on into later chunks: its tail and their
// heads, added in chunk order.  One block per chunk.
template <typename TG, int VE>
__global__ void __launch_bounds__(256)
    k_embed_join(const uint32_t *__restrict__ keys, int64_t T, int64_t V, int H, float scale, bool accumulate,
                 TG *__restrict__ dtable, int64_t ld, const float *__restrict__ partial, int64_t part_ld)
{
    pdl_begin();
    using PF = Pack<float, VE>;
    const int64_t chunks = (T + kChunk - 1) / kChunk;
    const int nstep = H / VE;
    for (int64_t c = blockIdx.x; c + 1 < chunks; c += gridDim.x) {
        const int64_t i0 = c * kChunk, i1 = i0 + kChunk;
        const uint32_t key = keys[i1 - 1];
        if (key == (uint32_t)V || keys[i1] != key) continue;
        if (i0 > 0 && keys[i0 - 1] == key) continue; // an earlier chunk's
        const int64_t last = (lower_bound(keys, T, key + 1) - 1) / kChunk;
        for (int s = threadIdx.x; s < nstep; s += blockDim.x) {
            PF a = reinterpret_cast<const PF *>(partial + (2 * c + 1) * part_ld)[s];
            for (int64_t q = c + 1; q <= last; ++q) {
                const PF b = reinterpret_cast<const PF *>(partial + 2 * q * part_ld)[s];
#pragma unroll
                for (int i = 0; i < VE; ++i) a.v[i] = __fadd_rn(a.v[i], b.v[i]);
            }
            finish_row<TG, VE>(dtable + (int64_t)key * ld, s, a.v, scale, accumulate);
        }
    }
}

// ---- host ------------------------------------------------------------------------
struct EmbedPlan {
    int passes, bits; // radix passes and bits per digit
    int64_t tiles, chunks, part_ld;
    int64_t off_k1, off_t0, off_t1, off_hist, off_part, bytes; // (keys 0 at offset 0)
};

EmbedPlan embed_plan(int64_t T, int64_t V, int32_t H)
{
    EmbedPlan p = {};
    int bits = 1;
    while (bits < 32 && (V >> bits)) ++bits; // keys 0 .. V
    p.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.tiles = (T + kSortTile - 1) / kSortTile;
    p.chunks = (T + kChunk - 1) / kChunk;
    p.part_ld = ((int64_t)H + 7) / 8 * 8;
    auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    p.off_k1 = up(T * 4);
    p.off_t0 = p.off_k1 + up(T * 4);
    p.off_t1 = p.off_t0 + up(T * 4);
    p.off_hist = p.off_t1 + up(T * 4);
    p.off_part = p.off_hist + up((p.tiles << p.bits) * 4);
    p.bytes = p.off_part + up(2 * p.chunks * p.part_ld * 4);
    return p;
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

template <typename TI, typename TO, int VE, int U>
void launch_embed(const void *table, int64_t V, int64_t ld, const void *ids, bool wide, int64_t T, int H, float scale,
                  void *out, int64_t out_ld, uint32_t *d_status, cudaStream_t st)
{
    static const int resident = resident_grid((const void *)k_embed<TI, TO, VE, U>, 256);
    const int64_t items = T * ((H / VE + U * kWarp - 1) / (U * kWarp));
    launch(k_embed<TI, TO, VE, U>, grid_for(items, resident), 256, 0, st, static_cast<const TI *>(table), V, ld, ids,
           wide, T, H, scale, static_cast<TO *>(out), out_ld, d_status);
}

template <typename TI, typename TO>
void embed_typed(const void *table, int64_t V, int64_t ld, int32_t tt, const void *ids, bool wide, int64_t T, int H,
                 float scale, void *out, int64_t out_ld, int32_t ot, uint32_t *d_status, cudaStream_t st)
{
    constexpr int VE = sizeof(TI) == 2 && sizeof(TO) == 2 ? 8 : 4;
    if (H % VE == 0 && vec_ok(table, ld, tt, VE) && vec_ok(out, out_ld, ot, VE))
        launch_embed<TI, TO, VE, 2>(table, V, ld, ids, wide, T, H, scale, out, out_ld, d_status, st);
    else
        launch_embed<TI, TO, 1, 4>(table, V, ld, ids, wide, T, H, scale, out, out_ld, d_status, st);
}

template <typename TD, typename TG, int VE>
ap_status embed_sums(const TD *dout, int64_t dout_ld, const uint32_t *keys, const uint32_t *toks, int64_t T, int64_t V,
                     int H, float scale, bool accumulate, TG *dtable, int64_t ld, float *partial, int64_t part_ld,
                     cudaStream_t st)
{
    if (!accumulate) {
        static const int resident = resident_grid((const void *)k_embed_fill<TG, VE>, 256);
        launch(k_embed_fill<TG, VE>, grid_for((V + kFillRows - 1) / kFillRows, resident), 256, 0, st, keys, T, V, H,
               dtable, ld);
        AP_CHECK_LAUNCH("embed_backward fill launch");
    }
    if (T == 0) return AP_OK;
    constexpr int U = VE == 1 ? 16 : 8;
    const int64_t chunks = (T + kChunk - 1) / kChunk;
    static const int resident = resident_grid((const void *)k_embed_sum<TD, TG, VE, U>, 256);
    const int64_t items = chunks * ((H / VE + kWarp - 1) / kWarp);
    launch(k_embed_sum<TD, TG, VE, U>, grid_for(items, resident), 256, 0, st, dout, dout_ld, keys, toks, T, V, H,
           scale, accumulate, dtable, ld, partial, part_ld);
    AP_CHECK_LAUNCH("embed_backward sum launch");
    if (chunks > 1) {
        static const int resident_j = resident_grid((const void *)k_embed_join<TG, VE>, 256);
        launch(k_embed_join<TG, VE>, (int)(chunks - 1 < resident_j ? chunks - 1 : resident_j), 256, 0, st, keys, T, V,
               H, scale, accumulate, dtable, ld, partial, part_ld);
        AP_CHECK_LAUNCH("embed_backward join launch");
    }
    return AP_OK;
}

template <typename TD, typename TG>
ap_status embed_backward_typed(const void *dout, int64_t dout_ld, int32_t dt, const uint32_t *keys,
                               const uint32_t *toks, int64_t T, int64_t V, int H, float scale, bool accumulate,
                               void *dtable, int64_t ld, int32_t gt, float *partial, int64_t part_ld, cudaStream_t st)
{
    constexpr int VE = sizeof(TD) == 2 ? 8 : 4;
    const TD *d = static_cast<const TD *>(dout);
    TG *g = static_cast<TG *>(dtable);
    if (H % VE == 0 && vec_ok(dout, dout_ld, dt, VE) && vec_ok(dtable, ld, gt, VE))
        return embed_sums<TD, TG, VE>(d, dout_ld, keys, toks, T, V, H, scale, accumulate, g, ld, partial, part_ld, st);
    return embed_sums<TD, TG, 1>(d, dout_ld, keys, toks, T, V, H, scale, accumulate, g, ld, partial, part_ld, st);
}

bool embed_sizes_ok(int64_t T, int64_t V, int32_t H)
{
    return T >= 0 && T < (int64_t(1) << 31) && V >= 1 && V < (int64_t(1) << 31) && H >= 1;
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
    if (!dtable || (T > 0 && (!dout || !ids || !scratch))) return fail(AP_EINVAL, "embed_backward: NULL pointer");
    if (reinterpret_cast<uintptr_t>(dout) % size_of(dout_dtype) || reinterpret_cast<uintptr_t>(ids) % id_bytes ||
        reinterpret_cast<uintptr_t>(dtable) % size_of(dtable_dtype) || (reinterpret_cast<uintptr_t>(scratch) & 15))
        return fail(AP_EINVAL, "embed_backward: pointer not aligned");
    const EmbedPlan p = embed_plan(T, V, H);
    if (T > 0 && scratch_bytes < p.bytes)
        return fail(AP_EINVAL, "embed_backward: scratch of %lld bytes, %lld needed", (long long)scratch_bytes,
                    (long long)p.bytes);
    cudaStream_t st = (cudaStream_t)stream;
    char *sc = static_cast<char *>(scratch);
    uint32_t *key[2] = {reinterpret_cast<uint32_t *>(sc), reinterpret_cast<uint32_t *>(sc + p.off_k1)};
    uint32_t *tok[2] = {reinterpret_cast<uint32_t *>(sc + p.off_t0), reinterpret_cast<uint32_t *>(sc + p.off_t1)};
    uint32_t *hist = reinterpret_cast<uint32_t *>(sc + p.off_hist);
    float *partial = reinterpret_cast<float *>(sc + p.off_part);
    const bool wide = id_bytes == 8;
    for (int q = 0; T > 0 && q < p.passes; ++q) {
        const uint32_t *kin = q ? key[(q - 1) & 1] : nullptr, *tin = q ? tok[(q - 1) & 1] : nullptr;
        launch(k_sort_count, (int)p.tiles, kSortThreads, 0, st, kin, ids, wide, T, V, padding_idx, q * p.bits, p.bits,
               hist, d_status);
        AP_CHECK_LAUNCH("embed_backward count launch");
        launch(k_sort_scan, 1, 1024, 0, st, hist, p.tiles << p.bits);
        AP_CHECK_LAUNCH("embed_backward scan launch");
        launch(k_sort_scatter, (int)p.tiles, kSortThreads, 0, st, kin, tin, ids, wide, T, V, padding_idx, q * p.bits,
               p.bits, hist, key[q & 1], tok[q & 1]);
        AP_CHECK_LAUNCH("embed_backward scatter launch");
    }
    const uint32_t *keys = key[(p.passes - 1) & 1], *toks = tok[(p.passes - 1) & 1];
#define AP_EMBED_BWD(TD, TG)                                                                                         \
    embed_backward_typed<TD, TG>(dout, dout_ld, dout_dtype, keys, toks, T, V, H, scale, accumulate != 0, dtable,      \
                                 dtable_ld, dtable_dtype, partial, p.part_ld, st)
    const bool fd = dout_dtype == AP_DTYPE_F32, fg = dtable_dtype == AP_DTYPE_F32;
    if (fd && fg) return AP_EMBED_BWD(float, float);
    if (fd) return AP_EMBED_BWD(float, bf16_t);
    if (fg) return AP_EMBED_BWD(bf16_t, float);
    return AP_EMBED_BWD(bf16_t, bf16_t);
#undef AP_EMBED_BWD
}
