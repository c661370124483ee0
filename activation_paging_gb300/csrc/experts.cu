// The experts' products: rows of expert e times its weights, on the rows that
// the dispatch leaves (counts and offsets on the GPU), with bias, activation and
// residual in the epilogue, and both gradients.
//
//   forward   z[r] = x[r] W[e]^T + b[e];  y[r] = act(z[r]) + res[r]
//   rows'     dx[r] = (dy[r] W[e] + res[r]) * act'(z[r])
//   weights'  dW[e] (+)= sum_r dy[r]^T x[r];  db[e] (+)= sum_r dy[r]
//
// All three run on the 5th-generation tensor cores: BF16 operands from shared
// memory, FP32 accumulators in tensor memory.  The first two put the features
// on the accumulator's 128 lanes and the rows on its columns: an expert's rows
// are ragged, and columns come by 16, so little of a product is wasted on rows
// that are not there (with rows on the lanes: by 128).  It also makes the
// epilogue's lanes neighbours in a row of the output.
// A block per SM walks the tiles: one warp fetches operands through a ring of
// stages, one issues the products, four read the accumulator and write the
// outputs while the next tile's products run into a second accumulator.
// Operands come by tensor map where base and pitch are multiples of 16 bytes;
// else (odd row lengths) three warps bring them element by element.
#include <cuda_bf16.h>
#include <math.h>

#include "umma.cuh"

namespace ap {
namespace {

using bf16_t = __nv_bfloat16;
using namespace umma;

constexpr int kExThreads = 256;    // warps: 0 fetches, 1 multiplies, 2 and 3 fetch odd rows, 4 to 7 write
constexpr int kFetchers = 96;      // threads of warps 0, 2 and 3
constexpr int kWriters = 128;
constexpr int kLanes = 128;        // features of a tile
constexpr int kDepth = 64;         // contraction of a stage: one line of 128 bytes
constexpr int kPanel = kDepth * 128; // 64 lines
constexpr int kMaxStages = 10;
constexpr int kMaxSmem = 232448;
constexpr int kMaxExperts = 1024;
constexpr int kSwapPitch = 33;     // of the gate's and the up product's exchange

enum Op { kForward, kRows, kWeights };

struct ExArgs {
    const bf16_t *x, *W;   // x: rows of the contraction; W: weights (kWeights: x = dy, W = x)
    int64_t ldx, ldw, lde; // pitches in elements
    const int32_t *seg, *live;
    const float *bias;
    const bf16_t *residual;
    bf16_t *pre;           // z: written forwards, read backwards
    void *out;
    int64_t ldres, ldpre, ldo;
    uint32_t *d_status;
    int64_t rows;
    int E, F, K;           // features of the output (of each half of a gated product), contraction
    int tiles_f, columns, stages, act;
    bool out_f32, add;     // add: kWeights, to what is there
    bool vec;              // kWeights: rows of the output on 32-byte boundaries
};

// ---- activations -----------------------------------------------------------------
__device__ __forceinline__ float ex_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
    return y;
}
__device__ __forceinline__ float sigmoid_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + ex_fast(-x)));
    return y;
}
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(-0.70710678f * x); }
__device__ __forceinline__ float act_of(int act, float z)
{
    if (act == AP_ACT_SILU) return z * sigmoid_fast(z);
    if (act == AP_ACT_GELU) return z * normal_cdf(z);
    return z;
}
__device__ __forceinline__ float act_slope(int act, float z)
{
    if (act == AP_ACT_GELU) return normal_cdf(z) + z * 0.39894228f * ex_fast(-0.5f * z * z);
    const float s = sigmoid_fast(z);
    return s * (1.f + z * (1.f - s));
}

// ---- the tiles of a block ----------------------------------------------------------
struct Table { // in shared memory
    int first[kMaxExperts + 1]; // tiles before each expert
    int seg[kMaxExperts], live[kMaxExperts];
};
struct Walk {
    const Table &tab;
    int t, e;
    __device__ __forceinline__ Walk(const Table &table) : tab(table), t((int)blockIdx.x), e(0) {}
    __device__ __forceinline__ bool find(int E)
    {
        if (t >= tab.first[E]) return false;
        while (t >= tab.first[e + 1]) ++e;
        return true;
    }
    __device__ __forceinline__ void next() { t += (int)gridDim.x; }
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Tiles of each expert, by one warp.  A segment outside the rows counts as empty.
template <Op OP> __device__ void count_tiles(const ExArgs &a, Table &tab)
{
    constexpr int64_t kMost = INT32_MAX - 65536; // segments that overlap could have more: cut off
    const int lane = (int)lane_id();
    int64_t before = 0;
    bool bad = false;
    for (int e0 = 0; e0 < a.E; e0 += kWarp) {
        const int e = e0 + lane;
        int n = 0, tiles = 0;
        if (e < a.E) {
            const int at = a.seg[e];
            n = a.live[e];
            if (n < 0 || at < 0 || (int64_t)at + n > a.rows) {
                n = 0;
                bad = true;
            }
            tab.seg[e] = at;
            tab.live[e] = n;
            if (OP == kWeights)
                tiles = n > 0 || !a.add ? a.tiles_f * ceil_div(a.K, a.columns) : 0;
            else
                tiles = a.tiles_f * ceil_div(n, a.columns);
        }
        int64_t upto = tiles;
#pragma unroll
        for (int off = 1; off < kWarp; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += o;
        }
        if (e < a.E) tab.first[e] = (int)min(before + upto - tiles, kMost);
        before += __shfl_sync(0xffffffffu, upto, kWarp - 1);
    }
    bad |= before > kMost;
    if (lane == 0) tab.first[a.E] = (int)min(before, kMost);
    if (bad && a.d_status && blockIdx.x == 0) atomicOr(a.d_status, AP_FLAG_BAD_COUNT);
}

// What a tile is: features from f0, columns (rows of the output, or kWeights:
// places of a weight's row) from c0, n of them; the contraction's steps.
struct Tile {
    int e, f0, c0, n, steps, row0, live;
};
template <Op OP> __device__ __forceinline__ Tile tile_of(const ExArgs &a, const Walk &w)
{
    Tile t;
    t.e = w.e;
    t.live = w.tab.live[w.e];
    const int at = w.t - w.tab.first[w.e];
    const int width = OP == kWeights ? a.K : t.live;
    const int across = ceil_div(width, a.columns);
    const int f = at / across, c = at - f * across;
    t.f0 = f * (OP == kForward && a.act == AP_ACT_SWIGLU ? kLanes / 2 : kLanes);
    t.c0 = c * a.columns;
    t.n = min(a.columns, width - t.c0);
    t.row0 = w.tab.seg[w.e] + (OP == kWeights ? 0 : t.c0);
    t.steps = OP == kWeights ? ceil_div(t.live, kDepth) : ceil_div(a.K, kDepth);
    return t;
}

// One panel of lines by plain loads: line r holds 64 values of row r of src from
// column c0 on, in swizzled pieces of 16 bytes; zeros outside rows and columns.
__device__ __forceinline__ void fill_panel(uint8_t *to, const bf16_t *src, int64_t ld, int lines, int64_t rows, int64_t columns,
                                           int thread)
{
    for (int i = thread; i < lines * 8; i += kFetchers) {
        const int r = i >> 3, c = i & 7;
        uint32_t w[4] = {0, 0, 0, 0};
        if (r < rows) {
            const unsigned short *p = reinterpret_cast<const unsigned short *>(src) + r * ld + c * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c * 8 + j < columns) w[j / 2] |= (uint32_t)p[j] << 16 * (j & 1);
        }
        *reinterpret_cast<uint4 *>(to + r * 128 + ((c ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// A stage: the features' operand (two panels, 16 KB), then the columns'.
template <Op OP, bool MAPS>
__device__ __forceinline__ void fetch(const ExArgs &a, const Tile &t, int step, uint8_t *stage, const CUtensorMap *mx,
                                      const CUtensorMap *mw, uint32_t full, int thread)
{
    const int k0 = step * kDepth;
    const bool gated = OP == kForward && a.act == AP_ACT_SWIGLU;
    const int half = gated ? a.F : 64; // where the second panel's features begin, behind the first's
    uint8_t *col = stage + 2 * kPanel;
    const int n = OP == kWeights ? ceil_div(t.n, 64) : ceil_div(t.n, 32);
    if constexpr (MAPS) {
        const uint32_t sa = smem_addr(stage), sb = smem_addr(col);
        bar_expect(full, 2 * kPanel + n * (OP == kWeights ? kPanel : kPanel / 2));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (OP == kForward) tma_3d(sa + h * kPanel, mw, k0, t.f0 + h * half, t.e, full);
            if (OP == kRows) tma_3d(sa + h * kPanel, mw, t.f0 + h * 64, k0, t.e, full);
            if (OP == kWeights) tma_2d(sa + h * kPanel, mx, t.f0 + h * 64, t.row0 + k0, full);
        }
        for (int i = 0; i < n; ++i) {
            if (OP == kWeights)
                tma_2d(sb + i * kPanel, mw, t.c0 + i * 64, t.row0 + k0, full);
            else
                tma_2d(sb + i * (kPanel / 2), mx, k0, t.row0 + i * 32, full);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int f = t.f0 + h * half;
            if (OP == kForward)
                fill_panel(stage + h * kPanel, a.W + t.e * a.lde + f * a.ldw + k0, a.ldw, 64, (gated ? 2 : 1) * a.F - f, a.K - k0,
                           thread);
            if (OP == kRows) fill_panel(stage + h * kPanel, a.W + t.e * a.lde + k0 * a.ldw + f, a.ldw, 64, a.K - k0, a.F - f, thread);
            if (OP == kWeights)
                fill_panel(stage + h * kPanel, a.x + (int64_t)(t.row0 + k0) * a.ldx + f, a.ldx, 64, t.live - k0, a.F - f, thread);
        }
        for (int i = 0; i < n; ++i) {
            if (OP == kWeights)
                fill_panel(col + i * kPanel, a.W + (int64_t)(t.row0 + k0) * a.ldw + t.c0 + i * 64, a.ldw, 64, t.live - k0,
                           a.K - t.c0 - i * 64, thread);
            else
                fill_panel(col + i * (kPanel / 2), a.x + (int64_t)(t.row0 + i * 32) * a.ldx + k0, a.ldx, 32, t.n - i * 32, a.K - k0,
                           thread);
        }
        fence_async();
        bar_arrive(full);
    }
}

__device__ __forceinline__ void writers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWriters) : "memory"); }

template <typename T> __device__ __forceinline__ void put(T *p, float v);
template <> __device__ __forceinline__ void put<float>(float *p, float v) { *p = v; }
template <> __device__ __forceinline__ void put<bf16_t>(bf16_t *p, float v) { *p = __float2bfloat16_rn(v); }

// 32 rows' values of a feature (lane), rows c .. c + count - 1 from row on.
template <typename T>
__device__ __forceinline__ void write_rows(const ExArgs &a, const Tile &t, int c, float (&v)[32], int f, int lane_row, float *swap)
{
    const int64_t row = (int64_t)t.row0 + c;
    const int count = min(32, t.n - c);
    const bool on = f < a.F;
    T *out = static_cast<T *>(a.out) + row * a.ldo + f;
    const bf16_t *res = a.residual + row * a.ldres + f;
    bf16_t *pre = a.pre + row * a.ldpre + f;
    const bool up = lane_row >= kLanes / 2;
    if (a.act == AP_ACT_SWIGLU) { // lanes 64 on hold the up product of the features of the lanes before
        if (a.bias && on) {
            const float b = a.bias[(int64_t)t.e * 2 * a.F + (up ? a.F : 0) + f];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += b;
        }
        if (a.pre && on) {
            bf16_t *p = pre + (up ? a.F : 0);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < count) p[j * a.ldpre] = __float2bfloat16_rn(v[j]);
        }
        float *mine = swap + (lane_row & (kLanes / 2 - 1)) * kSwapPitch;
        if (up)
#pragma unroll
            for (int j = 0; j < 32; ++j) mine[j] = v[j];
        writers_sync();
        if (!up && on)
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < count) {
                    float h = v[j] * sigmoid_fast(v[j]) * mine[j];
                    if (a.residual) h += __bfloat162float(res[j * a.ldres]);
                    put(out + j * a.ldo, h);
                }
        writers_sync();
        return;
    }
    if (!on) return;
    if (a.bias) {
        const float b = a.bias[(int64_t)t.e * a.F + f];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += b;
    }
    if (a.pre)
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < count) pre[j * a.ldpre] = __float2bfloat16_rn(v[j]);
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j < count) {
            float h = act_of(a.act, v[j]);
            if (a.residual) h += __bfloat162float(res[j * a.ldres]);
            put(out + j * a.ldo, h);
        }
}

template <typename T>
__device__ __forceinline__ void write_slopes(const ExArgs &a, const Tile &t, int c, float (&v)[32], int f)
{
    if (f >= a.F) return;
    const int64_t row = (int64_t)t.row0 + c;
    const int count = min(32, t.n - c);
    T *out = static_cast<T *>(a.out) + row * a.ldo + f;
    if (a.residual) {
        const bf16_t *res = a.residual + row * a.ldres + f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < count) v[j] += __bfloat162float(res[j * a.ldres]);
    }
    const bf16_t *pre = a.pre + row * a.ldpre + f;
    if (a.act == AP_ACT_SWIGLU) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < count) {
                const float g = __bfloat162float(pre[j * a.ldpre]), u = __bfloat162float(pre[j * a.ldpre + a.F]);
                put(out + j * a.ldo, v[j] * u * act_slope(AP_ACT_SILU, g));
                put(out + j * a.ldo + a.F, v[j] * g * sigmoid_fast(g));
            }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < count) {
                const float d = a.act == AP_ACT_NONE ? v[j] : v[j] * act_slope(a.act, __bfloat162float(pre[j * a.ldpre]));
                put(out + j * a.ldo, d);
            }
    }
}

// 32 places of a weight's row (lane), one after the other in memory.
template <typename T> __device__ __forceinline__ void write_weights(const ExArgs &a, const Tile &t, int c, float (&v)[32], int f)
{
    if (f >= a.F) return;
    const int count = min(32, t.n - c);
    T *out = static_cast<T *>(a.out) + ((int64_t)t.e * a.F + f) * a.K + t.c0 + c;
    if (a.vec && count == 32) {
        constexpr int kPer = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 32; j += kPer) {
            uint4 *p = reinterpret_cast<uint4 *>(out + j);
            T x[kPer];
            if (a.add) {
                const uint4 old = *p;
                memcpy(x, &old, 16);
            }
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                float s = v[j + q];
                if (a.add) s += (float)x[q];
                put(x + q, s);
            }
            uint4 n;
            memcpy(&n, x, 16);
            *p = n;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j < count) put(out + j, a.add ? (float)out[j] + v[j] : v[j]);
}

template <Op OP, bool MAPS>
__global__ void __launch_bounds__(kExThreads, 1)
    k_experts(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, const ExArgs a)
{
    pdl_begin();
    extern __shared__ __align__(1024) uint8_t s_mem[];
    __shared__ Table s_tab;
    __shared__ float s_swap[OP == kForward ? kLanes / 2 * kSwapPitch : 1];
    __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_done[2], s_free[2], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;
    const int wid = threadIdx.x / kWarp, lane = (int)lane_id();
    const int stage_bytes = 2 * kPanel + a.columns * 128;
    uint8_t *stages = s_mem + ((1024 - (smem_addr(s_mem) & 1023)) & 1023);
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            bar_init(smem_addr(&s_full[s]), MAPS ? 1 : kFetchers);
            bar_init(smem_addr(&s_empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(smem_addr(&s_done[s]), 1);
            bar_init(smem_addr(&s_free[s]), kWriters / kWarp);
        }
        bar_init(smem_addr(&s_drain), 1);
        bar_init_done();
        s_dead = 0;
    }
    if (wid == 1) tmem_alloc(smem_addr(&s_tmem), 512);
    if (wid == 2) count_tiles<OP>(a, s_tab);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *dead = &s_dead;
    Walk w(s_tab);

    if (wid == 0 || (!MAPS && (wid == 2 || wid == 3))) {
        // ---- fetch: stage by stage, as they fall empty
        const int thread = wid == 0 ? lane : threadIdx.x - kWarp;
        if (!MAPS || lane == 0) {
            if (MAPS) {
                tma_prefetch_map(&mx);
                tma_prefetch_map(&mw);
            }
            uint32_t count = 0, s = 0, turn = 0; // stages fetched; ring position and its turn
            bool ok = true;
            for (; ok && w.find(a.E); w.next()) {
                const Tile t = tile_of<OP>(a, w);
                for (int step = 0; step < t.steps; ++step) {
                    if (count >= (uint32_t)a.stages && !bar_wait(smem_addr(&s_empty[s]), (turn & 1) ^ 1, dead)) {
                        ok = false;
                        break;
                    }
                    fetch<OP, MAPS>(a, t, step, stages + (size_t)s * stage_bytes, &mx, &mw, smem_addr(&s_full[s]), thread);
                    ++count;
                    if (++s == (uint32_t)a.stages) {
                        s = 0;
                        ++turn;
                    }
                }
            }
            if (MAPS && !ok) { // copies on their way end before the block does
                volatile int none = 0;
                for (uint32_t i = 0; i < (uint32_t)a.stages && i < count; ++i) {
                    const uint32_t c = count - 1 - i;
                    none = 0;
                    (void)bar_wait(smem_addr(&s_full[c % a.stages]), c / a.stages & 1, &none);
                }
            }
        }
    } else if (wid == 1) {
        // ---- multiply
        uint32_t s = 0, turn = 0, count = 0; // ring; tiles so far
        bool ok = true;
        for (; ok && w.find(a.E); w.next()) {
            const Tile t = tile_of<OP>(a, w);
            if (t.steps == 0) continue;
            const uint32_t acc = count & 1;
            if (count >= 2 && !__all_sync(0xffffffffu, bar_wait(smem_addr(&s_free[acc]), (count >> 1 & 1) ^ 1, dead))) break;
            fence_after();
            const uint32_t shape = shape_of(kLanes, (t.n + 15) & ~15, OP != kForward, OP == kWeights);
            for (int step = 0; step < t.steps; ++step) {
                if (!__all_sync(0xffffffffu, bar_wait(smem_addr(&s_full[s]), turn & 1, dead))) {
                    ok = false;
                    break;
                }
                fence_after();
                uint8_t *stage = stages + (size_t)s * stage_bytes;
                if (OP == kWeights && MAPS && t.live - step * kDepth < kDepth) {
                    // the lines behind the expert's last row are others' rows: zeros
                    const int from = (t.live - step * kDepth) * 128, panels = 2 + ceil_div(t.n, 64);
                    for (int p = 0; p < panels; ++p)
                        for (int b = from + lane * 16; b < kPanel; b += kWarp * 16)
                            *reinterpret_cast<uint4 *>(stage + p * kPanel + b) = make_uint4(0, 0, 0, 0);
                    fence_async();
                    __syncwarp();
                }
                if (lane == 0) {
                    const uint32_t sa = smem_addr(stage), sb = sa + 2 * kPanel;
#pragma unroll
                    for (int k = 0; k < kDepth / 16; ++k)
                        mma(tmem + acc * 256, operand(sa + k * (OP == kForward ? 32 : 2048), kPanel),
                            operand(sb + k * (OP == kWeights ? 2048 : 32), kPanel), shape, step > 0 || k > 0);
                    mma_commit(smem_addr(&s_empty[s]));
                }
                __syncwarp();
                if (++s == (uint32_t)a.stages) {
                    s = 0;
                    ++turn;
                }
            }
            if (ok && lane == 0) mma_commit(smem_addr(&s_done[acc]));
            __syncwarp();
            ++count;
        }
        if (__any_sync(0xffffffffu, *dead)) { // products on their way end before tensor memory is freed
            volatile int none = 0;
            if (lane == 0) {
                mma_commit(smem_addr(&s_drain));
                (void)bar_wait(smem_addr(&s_drain), 0, &none);
            }
            __syncwarp();
        }
    } else if (wid >= 4) {
        // ---- write
        const int part = wid & 3, lane_row = part * kWarp + lane;
        uint32_t count = 0;
        bool ok = true;
        for (; w.find(a.E); w.next()) {
            const Tile t = tile_of<OP>(a, w);
            const uint32_t acc = count & 1;
            if (t.steps > 0) {
                if (ok && !bar_wait(smem_addr(&s_done[acc]), count >> 1 & 1, dead)) ok = false;
                ++count;
            }
            ok = __all_sync(0xffffffffu, ok);
            fence_after();
            const int f = t.f0 + (OP == kForward && a.act == AP_ACT_SWIGLU ? lane_row & (kLanes / 2 - 1) : lane_row);
            for (int c = 0; c < t.n; c += 32) {
                float v[32];
                if (t.steps > 0 && ok) {
                    acc_load(tmem + acc * 256 + c + ((uint32_t)part * kWarp << 16), v);
                } else { // nothing to add up, or products that did not come
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = t.steps > 0 ? NAN : 0.f;
                }
                if (c + 32 >= t.n) { // the accumulator is read
                    fence_before();
                    __syncwarp();
                    if (lane == 0 && t.steps > 0) bar_arrive(smem_addr(&s_free[acc]));
                }
                if (a.out_f32) {
                    if (OP == kForward) write_rows<float>(a, t, c, v, f, lane_row, s_swap);
                    if (OP == kRows) write_slopes<float>(a, t, c, v, f);
                    if (OP == kWeights) write_weights<float>(a, t, c, v, f);
                } else {
                    if (OP == kForward) write_rows<bf16_t>(a, t, c, v, f, lane_row, s_swap);
                    if (OP == kRows) write_slopes<bf16_t>(a, t, c, v, f);
                    if (OP == kWeights) write_weights<bf16_t>(a, t, c, v, f);
                }
            }
        }
        if (!ok && a.d_status && lane == 0) atomicOr(a.d_status, AP_FLAG_CORRUPT);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (wid == 1) {
        fence_after();
        tmem_free(tmem, 512);
    }
}

// db[e] (+)= the sum of the expert's rows of dy: a block takes 64 columns of an
// expert, eight warps every eighth row, two columns a lane.
__global__ void __launch_bounds__(256) k_expert_bias(const bf16_t *dy, int64_t ld, const int32_t *seg, const int32_t *live, int64_t rows,
                                                     int N, float *db, bool add)
{
    pdl_begin();
    __shared__ float s_sum[8][64];
    const int e = blockIdx.y, wid = threadIdx.x / kWarp, lane = (int)lane_id();
    const int at = seg[e];
    int n = live[e];
    if (n < 0 || at < 0 || (int64_t)at + n > rows) n = 0;
    const int c = blockIdx.x * 64 + lane;
    float s[2] = {0.f, 0.f};
    for (int r = wid; r < n; r += 8) {
        const bf16_t *p = dy + (int64_t)(at + r) * ld + c;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (c + 32 * q < N) s[q] += __bfloat162float(p[32 * q]);
    }
    s_sum[wid][lane] = s[0];
    s_sum[wid][lane + 32] = s[1];
    __syncthreads();
    const int col = blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < N) {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) sum += s_sum[q][threadIdx.x];
        float *to = db + (int64_t)e * N + col;
        *to = add ? *to + sum : sum;
    }
}

// ---- host ------------------------------------------------------------------------

// Whether a copy by tensor map takes rows of this base and pitch (in elements).
bool mappable(const void *p, int64_t ld, int64_t more = 0)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && more % 8 == 0;
}

template <Op OP, bool MAPS>
ap_status launch_experts(const char *who, const CUtensorMap &mx, const CUtensorMap &mw, ExArgs a, int64_t tiles, cudaStream_t st)
{
    const auto kernel = k_experts<OP, MAPS>;
    cudaFuncAttributes attr;
    static const int fixed = cudaFuncGetAttributes(&attr, (const void *)kernel) == cudaSuccess ? (int)attr.sharedSizeBytes : -1;
    if (fixed < 0) return cuda_fail(cudaGetLastError(), who);
    static const cudaError_t set =
        cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - fixed);
    if (set != cudaSuccess) return cuda_fail(set, who);
    const int stage = 2 * kPanel + a.columns * 128, room = kMaxSmem - fixed - 1024;
    a.stages = room / stage < kMaxStages ? room / stage : kMaxStages;
    const int sms = sm_count();
    launch(kernel, (int)(tiles < sms ? tiles : sms), kExThreads, (size_t)a.stages * stage + 1024, st, mx, mw, a);
    AP_CHECK_LAUNCH(who);
    return AP_OK;
}

ap_status check_rows(const char *who, int64_t rows, int32_t E, int32_t N, int32_t K, int64_t ldx, int64_t need_x, int64_t ldw,
                     int64_t need_w, int64_t lde, int64_t need_e)
{
    if (rows < 0 || rows >= (int64_t(1) << 31) || E < 1 || E > kMaxExperts || N < 1 || K < 1 || N > (1 << 20) || K > (1 << 20))
        return fail(AP_EINVAL, "%s: bad sizes rows=%lld E=%d N=%d K=%d", who, (long long)rows, E, N, K);
    if (ldx < need_x || ldw < need_w || lde < need_e || ldx >= (int64_t(1) << 38) || ldw >= (int64_t(1) << 38) ||
        lde >= (int64_t(1) << 38))
        return fail(AP_EINVAL, "%s: bad pitches %lld, %lld, %lld", who, (long long)ldx, (long long)ldw, (long long)lde);
    return AP_OK;
}
bool odd_address(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Columns of a tile: rows of the output at most, by what an expert has on the average.
int columns_for(int64_t rows, int32_t E)
{
    const int64_t each = rows / E;
    return each >= 96 ? 256 : each >= 24 ? 128 : 64;
}

ap_status rows_product(const char *who, Op op, ExArgs a, int halves, cudaStream_t st)
{
    if (a.E == 1) a.lde = a.ldw * (op == kForward ? a.F * halves : a.K); // (of no account)
    a.columns = columns_for(a.rows, a.E);
    const int per = op == kForward && halves == 2 ? kLanes / 2 : kLanes;
    a.tiles_f = (a.F + per - 1) / per;
    const int64_t tiles = (a.rows / a.columns + a.E) * (int64_t)a.tiles_f;
    if (tiles >= INT32_MAX) return fail(AP_EINVAL, "%s: %lld tiles are more than one launch takes", who, (long long)tiles);
    CUtensorMap mx = {}, mw = {};
    if (!mappable(a.x, a.ldx) || !mappable(a.W, a.ldw, a.lde))
        return op == kForward ? launch_experts<kForward, false>(who, mx, mw, a, tiles, st)
                              : launch_experts<kRows, false>(who, mx, mw, a, tiles, st);
    const int wide = op == kForward ? a.F * halves : a.K, deep = op == kForward ? a.K : a.F; // of W[e]
    const uint64_t ex[2] = {(uint64_t)a.K, (uint64_t)a.rows}, px[1] = {(uint64_t)a.ldx};
    const uint64_t ew[3] = {(uint64_t)deep, (uint64_t)wide, (uint64_t)a.E}, pw[2] = {(uint64_t)a.ldw, (uint64_t)a.lde};
    const uint32_t bx[2] = {64, 32}, bw[3] = {64, 64, 1};
    if (!make_map(&mx, a.x, 2, ex, px, bx) || !make_map(&mw, a.W, 3, ew, pw, bw))
        return fail(AP_ENOTSUP, "%s: no tensor map of these sizes", who);
    return op == kForward ? launch_experts<kForward, true>(who, mx, mw, a, tiles, st)
                          : launch_experts<kRows, true>(who, mx, mw, a, tiles, st);
}

} // namespace

bool umma::make_map(CUtensorMap *map, const void *base, int dims, const uint64_t *extent, const uint64_t *pitch, const uint32_t *box)
{
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        (void)cudaGetLastError();
        return reinterpret_cast<Encode>(p);
    }();
    if (!encode) return false;
    cuuint64_t strides[2], sizes[3];
    cuuint32_t ones[3] = {1, 1, 1};
    for (int i = 0; i < dims; ++i) sizes[i] = extent[i];
    for (int i = 0; i + 1 < dims; ++i) strides[i] = pitch[i] * 2;
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void *>(base), sizes, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

} // namespace ap

extern "C" ap_status ap_expert_linear(const void *x, int64_t ldx, int64_t rows, int32_t E, int32_t N, int32_t K,
                                      const int32_t *d_seg_off, const int32_t *d_live, const void *W, int64_t ldw, int64_t lde,
                                      const float *bias, int32_t act, const void *residual, int64_t ldres, void *pre,
                                      int64_t ldpre, void *out, int64_t ldo, int32_t out_dtype, uint32_t *d_status, void *stream)
{
    AP_NVTX_RANGE("ap_expert_linear");
    using namespace ap;
    const char *who = "expert_linear";
    if (act < AP_ACT_NONE || act > AP_ACT_SWIGLU) return fail(AP_EINVAL, "%s: unknown activation %d", who, act);
    const int halves = act == AP_ACT_SWIGLU ? 2 : 1;
    if (const ap_status s = check_rows(who, rows, E, N, K, ldx, K, ldw, K, lde, 0); s != AP_OK) return s;
    if (out_dtype != AP_DTYPE_BF16 && out_dtype != AP_DTYPE_F32) return fail(AP_EINVAL, "%s: type %d", who, out_dtype);
    if (ldo < N || (residual && ldres < N) || (pre && ldpre < (int64_t)halves * N)) return fail(AP_EINVAL, "%s: bad pitches", who);
    if (E > 1 && lde < ((int64_t)halves * N - 1) * ldw + K) return fail(AP_EINVAL, "%s: experts' weights overlap", who);
    if (rows == 0) return AP_OK;
    if (!x || !d_seg_off || !d_live || !W || !out) return fail(AP_EINVAL, "%s: NULL pointer", who);
    if (odd_address(x, 2) || odd_address(W, 2) || odd_address(residual, 2) || odd_address(pre, 2) || odd_address(bias, 4) ||
        odd_address(out, out_dtype == AP_DTYPE_BF16 ? 2 : 4))
        return fail(AP_EINVAL, "%s: not aligned", who);
    ExArgs a = {};
    a.x = (const bf16_t *)x, a.W = (const bf16_t *)W, a.ldx = ldx, a.ldw = ldw, a.lde = lde;
    a.seg = d_seg_off, a.live = d_live, a.bias = bias, a.residual = (const bf16_t *)residual, a.pre = (bf16_t *)pre, a.out = out;
    a.ldres = ldres, a.ldpre = ldpre, a.ldo = ldo, a.d_status = d_status, a.rows = rows, a.E = E, a.F = N, a.K = K, a.act = act;
    a.out_f32 = out_dtype == AP_DTYPE_F32;
    return rows_product(who, kForward, a, halves, (cudaStream_t)stream);
}

extern "C" ap_status ap_expert_linear_dx(const void *dy, int64_t ldy, int64_t rows, int32_t E, int32_t N, int32_t K,
                                         const int32_t *d_seg_off, const int32_t *d_live, const void *W, int64_t ldw, int64_t lde,
                                         int32_t act, const void *pre, int64_t ldpre, const void *residual, int64_t ldres, void *dx,
                                         int64_t ldx, int32_t dx_dtype, uint32_t *d_status, void *stream)
{
    AP_NVTX_RANGE("ap_expert_linear_dx");
    using namespace ap;
    const char *who = "expert_linear_dx";
    if (act < AP_ACT_NONE || act > AP_ACT_SWIGLU) return fail(AP_EINVAL, "%s: unknown activation %d", who, act);
    const int halves = act == AP_ACT_SWIGLU ? 2 : 1;
    if (const ap_status s = check_rows(who, rows, E, N, K, ldy, N, ldw, K, lde, 0); s != AP_OK) return s;
    if (dx_dtype != AP_DTYPE_BF16 && dx_dtype != AP_DTYPE_F32) return fail(AP_EINVAL, "%s: type %d", who, dx_dtype);
    if (ldx < (int64_t)halves * K || (residual && ldres < K) || (act != AP_ACT_NONE && ldpre < (int64_t)halves * K))
        return fail(AP_EINVAL, "%s: bad pitches", who);
    if (E > 1 && lde < ((int64_t)N - 1) * ldw + K) return fail(AP_EINVAL, "%s: experts' weights overlap", who);
    if (rows == 0) return AP_OK;
    if (!dy || !d_seg_off || !d_live || !W || !dx || (act != AP_ACT_NONE && !pre)) return fail(AP_EINVAL, "%s: NULL pointer", who);
    if (odd_address(dy, 2) || odd_address(W, 2) || odd_address(residual, 2) || odd_address(pre, 2) ||
        odd_address(dx, dx_dtype == AP_DTYPE_BF16 ? 2 : 4))
        return fail(AP_EINVAL, "%s: not aligned", who);
    ExArgs a = {};
    a.x = (const bf16_t *)dy, a.W = (const bf16_t *)W, a.ldx = ldy, a.ldw = ldw, a.lde = lde;
    a.seg = d_seg_off, a.live = d_live, a.residual = (const bf16_t *)residual, a.out = dx;
    a.pre = const_cast<bf16_t *>((const bf16_t *)pre);
    a.ldres = ldres, a.ldpre = ldpre, a.ldo = ldx, a.d_status = d_status, a.rows = rows, a.E = E, a.F = K, a.K = N, a.act = act;
    a.out_f32 = dx_dtype == AP_DTYPE_F32;
    return rows_product(who, kRows, a, halves, (cudaStream_t)stream);
}

extern "C" ap_status ap_expert_linear_dw(const void *dy, int64_t ldy, const void *x, int64_t ldx, int64_t rows, int32_t E, int32_t N,
                                         int32_t K, const int32_t *d_seg_off, const int32_t *d_live, int32_t accumulate, void *dW,
                                         int32_t dw_dtype, float *dbias, uint32_t *d_status, void *stream)
{
    AP_NVTX_RANGE("ap_expert_linear_dw");
    using namespace ap;
    const char *who = "expert_linear_dw";
    if (const ap_status s = check_rows(who, rows, E, N, K, ldy, N, ldx, K, 0, 0); s != AP_OK) return s;
    if (dw_dtype != AP_DTYPE_BF16 && dw_dtype != AP_DTYPE_F32) return fail(AP_EINVAL, "%s: type %d", who, dw_dtype);
    if (accumulate != 0 && accumulate != 1) return fail(AP_EINVAL, "%s: accumulate=%d", who, accumulate);
    if (!d_seg_off || !d_live || (!dW && !dbias) || (rows > 0 && (!dy || (dW && !x)))) return fail(AP_EINVAL, "%s: NULL pointer", who);
    if (odd_address(dy, 2) || odd_address(x, 2) || odd_address(dbias, 4) || odd_address(dW, dw_dtype == AP_DTYPE_BF16 ? 2 : 4))
        return fail(AP_EINVAL, "%s: not aligned", who);
    cudaStream_t st = (cudaStream_t)stream;
    if (dW) {
        ExArgs a = {};
        a.x = (const bf16_t *)dy, a.W = (const bf16_t *)x, a.ldx = ldy, a.ldw = ldx;
        a.seg = d_seg_off, a.live = d_live, a.out = dW, a.d_status = d_status, a.rows = rows, a.E = E, a.F = N, a.K = K;
        a.out_f32 = dw_dtype == AP_DTYPE_F32, a.add = accumulate != 0;
        a.columns = K > 128 ? 256 : K > 64 ? 128 : 64;
        a.tiles_f = (N + kLanes - 1) / kLanes;
        a.vec = !odd_address(dW, 16) && K % (a.out_f32 ? 4 : 8) == 0;
        const int64_t tiles = (int64_t)E * a.tiles_f * ((K + a.columns - 1) / a.columns);
        if (tiles >= INT32_MAX) return fail(AP_EINVAL, "%s: %lld tiles are more than one launch takes", who, (long long)tiles);
        CUtensorMap mx = {}, mw = {};
        ap_status s;
        if (rows > 0 && mappable(dy, ldy) && mappable(x, ldx)) {
            const uint64_t ey[2] = {(uint64_t)N, (uint64_t)rows}, py[1] = {(uint64_t)ldy};
            const uint64_t ex[2] = {(uint64_t)K, (uint64_t)rows}, px[1] = {(uint64_t)ldx};
            const uint32_t box[2] = {64, 64};
            if (!make_map(&mx, dy, 2, ey, py, box) || !make_map(&mw, x, 2, ex, px, box))
                return fail(AP_ENOTSUP, "%s: no tensor map of these sizes", who);
            s = launch_experts<kWeights, true>(who, mx, mw, a, tiles, st);
        } else {
            s = launch_experts<kWeights, false>(who, mx, mw, a, tiles, st);
        }
        if (s != AP_OK) return s;
    }
    if (dbias) {
        launch(k_expert_bias, dim3((unsigned)((N + 63) / 64), (unsigned)E), 256, 0, st, (const bf16_t *)dy, ldy, d_seg_off, d_live, rows,
               N, dbias, accumulate != 0);
        AP_CHECK_LAUNCH("expert_linear_dw bias launch");
    }
    return AP_OK;
}
