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
// stages, one issues the products, eight read the accumulator and write the
// outputs while the next tile's products run into a second accumulator.
// Outputs and what the epilogue reads (residual, pre-activations) pass through
// shared memory as 8 x 8 matrices, transposed, so that memory sees rows' pieces
// of 32 and 64 bytes.
// Operands come by tensor map, which wants bases and pitches that are multiples
// of 16 bytes.  Others (odd row lengths) are copied to rows that begin on such
// boundaries first (k_repitch).
#include <cuda_bf16.h>
#include <math.h>

#include "umma.cuh"

namespace ap {
namespace {

using bf16_t = __nv_bfloat16;
using namespace umma;

constexpr int kExThreads = 384;    // warps: 0 fetches, 1 multiplies, 2 and 3 pass stages on, 4 to 11 write
constexpr int kWriters = 8;        // warps: two for each quarter of the lanes, with every other 32 columns
constexpr int kLanes = 128;        // features of a tile
constexpr int kDepth = 64;         // contraction of a stage: one line of 128 bytes
constexpr int kPanel = kDepth * 128; // 64 lines
constexpr int kMaxStages = 10;
// The tensor cores cut what they add to an accumulator: its error grows with the
// contraction, 1.1e-9 of it for each place (9.2e-6 at 8192).  FP32 weights'
// gradients are therefore added up over sections of 2048 rows, which the writers
// add with rounding (2.1e-6; by 1024 1.1e-6, but then the products do not hide the
// writing: 262144 rows over 128 experts, 1024 x 2048 1135 us for 1011).
constexpr int kSection = 32; // stages
// FP32 results of the other two (PARTS) likewise, over 1024 places, where the
// contraction is longer: error 1e-6 whatever its length, for 2.1e-6 at 2048 and
// 4.4e-6 at 4096.  The writers add a section to the sums so far, which stand in
// place of the second accumulator, while the products wait: 65536 rows of 2048 to
// 1024 over 128 experts 229 us for 198, 8192 of 4096 to 4096 over 8 215 for 180.
// (By 512 4.7e-7, 275 and 244 us; by 2048 199 and 218.  Two accumulators of 160
// columns beside the sums, by 512: 320 and 249.)
constexpr int kPart = 16; // stages
constexpr int kMaxSmem = 232448;
constexpr int kMaxExperts = 1024;
constexpr int kPassPitch = 80;     // bytes of 32 lanes' values on their way, with what keeps banks apart
constexpr int kPass = 32 * kPassPitch; // of a writer
constexpr int kHalf = 16 * 128;    // (of weights: 16 rows of 32 FP32)

enum Op { kForward, kRows, kWeights };

struct ExArgs {
    const bf16_t *x, *W;   // x: rows of the contraction; W: weights (kWeights: x = dy, W = x)
    int64_t ldx, ldw, lde; // pitches in elements
    const int32_t *seg, *live;
    const float *bias;
    const bf16_t *residual;
    float *db;             // kWeights: the bias's gradient or nullptr
    bf16_t *pre;           // z: written forwards, read backwards
    void *out;
    int64_t ldres, ldpre, ldo;
    uint32_t *d_status;
    int64_t rows;
    int E, F, K;           // features of the output (of each half of a gated product), contraction
    int tiles_f, columns, stages, act;
    bool out_f32, add;     // add: kWeights, to what is there
    bool chunk_x, chunk_w; // kWeights: rows of whole 64s, two of them in a copy
    bool by16;             // a gated product's map takes 16 features of either half in turn
    bool vec_out, vec_pre, vec_res; // rows on 16-byte boundaries, of whole pieces
};

// Where operands come from: x in small and in large copies, the weights (kWeights:
// x is dy, w is x).
struct ExMaps {
    CUtensorMap x, xx, w, ww;
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
// The normal distribution: its value Phi(x) and e^(-x^2 / 2).  Of the smaller
// tail, Phi(-|x|) = t P(t) e^(-x^2 / 2) with t = 1 / (1 + |x| / sqrt 8): a
// least-squares fit of P to erfc's scaled form, reweighted to even errors of
// 4.3e-8; with FP32's roundings 2e-7 and (0.75 x^2 + 4) 2^-24 of the exponential,
// relative to the tail.  (erfc in its place: 44.5 us for 32
// at 5994 rows of 1000 to 520, whose epilogue bounds them.)
struct Normal {
    float cdf, bell;
};
__device__ __forceinline__ Normal normal_of(float x)
{
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(fabsf(x), 0.353553391f, 1.f)));
    float p = -0.0295344745f;
    p = fmaf(p, t, 0.142287454f);
    p = fmaf(p, t, -0.243599892f);
    p = fmaf(p, t, 0.139033515f);
    p = fmaf(p, t, -0.0133127892f);
    p = fmaf(p, t, 0.101343417f);
    p = fmaf(p, t, 0.121551885f);
    p = fmaf(p, t, 0.141187654f);
    p = fmaf(p, t, 0.141043209f);
    Normal n;
    n.bell = ex_fast(-0.5f * x * x);
    const float tail = t * p * n.bell;
    n.cdf = x < 0.f ? tail : 1.f - tail;
    return n;
}
__device__ __forceinline__ float gelu_of(float x) { return x * normal_of(x).cdf; }
__device__ __forceinline__ float act_slope(int act, float z)
{
    if (act == AP_ACT_GELU) {
        const Normal n = normal_of(z);
        return fmaf(z * 0.39894228f, n.bell, n.cdf);
    }
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
    int t, e, step;
    __device__ __forceinline__ Walk(const Table &table, int from, int by) : tab(table), t(from), e(0), step(by) {}
    __device__ __forceinline__ bool find(int E)
    {
        if (t >= tab.first[E]) return false;
        while (t >= tab.first[e + 1]) ++e;
        return true;
    }
    __device__ __forceinline__ void next() { t += step; }
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

// What a tile is: features from f0 (this block's, of a pair's), columns (rows of
// the output, or kWeights: places of a weight's row) from c0, n of them; the
// contraction's steps.  An expert's rows are shared out evenly among its tiles.
struct Tile {
    int e, f0, c0, n, steps, row0, live, sections;
};
template <Op OP, bool PAIR, bool PARTS> __device__ __forceinline__ Tile tile_of(const ExArgs &a, const Walk &w, int rank)
{
    Tile t;
    t.e = w.e;
    t.live = w.tab.live[w.e];
    const int at = w.t - w.tab.first[w.e];
    const int width = OP == kWeights ? a.K : t.live;
    const int across = ceil_div(width, a.columns);
    const int f = at / across, c = at - f * across;
    const int each = OP == kWeights ? a.columns : (ceil_div(width, across) + 31) & ~31;
    t.f0 = ((PAIR ? 2 : 1) * f + rank) * (OP == kForward && a.act == AP_ACT_SWIGLU ? kLanes / 2 : kLanes);
    t.c0 = c * each;
    t.n = min(each, width - t.c0);
    t.row0 = w.tab.seg[w.e] + (OP == kWeights ? 0 : t.c0);
    t.steps = OP == kWeights ? ceil_div(t.live, kDepth) : ceil_div(a.K, kDepth);
    t.sections = PARTS ? ceil_div(t.steps, kPart) : OP == kWeights && a.out_f32 ? ceil_div(t.steps, kSection) : t.steps > 0;
    return t;
}

// A stage: the features' operand (16 KB), then the columns'.  A gated product's
// features alternate by 16 between the gate's and the up product's, so that a
// writing lane finds both.
template <Op OP, bool PAIR>
__device__ __forceinline__ void fetch(const ExArgs &a, const Tile &t, int step, uint8_t *stage, const ExMaps &m, uint32_t full, int rank)
{
    const int k0 = step * kDepth;
    const bool gated = OP == kForward && a.act == AP_ACT_SWIGLU;
    uint8_t *col = stage + 2 * kPanel;
    const uint32_t sa = smem_addr(stage), sb = smem_addr(col);
    // a pair's blocks bring half of the tile's columns each, and all tell the first one's barrier
    const int half = (t.n + 31) / 32 * 16, most = PAIR ? a.columns / 2 : a.columns, cols = PAIR ? half : t.n;
    const int from = PAIR ? rank * half : 0; // of the tile's columns
    const int small = a.columns >= 128 ? 64 : 32, boxes = ceil_div(cols, small);
    const bool all = OP == kWeights || cols > most - small; // as many as there may be
    const int bytes = 2 * kPanel + (all ? most : boxes * small) * 128;
    if (rank == 0) bar_expect(full, PAIR ? 2 * bytes : bytes);
    const uint32_t bar = PAIR ? cluster_addr(full, 0) : full;
    if constexpr (OP == kForward) {
        if (!gated)
            tma_3d<PAIR>(sa, &m.w, k0, t.f0, t.e, bar);
        else if (a.by16)
            tma_5d<PAIR>(sa, &m.w, k0, 0, 0, t.f0 >> 4, t.e, bar);
        else
            for (int b = 0; b < 8; ++b) tma_3d<PAIR>(sa + b * 2048, &m.w, k0, t.f0 + (b >> 1) * 16 + (b & 1) * a.F, t.e, bar);
    } else if constexpr (OP == kRows) {
        tma_3d<PAIR>(sa, &m.w, t.f0, k0, t.e, bar);
        tma_3d<PAIR>(sa + kPanel, &m.w, t.f0 + 64, k0, t.e, bar);
    }
    if constexpr (OP == kWeights) {
        const int row = t.row0 + k0, c = t.c0 + from;
        if (a.chunk_x) {
            tma_3d<PAIR>(sa, &m.xx, 0, row, t.f0 >> 6, bar);
        } else {
            tma_2d<PAIR>(sa, &m.x, t.f0, row, bar);
            tma_2d<PAIR>(sa + kPanel, &m.x, t.f0 + 64, row, bar);
        }
        for (int i = 0; i < most; i += 128) {
            const uint32_t to = sb + i * 128;
            if (a.chunk_w && most >= 128 && c % 64 == 0) {
                tma_3d<PAIR>(to, &m.ww, 0, row, (c + i) >> 6, bar);
            } else {
                tma_2d<PAIR>(to, &m.w, c + i, row, bar);
                if (most >= 128) tma_2d<PAIR>(to + kPanel, &m.w, c + i + 64, row, bar);
            }
        }
    } else if (all) {
        tma_2d<PAIR>(sb, &m.xx, k0, t.row0 + from, bar);
    } else {
        for (int i = 0; i < boxes; ++i) tma_2d<PAIR>(sb + i * small * 128, &m.x, k0, t.row0 + from + i * small, bar);
    }
}

__device__ __forceinline__ uint32_t pack(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A writer's 32 rows (columns of the accumulator) of 32 features (lanes) from f
// on, of which those below F count.  Values in the tiles' layout of
// acc_load_tiles: v[h][4 i + 2 s + c] is feature f + 16 h + 8 s + lane / 4 of row
// 8 i + 2 (lane % 4) + c; as 16-bit pairs: p[i][2 h + s].
using Frag = float[2][16];
using Pairs = uint32_t[4][4];

// Memory's rows of 32 features: lane l holds 16 bytes of row 8 q + l / 4, piece l % 4.
struct Piece {
    uint4 w[4];
};
// Which of the 32 features count: those below `left` of the first 16 and below
// `left2` of the others, which begin `second` elements on (16, or a gated product's other half).
struct Span {
    int left, left2;
    int64_t second;
};
__device__ __forceinline__ Span together(int left) { return {left, left - 16, 16}; }
__device__ __forceinline__ void piece_load(Piece &x, const bf16_t *rows, int64_t ld, int count, const Span &n, bool vec)
{
    const int lane = (int)lane_id();
    const int at = (lane & 1) * 8; // of the 16 features of a half
    const int64_t off = (lane & 2 ? n.second : 0) + at;
    const int in = (lane & 2 ? n.left2 : n.left) - at; // features from this piece on that count
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = q * 8 + (lane >> 2);
        x.w[q] = make_uint4(0, 0, 0, 0);
        if (r >= count) continue;
        const bf16_t *p = rows + r * ld + off;
        if (vec) {
            // (volatile: the load stays here, ahead of the work on the rows before)
            asm volatile("{ .reg .pred q; setp.gt.s32 q, %5, 0; @q ld.global.v4.u32 {%0, %1, %2, %3}, [%4]; }"
                         : "+r"(x.w[q].x), "+r"(x.w[q].y), "+r"(x.w[q].z), "+r"(x.w[q].w)
                         : "l"(p), "r"(in)
                         : "memory");
        } else {
            const unsigned short *s = reinterpret_cast<const unsigned short *>(p);
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < in) w[j / 2] |= (uint32_t)s[j] << 16 * (j & 1);
            x.w[q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}
__device__ __forceinline__ void piece_to_pairs(const Piece &x, uint8_t *pass, Pairs &p)
{
    const int lane = (int)lane_id();
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4 *>(pass + (q * 8 + (lane >> 2)) * kPassPitch + (lane & 3) * 16) = x.w[q];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) matrices_load(smem_addr(pass) + (i * 8 + (lane & 7)) * kPassPitch + (lane >> 3) * 16, p[i]);
}
__device__ __forceinline__ void pairs_store(const Pairs &p, uint8_t *pass, bf16_t *rows, int64_t ld, int count, const Span &n, bool vec)
{
    const int lane = (int)lane_id();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) matrices_store(smem_addr(pass) + (i * 8 + (lane & 7)) * kPassPitch + (lane >> 3) * 16, p[i]);
    __syncwarp();
    if (vec) {
        const int at = (lane & 1) * 8;
        const int64_t off = (lane & 2 ? n.second : 0) + at;
        const int in = (lane & 2 ? n.left2 : n.left) - at;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = q * 8 + (lane >> 2);
            const uint4 w = *reinterpret_cast<const uint4 *>(pass + r * kPassPitch + (lane & 3) * 16);
            if (r < count && in > 0) *reinterpret_cast<uint4 *>(rows + r * ld + off) = w;
        }
    } else { // a row at a time, a feature a lane
        const int in = (lane < 16 ? n.left : n.left2) - (lane & 15);
        unsigned short *to = reinterpret_cast<unsigned short *>(rows) + (lane & 15) + (lane < 16 ? 0 : n.second);
        for (int r = 0; r < count; ++r)
            if (in > 0) to[r * ld] = *reinterpret_cast<const unsigned short *>(pass + r * kPassPitch + lane * 2);
    }
}
// The first halves alone (16 features).
__device__ __forceinline__ void half_store(const uint32_t (&p)[4][2], uint8_t *pass, bf16_t *rows, int64_t ld, int count, int left,
                                           bool vec)
{
    const int lane = (int)lane_id();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t r[4] = {p[2 * i][0], p[2 * i][1], p[2 * i + 1][0], p[2 * i + 1][1]};
        matrices_store(smem_addr(pass) + ((2 * i + (lane >> 4)) * 8 + (lane & 7)) * kPassPitch + (lane >> 3 & 1) * 16, r);
    }
    __syncwarp();
    if (vec) {
        const int at = (lane & 1) * 8;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = q * 16 + (lane >> 1);
            const uint4 w = *reinterpret_cast<const uint4 *>(pass + r * kPassPitch + (lane & 1) * 16);
            if (r < count && left > at) *reinterpret_cast<uint4 *>(rows + r * ld + at) = w;
        }
    } else {
        unsigned short *to = reinterpret_cast<unsigned short *>(rows) + (lane & 15);
        for (int r = lane >> 4; r < count; r += 2)
            if (left > (lane & 15)) to[r * ld] = *reinterpret_cast<const unsigned short *>(pass + r * kPassPitch + (lane & 15) * 2);
    }
}
// FP32 results go straight to memory: eight lanes hold 32 bytes of a row.
__device__ __forceinline__ void floats_store(const float (&v)[16], float *rows, int64_t ld, int count, int left)
{
    const int lane = (int)lane_id();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 8 * i + 2 * (lane & 3) + c, f = 8 * s + (lane >> 2);
                if (r < count && f < left) rows[r * ld + f] = v[4 * i + 2 * s + c];
            }
}
__device__ __forceinline__ void to_pairs(const Frag &v, Pairs &p)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < 2; ++s) p[i][2 * h + s] = pack(v[h][4 * i + 2 * s], v[h][4 * i + 2 * s + 1]);
}
// fn(value, what the pairs hold there) for all 32 values.
template <typename Fn> __device__ __forceinline__ void with_pairs(Frag &v, const Pairs &p, Fn fn)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                v[h][4 * i + 2 * s] = fn(v[h][4 * i + 2 * s], low(p[i][2 * h + s]));
                v[h][4 * i + 2 * s + 1] = fn(v[h][4 * i + 2 * s + 1], high(p[i][2 * h + s]));
            }
}
__device__ __forceinline__ void result_store(const ExArgs &a, const Frag &v, uint8_t *pass, int64_t at, int count, int left)
{
    if (a.out_f32) {
        float *out = static_cast<float *>(a.out) + at;
        floats_store(v[0], out, a.ldo, count, left);
        floats_store(v[1], out + 16, a.ldo, count, left - 16);
    } else {
        Pairs p;
        to_pairs(v, p);
        pairs_store(p, pass, static_cast<bf16_t *>(a.out) + at, a.ldo, count, together(left), a.vec_out);
    }
}

// What the epilogue reads of 32 rows, on its way while the products still run.
struct Ahead {
    Piece residual, first, second;
};
template <Op OP>
__device__ __forceinline__ void read_ahead(const ExArgs &a, const Tile &t, int c, int part, Ahead &x)
{
    if (c >= t.n) return;
    const int64_t row = (int64_t)t.row0 + c;
    const int count = min(32, t.n - c);
    const bool gated = a.act == AP_ACT_SWIGLU;
    const int f = t.f0 + part * (OP == kForward && gated ? 16 : 32), left = a.F - f;
    if (a.residual) piece_load(x.residual, a.residual + row * a.ldres + f, a.ldres, count,
                               together(OP == kForward && gated ? min(left, 16) : left), a.vec_res);
    if (OP == kRows && a.act != AP_ACT_NONE) {
        piece_load(x.first, a.pre + row * a.ldpre + f, a.ldpre, count, together(left), a.vec_pre);
        if (gated) piece_load(x.second, a.pre + row * a.ldpre + f + a.F, a.ldpre, count, together(left), a.vec_pre);
    }
}

// The epilogue of 32 rows from c on: forwards.
__device__ __forceinline__ void write_rows(const ExArgs &a, const Tile &t, int c, int part, Frag &v, const Ahead &x, uint8_t *pass)
{
    const int lane = (int)lane_id();
    const int64_t row = (int64_t)t.row0 + c;
    const int count = min(32, t.n - c);
    const bool gated = a.act == AP_ACT_SWIGLU;
    const int f = t.f0 + part * (gated ? 16 : 32), left = a.F - f;
    if (left <= 0) return;
    if (a.bias) {
        const float *b = a.bias + (int64_t)t.e * (gated ? 2 : 1) * a.F + f + (lane >> 2);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bool in = (gated ? 0 : 16 * h) + 8 * s + (lane >> 2) < left;
                const float add = in ? b[(gated ? h * a.F : 16 * h) + 8 * s] : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[h][4 * i + 2 * s] += add;
                    v[h][4 * i + 2 * s + 1] += add;
                }
            }
    }
    Pairs p;
    if (a.pre) {
        to_pairs(v, p);
        pairs_store(p, pass, a.pre + row * a.ldpre + f, a.ldpre, count, gated ? Span{left, left, a.F} : together(left), a.vec_pre);
    }
    if (gated) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[0][i] = v[0][i] * sigmoid_fast(v[0][i]) * v[1][i];
    } else if (a.act == AP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i / 16][i % 16] *= sigmoid_fast(v[i / 16][i % 16]);
    } else if (a.act == AP_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i / 16][i % 16] = gelu_of(v[i / 16][i % 16]);
    }
    if (a.residual) {
        piece_to_pairs(x.residual, pass, p);
        with_pairs(v, p, [](float y, float r) { return y + r; });
    }
    const int64_t at = row * a.ldo + f;
    if (!gated) {
        result_store(a, v, pass, at, count, left);
    } else if (a.out_f32) {
        floats_store(v[0], static_cast<float *>(a.out) + at, a.ldo, count, left);
    } else {
        uint32_t q[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s) q[i][s] = pack(v[0][4 * i + 2 * s], v[0][4 * i + 2 * s + 1]);
        half_store(q, pass, static_cast<bf16_t *>(a.out) + at, a.ldo, count, left, a.vec_out);
    }
}

// Backwards to the rows.
__device__ __forceinline__ void write_slopes(const ExArgs &a, const Tile &t, int c, int part, Frag &v, const Ahead &x, uint8_t *pass)
{
    const int64_t row = (int64_t)t.row0 + c;
    const int count = min(32, t.n - c);
    const int f = t.f0 + part * 32, left = a.F - f;
    if (left <= 0) return;
    Pairs p;
    if (a.residual) {
        piece_to_pairs(x.residual, pass, p);
        with_pairs(v, p, [](float y, float r) { return y + r; });
    }
    const int64_t at = row * a.ldo + f;
    if (a.act == AP_ACT_SWIGLU) {
        Pairs u;
        piece_to_pairs(x.first, pass, p);
        piece_to_pairs(x.second, pass, u);
        Frag d;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float g = e ? high(p[i][2 * h + s]) : low(p[i][2 * h + s]);
                        const float w = e ? high(u[i][2 * h + s]) : low(u[i][2 * h + s]);
                        const float q = sigmoid_fast(g), y = v[h][4 * i + 2 * s + e];
                        v[h][4 * i + 2 * s + e] = y * w * (q * (1.f + g * (1.f - q)));
                        d[h][4 * i + 2 * s + e] = y * g * q;
                    }
        result_store(a, v, pass, at, count, left);
        result_store(a, d, pass, at + a.F, count, left);
        return;
    }
    if (a.act == AP_ACT_SILU) {
        piece_to_pairs(x.first, pass, p);
        with_pairs(v, p, [](float y, float z) { return y * act_slope(AP_ACT_SILU, z); });
    } else if (a.act == AP_ACT_GELU) {
        piece_to_pairs(x.first, pass, p);
        with_pairs(v, p, [](float y, float z) { return y * act_slope(AP_ACT_GELU, z); });
    }
    result_store(a, v, pass, at, count, left);
}

// Weights: rows are the lanes, 32 of their places the columns.  Sixteen rows at a
// time pass through shared memory (lines of 128 bytes, swizzled in pieces of 16),
// so that memory sees pieces of 128 bytes (BF16: 64) of a row.  FP32 sums to what
// is there are left to memory: its vector reductions need no answer.
__device__ __forceinline__ void add_vector(float *p, float4 v)
{
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void add_one(float *p, float v) { asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory"); }

template <typename T> __device__ __forceinline__ T *weights_at(const ExArgs &a, const Tile &t, int c, int f)
{
    return static_cast<T *>(a.out) + ((int64_t)t.e * a.F + f) * a.K + t.c0 + c;
}
// BF16 weights that are there, read while the products run: 8 of row 8 q + lane / 4.
struct Kept {
    uint4 w[4];
};
__device__ __forceinline__ void read_weights(const ExArgs &a, const Tile &t, int c, int f, Kept &x)
{
    const int lane = (int)lane_id(), k = c + (lane & 3) * 8;
    if (!a.add || a.out_f32 || !a.vec_out || k >= t.n) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int row = f + q * 8 + (lane >> 2);
        if (row < a.F) x.w[q] = *reinterpret_cast<const uint4 *>(weights_at<bf16_t>(a, t, k, row));
    }
}
__device__ __forceinline__ void write_weights(const ExArgs &a, const Tile &t, int c, int f, const float (&v)[32], const Kept &kept,
                                              bool add, uint8_t *pass)
{
    const int lane = (int)lane_id();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int f0 = f + h * 16;
        __syncwarp();
        if (lane >> 4 == h)
#pragma unroll
            for (int q = 0; q < 8; ++q)
                *reinterpret_cast<float4 *>(pass + (lane & 15) * 128 + ((q ^ (lane & 7)) << 4)) =
                    make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        __syncwarp();
        const auto piece = [&](int r, int q) { return *reinterpret_cast<const float4 *>(pass + r * 128 + ((q ^ (r & 7)) << 4)); };
        if (a.vec_out && a.out_f32) {
            const int k = c + (lane & 7) * 4;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = q * 4 + (lane >> 3);
                const float4 x = piece(r, lane & 7);
                if (f0 + r < a.F && k < t.n) {
                    float *p = weights_at<float>(a, t, k, f0 + r);
                    if (add)
                        add_vector(p, x);
                    else
                        *reinterpret_cast<float4 *>(p) = x;
                }
            }
        } else if (a.vec_out) {
            const int k = c + (lane & 3) * 8;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = q * 8 + (lane >> 2);
                float4 x = piece(r, (lane & 3) * 2), y = piece(r, (lane & 3) * 2 + 1);
                if (add) {
                    const uint4 o = kept.w[h * 2 + q];
                    x.x += low(o.x), x.y += high(o.x), x.z += low(o.y), x.w += high(o.y);
                    y.x += low(o.z), y.y += high(o.z), y.z += low(o.w), y.w += high(o.w);
                }
                if (f0 + r < a.F && k < t.n)
                    *reinterpret_cast<uint4 *>(weights_at<bf16_t>(a, t, k, f0 + r)) =
                        make_uint4(pack(x.x, x.y), pack(x.z, x.w), pack(y.x, y.y), pack(y.z, y.w));
            }
        } else { // a row at a time, a place a lane
            const int rows = min(16, a.F - f0);
            if (c + lane < t.n)
#pragma unroll 4
                for (int r = 0; r < rows; ++r) {
                    const float x = *reinterpret_cast<const float *>(pass + r * 128 + ((lane >> 2 ^ (r & 7)) << 4) + (lane & 3) * 4);
                    if (a.out_f32) {
                        float *p = weights_at<float>(a, t, c + lane, f0 + r);
                        if (add)
                            add_one(p, x);
                        else
                            *p = x;
                    } else {
                        bf16_t *p = weights_at<bf16_t>(a, t, c + lane, f0 + r);
                        *p = __float2bfloat16_rn(add ? __bfloat162float(*p) + x : x);
                    }
                }
        }
    }
}

// One writer: two for each quarter of the accumulator's lanes.
template <Op OP, bool PAIR, bool PARTS>
__device__ __forceinline__ void write_tiles(const ExArgs &a, Walk &w, int rank, int writer, uint32_t tmem, uint64_t *s_done,
                                            uint64_t *s_free, uint8_t *pass, volatile int *dead, const volatile uint32_t *fetched)
{
    const int part = writer & 3, lane = (int)lane_id();
    uint32_t count = 0;
    bool ok = true;
    const auto release = [&](uint32_t acc) { // the accumulator is read
        __syncwarp();
        if (lane == 0) {
            if (PAIR)
                bar_arrive_at(cluster_addr(smem_addr(&s_free[acc]), 0));
            else
                bar_arrive(smem_addr(&s_free[acc]));
        }
    };
    for (; w.find(a.E); w.next()) {
        const Tile t = tile_of<OP, PAIR, PARTS>(a, w, rank);
        const int f = t.f0 + part * kWarp; // (of weights)
        const uint32_t own = tmem + ((uint32_t)part * kWarp << 16);
        if constexpr (PARTS) { // sections to their sums, which the epilogue takes
            for (int section = 0; section < t.sections; ++section, ++count) {
                ok = __all_sync(0xffffffffu, ok && bar_wait(smem_addr(&s_done[0]), count & 1, dead, fetched));
                fence_after();
                if (ok) {
                    for (int c = (writer >> 2) * 32; c < t.n; c += 64) acc_fold(own + c, own + 256 + c, section > 0);
                    acc_folded();
                }
                fence_before();
                release(0);
            }
        }
        for (int section = 0; section == 0 || (!PARTS && section < t.sections); ++section) {
            const uint32_t acc = count & 1, at = own + (PARTS ? 1 : acc) * 256;
            const bool waits = t.steps > 0 && !PARTS;
            int c = (writer >> 2) * 32;
            Ahead x;
            Kept kept;
            if constexpr (OP == kWeights)
                read_weights(a, t, c, f, kept);
            else
                read_ahead<OP>(a, t, c, part, x);
            if (waits) {
                // (for all of a section, which may be a whole expert's rows: as long as stages come)
                ok = __all_sync(0xffffffffu, ok && bar_wait(smem_addr(&s_done[acc]), count >> 1 & 1, dead, fetched));
                ++count;
            }
            fence_after();
            if (c >= t.n && waits) release(acc);
            for (; c < t.n; c += 64) {
                const bool last = c + 64 >= t.n;
                float v[32];
                Frag y;
                if (t.steps > 0 && ok) {
                    if constexpr (OP == kWeights)
                        acc_load(at + c, v);
                    else
                        acc_load_tiles(at + c, y);
                } else { // nothing to add up, or products that did not come
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        v[j] = t.steps > 0 ? NAN : 0.f;
                        y[j / 16][j % 16] = NAN;
                    }
                }
                if (last) {
                    fence_before();
                    if (waits) release(acc);
                }
                if constexpr (OP == kWeights) {
                    const Kept now = kept;
                    if (!last) read_weights(a, t, c + 64, f, kept);
                    if (f < a.F) write_weights(a, t, c, f, v, now, a.add || section > 0, pass);
                } else {
                    const Ahead now = x;
                    if (!last) read_ahead<OP>(a, t, c + 64, part, x);
                    if constexpr (OP == kForward)
                        write_rows(a, t, c, part, y, now, pass);
                    else
                        write_slopes(a, t, c, part, y, now, pass);
                }
            }
        }
    }
    if (!ok && a.d_status && lane == 0) atomicOr(a.d_status, AP_FLAG_CORRUPT);
}

template <Op OP, bool PAIR, bool PARTS>
__global__ void __launch_bounds__(kExThreads, 1)
    k_experts(const __grid_constant__ ExMaps m, const ExArgs a)
{
    pdl_begin();
    constexpr bool kPass2 = OP == kWeights; // two warps pass stages on to the products
    extern __shared__ __align__(1024) uint8_t s_mem[];
    __shared__ Table s_tab;
    constexpr int kPassOf = OP == kWeights ? kHalf : kPass;
    __shared__ __align__(16) uint8_t s_pass[kWriters * kPassOf];
    __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_ready[kPass2 ? kMaxStages : 1], s_done[2], s_free[2], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;
    __shared__ uint32_t s_fetched; // stages so far
    const int wid = threadIdx.x / kWarp, lane = (int)lane_id();
    const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;
    const int stage_bytes = 2 * kPanel + a.columns * (PAIR ? 64 : 128);
    uint8_t *stages = s_mem + ((1024 - (smem_addr(s_mem) & 1023)) & 1023);
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            bar_init(smem_addr(&s_full[s]), 1);
            bar_init(smem_addr(&s_empty[s]), kPass2 && a.db ? 3 : 1);
            if (kPass2) bar_init(smem_addr(&s_ready[s]), 2);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(smem_addr(&s_done[s]), 1);
            bar_init(smem_addr(&s_free[s]), (PAIR ? 2 : 1) * kWriters);
        }
        bar_init(smem_addr(&s_drain), 1);
        bar_init_done();
        s_dead = 0;
        s_fetched = 0;
    }
    if (wid == 1) tmem_alloc<PAIR>(smem_addr(&s_tmem), 512);
    if (wid == 2) count_tiles<OP>(a, s_tab);
    fence_before();
    __syncthreads();
    if (PAIR) cluster_sync(); // the other block's barriers are ready, and it has the table of its own
    fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *dead = &s_dead;
    Walk w(s_tab, (int)blockIdx.x / (PAIR ? 2 : 1), (int)gridDim.x / (PAIR ? 2 : 1));

    if (wid == 0) {
        // ---- fetch: stage by stage, as they fall empty
        if (elect_one()) {
            if (a.rows > 0) {
                tma_prefetch_map(OP == kWeights && !a.chunk_x ? &m.x : &m.xx);
                tma_prefetch_map(OP == kWeights && a.chunk_w ? &m.ww : &m.w);
            }
            uint32_t count = 0, s = 0, turn = 0; // stages fetched; ring position and its turn
            bool ok = true;
            for (; ok && w.find(a.E); w.next()) {
                const Tile t = tile_of<OP, PAIR, PARTS>(a, w, rank);
                for (int step = 0; step < t.steps; ++step) {
                    if (count >= (uint32_t)a.stages && !bar_wait(smem_addr(&s_empty[s]), (turn & 1) ^ 1, dead)) {
                        ok = false;
                        break;
                    }
                    fetch<OP, PAIR>(a, t, step, stages + (size_t)s * stage_bytes, m, smem_addr(&s_full[s]), rank);
                    *(volatile uint32_t *)&s_fetched = ++count;
                    if (++s == (uint32_t)a.stages) {
                        s = 0;
                        ++turn;
                    }
                }
            }
            if (PAIR || !ok) {
                // Copies on their way end before the block does (a pair's are told to the first block, which the second
                // waits for below), and so do the arrivals that the other block's products send here.
                volatile int none = 0;
                for (uint32_t i = 0; i < (uint32_t)a.stages && i < count; ++i) {
                    const uint32_t c = count - 1 - i, at = c % a.stages, parity = c / a.stages & 1;
                    none = 0;
                    if (ok)
                        (void)bar_wait(smem_addr(&s_empty[at]), parity, dead);
                    else if (rank == 0)
                        (void)bar_wait(smem_addr(&s_full[at]), parity, &none);
                }
            }
        }
    } else if (wid == 1) {
        // ---- multiply (a pair's first block for both)
        if (rank == 0 && elect_one()) {
            uint32_t s = 0, turn = 0, count = 0; // ring; tiles so far
            bool ok = true;
            for (; ok && w.find(a.E); w.next()) {
                const Tile t = tile_of<OP, PAIR, PARTS>(a, w, rank);
                if (t.steps == 0) continue;
                const uint32_t shape = shape_of(PAIR ? 2 * kLanes : kLanes, PAIR ? (t.n + 31) & ~31 : (t.n + 15) & ~15,
                                                OP != kForward, OP == kWeights);
                const int section = t.sections <= 1 ? t.steps : PARTS ? kPart : kSection;
                constexpr int two = !PARTS; // accumulators in turn, or one
                for (int from = 0; ok && from < t.steps; from += section, ++count) {
                    const uint32_t acc = two ? count & 1 : 0;
                    ok = count < 1u + two || bar_wait(smem_addr(&s_free[acc]), (count >> two & 1) ^ 1, dead);
                    fence_after();
                    const int end = min(from + section, t.steps);
                    for (int step = from; ok && step < end; ++step) {
                        ok = bar_wait(smem_addr(kPass2 ? &s_ready[s] : &s_full[s]), turn & 1, dead);
                        if (!ok) break;
                        fence_after();
                        const uint32_t sa = smem_addr(stages) + s * stage_bytes, sb = sa + 2 * kPanel;
#pragma unroll
                        for (int k = 0; k < kDepth / 16; ++k)
                            mma<PAIR>(tmem + acc * 256, operand(sa + k * (OP == kForward ? 32 : 2048), kPanel),
                                      operand(sb + k * (OP == kWeights ? 2048 : 32), kPanel), shape, step > from || k > 0);
                        mma_commit<PAIR>(smem_addr(&s_empty[s]));
                        if (++s == (uint32_t)a.stages) {
                            s = 0;
                            ++turn;
                        }
                    }
                    if (ok) mma_commit<PAIR>(smem_addr(&s_done[acc]));
                }
            }
            if (*dead) { // products on their way end before tensor memory is freed
                volatile int none = 0;
                mma_commit<PAIR>(smem_addr(&s_drain));
                (void)bar_wait(smem_addr(&s_drain), 0, &none);
            }
        }
    } else if (kPass2 && wid < 4) {
        // ---- pass stages on, with zeros for the lines behind an expert's last row, which are others' rows; and add up the
        // bias's gradient, each row of tiles in one of them: always the first would be the same SMs' wherever `across` and the
        // grid have a factor in common, so it moves on from round to round of the grid, or else from row to row (65536 rows, 128
        // experts, 2048 x 1024: 463 us for 546; without a bias 462). A warp takes a panel of 64 features, a lane 8 of them of
        // every fourth line, in two sums a stage
        uint32_t s = 0, turn = 0;
        bool ok = true;
        for (; w.find(a.E); w.next()) {
            const Tile t = tile_of<OP, PAIR, PARTS>(a, w, rank);
            const uint32_t across = ceil_div(a.K, a.columns), c = t.c0 / a.columns, first = w.t - c, by = w.step;
            const bool adds = a.db && c == first / (by % across ? across : by) % across;
            float sum[8] = {};
            for (int step = 0; ok && step < t.steps; ++step) {
                ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&s_full[s]), turn & 1, dead));
                if (!ok) break;
                const int left = t.live - step * kDepth;
                if (left < kDepth) {
                    uint8_t *stage = stages + (size_t)s * stage_bytes;
                    const int panels = 2 + a.columns / 64;
                    for (int p = wid - 2; p < panels; p += 2)
                        for (int b = left * 128 + lane * 16; b < kPanel; b += kWarp * 16)
                            *reinterpret_cast<uint4 *>(stage + p * kPanel + b) = make_uint4(0, 0, 0, 0);
                    fence_async();
                    __syncwarp();
                }
                if (lane == 0) bar_arrive(smem_addr(&s_ready[s]));
                if (a.db) {
                    if (adds) {
                        const uint8_t *panel = stages + (size_t)s * stage_bytes + (wid - 2) * kPanel;
                        float part[2][8] = {};
#pragma unroll
                        for (int i = 0; i < kDepth / 4; ++i) {
                            const int r = 4 * i + (lane >> 3);
                            const uint4 x = *reinterpret_cast<const uint4 *>(panel + r * 128 + (((lane ^ r) & 7) << 4));
                            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                part[i & 1][2 * j] += low(y[j]);
                                part[i & 1][2 * j + 1] += high(y[j]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) sum[j] += part[0][j] + part[1][j];
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(smem_addr(&s_empty[s])); // (the stage is read)
                }
                if (++s == (uint32_t)a.stages) {
                    s = 0;
                    ++turn;
                }
            }
            if (adds)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 8);
                    sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
                    const int f = t.f0 + (wid - 2) * 64 + lane * 8 + j;
                    float *to = a.db + (int64_t)t.e * a.F + f;
                    if (lane < 8 && f < a.F) *to = ok ? a.add ? *to + sum[j] : sum[j] : NAN;
                }
        }
    } else if (wid >= 4) {
        // ---- write
        write_tiles<OP, PAIR, PARTS>(a, w, rank, wid - 4, tmem, s_done, s_free, s_pass + (wid - 4) * kPassOf, dead, &s_fetched);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (PAIR) cluster_sync(); // neither block's memory is used by the other any more
    if (wid == 1) {
        fence_after();
        tmem_free<PAIR>(tmem, 512);
    }
}

// 16 bytes from an address between granules: of the two granules a and b those
// from byte `off` (even) on.
__device__ __forceinline__ uint4 cut(uint4 a, uint4 b, uint32_t off)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
    if (off & 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows of `cols` values, ld apart (per of them to an expert, experts lde apart),
// to rows that begin on 16-byte boundaries; experts without rows are left out.  A
// warp per row, a lane per 16 bytes there: it cuts them out of the granules that
// hold them, which are read whole where they lie inside the buffer, and by
// elements where its ends cut them.  Two operands go in one launch (999 tokens'
// rows and 60 experts' weights of 1003 x 517 with their product: 59.6 us for 61.1).  Bound by HBM.
struct Lot {
    const bf16_t *src;
    int64_t ld, lde, per, rows;
    const int32_t *live;
    bf16_t *dst;
    int64_t pitch;
    int cols;
};
__global__ void __launch_bounds__(256) k_repitch(const Lot first, const Lot second)
{
    pdl_begin();
    const int lane = (int)lane_id();
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / kWarp; i < first.rows + second.rows; i += step) {
        const bool other = i >= first.rows;
        const int64_t r = other ? i - first.rows : i, rows = other ? second.rows : first.rows, per = other ? second.per : first.per,
                      ld = other ? second.ld : first.ld, lde = other ? second.lde : first.lde;
        const bf16_t *src = other ? second.src : first.src;
        const int32_t *live = other ? second.live : first.live;
        const int cols = other ? second.cols : first.cols, pieces = (cols + 7) / 8;
        const int64_t e = r / per;
        if (live && live[e] <= 0) continue;
        const char *begin = reinterpret_cast<const char *>(src);
        const char *end = reinterpret_cast<const char *>(src + (rows - 1) / per * lde + (rows - 1) % per * ld + cols);
        const char *row = reinterpret_cast<const char *>(src + e * lde + (r - e * per) * ld);
        uint4 *to = reinterpret_cast<uint4 *>(other ? second.dst + r * second.pitch : first.dst + r * first.pitch);
        const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(row) & 15; // of every piece
        constexpr int kEach = 4;
        for (int c0 = lane; c0 < pieces; c0 += kEach * kWarp) {
            uint4 lo[kEach], hi[kEach];
            bool whole[kEach];
#pragma unroll
            for (int u = 0; u < kEach; ++u) {
                const int c = c0 + u * kWarp, n = min(cols - c * 8, 8);
                const char *at = row + c * 16 - off;
                const bool second = (int)off + 2 * n > 16;
                lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
                whole[u] = at >= begin && at + (second ? 32 : 16) <= end;
                if (n > 0 && whole[u]) {
                    lo[u] = *reinterpret_cast<const uint4 *>(at);
                    if (second) hi[u] = *reinterpret_cast<const uint4 *>(at + 16);
                }
            }
#pragma unroll
            for (int u = 0; u < kEach; ++u) {
                const int c = c0 + u * kWarp, n = min(cols - c * 8, 8);
                if (n <= 0) continue;
                uint4 w = cut(lo[u], hi[u], off);
                if (!whole[u]) {
                    const unsigned short *p = reinterpret_cast<const unsigned short *>(row) + c * 8;
                    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < n) v[j / 2] |= (uint32_t)p[j] << 16 * (j & 1);
                    w = make_uint4(v[0], v[1], v[2], v[3]);
                }
                to[c] = w; // (what lies behind the last value is no part of a row to the tensor maps)
            }
        }
    }
}

// db[e] (+)= the sum of the expert's rows of dy, where the weights' gradient is
// not wanted (with it, its stages are added up): a block takes 64 columns of an
// expert, eight warps every eighth row, two columns a lane.
__global__ void __launch_bounds__(256) k_expert_bias(const bf16_t *dy, int64_t ld, const int32_t *seg, const int32_t *live, int64_t rows,
                                                     int N, float *db, bool add, uint32_t *d_status)
{
    pdl_begin();
    __shared__ float s_sum[8][64];
    const int e = blockIdx.y, wid = threadIdx.x / kWarp, lane = (int)lane_id();
    const int at = seg[e];
    int n = live[e];
    if (n < 0 || at < 0 || (int64_t)at + n > rows) {
        n = 0;
        if (d_status && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(d_status, AP_FLAG_BAD_COUNT);
    }
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

// The stages that fit the shared memory, and its bytes: as many as the kernel's attribute allows (0: an error).
template <Op OP, bool PAIR, bool PARTS> size_t stages_of(ExArgs &a)
{
    const auto kernel = k_experts<OP, PAIR, PARTS>;
    static const int fixed = [&] {
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, (const void *)kernel) != cudaSuccess) return -1;
        const int n = (int)attr.sharedSizeBytes;
        return cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - n) == cudaSuccess ? n
                                                                                                                                    : -1;
    }();
    if (fixed < 0) return 0;
    const int stage = 2 * kPanel + a.columns * (PAIR ? 64 : 128), room = kMaxSmem - fixed - 1024;
    a.stages = room / stage < kMaxStages ? room / stage : kMaxStages;
    return (size_t)a.stages * stage + 1024;
}
// Pairs of blocks that the stream's SMs take at once (a partition may take none).
template <Op OP, bool PARTS> int pairs_of(ExArgs a, cudaStream_t st)
{
    const size_t smem = stages_of<OP, true, PARTS>(a);
    return smem ? cluster_count((const void *)k_experts<OP, true, PARTS>, kExThreads, smem, 2, st) : 0;
}

// `pairs`: that many at most, of two blocks each; 0: single blocks
template <Op OP, bool PAIR, bool PARTS>
ap_status launch_experts(const char *who, const ExMaps &m, ExArgs a, int64_t tiles, int pairs, cudaStream_t st)
{
    const auto kernel = k_experts<OP, PAIR, PARTS>;
    const size_t smem = stages_of<OP, PAIR, PARTS>(a);
    if (!smem) return cuda_fail(cudaGetLastError(), who);
    if constexpr (PAIR) {
        launch_cluster(kernel, 2 * (int)(tiles < pairs ? tiles : pairs), kExThreads, smem, 2, st, m, a);
    } else {
        const int sms = sm_count();
        launch(kernel, (int)(tiles < sms ? tiles : sms), kExThreads, smem, st, m, a);
    }
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
int64_t repitch_bytes(const void *p, int64_t ld, int64_t lde, int64_t rows, int cols)
{
    return mappable(p, ld, lde) ? 0 : (rows * ((cols + 7) / 8 * 16) + 255) / 256 * 256;
}
// Copies operands that tensor maps do not take into the work space, one after the other.
struct Repitch {
    char *scratch;
    Lot lot[2] = {};
    // `count` lots of `per` rows, *lde apart (nullptr: one lot)
    void take(int i, const bf16_t **p, int64_t *ld, int64_t *lde, int64_t per, int count, int cols, const int32_t *live)
    {
        const int64_t rows = per * count, need = repitch_bytes(*p, *ld, lde ? *lde : 0, rows, cols), pitch = (cols + 7) / 8 * 8;
        if (!need) return;
        bf16_t *to = reinterpret_cast<bf16_t *>(scratch);
        lot[i] = {*p, *ld, lde ? *lde : 0, per, rows, live, to, pitch, cols};
        scratch += need;
        *p = to;
        *ld = pitch;
        if (lde) *lde = per * pitch;
    }
    ap_status run(const char *who, cudaStream_t st)
    {
        const int64_t want = (lot[0].rows + lot[1].rows + 7) / 8, most = (int64_t)sm_count() * 8;
        if (!want) return AP_OK;
        launch(k_repitch, (int)(want < most ? want : most), 256, 0, st, lot[0], lot[1]);
        AP_CHECK_LAUNCH(who);
        return AP_OK;
    }
};
ap_status scratch_ok(const char *who, const void *scratch, int64_t have, int64_t need)
{
    if (!need) return AP_OK;
    if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 15)) return fail(AP_EINVAL, "%s: scratch is NULL or not aligned", who);
    if (have < need) return fail(AP_EINVAL, "%s: scratch of %lld bytes, %lld needed", who, (long long)have, (long long)need);
    return AP_OK;
}
bool odd_address(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Columns of a tile: rows of the output at most, by what an expert has on the average.
int columns_for(int64_t rows, int32_t E)
{
    const int64_t each = rows / E;
    return each > 128 ? 256 : each > 32 ? 128 : 64;
}

template <Op OP, bool PARTS>
ap_status rows_launch(const char *who, const ExMaps &m, const ExArgs &a, int64_t tiles, int pairs, cudaStream_t st)
{
    return pairs ? launch_experts<OP, true, PARTS>(who, m, a, tiles, pairs, st) : launch_experts<OP, false, PARTS>(who, m, a, tiles, 0, st);
}

ap_status rows_product(const char *who, Op op, ExArgs a, int halves, void *scratch, int64_t scratch_bytes, cudaStream_t st)
{
    if (a.E == 1) a.lde = a.ldw * (op == kForward ? a.F * halves : a.K); // (of no account)
    const int wide = op == kForward ? a.F * halves : a.K, deep = op == kForward ? a.K : a.F; // of W[e]
    if (const ap_status r = scratch_ok(who, scratch, scratch_bytes,
                                       repitch_bytes(a.x, a.ldx, 0, a.rows, a.K) +
                                           repitch_bytes(a.W, a.ldw, a.lde, (int64_t)wide * a.E, deep));
        r != AP_OK)
        return r;
    a.columns = columns_for(a.rows, a.E);
    const bool parts = a.out_f32 && a.K > kPart * kDepth;
    a.vec_out = !odd_address(a.out, 16) && a.ldo % 8 == 0 && a.F % 8 == 0;
    a.vec_pre = !odd_address(a.pre, 16) && a.ldpre % 8 == 0 && a.F % 8 == 0;
    a.vec_res = !odd_address(a.residual, 16) && a.ldres % 8 == 0 && a.F % 8 == 0;
    // Two blocks to a tile of 256 features share its rows' operand: 32 KB from L2 for 48 a product (65536 rows of 2048 over
    // 128 experts: 476 us for 545).
    int pairs = 0;
    if (a.columns == 256 && a.F * (op == kForward ? halves : 1) > kLanes)
        pairs = op == kForward ? (parts ? pairs_of<kForward, true>(a, st) : pairs_of<kForward, false>(a, st))
                               : (parts ? pairs_of<kRows, true>(a, st) : pairs_of<kRows, false>(a, st));
    const int per = (op == kForward && halves == 2 ? kLanes / 2 : kLanes) * (pairs ? 2 : 1);
    a.tiles_f = (a.F + per - 1) / per;
    const int64_t tiles = (a.rows / a.columns + a.E) * (int64_t)a.tiles_f;
    if (tiles >= INT32_MAX) return fail(AP_EINVAL, "%s: %lld tiles are more than one launch takes", who, (long long)tiles);
    Repitch re = {static_cast<char *>(scratch)};
    re.take(0, &a.x, &a.ldx, nullptr, a.rows, 1, a.K, nullptr);
    re.take(1, &a.W, &a.ldw, &a.lde, wide, a.E, deep, a.live);
    if (const ap_status r = re.run(who, st); r != AP_OK) return r;
    ExMaps m = {};
    const uint64_t ex[2] = {(uint64_t)a.K, (uint64_t)a.rows}, px[1] = {(uint64_t)a.ldx};
    const uint32_t bx[2] = {64, a.columns >= 128 ? 64u : 32u}, ball[2] = {64, (uint32_t)(pairs ? a.columns / 2 : a.columns)};
    bool ok = make_map(&m.x, a.x, 2, ex, px, bx) && make_map(&m.xx, a.x, 2, ex, px, ball);
    // One copy for a gated product's features needs whole sixteens: 8 copies of 16 lines took 957 us where one takes 590
    a.by16 = op == kForward && halves == 2 && a.F % 16 == 0;
    if (a.by16) {
        const uint64_t ew[5] = {(uint64_t)deep, 16, 2, (uint64_t)a.F / 16, (uint64_t)a.E};
        const uint64_t pw[4] = {(uint64_t)a.ldw, (uint64_t)(a.F * a.ldw), (uint64_t)(16 * a.ldw), (uint64_t)a.lde};
        const uint32_t bw[5] = {64, 16, 2, 4, 1};
        ok = ok && make_map(&m.w, a.W, 5, ew, pw, bw);
    } else {
        const uint64_t ew[3] = {(uint64_t)deep, (uint64_t)wide, (uint64_t)a.E}, pw[2] = {(uint64_t)a.ldw, (uint64_t)a.lde};
        const uint32_t bw[3] = {64, op == kRows ? 64u : halves == 2 ? 16u : 128u, 1};
        ok = ok && make_map(&m.w, a.W, 3, ew, pw, bw);
    }
    if (!ok) return fail(AP_ENOTSUP, "%s: no tensor map of these sizes", who);
    if (op == kForward)
        return parts ? rows_launch<kForward, true>(who, m, a, tiles, pairs, st) : rows_launch<kForward, false>(who, m, a, tiles, pairs, st);
    return parts ? rows_launch<kRows, true>(who, m, a, tiles, pairs, st) : rows_launch<kRows, false>(who, m, a, tiles, pairs, st);
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
    cuuint64_t strides[4], sizes[5];
    cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i < dims; ++i) sizes[i] = extent[i];
    for (int i = 0; i + 1 < dims; ++i) strides[i] = pitch[i] * 2;
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void *>(base), sizes, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

} // namespace ap

extern "C" ap_status ap_expert_linear_scratch_bytes(const void *a, int64_t lda, int64_t rows_a, int32_t cols_a, const void *b,
                                                    int64_t ldb, int64_t lde, int64_t rows_b, int32_t cols_b, int64_t *bytes)
{
    using namespace ap;
    if (!bytes || rows_a < 0 || rows_b < 0 || cols_a < 1 || cols_b < 1 || cols_a > (1 << 20) || cols_b > (1 << 20) ||
        rows_a >= (int64_t(1) << 31) || rows_b >= (int64_t(1) << 32))
        return fail(AP_EINVAL, "expert_linear_scratch_bytes: bad sizes");
    *bytes = repitch_bytes(a, lda, 0, rows_a, cols_a) + repitch_bytes(b, ldb, lde, rows_b, cols_b);
    return AP_OK;
}

extern "C" ap_status ap_expert_linear(const void *x, int64_t ldx, int64_t rows, int32_t E, int32_t N, int32_t K,
                                      const int32_t *d_seg_off, const int32_t *d_live, const void *W, int64_t ldw, int64_t lde,
                                      const float *bias, int32_t act, const void *residual, int64_t ldres, void *pre,
                                      int64_t ldpre, void *out, int64_t ldo, int32_t out_dtype, void *scratch, int64_t scratch_bytes,
                                      uint32_t *d_status, void *stream)
{
    AP_NVTX_RANGE("ap_expert_linear");
    using namespace ap;
    const char *who = "expert_linear";
    if (act < AP_ACT_NONE || act > AP_ACT_SWIGLU) return fail(AP_EINVAL, "%s: unknown activation %d", who, act);
    const int halves = act == AP_ACT_SWIGLU ? 2 : 1;
    if (const ap_status s = check_rows(who, rows, E, N, K, ldx, K, ldw, K, lde, 0); s != AP_OK) return s;
    if (out_dtype != AP_DTYPE_BF16 && out_dtype != AP_DTYPE_F32) return fail(AP_EINVAL, "%s: type %d", who, out_dtype);
    if (ldo < N || (residual && ldres < N) || (pre && ldpre < (int64_t)halves * N)) return fail(AP_EINVAL, "%s: bad pitches", who);
    if (E > 1 && lde < ((int64_t)halves * N - 1) * ldw + K) return fail(AP_EINVAL, "%s: experts' weights overlap or interleave", who);
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
    return rows_product(who, kForward, a, halves, scratch, scratch_bytes, (cudaStream_t)stream);
}

extern "C" ap_status ap_expert_linear_dx(const void *dy, int64_t ldy, int64_t rows, int32_t E, int32_t N, int32_t K,
                                         const int32_t *d_seg_off, const int32_t *d_live, const void *W, int64_t ldw, int64_t lde,
                                         int32_t act, const void *pre, int64_t ldpre, const void *residual, int64_t ldres, void *dx,
                                         int64_t ldx, int32_t dx_dtype, void *scratch, int64_t scratch_bytes, uint32_t *d_status,
                                         void *stream)
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
    if (E > 1 && lde < ((int64_t)N - 1) * ldw + K) return fail(AP_EINVAL, "%s: experts' weights overlap or interleave", who);
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
    return rows_product(who, kRows, a, halves, scratch, scratch_bytes, (cudaStream_t)stream);
}

extern "C" ap_status ap_expert_linear_dw(const void *dy, int64_t ldy, const void *x, int64_t ldx, int64_t rows, int32_t E, int32_t N,
                                         int32_t K, const int32_t *d_seg_off, const int32_t *d_live, int32_t accumulate, void *dW,
                                         int32_t dw_dtype, float *dbias, void *scratch, int64_t scratch_bytes, uint32_t *d_status,
                                         void *stream)
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
        a.out_f32 = dw_dtype == AP_DTYPE_F32, a.add = accumulate != 0, a.db = dbias;
        a.tiles_f = (N + kLanes - 1) / kLanes;
        const auto tiles_of = [&](int columns) { return (int64_t)E * a.tiles_f * ((K + columns - 1) / columns); };
        const auto rounds = [&](int columns) { return (tiles_of(columns) + sm_count() - 1) / sm_count(); };
        // A stage of 256 columns takes 0.43 us, of 128 or 64 0.34 (issuing bounds these): by rounds of tiles over the SMs. 8
        // experts of 4096 rows, 1024 x 1024 (256 or 512 tiles): 79 us by 256, 96 by 128; of 8192, 512 x 512 (64 or 128): 99 and 75.
        a.columns = K <= 64 ? 64 : K > 128 && 4 * rounds(256) <= 3 * rounds(128) ? 256 : 128;
        a.vec_out = !odd_address(dW, 16) && K % (a.out_f32 ? 4 : 8) == 0;
        const int64_t tiles = tiles_of(a.columns);
        if (tiles >= INT32_MAX) return fail(AP_EINVAL, "%s: %lld tiles are more than one launch takes", who, (long long)tiles);
        ExMaps m = {};
        if (rows > 0) {
            if (const ap_status r = scratch_ok(who, scratch, scratch_bytes,
                                               repitch_bytes(dy, ldy, 0, rows, N) + repitch_bytes(x, ldx, 0, rows, K));
                r != AP_OK)
                return r;
            Repitch re = {static_cast<char *>(scratch)};
            re.take(0, &a.x, &a.ldx, nullptr, rows, 1, N, nullptr);
            re.take(1, &a.W, &a.ldw, nullptr, rows, 1, K, nullptr);
            if (const ap_status r = re.run(who, st); r != AP_OK) return r;
            // two chunks of 64 columns in a copy where rows are whole chunks: a row's end is no border to such a map
            a.chunk_x = N % 64 == 0, a.chunk_w = K % 64 == 0;
            const uint64_t ey[3] = {a.chunk_x ? 64 : (uint64_t)N, (uint64_t)rows, (uint64_t)N / 64}, py[2] = {(uint64_t)a.ldx, 64};
            const uint64_t ex[3] = {a.chunk_w ? 64 : (uint64_t)K, (uint64_t)rows, (uint64_t)K / 64}, px[2] = {(uint64_t)a.ldw, 64};
            const uint32_t box[3] = {64, 64, 2};
            const uint64_t e1[2] = {(uint64_t)N, (uint64_t)rows}, e2[2] = {(uint64_t)K, (uint64_t)rows};
            if (!make_map(&m.x, a.x, 2, e1, py, box) || !make_map(&m.w, a.W, 2, e2, px, box) ||
                (a.chunk_x && !make_map(&m.xx, a.x, 3, ey, py, box)) || (a.chunk_w && !make_map(&m.ww, a.W, 3, ex, px, box)))
                return fail(AP_ENOTSUP, "%s: no tensor map of these sizes", who);
        }
        if (const ap_status s = launch_experts<kWeights, false, false>(who, m, a, tiles, 0, st); s != AP_OK) return s;
    }
    if (dbias && !dW) {
        launch(k_expert_bias, dim3((unsigned)((N + 63) / 64), (unsigned)E), 256, 0, st, (const bf16_t *)dy, ldy, d_seg_off, d_live, rows,
               N, dbias, accumulate != 0, d_status);
        AP_CHECK_LAUNCH("expert_linear_dw bias launch");
    }
    return AP_OK;
}
