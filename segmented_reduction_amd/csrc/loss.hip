// loss.hip -- the softmax cross entropy of rows against a vocabulary's weights,
// and its gradient, by pieces of the vocabulary: the logits are never kept.
//
// With z_v = scale <x, W_v>, targets v_j of probability t_j and s = sum t_j,
//   loss = s lse - sum_j t_j z_(v_j), lse = log sum_v exp z_v
//   dz_v = g scale (s exp(z_v - lse) - sum of the t_j with v_j = v)
//   dx = sum_v dz_v W_v, dW_v = sum over rows of dz_v x.
// Forward: tiles of x W^T leave one pair (largest, sum of exponentials) per row
// and tile; a second kernel joins a row's pairs and forms its targets' logits.
// Back, for each piece of the vocabulary: the tiles again, whose epilogue makes
// dz of them, then the two products of dz.  dz is rounded to the inputs' type, which
// the matrix units take: half a step of each term, which adds about as much to the
// results as their own rounding does (bfloat16: 0.0024 off 64 bits in all, 0.0017
// with dz in 32 bits; a caller who wants that calls with float32 values and weights, 1,256
// us against 268 for 4,096 rows x 1,024, 8,192 entries); float32 stays float32.  dx is added up in float32 over the
// pieces and rounded at the end.
// Many rows are bound by the matrix units (4,096 rows x 2,048, 65,536 entries,
// bfloat16: 820 to 860 us forward, 1,280 to 1,340 TFLOP/s; 2,780 to 2,880 back for three
// products, 1,150 to 1,190), few by the weights (8 rows x 2,048, 32,000 entries: 28 us, 4.6
// TB/s; float32 55, 4.8).  Float32, 256 rows x 1,024, 32,000 entries: 105 us forward and 331
// back, what float products take at the rate of a large one; 4,096 rows, 8,192 entries 374
// and 1,214, 184 TFLOP/s by bf16 parts.
// Exponentials are powers of two: z scale log2(e) minus the base in one fma.
#include <algorithm>
#include <cmath>

#include "internal.hpp"
#include "outer.hpp"
#include "rowtile.hpp"

namespace segred {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

struct LossArgs {
    const char *values, *weights;
    const int64_t *target;  // [N, picks]
    const float *probs;     // [N, picks], or null: 1
    int64_t N, V, K, picks;
    int64_t KO;  // columns of the gradients: K, or fewer where the operands are copies of wider rows
    float scale, bend;  // bend = scale log2(e)
    int64_t v0, vc;     // the piece of the vocabulary
    int64_t mtiles, ntiles;
    // forward
    float2 *partial;  // [N, parts] of (base, sum of 2^(z bend - base))
    int64_t parts;
    float *loss, *lse, *picked;  // picked: [N, picks], also the gradient call's
    // back
    const float *grad;
    float *share, *hit;  // [N]: grad scale s (by `factor`) and grad scale
    float *bound;        // [N]: what |dz| of a row is at most
    int64_t *live;       // [N]: the row, or -1 where it has no target
    float *factor;       // what dz is multiplied by before it is rounded, and 1 / factor
    char *slope;         // [N, ld]: dz of the piece
    char *turned;        // [vc, ldn]: the same turned, or null
    int64_t ld, ldn;
    float *hits;         // [N, picks]: dz of the targets, before `factor`
    const char *rows_turned, *words_turned;  // [K, ldn] of the values, [K, ld] of the piece's weights
    float *sums;  // [parts_k, N, K]: dx so far
    int64_t cuts;
    int first;  // the first piece
    void *grad_values;
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Over the four rows of 16 lanes.
template <typename F>
__device__ __forceinline__ float quarters_fold(float v, F f) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return f(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// A tile: rows row0 .. row0 + rows - 1, columns of the piece from n0.
struct LossPlace {
    int64_t row0, n0, tile;  // tile: of the columns
    int rows;
};
template <int BM, int BN>
__device__ __forceinline__ LossPlace loss_place(const LossArgs &a) {
    const int64_t id = xcd_tile(a.mtiles * a.ntiles);
    if (id >= a.mtiles * a.ntiles) return {0, 0, 0, 0};
    const TilePlace at = tile_place(id, a.mtiles, a.ntiles);
    return {at.m * BM, at.n * BN, at.n, (int)min((int64_t)BM, a.N - at.m * BM)};
}
template <typename T>
__device__ __forceinline__ const char *loss_row(const LossArgs &a, const LossPlace &p, int r) {
    return r < p.rows ? a.values + (p.row0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
}
template <typename T>
__device__ __forceinline__ const char *loss_word(const LossArgs &a, const LossPlace &p, int c) {
    return p.n0 + c < a.vc ? a.weights + (a.v0 + p.n0 + c) * a.K * (int64_t)sizeof(T) : nullptr;
}

// The pair of each row of a tile: RI x CJ quads per lane, get(i, j) at row(i)
// and column col(j); WN waves (this one is `wn`) share a row.  `part` is the
// place of the pair among the row's.
template <int RI, int CJ, int WN, int BM, int BN, typename G, typename R, typename C>
__device__ __forceinline__ void loss_pairs(const LossArgs &a, const LossPlace &p, int64_t part, lds_char *lds, int wn,
                                           int lane, G get, R row, C col) {
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    typedef __attribute__((address_space(3))) f32x2 lds_pair;
    lds_pair *s = reinterpret_cast<lds_pair *>(lds);
    const bool cut = p.n0 + BN > a.vc;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
            f32x4 &z = get(i, j);
            if (cut)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (p.n0 + col(j) + e >= a.vc) z[e] = -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, z[e]);
        }
        m = quarters_fold(m, [](float x, float y) { return fmaxf(x, y); }) * a.bend;
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
            const f32x4 &z = get(i, j);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += exp2_fast(fmaf(z[e], a.bend, -base));
        }
        sum = quarters_fold(sum, [](float x, float y) { return x + y; });
        if (lane < 16) s[wn * BM + row(i)] = f32x2{m, sum};
    }
    __syncthreads();
    for (int r = threadIdx.x; r < p.rows; r += blockDim.x) {
        f32x2 v = s[r];
#pragma unroll
        for (int w = 1; w < WN; ++w) {
            const f32x2 o = s[w * BM + r];
            const float m = fmaxf(v[0], o[0]), base = m == -INFINITY ? 0.f : m;
            v = f32x2{m, v[1] * exp2_fast(v[0] - base) + o[1] * exp2_fast(o[0] - base)};
        }
        a.partial[(p.row0 + r) * a.parts + part] = make_float2(v[0], v[1]);
    }
}

// dz of a row's logits, without its targets.
struct LossRow {
    float share, base;
    bool live;
};
__device__ __forceinline__ LossRow loss_row_of(const LossArgs &a, int64_t row) {
    return {a.share[row], a.lse[row] * kLog2e, a.live[row] >= 0};
}
__device__ __forceinline__ f32x4 loss_slopes(const LossArgs &a, const LossRow &o, f32x4 z, int64_t n) {
    f32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        y[e] = o.live && n + e < a.vc ? o.share * exp2_fast(fmaf(z[e], a.bend, -o.base)) : 0.f;
    return y;
}
// Calls put(r, c, dz) for the targets of the tile's rows in its columns.
template <int BM, int BN, int THREADS, typename P>
__device__ __forceinline__ void loss_targets(const LossArgs &a, const LossPlace &p, P put) {
    constexpr int kEach = THREADS / BM, kBatch = 8;  // threads of a row, targets that a thread looks at at a time
    const int picks = (int)a.picks, r = threadIdx.x / kEach;
    if (r >= p.rows) return;
    const int64_t begin = a.v0 + p.n0, row = p.row0 + r;
    const uint64_t left = min((int64_t)BN, a.vc - p.n0);
    const int64_t *target = a.target + row * picks;
    const float f = a.factor ? a.factor[0] : 1.f;
    for (int j0 = threadIdx.x % kEach; j0 < picks; j0 += kBatch * kEach) {
        int64_t t[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) t[b] = j0 + b * kEach < picks ? target[j0 + b * kEach] - begin : -1;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if ((uint64_t)t[b] >= left) continue;
            put(r, (int)t[b], f * a.hits[row * picks + j0 + b * kEach]);
        }
    }
}

// Leaves dz of a tile in the piece, and turned (TURN).
template <typename T, int RI, int CJ, int BM, int BN, int THREADS, bool TURN, typename G, typename R, typename C>
__device__ __forceinline__ void loss_slope(const LossArgs &a, const LossPlace &p, lds_char *lds, int lane, G get, R row,
                                           C col) {
    T *out = reinterpret_cast<T *>(a.slope) + p.row0 * a.ld;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const int r = row(i);
        const LossRow o = r < p.rows ? loss_row_of(a, p.row0 + r) : LossRow{0.f, 0.f, false};
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
            const f32x4 y = loss_slopes(a, o, get(i, j), p.n0 + col(j));
            if constexpr (sizeof(T) == 2) tile_put<T, BN>(lds, r, col(j), y);
            else if (r < p.rows) store_quad<T>(out + r * a.ld, p.n0 + col(j), a.ld, y, true);
        }
    }
    if constexpr (sizeof(T) == 2) {
        __syncthreads();
        loss_targets<BM, BN, THREADS>(a, p, [&](int r, int c, float y) {
            *reinterpret_cast<__attribute__((address_space(3))) T *>(lds + tile_unit<T, BN>(r, c >> 3) + (c & 7) * 2) = (T)y;
        });
        __syncthreads();
        tile_write<T, BM, BN, THREADS>(lds, out, p.rows, p.n0, a.ld, a.ld);
        if constexpr (TURN)
            if (a.turned) {
                tile_turn<T, BM, BN, THREADS>(lds, threadIdx.x >> 6, lane);
                tile_write<T, BN, BM, THREADS>(lds, reinterpret_cast<T *>(a.turned) + p.n0 * a.ldn,
                                               (int)min((int64_t)BN, a.vc - p.n0), p.row0, a.ldn, a.ldn);
            }
    } else {
        // the stores of other waves to the same places must have gone before
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        loss_targets<BM, BN, THREADS>(a, p, [&](int r, int c, float y) { out[r * a.ld + p.n0 + c] = (T)y; });
    }
}

template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool DIRECT, bool SLOPE>
struct LossTile {
    using Tile = RowTile<T, BM, BN, WM, WN, STAGES, DIRECT>;
    static constexpr int kLds = std::max(Tile::kLds, sizeof(T) == 2 && SLOPE ? BM * BN * 2 : WN * BM * 8);
    static __device__ __forceinline__ void run(const LossArgs &a, const LossPlace &p, int64_t part, lds_char *lds,
                                               int wave, int lane) {
        f32x4 acc[Tile::MT][Tile::NT] = {};
        Tile::run(acc, (int)a.K, lds, wave, lane, [&](int r) { return loss_row<T>(a, p, r); },
                  [&](int c) { return loss_word<T>(a, p, c); });
        auto get = [&](int i, int j) -> f32x4 & { return acc[i][j]; };
        auto row = [&](int i) { return Tile::m0(wave) + 16 * i + (lane & 15); };
        auto col = [&](int j) { return Tile::n0(wave) + 16 * j + (lane >> 4) * 4; };
        if constexpr (SLOPE) loss_slope<T, Tile::MT, Tile::NT, BM, BN, Tile::kThreads, DIRECT>(a, p, lds, lane, get, row, col);
        else loss_pairs<Tile::MT, Tile::NT, WN, BM, BN>(a, p, part, lds, wave % WN, lane, get, row, col);
    }
};

template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool DIRECT, bool SLOPE>
__global__ __launch_bounds__(64 * WM * WN) void loss_tiles(LossArgs a) {
    using Tile = LossTile<T, BM, BN, WM, WN, STAGES, DIRECT, SLOPE>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LossPlace p = loss_place<BM, BN>(a);
    if (p.rows > 0) Tile::run(a, p, p.tile, (lds_char *)lds_mem, wave, lane);
}

// Float in bf16 parts, 64 x 128; a tile with a sum that is not finite is computed
// again with float products, 64 columns at a time: a pair covers 64 columns, and
// where there is one for 128 the second is empty.
template <bool WHOLE, bool SLOPE>
__global__ __launch_bounds__(kRowSplitThreads, 3) void loss_split(LossArgs a) {
    using Tile = SplitTile<64, 128, WHOLE>;
    using Plain = LossTile<float, 64, 64, 2, 2, 2, false, SLOPE>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds > Plain::kLds ? Tile::kLds : Plain::kLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LossPlace p = loss_place<64, 128>(a);
    if (p.rows <= 0) return;
    f32x4 acc[Tile::MT][Tile::NT] = {};
    if (!Tile::run(acc, (int)a.K, lds, threadIdx.x, [&](int r) { return loss_row<float>(a, p, r); },
                   [&](int c) { return loss_word<float>(a, p, c); })) {
        for (int c = 0; c < 128; c += 64) {
            const LossPlace q{p.row0, p.n0 + c, 0, p.rows};
            __syncthreads();
            if (q.n0 < a.vc) Plain::run(a, q, q.n0 >> 6, lds, wave, lane);
            else if (!SLOPE)
                for (int r = threadIdx.x; r < p.rows; r += kRowSplitThreads)
                    a.partial[(p.row0 + r) * a.parts + (q.n0 >> 6)] = make_float2(-INFINITY, 0.f);
        }
        return;
    }
    auto get = [&](int i, int j) -> f32x4 & { return acc[i][j]; };
    auto row = [&](int i) { return Tile::m0(wave) + 16 * i + (lane & 15); };
    auto col = [&](int j) { return Tile::n0(wave) + 16 * j + (lane >> 4) * 4; };
    if constexpr (SLOPE) {
        loss_slope<float, Tile::MT, Tile::NT, 64, 128, kRowSplitThreads, false>(a, p, lds, lane, get, row, col);
    } else {
        loss_pairs<Tile::MT, Tile::NT, 2, 64, 128>(a, p, p.n0 >> 6, lds, wave % 2, lane, get, row, col);
        for (int r = threadIdx.x; r < p.rows; r += kRowSplitThreads)
            a.partial[(p.row0 + r) * a.parts + (p.n0 >> 6) + 1] = make_float2(-INFINITY, 0.f);
    }
}

// Many rows, 16-bit types: AH * 128 rows x 256 columns in phases.
template <typename T, int AH, bool SLOPE>
__global__ __launch_bounds__(kPhaseThreads) void loss_many(LossArgs a) {
    using Tile = PhaseTile<T, AH>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[kPhaseLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LossPlace p = loss_place<AH * kHalf, 2 * kHalf>(a);
    if (p.rows <= 0) return;
    f32x4 acc[2][2][4][2] = {};
    Tile::run(acc, p.rows, (int)a.K, lds, wave, lane, [&](int r) { return loss_row<T>(a, p, r); },
              [&](int c) { return loss_word<T>(a, p, c); });
    auto get = [&](int i, int j) -> f32x4 & { return acc[i >> 2][j >> 1][i & 3][j & 1]; };
    auto row = [&](int i) { return phase_row(i >> 2, i & 3, wave) + (lane & 15); };
    auto col = [&](int j) { return phase_col(j >> 1, j & 1, wave) + (lane >> 4) * 4; };
    if constexpr (SLOPE) loss_slope<T, 4 * AH, 4, AH * kHalf, 2 * kHalf, kPhaseThreads, true>(a, p, lds, lane, get, row, col);
    else loss_pairs<4 * AH, 4, 4, AH * kHalf, 2 * kHalf>(a, p, p.tile, lds, wave & 3, lane, get, row, col);
}

// Up to 16 rows: 64 columns per workgroup, the contraction split over its waves.
template <typename T, int NT, int NW, int STAGES, bool DIRECT, bool SLOPE>
__global__ __launch_bounds__(64 * NW) void loss_few(LossArgs a) {
    using Tile = FewTile<T, NT, NW, STAGES, DIRECT>;
    static_assert(NT == NW, "a wave per block of columns");
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LossPlace p = loss_place<16, 16 * NT>(a);
    if (p.rows <= 0) return;
    Tile::run((int)a.K, lds, wave, lane, [&](int r) { return loss_row<T>(a, p, r); },
              [&](int c) { return loss_word<T>(a, p, c); });
    f32x4 z = Tile::sum(lds, wave, lane);
    const int r = lane & 15, c = 16 * wave + (lane >> 4) * 4;
    if constexpr (SLOPE) {
        T *out = reinterpret_cast<T *>(a.slope) + p.row0 * a.ld;
        if (r < p.rows) store_quad<T>(out + r * a.ld, p.n0 + c, a.ld, loss_slopes(a, loss_row_of(a, p.row0 + r), z, p.n0 + c), true);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        loss_targets<16, 16 * NT, 64 * NW>(a, p, [&](int i, int j, float y) { out[i * a.ld + p.n0 + j] = (T)y; });
    } else {
        auto get = [&](int, int) -> f32x4 & { return z; };
        auto row = [&](int) { return r; };
        auto col = [&](int) { return c; };
        loss_pairs<1, 1, NW, 16, 16 * NT>(a, p, p.tile, lds + NW * NT * 1024, wave, lane, get, row, col);
    }
}

// Joins a row's pairs and forms its targets' logits, kDots at a time; WAVES waves
// per row.
constexpr int kDots = 4;
template <typename T>
__device__ __forceinline__ void loss_dots(float (&sum)[kDots], const char *x, const char *const (&w)[kDots], int K, int lane) {
#pragma unroll
    for (int d = 0; d < kDots; ++d) sum[d] = 0.f;
#pragma unroll 2
    for (int c = lane * kUnit<T>; c < K; c += 64 * kUnit<T>) {
        const u32x4 p = load_unit<T>((uint64_t)(x + (int64_t)c * sizeof(T)), K - c);
        u32x4 q[kDots];
#pragma unroll
        for (int d = 0; d < kDots; ++d) q[d] = load_unit<T>((uint64_t)(w[d] + (int64_t)c * sizeof(T)), w[d] ? K - c : 0);
#pragma unroll
        for (int d = 0; d < kDots; ++d)
#pragma unroll
            for (int e = 0; e < kUnit<T>; ++e) sum[d] = fmaf(element<T>(p, e), element<T>(q[d], e), sum[d]);
    }
#pragma unroll
    for (int d = 0; d < kDots; ++d) sum[d] = lanes_sum<64>(sum[d]);
}
template <typename T, int WAVES>
__global__ __launch_bounds__(256) void loss_join(LossArgs a) {
    __shared__ float s_part[4][5];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (4 / WAVES) + wave / WAVES;
    const int part = wave % WAVES;
    if (row >= a.N) return;
    // the pairs
    const float2 *pair = a.partial + row * a.parts;
    float m = -INFINITY, sum = 0.f;
#pragma unroll 4
    for (int64_t i = part * 64 + lane; i < a.parts; i += 64 * WAVES) m = fmaxf(m, pair[i].x);
    m = lanes_fold<64>(m, [](float p, float q) { return fmaxf(p, q); });
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 4
    for (int64_t i = part * 64 + lane; i < a.parts; i += 64 * WAVES) sum = fmaf(pair[i].y, exp2_fast(pair[i].x - base), sum);
    sum = lanes_sum<64>(sum);
    // the targets
    const int64_t *target = a.target + row * a.picks;
    const char *x = a.values + row * a.K * (int64_t)sizeof(T);
    float share = 0.f, at = 0.f;
    bool live = false;
    for (int64_t j0 = part; j0 < a.picks; j0 += kDots * WAVES) {
        const char *w[kDots];
        float prob[kDots], z[kDots];
#pragma unroll
        for (int d = 0; d < kDots; ++d) {
            const int64_t j = j0 + d * WAVES, t = j < a.picks ? target[j] : -1;
            const bool there = t >= 0 && t < a.V;
            w[d] = there ? a.weights + t * a.K * (int64_t)sizeof(T) : nullptr;
            prob[d] = !there ? 0.f : a.probs ? a.probs[row * a.picks + j] : 1.f;
            live = live || there;
        }
        if (a.picks == 1) {
            const char *one[kDots] = {w[0], nullptr, nullptr, nullptr};
            loss_dots<T>(z, x, one, (int)a.K, lane);
        } else {
            loss_dots<T>(z, x, w, (int)a.K, lane);
        }
#pragma unroll
        for (int d = 0; d < kDots; ++d) {
            const int64_t j = j0 + d * WAVES;
            const float y = w[d] ? a.scale * z[d] : 0.f;
            share += prob[d];
            if (w[d]) at = fmaf(prob[d], y, at);
            if (lane == 0 && j < a.picks) a.picked[row * a.picks + j] = y;
        }
    }
    if constexpr (WAVES > 1) {
        // the waves of the row in order
        if (lane == 0) {
            s_part[wave][0] = m;
            s_part[wave][1] = sum;
            s_part[wave][2] = share;
            s_part[wave][3] = at;
            s_part[wave][4] = live ? 1.f : 0.f;
        }
        __syncthreads();
        if (part > 0) return;
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < WAVES; ++q) top = fmaxf(top, s_part[wave + q][0]);
        const float low = top == -INFINITY ? 0.f : top;
        m = top;
        sum = share = at = 0.f;
        live = false;
#pragma unroll
        for (int q = 0; q < WAVES; ++q) {
            const float *o = s_part[wave + q];
            sum = fmaf(o[1], exp2_fast(o[0] - low), sum);
            share += o[2];
            at += o[3];
            live = live || o[4] != 0.f;
        }
    }
    if (lane == 0) {
        const float lse = kLn2 * (m + __log2f(sum));
        a.lse[row] = lse;
        // a row without a target has no loss, whatever its logits are
        a.loss[row] = live ? fmaf(share, lse, -at) : 0.f;
    }
}

// dz of a row's target `i` that has probability p in all.
__device__ __forceinline__ float loss_hit(const LossArgs &a, int64_t row, int64_t i, float p) {
    const float e = exp2_fast(fmaf(a.picked[i], kLog2e, -a.lse[row] * kLog2e));
    return fmaf(a.share[row], e, -a.hit[row] * p);
}

// What the gradient's tiles need of row `row`, from the LANES lanes it has (lane
// `l`): left in `share`, `hit`, `bound` and `live`.
template <int LANES>
__device__ __forceinline__ void loss_row_prepare(const LossArgs &a, int64_t row, int l) {
    float share = 0.f, size = 0.f, any = 0.f;
    for (int64_t j = l; j < a.picks; j += LANES) {
        const int64_t t = a.target[row * a.picks + j];
        if (t < 0 || t >= a.V) continue;
        const float p = a.probs ? a.probs[row * a.picks + j] : 1.f;
        share += p;
        size += fabsf(p);
        any = 1.f;
    }
    if constexpr (LANES > 1) {
        share = lanes_sum<LANES>(share);
        size = lanes_sum<LANES>(size);
        any = lanes_sum<LANES>(any);
    }
    if (l > 0) return;
    const bool live = any > 0.f;
    const float g = a.grad[row] * a.scale, bound = fabsf(g) * size;
    a.share[row] = live ? g * share : 0.f;
    a.hit[row] = g;
    a.bound[row] = bound < INFINITY ? bound : 0.f;
    a.live[row] = live ? row : -1;
    if constexpr (LANES == 1) a.hits[row] = live ? loss_hit(a, row, row, share) : 0.f;
}
// The one segment of the weights' sums.
__device__ __forceinline__ void loss_bounds(int64_t *offsets, int64_t n) {
    offsets[0] = 0;
    offsets[1] = n;
}
template <int LANES>
__global__ __launch_bounds__(256) void loss_rows_prepare(LossArgs a, int64_t *offsets) {
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
    if (row == 0) loss_bounds(offsets, a.N);
    if (row < a.N) loss_row_prepare<LANES>(a, row, threadIdx.x % LANES);  // whole groups of LANES
}
// dz of target i (of all rows) from the logits that the forward call kept; a target
// named twice in a row gets both shares.
__device__ __forceinline__ void loss_target_hit(const LossArgs &a, int64_t i) {
    const int64_t row = i / a.picks, t = a.target[i];
    const int64_t *target = a.target + row * a.picks;
    float sum = 0.f;
    if (t >= 0 && t < a.V) {
#pragma unroll 8
        for (int64_t j = 0; j < a.picks; ++j)
            sum += target[j] == t ? (a.probs ? a.probs[row * a.picks + j] : 1.f) : 0.f;
        sum = loss_hit(a, row, i, sum);
    }
    a.hits[i] = sum;
}
__global__ __launch_bounds__(256) void loss_hits(LossArgs a) {
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    if (i < a.N * a.picks) loss_target_hit(a, i);
}

// float16 holds 2^-24 to 2^16, so dz is brought near 2^13 by a power of two that
// all rows share (|dz| is at most twice its bound, so below 2^15), and the products take it out again:
// of the row with the largest bound, probabilities from 2^-37 on are kept, those
// from 2^-27 on with all bits.  By one workgroup.
constexpr int kOnce = 1024;
__device__ __forceinline__ void loss_scale(const LossArgs &a) {
    __shared__ float s[kOnce / 64];
    float m = 0.f;
    for (int64_t i = threadIdx.x; i < a.N; i += kOnce) m = fmaxf(m, a.bound[i]);
    m = lanes_fold<64>(m, [](float p, float q) { return fmaxf(p, q); });
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = m;
    __syncthreads();
    m = 0.f;
#pragma unroll
    for (int w = 0; w < kOnce / 64; ++w) m = fmaxf(m, s[w]);
    const int up = m > 0.f ? min(max(13 - ilogbf(m), -126), 126) : 0;
    const float f = ldexpf(1.f, up);
    for (int64_t i = threadIdx.x; i < a.N; i += kOnce) a.share[i] *= f;
    if (threadIdx.x == 0) {
        a.factor[0] = f;
        a.factor[1] = ldexpf(1.f, -up);
    }
}
__global__ __launch_bounds__(kOnce) void loss_factor(LossArgs a) { loss_scale(a); }

// All of these by one workgroup, for calls whose launches are what they take (15 rows
// of 4 targets, 144 columns, 876 entries, float16: the call 22 us, 29 with kernels of their
// own and dz turned; 5 rows of one 22.5 and 28; but 128 rows of 32 66 and 51, so rows of several
// only where each thread has one).
constexpr bool loss_once(int64_t n, int64_t picks) {
    return picks == 1 ? n <= 4 * kOnce : n <= kOnce / 16 && n * picks <= kOnce;
}
__global__ __launch_bounds__(kOnce) void loss_prepare_once(LossArgs a, int64_t *offsets) {
    if (threadIdx.x == 0) loss_bounds(offsets, a.N);
    if (a.picks == 1) {
        for (int64_t row = threadIdx.x; row < a.N; row += kOnce) loss_row_prepare<1>(a, row, 0);
    } else {
        for (int64_t row = threadIdx.x / 16; row < a.N; row += kOnce / 16) loss_row_prepare<16>(a, row, threadIdx.x % 16);
        __syncthreads();
        for (int64_t i = threadIdx.x; i < a.N * a.picks; i += kOnce) loss_target_hit(a, i);
    }
    __syncthreads();
    if (a.factor) loss_scale(a);
}

// dx += dz W of a piece: rows of dz in row form, rows of W across the
// contraction.  `cuts` workgroups share a tile's contraction, each with sums of its
// own.
struct LossBack {
    int64_t row0, n0, cut;
    int rows;
};
template <int BM, int BN>
__device__ __forceinline__ LossBack loss_back_place(const LossArgs &a) {
    const int64_t tiles = a.mtiles * a.ntiles, id = xcd_tile(tiles * a.cuts);
    if (id >= tiles * a.cuts) return {0, 0, 0, 0};
    const int64_t cut = id / tiles;
    const TilePlace at = tile_place(id - cut * tiles, a.mtiles, a.ntiles);
    return {at.m * BM, at.n * BN, cut, (int)min((int64_t)BM, a.N - at.m * BM)};
}
__device__ __forceinline__ void loss_add(const LossArgs &a, const LossBack &p, int r, int64_t n, f32x4 c) {
    if (r >= p.rows) return;
    float *row = a.sums + (p.cut * a.N + p.row0 + r) * a.KO;
    store_four<float>(row, n, a.KO, a.first ? c : load_four<float>(row, n, a.KO) + c);
}

template <typename T, int BM, int BN, int WM, int WN, bool DIRECT>
struct LossBackTile {
    static constexpr int kThreads = 64 * WM * WN, kStages = DIRECT ? 3 : 2;
    static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    using AStage = RowStage<T, BM, kThreads, DIRECT>;
    using BStage = ColStage<T, BN, kThreads, DIRECT>;
    static constexpr int kStageBytes = AStage::kBytes + BStage::kBytes, kLds = kStages * kStageBytes;

    static __device__ __forceinline__ void run(const LossArgs &a, const LossBack &p, int t0, int t1, lds_char *lds,
                                               int wave, int lane) {
        constexpr int kLoads = AStage::kLoads + BStage::kLoads;
        AStage sa;
        BStage sb;
        sa.init(wave, lane, (int)a.ld, [&](int r) -> const char * {
            return r < p.rows ? a.slope + (p.row0 + r) * a.ld * (int64_t)sizeof(T) : nullptr;
        });
        uint64_t wp[BStage::kLoads];
        int left[BStage::kLoads];
#pragma unroll
        for (int i = 0; i < BStage::kLoads; ++i) {
            const int64_t n = p.n0 + BStage::col(i, wave, lane);
            wp[i] = (uint64_t)(a.weights + ((a.v0 + BStage::row(i, wave, lane)) * a.K + n) * (int64_t)sizeof(T));
            left[i] = (int)(a.K - n);
        }
        auto issue = [&](int t, lds_char *buf) {
            const int k0 = t * kStep<T>;
            const uint64_t step = (uint64_t)k0 * a.K * sizeof(T);
            sa.issue(buf, wave, k0);
            sb.issue(
                buf + AStage::kBytes, wave, [&](int i) { return wp[i] + step; },
                [&](int i) { return k0 + BStage::row(i, wave, lane) < a.vc ? left[i] : 0; });
        };
        f32x4 acc[MT][NT] = {};
        const int m_w = wave / WN * (MT * 16), n_w = wave % WN * (NT * 16);
        auto products = [&](const lds_char *buf) {
            step_products<T, MT, NT, false, BM, true, BN>(acc, buf, buf + AStage::kBytes, m_w, n_w, lane);
        };
        if constexpr (DIRECT) {
#pragma unroll
            for (int t = 0; t < kStages - 1; ++t) issue(t0 + t, lds + t * kStageBytes);
            int cur = 0, fill = kStages - 1;
            for (int t = t0; t < t1; ++t) {
                wait_and_meet<(kStages - 2) * kLoads>();
                issue(t + kStages - 1, lds + fill * kStageBytes);
                products(lds + cur * kStageBytes);
                cur = cur + 1 == kStages ? 0 : cur + 1;
                fill = fill + 1 == kStages ? 0 : fill + 1;
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
            issue(t0, lds);
            sa.commit(lds, wave, lane);
            sb.commit(lds + AStage::kBytes, wave, lane);
            for (int t = t0; t < t1; ++t) {
                lds_char *next = lds + ((t + 1 - t0) & 1) * kStageBytes;
                __syncthreads();
                if (t + 1 < t1) issue(t + 1, next);
                products(lds + ((t - t0) & 1) * kStageBytes);
                if (t + 1 < t1) {
                    sa.commit(next, wave, lane);
                    sb.commit(next + AStage::kBytes, wave, lane);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                loss_add(a, p, m_w + 16 * i + (lane & 15), p.n0 + n_w + 16 * j + (lane >> 4) * 4, acc[i][j]);
    }
};
template <typename T, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN) void loss_back(LossArgs a) {
    using Tile = LossBackTile<T, BM, BN, WM, WN, DIRECT>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LossBack p = loss_back_place<BM, BN>(a);
    if (p.rows <= 0) return;
    const int64_t steps = (a.vc + kStep<T> - 1) / kStep<T>;
    Tile::run(a, p, (int)(p.cut * steps / a.cuts), (int)((p.cut + 1) * steps / a.cuts), (lds_char *)lds_mem, wave, lane);
}

// Float in bf16 parts, as above where a sum is not finite.
template <bool WHOLE>
__global__ __launch_bounds__(kRowSplitThreads, 3) void loss_back_split(LossArgs a) {
    constexpr int BM = 64, BN = 128, MT = 2, NT = 4;
    using Plain = LossBackTile<float, 64, 64, 2, 2, false>;
    using SA = SplitStage<BM, kRowSplitThreads, false, true>;  // rows of dz hold whole parts
    using SB = SplitStage<BN, kRowSplitThreads, true, WHOLE>;
    constexpr int kLds = SA::kLds + SB::kLds;
    __shared__ __attribute__((aligned(1024))) char lds_mem[kLds > Plain::kLds ? kLds : Plain::kLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const LossBack p = loss_back_place<BM, BN>(a);
    if (p.rows <= 0) return;
    const int64_t steps = (a.vc + kSplitK - 1) / kSplitK;
    const int64_t t0 = p.cut * steps / a.cuts, t1 = (p.cut + 1) * steps / a.cuts;
    SA sa;
    SB sb;
    uint64_t ap[SA::kParts], bp[SB::kParts];
    int aleft[SA::kParts], bleft[SB::kParts];
#pragma unroll
    for (int i = 0; i < SA::kParts; ++i) {
        const int r = SA::row(i, tid);
        ap[i] = (uint64_t)(a.slope + ((p.row0 + r) * a.ld + SA::at(i, tid)) * 4);
        aleft[i] = r < p.rows ? (int)a.ld - SA::at(i, tid) : 0;
    }
#pragma unroll
    for (int i = 0; i < SB::kParts; ++i) {
        const int64_t n = p.n0 + SB::at(i, tid);
        bp[i] = (uint64_t)(a.weights + ((a.v0 + SB::row(i, tid)) * a.K + n) * 4);
        bleft[i] = (int)(a.K - n);
    }
    f32x4 acc[MT][NT] = {};
    const int m_w = wave / 2 * (BM / 2), n_w = wave % 2 * (BN / 2);
    split_steps(
        t1 - t0,
        [&](int64_t t) {
            const int64_t k0 = (t0 + t) * kSplitK;
            sa.issue([&](int i) { return ap[i] + (uint64_t)k0 * 4; }, [&](int i) { return aleft[i] - (int)k0; });
            sb.issue([&](int i) { return bp[i] + (uint64_t)k0 * a.K * 4; },
                     [&](int i) { return k0 + SB::row(i, tid) < a.vc ? bleft[i] : 0; });
        },
        [&] {
            sa.commit(lds, tid);
            sb.commit(lds + SA::kLds, tid);
        },
        [&] { split_step<MT, NT, false, BM, true, BN>(acc, lds, lds + SA::kLds, m_w, n_w, lane); });
    if (__syncthreads_or(any_not_finite(acc))) {
        // in steps of the same length
        static_assert(kStep<float> == kSplitK, "cuts agree");
        for (int c = 0; c < BN && p.n0 + c < a.K; c += 64) {
            const LossBack q{p.row0, p.n0 + c, p.cut, p.rows};
            __syncthreads();
            Plain::run(a, q, (int)t0, (int)t1, lds, wave, lane);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            loss_add(a, p, m_w + 16 * i + (lane & 15), p.n0 + n_w + 16 * j + (lane >> 4) * 4, acc[i][j]);
}

// 128 rows x 256 columns in phases, 16-bit types.
template <typename T>
__global__ __launch_bounds__(kPhaseThreads) void loss_back_many(LossArgs a) {
    using AStage = RowStage<T, kHalf, kPhaseThreads, true>;
    using BStage = ColStage<T, kHalf, kPhaseThreads, true>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[kPhaseLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LossBack p = loss_back_place<kHalf, 2 * kHalf>(a);
    if (p.rows <= 0) return;
    const int64_t steps = (a.vc + kStep<T> - 1) / kStep<T>;
    const int t0 = (int)(p.cut * steps / a.cuts), t1 = (int)((p.cut + 1) * steps / a.cuts);
    AStage sa;
    sa.init(wave, lane, (int)a.ld, [&](int r) -> const char * {
        return r < p.rows ? a.slope + (p.row0 + r) * a.ld * (int64_t)sizeof(T) : nullptr;
    });
    BStage sb;
    uint64_t wp[2][BStage::kLoads];
    int left[2][BStage::kLoads];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < BStage::kLoads; ++i) {
            const int64_t n = p.n0 + h * kHalf + BStage::col(i, wave, lane);
            wp[h][i] = (uint64_t)(a.weights + ((a.v0 + BStage::row(i, wave, lane)) * a.K + n) * (int64_t)sizeof(T));
            left[h][i] = (int)(a.K - n);
        }
    f32x4 acc[2][2][4][2] = {};
    auto fetch_a = [&](int, int t, lds_char *place) { sa.issue(place, wave, (t0 + t) * kStep<T>); };
    auto fetch_b = [&](int h, int t, lds_char *place) {
        const int k0 = (t0 + t) * kStep<T>;
        const uint64_t step = (uint64_t)k0 * a.K * sizeof(T);
        sb.issue(
            place, wave, [&](int i) { return wp[h][i] + step; },
            [&](int i) { return k0 + BStage::row(i, wave, lane) < a.vc ? left[h][i] : 0; });
    };
    auto products = [](f32x4 (&c)[4][2], const u32x4 (&x)[2][4], const u32x4 (&y)[2][2]) { quadrant<T>(c, x, y); };
    phase_steps<T, 1, true>(acc, lds, t1 - t0, wave, lane, fetch_a, fetch_b, products);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                loss_add(a, p, phase_row(0, i, wave) + (lane & 15), p.n0 + phase_col(q, j, wave) + (lane >> 4) * 4,
                         acc[0][q][i][j]);
}

// The same from the piece's weights turned: both operands run along the
// contraction, AH * 128 x 256.
template <typename T, int AH>
__global__ __launch_bounds__(kPhaseThreads) void loss_back_turned(LossArgs a) {
    using Tile = PhaseTile<T, AH>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[kPhaseLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LossBack p = loss_back_place<AH * kHalf, 2 * kHalf>(a);
    if (p.rows <= 0) return;
    const int64_t steps = (a.vc + kStep<T> - 1) / kStep<T>, k0 = p.cut * steps / a.cuts * kStep<T>;
    const int64_t k1 = min((p.cut + 1) * steps / a.cuts * kStep<T>, a.ld);
    f32x4 acc[2][2][4][2] = {};
    Tile::run(
        acc, p.rows, (int)(k1 - k0), lds, wave, lane,
        [&](int r) -> const char * {
            return r < p.rows ? a.slope + ((p.row0 + r) * a.ld + k0) * (int64_t)sizeof(T) : nullptr;
        },
        [&](int c) -> const char * {
            return p.n0 + c < a.K ? a.words_turned + ((p.n0 + c) * a.ld + k0) * (int64_t)sizeof(T) : nullptr;
        });
#pragma unroll
    for (int h = 0; h < AH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    loss_add(a, p, phase_row(h, i, wave) + (lane & 15), p.n0 + phase_col(q, j, wave) + (lane >> 4) * 4,
                             acc[h][q][i][j]);
}

// dW of a piece from dz and the values, both turned.  BM: 256 (in phases) or less.
template <typename T, int BM, int BN, int THREADS, typename F>
__device__ __forceinline__ void loss_words_store(const LossArgs &a, char *out, int f32, int64_t m0, int64_t n0, int rows,
                                                 lds_char *lds, F quads) {
    const float f = a.factor ? a.factor[1] : 1.f;
    if (f32) {
        float *to = reinterpret_cast<float *>(out) + m0 * a.KO;
        quads([&](int r, int c, f32x4 y) {
            if (r < rows) store_four<float>(to + r * a.KO, n0 + c, a.KO, y * f);
        });
    } else {
        quads([&](int r, int c, f32x4 y) { tile_put<T, BN>(lds, r, c, y * f); });
        __syncthreads();
        tile_write<T, BM, BN, THREADS>(lds, reinterpret_cast<T *>(out) + m0 * a.KO, rows, n0, a.KO, a.KO);
    }
}
template <typename T, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(64 * WM * WN) void loss_words(LossArgs a, char *out, int f32) {
    using Tile = RowTile<T, BM, BN, WM, WN, STAGES, true>;
    static_assert(BM * BN * 2 <= Tile::kLds, "the results fit");
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = xcd_tile(a.mtiles * a.ntiles);
    if (id >= a.mtiles * a.ntiles) return;
    const TilePlace at = tile_place(id, a.mtiles, a.ntiles);
    const int64_t m0 = at.m * BM, n0 = at.n * BN;
    const int rows = (int)min((int64_t)BM, a.vc - m0);
    f32x4 acc[Tile::MT][Tile::NT] = {};
    Tile::run(
        acc, (int)a.ldn, lds, wave, lane,
        [&](int r) -> const char * { return r < rows ? a.turned + (m0 + r) * a.ldn * (int64_t)sizeof(T) : nullptr; },
        [&](int c) -> const char * {
            return n0 + c < a.K ? a.rows_turned + (n0 + c) * a.ldn * (int64_t)sizeof(T) : nullptr;
        });
    loss_words_store<T, BM, BN, Tile::kThreads>(a, out, f32, m0, n0, rows, lds, [&](auto put) {
#pragma unroll
        for (int i = 0; i < Tile::MT; ++i)
#pragma unroll
            for (int j = 0; j < Tile::NT; ++j)
                put(Tile::m0(wave) + 16 * i + (lane & 15), Tile::n0(wave) + 16 * j + (lane >> 4) * 4, acc[i][j]);
    });
}
template <typename T>
__global__ __launch_bounds__(kPhaseThreads) void loss_words_many(LossArgs a, char *out, int f32) {
    using Tile = PhaseTile<T, 2>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[kPhaseLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = xcd_tile(a.mtiles * a.ntiles);
    if (id >= a.mtiles * a.ntiles) return;
    const TilePlace at = tile_place(id, a.mtiles, a.ntiles);
    const int64_t m0 = at.m * 256, n0 = at.n * 256;
    const int rows = (int)min((int64_t)256, a.vc - m0);
    f32x4 acc[2][2][4][2] = {};
    Tile::run(
        acc, rows, (int)a.ldn, lds, wave, lane,
        [&](int r) -> const char * { return r < rows ? a.turned + (m0 + r) * a.ldn * (int64_t)sizeof(T) : nullptr; },
        [&](int c) -> const char * {
            return n0 + c < a.K ? a.rows_turned + (n0 + c) * a.ldn * (int64_t)sizeof(T) : nullptr;
        });
    loss_words_store<T, 256, 256, kPhaseThreads>(a, out, f32, m0, n0, rows, lds, [&](auto put) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        put(phase_row(h, i, wave) + (lane & 15), phase_col(q, j, wave) + (lane >> 4) * 4, acc[h][q][i][j]);
    });
}

// out[c][r] = in[r][c] for `rows` rows of `cols` (whole units), `ld` and `old`
// elements apart; rows that `live` leaves out and the columns up to `old` are zeros.
// (32,000 x 2,048: 58 us in tiles of 128 columns, 66 of 64; 4,096 x 2,048 in 11 and 8,
// with twice the workgroups.)
constexpr int kTurnRows = 128;
template <typename T, int kTurnCols>
__global__ __launch_bounds__(256) void loss_turn(const T *in, int64_t rows, int64_t cols, int64_t ld, const int64_t *live,
                                                 T *out, int64_t old) {
    __shared__ __attribute__((aligned(1024))) char lds_mem[kTurnRows * kTurnCols * 2];
    lds_char *lds = (lds_char *)lds_mem;
    const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, high = (old + kTurnRows - 1) / kTurnRows;
    const int64_t r0 = id % high * kTurnRows, c0 = id / high * kTurnCols;
    if (c0 >= cols) return;
#pragma unroll
    for (int i = threadIdx.x; i < kTurnRows * kTurnCols / 8; i += 256) {
        const int r = i / (kTurnCols / 8), u = i % (kTurnCols / 8);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (r0 + r < rows && c0 + u * 8 < cols && (!live || live[r0 + r] >= 0))
            v = *reinterpret_cast<const u32x4 *>(in + (r0 + r) * ld + c0 + u * 8);
        *reinterpret_cast<__attribute__((address_space(3))) u32x4 *>(lds + tile_unit<T, kTurnCols>(r, u)) = v;
    }
    __syncthreads();
    tile_turn<T, kTurnRows, kTurnCols, 256>(lds, threadIdx.x >> 6, threadIdx.x & 63);
    tile_write<T, kTurnCols, kTurnRows, 256>(lds, out + c0 * old, (int)min((int64_t)kTurnCols, cols - c0), r0, old, old);
}

// Copies `rows` rows of `cols` 16-bit elements, of any width and place, to rows of
// whole 16-byte units, zeros behind their end.
template <typename T>
__global__ __launch_bounds__(256) void loss_pad(const T *in, int64_t rows, int64_t cols, u32x4 *out) {
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x, units = (cols + 7) / 8;
    if (i >= rows * units) return;
    const int64_t r = i / units, u = i - r * units;
    out[i] = load_unit<T>((uint64_t)(in + r * cols + u * 8), (int)min(cols - u * 8, (int64_t)8));
}

// Four neighbouring sums of dx from element i on, zeros in rows without a target: their dz is
// zero, but a product with an infinite weight or a NaN is not.
__device__ __forceinline__ f32x4 loss_live(const LossArgs &a, int64_t i, f32x4 s) {
    int64_t r = a.N * a.KO <= UINT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)a.KO) : i / a.KO, left = (r + 1) * a.KO - i;
    bool live = a.live[r] >= 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (e == left) {
            if (++r >= a.N) break;
            left += a.KO;
            live = a.live[r] >= 0;
        }
        s[e] = live ? s[e] : 0.f;
    }
    return s;
}

// Adds the cuts' sums and rounds once: PARTS threads share four elements, each
// adds its part of the cuts in order, and these sums are added in order.  (8 rows of
// 2,048 from 32 cuts: 4.8 us by four threads, 10.5 by one; 4,096 rows of 1,024 from 4
// cuts 14 and 7.7.)
constexpr int kBackJoin = 256, kBackParts = 4, kBackCuts = 16;
template <typename T, int PARTS>
__global__ __launch_bounds__(kBackJoin) void loss_back_join(LossArgs a) {
    constexpr int kEach = kBackJoin / PARTS;
    __shared__ f32x4 s_part[PARTS > 1 ? PARTS - 1 : 1][kEach];
    const int part = threadIdx.x / kEach, at = threadIdx.x % kEach;
    const int64_t i = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kEach + at) * 4, all = a.N * a.KO;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    const int64_t c0 = part * a.cuts / PARTS, c1 = (part + 1) * a.cuts / PARTS;
    if (i < all)
#pragma unroll 8
        for (int64_t c = c0; c < c1; ++c) s += load_four<float>(a.sums + c * all, i, all);
    if constexpr (PARTS > 1) {
        if (part > 0) s_part[part - 1][at] = s;
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int q = 0; q < PARTS - 1; ++q) s += s_part[q][at];
    }
    if (i < all) store_four<T>(static_cast<T *>(a.grad_values), i, all, loss_live(a, i, s) * (a.factor ? a.factor[1] : 1.f));
}

// --------------------------------------------------------------------- host

// Rows up to 2^27: 16 lanes prepare one, and a launch has fewer than 2^32; the products
// over them count in 32 bits.
constexpr int64_t kLossFewRows = 16, kLossFewWords = 192 * 64, kLossRows = 1 << 27, kLossVocab = 1 << 30, kLossPicks = 4096;
// Kernels of the tiles.  Times in us of the forward call (bfloat16, the joining
// kernel's 6 to 10 among them):
//
//   rows, k, vocabulary       16   64  128  256  512 1024  4096     4096   2048    8192
//                             2048, 32,000                       1024, 5,000  512, 32,000
//   few                       33   69  121  229  445  783
//   64 x 64                   34   35   48   74  125  232   796       79    127     466
//   128 x 128                 42   42   43   50   82  143   538       56     84     311
//   128 x 256                 40   41   43   43   80  143   529       65     95     349
//   256 x 256                 42   43   45   54   64  114   432       66     75     279
//
// Up to 16 rows waves split the contraction, else the rule is the least of
// tile_time(), less 3 us a round for the largest tiles (rows are not gathered and
// need no search).
enum LossKind { kLossFew, kLossSmall, kLossMiddle, kLossOne, kLossTwo, kLossSplit, kLossFewAny, kLossAny };
LossKind loss_kind(int32_t dtype, int64_t n, int64_t k, int64_t v, bool direct) {
    if (dtype == SEGRED_F32) {
        // bf16 parts need tiles enough for every CU to be worth their splitting
        if (!direct) return kLossSplit;
        if (n <= kLossFewRows) return kLossFew;
        return n <= 64 || ((n + 63) / 64) * ((v + 127) / 128) < 224 ? kLossSmall : kLossSplit;
    }
    // (10 rows, k = 1,711, rows of no whole units: 7,143 entries 30 us against 44 in tiles of
    // 64 x 128; 8 rows, k = 2,047, 32,000 entries 69 and 62)
    if (!direct) return n <= kLossFewRows && v <= kLossFewWords ? kLossFewAny : kLossAny;
    if (n <= kLossFewRows) return kLossFew;
    constexpr LossKind kKinds[] = {kLossTwo, kLossOne, kLossMiddle, kLossSmall};
    auto time = [&](int i) {
        const TileCost &g = kTileCosts[i];
        return tile_time(g, i == 0 ? -3 : 0, k, (double)((n + g.rows - 1) / g.rows) * ((v + g.columns - 1) / g.columns), true);
    };
    int best = 0;
    for (int i = 1; i < 4; ++i)
        if (time(i) < time(best)) best = i;
    return kKinds[best];
}
// Columns that a pair covers.
int64_t loss_columns(LossKind kind) {
    return kind == kLossOne || kind == kLossTwo ? 256 : kind == kLossMiddle || kind == kLossAny ? 128 : 64;
}

template <typename T, bool SLOPE>
int loss_tiles_launch(LossArgs a, LossKind kind, hipStream_t st) {
    const int64_t bm = kind == kLossTwo ? 256 : kind == kLossOne || kind == kLossMiddle ? 128 : kind == kLossFew || kind == kLossFewAny ? 16 : sizeof(T) == 4 && kind == kLossSmall ? 32 : 64;
    const int64_t bn = kind == kLossSplit ? 128 : loss_columns(kind);
    a.mtiles = (a.N + bm - 1) / bm;
    a.ntiles = (a.vc + bn - 1) / bn;
    dim3 grid;
    if (!tile_grid(a.mtiles * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    if constexpr (sizeof(T) == 4) {
        if (kind == kLossFew) timed_launch_ggl(true, (loss_few<T, 4, 4, 3, true, SLOPE>), grid, dim3(256), 0, st, a);
        else if (kind == kLossSmall) timed_launch_ggl(true, (loss_tiles<T, 32, 64, 1, 4, 4, true, SLOPE>), grid, dim3(256), 0, st, a);
        else if (a.K % 8 == 0) timed_launch_ggl(true, (loss_split<true, SLOPE>), grid, dim3(kRowSplitThreads), 0, st, a);
        else timed_launch_ggl(true, (loss_split<false, SLOPE>), grid, dim3(kRowSplitThreads), 0, st, a);
    } else {
        switch (kind) {
        case kLossFew: timed_launch_ggl(true, (loss_few<T, 4, 4, 3, true, SLOPE>), grid, dim3(256), 0, st, a); break;
        case kLossFewAny: timed_launch_ggl(true, (loss_few<T, 4, 4, 3, false, SLOPE>), grid, dim3(256), 0, st, a); break;
        case kLossSmall:
            timed_launch_ggl(true, (loss_tiles<T, 64, 64, 2, 2, 3, true, SLOPE>), grid, dim3(256), 0, st, a);
            break;
        case kLossMiddle:
            timed_launch_ggl(true, (loss_tiles<T, 128, 128, 2, 4, 2, true, SLOPE>), grid, dim3(512), 0, st, a);
            break;
        case kLossOne: timed_launch_ggl(true, (loss_many<T, 1, SLOPE>), grid, dim3(kPhaseThreads), 0, st, a); break;
        case kLossTwo: timed_launch_ggl(true, (loss_many<T, 2, SLOPE>), grid, dim3(kPhaseThreads), 0, st, a); break;
        default: timed_launch_ggl(true, (loss_tiles<T, 64, 128, 2, 2, 2, false, SLOPE>), grid, dim3(256), 0, st, a); break;
        }
    }
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

int64_t loss_parts(LossKind kind, int64_t v) {
    const int64_t c = loss_columns(kind);
    // in pairs of 64 columns of 128
    return kind == kLossSplit ? (v + 127) / 128 * 2 : (v + c - 1) / c;
}

// What both calls ask of the arguments that they share.
int loss_check(const void *values, int32_t dtype, int64_t k, int64_t rows, const void *weights, int64_t vocab,
               const int64_t *target, const float *probs, int64_t picks, float scale, const void *workspace) {
    const int64_t e = float_size(dtype);
    if (dtype < SEGRED_U32 || dtype > SEGRED_F16 || k < 1 || rows < 0 || vocab < 1 || picks < 1)
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (!(scale > 0.f) || std::isinf(scale)) return SEGRED_ERR_INVALID_ARGUMENT;
    if (!weights || (rows > 0 && (!values || !target))) return SEGRED_ERR_INVALID_ARGUMENT;
    if (e == 0 || k > kMaxWidth || vocab > kLossVocab || picks > kLossPicks || rows > kLossRows)
        return SEGRED_ERR_UNSUPPORTED;
    if (!aligned(values, e) || !aligned(weights, e) || !aligned(target, 8) || !aligned(probs, 4) || !aligned(workspace, 16))
        return SEGRED_ERR_INVALID_ARGUMENT;
    return SEGRED_OK;
}

bool loss_direct(const void *values, const void *weights, int32_t dtype, int64_t k) {
    return (k * float_size(dtype)) % 16 == 0 && aligned(values, 16) && aligned(weights, 16);
}

LossArgs loss_args(const void *values, int64_t k, int64_t rows, const void *weights, int64_t vocab,
                   const int64_t *target, const float *probs, int64_t picks, float scale) {
    LossArgs a{};
    a.values = static_cast<const char *>(values);
    a.weights = static_cast<const char *>(weights);
    a.target = target;
    a.probs = probs;
    a.N = rows;
    a.V = a.vc = vocab;
    a.K = a.KO = k;
    a.picks = picks;
    a.scale = scale;
    a.bend = scale * kLog2e;
    return a;
}

// 16-bit rows that are not whole 16-byte units are copied to rows that are, the
// weights a piece at a time: read as they are, through registers, they made the
// kernels several times slower (4,096 rows, 32,000 entries, bfloat16: k = 2,047 took
// 1,156 us forward and 5,787 back, 2,048 472 and 1,445).  Few rows go as they are
// in the forward call (1 row: 65 us against 33 and 65 for the copy).
//
// A piece: 256 MiB of dz, and 4,096 entries at least.  The gradient call in us:
//
//   MiB                                       32    64   128   256   512
//   bfloat16  4,096 x 2,048, 65,536         3416  2998  2926  2872  2829
//   bfloat16 16,384 x 1,024, 32,000         4298  4296  4292  3341  3014
//   float16   1,500 x 1,024, 32,011, 32      445   427   389   389   389
//   bfloat16  2,166 x 88, 54,570, 16         447   367   287   225   224
//   float32   4,096 x 1,024, 32,000         5062  5056  4896  4850  4945
//   entries at least                         256  1024  2048  4096  8192
//   bfloat16 65,536 x 512, 16,000           6574  6565  6567  5184  4706
//   float32  32,768 x 256, 16,000           5685  5759  5742  5650  5920
//
// (equal times on the left: a piece has the least 4,096 entries already, or, below, the 2,048
// that 256 MiB hold).  Twice the memory
// would gain 0 to 10 %; dz may have a turned copy beside it, so a call holds up to two pieces.
constexpr int64_t kPieceBytes = int64_t(256) << 20, kPieceLeast = 4096, kPadRows = 256;
bool loss_padded(int32_t dtype, int64_t k) { return dtype != SEGRED_F32 && k % 8 != 0; }
template <typename T>
int loss_pad_launch(const void *in, int64_t rows, int64_t cols, void *out, hipStream_t st) {
    dim3 grid;
    if (!tile_grid((rows * ((cols + 7) / 8) + 255) / 256, grid)) return SEGRED_ERR_UNSUPPORTED;
    timed_launch_ggl(false, (loss_pad<T>), grid, dim3(256), 0, st, static_cast<const T *>(in), rows, cols,
                     static_cast<u32x4 *>(out));
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

// The forward call's working memory: the pairs, and the copies.
struct LossRoom {
    bool pad;
    int64_t wide, piece;  // columns of a copy, rows of one of the weights
    int64_t values, words, bytes;  // places
};
LossRoom loss_room(int32_t dtype, int64_t k, int64_t n, int64_t v) {
    LossRoom r{};
    r.pad = loss_padded(dtype, k) && n >= kPadRows;
    r.wide = (k + 7) / 8 * 8;
    r.piece = std::min(v, std::max(kPieceLeast, kPieceBytes / (r.wide * 2) / 256 * 256));
    // the smallest pairs, whatever kernel is taken
    const int64_t pairs = n * ((v + 127) / 128 * 2) * 8;
    r.values = (pairs + 255) / 256 * 256;
    r.words = r.values + n * r.wide * 2;
    r.bytes = r.pad ? r.words + r.piece * r.wide * 2 : pairs;
    return r;
}

template <typename T>
int loss_forward(const LossArgs &a, LossKind kind, const LossRoom &room, hipStream_t st) {
    int rc = SEGRED_OK;
    char *work = reinterpret_cast<char *>(a.partial);
    if (!room.pad) {
        rc = loss_tiles_launch<T, false>(a, kind, st);
    } else if constexpr (sizeof(T) == 2) {
        rc = loss_pad_launch<T>(a.values, a.N, a.K, work + room.values, st);
        LossArgs b = a;
        b.values = work + room.values;
        b.K = room.wide;
        for (; b.v0 < a.V && rc == SEGRED_OK; b.v0 += room.piece) {
            b.vc = std::min(room.piece, a.V - b.v0);
            rc = loss_pad_launch<T>(a.weights + b.v0 * a.K * 2, b.vc, a.K, work + room.words, st);
            b.weights = work + room.words - b.v0 * b.K * 2;
            b.partial = a.partial + b.v0 / loss_columns(kind);
            if (rc == SEGRED_OK) rc = loss_tiles_launch<T, false>(b, kind, st);
        }
    }
    if (rc != SEGRED_OK) return rc;
    dim3 grid;
    const bool shared = a.picks > 1 || a.N <= 1024;  // four waves a row
    if (!tile_grid(shared ? a.N : (a.N + 3) / 4, grid)) return SEGRED_ERR_UNSUPPORTED;
    if (shared) timed_launch_ggl(false, (loss_join<T, 4>), grid, dim3(256), 0, st, a);
    else timed_launch_ggl(false, (loss_join<T, 1>), grid, dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

// The gradient's pieces and its working memory.
//
// Products whose operands both run along the contraction are the fastest (bfloat16,
// 4,096 rows, 2,048 columns, 32,768 entries: 410 us against 580 and 673 with one or
// both across it), so operands are turned where that is less than it saves: dz
// as the tiles write it, the values once, the weights a piece at a time.
struct LossPlan {
    int64_t piece, cuts;  // columns of a piece; workgroups that share a tile of dx
    int64_t wide;         // columns of the copies
    bool pad;             // the operands are copied to whole units
    bool many;            // dx in tiles of 128 x 256
    bool turn_rows, turn_words;  // dW from dz and the values turned; dx from the weights turned
    // places in the working memory
    int64_t slope, turned, rows_turned, words_turned, values, words, sums, share, hit, bound, live, hits, offsets, factor, outer, bytes;
};
constexpr int64_t kTurnWords = 12 << 20;
LossPlan loss_plan(int32_t dtype, int64_t columns, int64_t n, int64_t v, int64_t picks) {
    const int64_t e = float_size(dtype);
    LossPlan p{};
    p.pad = loss_padded(dtype, columns);
    const int64_t k = p.pad ? (columns + 7) / 8 * 8 : columns;
    p.wide = k;
    p.piece = std::min(v, std::max(kPieceLeast, kPieceBytes / (std::max<int64_t>(n, 1) * e) / 256 * 256));
    // pieces of about the same size
    const int64_t pieces = (v + p.piece - 1) / p.piece;
    p.piece = std::min(v, ((v + pieces - 1) / pieces + 255) / 256 * 256);
    p.many = e == 2 && n > 64 && k > 128;
    const bool whole = e == 2 && k % 8 == 0 && n > 0;
    // (16 / 64 / 256 rows, 512 columns, 4,000 entries: the call 28 / 30 / 42 us with dz and
    // values turned, 22 / 27 / 39 without; 8 x 1,024 x 32,000 65 and 70, 64 x 2,048 x 16,000 68
    // and 75; 1,024 x 512 x 4,000 55 and 64)
    p.turn_rows = whole && (p.pad || (n <= 256 ? k >= 128 && k * v >= kTurnWords : k >= 512 || (n <= 512 && k >= 128)));
    // (32,000 entries, bfloat16, the call without / with the weights turned:
    //   rows    512        1,024      1,500      2,048      3,000        4,096
    //   k 512   100 / 122  158 / 181  221 / 254  283 / 310  417 / 429    528 / 516
    //   1,024   156 / 188  253 / 284  353 / 381  451 / 459  709 / 665    833 / 806
    //   2,048   253 / 313  427 / 459  661 / 623  787 / 772  1281 / 1176  1499 / 1418
    // so 1,500 x 2,048 and 3,000 x 1,024 would be 6 % faster on the other side)
    p.turn_words = whole && n >= 2048 && ((n + 255) / 256) * ((k + 255) / 256) >= 64;
    const int64_t tiles = p.turn_words ? ((n + 255) / 256) * ((k + 255) / 256)
                          : p.many     ? ((n + 127) / 128) * ((k + 255) / 256)
                                       : (n <= 16 && e == 2 ? 1 : (n + 63) / 64) * ((k + 127) / 128);
    const int64_t room = p.many ? 256 : 512, steps = (p.piece + 63) / 64;
    p.cuts = std::max<int64_t>(1, std::min({room / std::max<int64_t>(tiles, 1), steps / 8, (int64_t)64}));
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const int64_t ld = (p.piece + 7) / 8 * 8, ldn = (n + 7) / 8 * 8;
    p.slope = take(n * ld * e);
    p.turned = take(p.turn_rows ? p.piece * ldn * e : 0);
    p.rows_turned = take(p.turn_rows ? k * ldn * e : 0);
    p.words_turned = take(p.turn_words ? k * ld * e : 0);
    p.values = take(p.pad ? n * k * e : 0);
    p.words = take(p.pad ? p.piece * k * e : 0);
    p.sums = take(p.cuts * n * columns * 4);
    p.share = take(n * 4);
    p.hit = take(n * 4);
    p.bound = take(n * 4);
    p.live = take(n * 8);
    p.hits = take(n * picks * 4);
    p.offsets = take(16);
    p.factor = take(8);
    // the last piece is no wider than the others, but may be cut otherwise
    const int64_t last = v - (pieces - 1) * p.piece;
    p.outer = take(std::max(segred_outer_workspace(p.piece, k, 1, n), last > 0 ? segred_outer_workspace(last, k, 1, n) : 0));
    p.bytes = at;
    return p;
}

template <typename T>
int loss_turn_launch(const void *in, int64_t rows, int64_t cols, int64_t ld, const int64_t *live, void *out, int64_t old,
                     hipStream_t st) {
    const int64_t high = (old + kTurnRows - 1) / kTurnRows;
    const bool wide = high * ((cols + 127) / 128) >= 1024;
    dim3 grid;
    if (!tile_grid(high * (wide ? (cols + 127) / 128 : (cols + 63) / 64), grid)) return SEGRED_ERR_UNSUPPORTED;
    if (wide)
        timed_launch_ggl(false, (loss_turn<T, 128>), grid, dim3(256), 0, st, static_cast<const T *>(in), rows, cols, ld, live,
                         static_cast<T *>(out), old);
    else
        timed_launch_ggl(false, (loss_turn<T, 64>), grid, dim3(256), 0, st, static_cast<const T *>(in), rows, cols, ld, live,
                         static_cast<T *>(out), old);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

// dx += dz W of a piece.
template <typename T>
int loss_back_launch(LossArgs a, const LossPlan &p, bool direct, hipStream_t st) {
    const int64_t e = sizeof(T);
    const bool turned = p.turn_words && direct;
    const int64_t bm = turned ? 256 : p.many ? 128 : a.N <= 16 && e == 2 ? 16 : 64, bn = p.many && direct ? 256 : 128;
    a.mtiles = (a.N + bm - 1) / bm;
    a.ntiles = (a.K + bn - 1) / bn;
    dim3 grid;
    if (!tile_grid(a.mtiles * a.ntiles * a.cuts, grid)) return SEGRED_ERR_UNSUPPORTED;
    if constexpr (sizeof(T) == 4) {
        if (a.K % 8 == 0) timed_launch_ggl(true, (loss_back_split<true>), grid, dim3(kRowSplitThreads), 0, st, a);
        else timed_launch_ggl(true, (loss_back_split<false>), grid, dim3(kRowSplitThreads), 0, st, a);
    } else if (turned) {
        const int rc = loss_turn_launch<T>(a.weights + a.v0 * a.K * e, a.vc, a.K, a.K, nullptr,
                                           const_cast<char *>(a.words_turned), a.ld, st);
        if (rc != SEGRED_OK) return rc;
        timed_launch_ggl(true, (loss_back_turned<T, 2>), grid, dim3(kPhaseThreads), 0, st, a);
    } else if (p.many && direct) {
        timed_launch_ggl(true, (loss_back_many<T>), grid, dim3(kPhaseThreads), 0, st, a);
    } else if (p.many) {
        timed_launch_ggl(true, (loss_back<T, 128, 128, 2, 2, false>), grid, dim3(256), 0, st, a);
    } else if (bm == 16) {
        if (direct) timed_launch_ggl(true, (loss_back<T, 16, 128, 1, 4, true>), grid, dim3(256), 0, st, a);
        else timed_launch_ggl(true, (loss_back<T, 16, 128, 1, 4, false>), grid, dim3(256), 0, st, a);
    } else {
        if (direct) timed_launch_ggl(true, (loss_back<T, 64, 128, 2, 2, true>), grid, dim3(256), 0, st, a);
        else timed_launch_ggl(true, (loss_back<T, 64, 128, 2, 2, false>), grid, dim3(256), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

// dW of a piece; `later`: dz is still to be turned.
template <typename T>
int loss_words_launch(LossArgs a, bool later, char *to, int f32, hipStream_t st) {
    if (later) {
        const int rc = loss_turn_launch<T>(a.slope, a.N, a.vc, a.ld, nullptr, a.turned, a.ldn, st);
        if (rc != SEGRED_OK) return rc;
    }
    // few rows are a short contraction: then the small tiles store while others load
    int best = 0;
    auto time = [&](int i) {
        const TileCost &g = kTileCosts[i];
        const int64_t tiles = ((a.vc + g.rows - 1) / g.rows) * ((a.K + g.columns - 1) / g.columns);
        return tile_time(g, i == 0 ? -3 : 0, a.N, (double)tiles, true);
    };
    for (int i : {2, 3})
        if (time(i) < time(best)) best = i;
    a.mtiles = (a.vc + kTileCosts[best].rows - 1) / kTileCosts[best].rows;
    a.ntiles = (a.K + kTileCosts[best].columns - 1) / kTileCosts[best].columns;
    dim3 grid;
    if (!tile_grid(a.mtiles * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    if (best == 0) timed_launch_ggl(true, (loss_words_many<T>), grid, dim3(kPhaseThreads), 0, st, a, to, f32);
    else if (best == 2) timed_launch_ggl(true, (loss_words<T, 128, 128, 2, 4, 2>), grid, dim3(512), 0, st, a, to, f32);
    else timed_launch_ggl(true, (loss_words<T, 64, 64, 2, 2, 3>), grid, dim3(256), 0, st, a, to, f32);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

template <typename T>
int loss_backward(LossArgs a, const LossPlan &p, LossKind kind, bool direct, int32_t dtype, void *grad_weights,
                  int32_t grad_weights_dtype, char *work, hipStream_t st) {
    const int64_t ge = float_size(grad_weights_dtype);
    int64_t *offsets = reinterpret_cast<int64_t *>(work + p.offsets);
    const bool turn_rows = p.turn_rows && direct && grad_weights;
    a.ldn = (a.N + 7) / 8 * 8;
    a.turned = turn_rows ? work + p.turned : nullptr;
    a.rows_turned = work + p.rows_turned;
    a.words_turned = work + p.words_turned;
    const bool several = a.picks > 1;
    if (loss_once(a.N, a.picks) && (several || a.factor || a.N == 0)) {
        timed_launch_ggl(false, loss_prepare_once, dim3(1), dim3(kOnce), 0, st, a, offsets);
    } else {
        if (several) {
            dim3 grid;
            if (!tile_grid((a.N * a.picks + 255) / 256, grid)) return SEGRED_ERR_UNSUPPORTED;
            timed_launch_ggl(false, (loss_rows_prepare<16>), dim3((unsigned)((a.N + 15) / 16)), dim3(256), 0, st, a, offsets);
            timed_launch_ggl(false, loss_hits, grid, dim3(256), 0, st, a);
        } else {
            timed_launch_ggl(false, (loss_rows_prepare<1>), dim3((unsigned)((a.N + 255) / 256)), dim3(256), 0, st, a, offsets);
        }
        if (a.factor) timed_launch_ggl(false, loss_factor, dim3(1), dim3(kOnce), 0, st, a);
    }
    if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    int rc = SEGRED_OK;
    const char *const weights = a.weights;
    if constexpr (sizeof(T) == 2) {
        if (p.pad) {
            if (a.N > 0) rc = loss_pad_launch<T>(a.values, a.N, a.K, work + p.values, st);
            if (rc != SEGRED_OK) return rc;
            a.values = work + p.values;
            a.K = p.wide;
        }
    }
    if constexpr (sizeof(T) == 2)
        if (turn_rows) rc = loss_turn_launch<T>(a.values, a.N, a.K, a.K, a.live, work + p.rows_turned, a.ldn, st);
    for (a.v0 = 0; a.v0 < a.V && rc == SEGRED_OK; a.v0 += p.piece) {
        a.vc = std::min(p.piece, a.V - a.v0);
        a.ld = (a.vc + 7) / 8 * 8;
        a.first = a.v0 == 0;
        if constexpr (sizeof(T) == 2)
            if (p.pad && a.N > 0) {
                rc = loss_pad_launch<T>(weights + a.v0 * a.KO * 2, a.vc, a.KO, work + p.words, st);
                if (rc != SEGRED_OK) return rc;
                a.weights = work + p.words - a.v0 * a.K * 2;
            }
        if (a.N > 0) rc = loss_tiles_launch<T, true>(a, kind, st);
        if (rc == SEGRED_OK && a.grad_values && a.N > 0) rc = loss_back_launch<T>(a, p, direct, st);
        if (rc != SEGRED_OK || !grad_weights) continue;
        char *to = static_cast<char *>(grad_weights) + a.v0 * a.KO * ge;
        if constexpr (sizeof(T) == 2) {
            if (turn_rows) {
                rc = loss_words_launch<T>(a, kind == kLossFew || kind == kLossFewAny, to, ge == 4 ? 1 : 0, st);
                continue;
            }
        }
        rc = outer_scaled(a.slope, a.ld, a.vc, a.values, a.live, a.N, a.KO, dtype, offsets, to, grad_weights_dtype,
                          a.factor ? a.factor + 1 : nullptr, work + p.outer, st);
    }
    if (rc != SEGRED_OK) return rc;
    if (a.grad_values && a.N > 0) {
        dim3 grid;
        const bool shared = p.cuts >= kBackCuts;
        const int64_t each = 4 * kBackJoin / (shared ? kBackParts : 1);
        if (!tile_grid((a.N * a.KO + each - 1) / each, grid)) return SEGRED_ERR_UNSUPPORTED;
        if (shared) timed_launch_ggl(false, (loss_back_join<T, kBackParts>), grid, dim3(kBackJoin), 0, st, a);
        else timed_launch_ggl(false, (loss_back_join<T, 1>), grid, dim3(kBackJoin), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

}  // namespace segred

using namespace segred;

extern "C" int64_t segred_cross_entropy_workspace(int32_t dtype, int64_t k, int64_t rows, int64_t vocab) {
    if (float_size(dtype) == 0 || k < 1 || k > kMaxWidth || rows < 1 || rows > kLossRows || vocab < 1 || vocab > kLossVocab)
        return 0;
    return loss_room(dtype, k, rows, vocab).bytes;
}

extern "C" int segred_cross_entropy(const void *values, int32_t dtype, int64_t k, int64_t rows, const void *weights,
                                    int64_t vocab, const int64_t *target, const float *probs, int64_t picks,
                                    float scale, float *loss, float *lse, float *picked, void *workspace,
                                    int64_t workspace_bytes, hipStream_t stream) {
    const int rc = loss_check(values, dtype, k, rows, weights, vocab, target, probs, picks, scale, workspace);
    if (rc != SEGRED_OK) return rc;
    if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(picked, 4)) return SEGRED_ERR_INVALID_ARGUMENT;
    if (rows == 0) return SEGRED_OK;
    if (!loss || !lse || !picked || !workspace ||
        workspace_bytes < segred_cross_entropy_workspace(dtype, k, rows, vocab))
        return SEGRED_ERR_INVALID_ARGUMENT;
    LossArgs a = loss_args(values, k, rows, weights, vocab, target, probs, picks, scale);
    const LossRoom room = loss_room(dtype, k, rows, vocab);
    const LossKind kind = room.pad ? loss_kind(dtype, rows, room.wide, room.piece, true)
                                   : loss_kind(dtype, rows, k, vocab, loss_direct(values, weights, dtype, k));
    a.partial = static_cast<float2 *>(workspace);
    a.parts = loss_parts(kind, vocab);
    a.loss = loss;
    a.lse = lse;
    a.picked = picked;
    switch (dtype) {
    case SEGRED_BF16: return loss_forward<__bf16>(a, kind, room, stream);
    case SEGRED_F16: return loss_forward<_Float16>(a, kind, room, stream);
    default: return loss_forward<float>(a, kind, room, stream);
    }
}

extern "C" int64_t segred_cross_entropy_grad_workspace(int32_t dtype, int64_t k, int64_t rows, int64_t vocab,
                                                       int64_t picks) {
    if (float_size(dtype) == 0 || k < 1 || k > kMaxWidth || rows < 0 || rows > kLossRows || vocab < 1 ||
        vocab > kLossVocab || picks < 1 || picks > kLossPicks)
        return 0;
    return loss_plan(dtype, k, rows, vocab, picks).bytes;
}

extern "C" int segred_cross_entropy_grad(const float *grad, const void *values, int32_t dtype, int64_t k, int64_t rows,
                                         const void *weights, int64_t vocab, const int64_t *target,
                                         const float *probs, int64_t picks, float scale, const float *lse,
                                         const float *picked, void *grad_values, void *grad_weights,
                                         int32_t grad_weights_dtype, void *workspace, int64_t workspace_bytes,
                                         hipStream_t stream) {
    const int rc = loss_check(values, dtype, k, rows, weights, vocab, target, probs, picks, scale, workspace);
    if (rc != SEGRED_OK) return rc;
    const int64_t e = float_size(dtype);
    if (grad_weights_dtype != dtype && grad_weights_dtype != SEGRED_F32) return SEGRED_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!grad || !lse || !picked)) return SEGRED_ERR_INVALID_ARGUMENT;
    if (!aligned(grad, 4) || !aligned(lse, 4) || !aligned(picked, 4) || !aligned(grad_values, e) ||
        !aligned(grad_weights, float_size(grad_weights_dtype)))
        return SEGRED_ERR_INVALID_ARGUMENT;
    const LossPlan p = loss_plan(dtype, k, rows, vocab, picks);
    if (!workspace || workspace_bytes < p.bytes) return SEGRED_ERR_INVALID_ARGUMENT;
    LossArgs a = loss_args(values, k, rows, weights, vocab, target, probs, picks, scale);
    char *work = static_cast<char *>(workspace);
    a.grad = grad;
    a.lse = const_cast<float *>(lse);
    a.picked = const_cast<float *>(picked);
    a.grad_values = grad_values;
    a.slope = work + p.slope;
    a.sums = reinterpret_cast<float *>(work + p.sums);
    a.share = reinterpret_cast<float *>(work + p.share);
    a.hit = reinterpret_cast<float *>(work + p.hit);
    a.bound = reinterpret_cast<float *>(work + p.bound);
    a.live = reinterpret_cast<int64_t *>(work + p.live);
    a.hits = reinterpret_cast<float *>(work + p.hits);
    a.factor = dtype == SEGRED_F16 && rows > 0 ? reinterpret_cast<float *>(work + p.factor) : nullptr;
    a.cuts = p.cuts;
    const bool direct = p.pad || loss_direct(values, weights, dtype, k);
    const LossKind kind = loss_kind(dtype, rows, p.wide, p.piece, direct);
    switch (dtype) {
    case SEGRED_BF16: return loss_backward<__bf16>(a, p, kind, direct, dtype, grad_weights, grad_weights_dtype, work, stream);
    case SEGRED_F16: return loss_backward<_Float16>(a, p, kind, direct, dtype, grad_weights, grad_weights_dtype, work, stream);
    default: return loss_backward<float>(a, p, kind, direct, dtype, grad_weights, grad_weights_dtype, work, stream);
    }
}
