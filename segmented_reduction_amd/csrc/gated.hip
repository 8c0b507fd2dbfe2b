// gated.hip -- the gated pair of projections of each segment's rows and its
// gradient: with g = x G[s]^T and u = x U[s]^T, G[s] and U[s] the first and the
// last m rows of weights[s],
//   out  = act(g) u
//   grad = (d u act'(g), d act(g)) from d, the gradient of out: the gradient of the
//          pair (g, u), [., 2 m], whose products with the weights and the rows are
//          segred_matmul's and segred_outer's.
// One kernel forms both projections side by side: of a tile's columns one half are
// rows of G and the other the same rows of U, so that a lane holds g and u of the
// same outputs and neither goes to memory.  The gradient forms them again: kept in
// float32 they would take 16 bytes an output to write and read, against 4 k
// operations to form them again (8,192 rows, 1,024 -> 2 x 2,560: 336 MB, 65 us at the
// rate of a copy, against 90).
// Few rows per segment are bound by the weights (64 rows over 64 segments, 2,048 x
// 1,024: 5 TB/s), many by the matrix units (64 segments of 512 rows on average: 312 to 321 us,
// 855 to 880 TFLOP/s; one segment of 8,192, 4,096 x 4,096: 1,340; float32, 8 segments of 1,024
// rows, 1,024 -> 2 x 2,560: 505 us and the gradient 544, 170 and 158 by bf16 parts).
#include <algorithm>

#include "internal.hpp"
#include "rowtile.hpp"

namespace segred {

struct GatedArgs {
    const char *values;
    const int64_t *rows;  // row of `values` behind each row, or null
    int64_t value_rows;
    const char *weights;  // [S, 2 M, K]
    const int64_t *offsets;
    int64_t S, N, K, M;
    int64_t slots, ntiles;
    const char *grad;  // [N, M], the gradient call's
    void *out;         // [N, M], or [N, 2 M]
    float c1, c2;      // act(x) = x / (1 + exp(-x (c1 + c2 x^2))) where it is neither of the others
    int relu;
};

// An activation and its slope.  ERF: x Phi(x), Phi of the normal distribution.  Phi(-z) =
// exp(-z^2 / 2) R(z), and R(z) = t P(t) with t = 1 / (1 + 0.34375 z): R falls as 1 / z, so P
// is smooth up to t = 0, and a polynomial of degree 8 (least relative error over z = 0 .. 15)
// is off by 2.9e-8 of R.  So Phi keeps its relative accuracy where it is small: R to 6 u
// in float arithmetic, u = 2^-24, and the exponential to x^2 u, its argument's roundings.
// The slope needs the exponential as well.  (A float call of 40,000 rows, 96 x 130, 30.3 us
// and its gradient 32.3, 29.7 and 31.6 with half the terms and 7e-8 of 1 in place of Phi; with
// the C library's erfc the epilogue took a quarter of the time.)
struct Bend {
    float value, slope;
};
template <bool ERF>
__device__ __forceinline__ Bend bend(float x, const GatedArgs &a) {
    if constexpr (ERF) {
        const float z = fabsf(x), e = __builtin_amdgcn_exp2f(x * x * -0.72134752044448170f);
        const float t = __builtin_amdgcn_rcpf(fmaf(0.34375f, z, 1.f));
        float q = -0.02736702f;
        q = fmaf(q, t, 0.141812742f);
        q = fmaf(q, t, -0.267751813f);
        q = fmaf(q, t, 0.186679602f);
        q = fmaf(q, t, -0.0365845561f);
        q = fmaf(q, t, 0.11158856f);
        q = fmaf(q, t, 0.116990633f);
        q = fmaf(q, t, 0.137510493f);
        q = fmaf(q, t, 0.13712135f);
        const float tail = q * t * e;  // Phi(-|x|)
        const float phi = x > 0.f ? 1.f - tail : tail;
        return {x * phi, fmaf(x * 0.39894228040143268f, e, phi)};
    } else {
        if (a.relu) return {x < 0.f ? 0.f : x, x <= 0.f ? 0.f : 1.f};
        const float q = fminf(x * x, 1e6f);  // beyond that s is 0 or 1 already
        const float p = x * fmaf(a.c2, q, a.c1);
        const float e = __expf(-p), s = __builtin_amdgcn_rcpf(1.f + e);
        const float rest = p > 0.f ? e * s : 1.f - s;  // 1 - s
        return {x * s, fmaf(x * s * rest, fmaf(3.f * a.c2, q, a.c1), s)};
    }
}
template <bool ERF>
__device__ __forceinline__ f32x4 gated_value(f32x4 g, f32x4 u, const GatedArgs &a) {
    f32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = bend<ERF>(g[e], a).value * u[e];
    return y;
}
template <bool ERF>
__device__ __forceinline__ void gated_slope(f32x4 &g, f32x4 &u, f32x4 d, const GatedArgs &a) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const Bend b = bend<ERF>(g[e], a);
        g[e] = d[e] * u[e] * b.slope;
        u[e] = d[e] * b.value;
    }
}

// A tile of one segment: rows row0 .. row0 + rows - 1, outputs from n0.
struct GatedPlace {
    int64_t s, row0, n0;
    int rows;  // 0: nothing to do
};
// BM rows x BN outputs.
template <int BM, int BN>
__device__ __forceinline__ GatedPlace gated_place(const GatedArgs &a, int lane) {
    constexpr int kLg = __builtin_ctz(BM);
    GatedPlace p{0, 0, 0, 0};
    const int64_t id = xcd_tile(a.slots * a.ntiles);
    if (id >= a.slots * a.ntiles) return p;
    const TilePlace at = tile_place(id, a.slots, a.ntiles);
    p.s = tight_segment(a.offsets, a.S, kLg, at.m, lane);
    p.n0 = at.n * BN;
    p.row0 = a.offsets[p.s] + ((at.m - tight_key(a.offsets, p.s, kLg)) << kLg);
    const int64_t end = min(a.offsets[p.s + 1], a.N);
    if (p.row0 < end && p.row0 >= 0) p.rows = (int)min((int64_t)BM, end - p.row0);
    return p;
}
template <typename T>
__device__ __forceinline__ const char *gated_row(const GatedArgs &a, const GatedPlace &p, int r) {
    if (r >= p.rows) return nullptr;
    int64_t v = p.row0 + r;
    if (a.rows) v = a.rows[v];
    return v >= 0 && v < a.value_rows ? a.values + v * a.K * (int64_t)sizeof(T) : nullptr;
}
// Row of the weights for output n of the tile's segment, half 0 (G) or 1 (U).
template <typename T>
__device__ __forceinline__ const char *gated_weight(const GatedArgs &a, const GatedPlace &p, int64_t n, int half) {
    n += p.n0;
    return n < a.M ? a.weights + ((2 * p.s + half) * a.M + n) * a.K * (int64_t)sizeof(T) : nullptr;
}
// The same for tile column c where blocks of 16 of G and U take turns.
template <typename T>
__device__ __forceinline__ const char *gated_pair(const GatedArgs &a, const GatedPlace &p, int c) {
    return gated_weight<T>(a, p, (c >> 5) * 16 + (c & 15), (c >> 4) & 1);
}

// Quads of 16-bit results pass through LDS so that whole stretches are moved; a
// tile of the output's gradient enters the same way, and each quad of it is
// replaced by the result's.  quad(f) calls f(row, column, g, u) for each of a
// lane's; BM x BN outputs.
template <typename T, int BM, int BN, int THREADS, bool GRAD, bool ERF, typename Q>
__device__ __forceinline__ void gated_store(const GatedArgs &a, const GatedPlace &p, lds_char *lds, Q quad) {
    T *out = reinterpret_cast<T *>(a.out);
    if constexpr (sizeof(T) == 4) {
        quad([&](int r, int c, f32x4 g, f32x4 u) {
            if (r >= p.rows) return;
            const int64_t n = p.n0 + c, row = p.row0 + r;
            if constexpr (GRAD) {
                gated_slope<ERF>(g, u, load_four<T>(reinterpret_cast<const T *>(a.grad) + row * a.M, n, a.M), a);
                store_four<T>(out + row * 2 * a.M, n, a.M, g);
                store_four<T>(out + row * 2 * a.M + a.M, n, a.M, u);
            } else {
                store_four<T>(out + row * a.M, n, a.M, gated_value<ERF>(g, u, a));
            }
        });
    } else if constexpr (GRAD) {
        lds_char *second = lds + BM * BN * 2;
        tile_in<T, BM, BN, THREADS>(lds, reinterpret_cast<const T *>(a.grad) + p.row0 * a.M, p.rows, p.n0, a.M);
        __syncthreads();
        quad([&](int r, int c, f32x4 g, f32x4 u) {
            gated_slope<ERF>(g, u, tile_get<T, BN>(lds, r, c), a);
            tile_put<T, BN>(lds, r, c, g);
            tile_put<T, BN>(second, r, c, u);
        });
        __syncthreads();
        tile_write<T, BM, BN, THREADS>(lds, out + p.row0 * 2 * a.M, p.rows, p.n0, a.M, 2 * a.M);
        tile_write<T, BM, BN, THREADS>(second, out + p.row0 * 2 * a.M + a.M, p.rows, p.n0, a.M, 2 * a.M);
    } else {
        quad([&](int r, int c, f32x4 g, f32x4 u) { tile_put<T, BN>(lds, r, c, gated_value<ERF>(g, u, a)); });
        __syncthreads();
        tile_write<T, BM, BN, THREADS>(lds, out + p.row0 * a.M, p.rows, p.n0, a.M, a.M);
    }
}

// BM rows x BN / 2 outputs per workgroup.
template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool DIRECT, bool GRAD, bool ERF>
struct GatedTile {
    using Tile = RowTile<T, BM, BN, WM, WN, STAGES, DIRECT>;
    static constexpr int kOut = GRAD ? 2 : 1;
    static constexpr int kLds = std::max(Tile::kLds, sizeof(T) == 2 ? kOut * BM * BN : 0);

    static __device__ __forceinline__ void run(const GatedArgs &a, const GatedPlace &p, lds_char *lds, int wave, int lane) {
        f32x4 acc[Tile::MT][Tile::NT] = {};
        Tile::run(acc, (int)a.K, lds, wave, lane, [&](int r) { return gated_row<T>(a, p, r); },
                  [&](int c) { return gated_pair<T>(a, p, c); });
        gated_store<T, BM, BN / 2, Tile::kThreads, GRAD, ERF>(a, p, lds, [&](auto f) {
#pragma unroll
            for (int i = 0; i < Tile::MT; ++i)
#pragma unroll
                for (int j = 0; j < Tile::NT; j += 2)
                    f(Tile::m0(wave) + 16 * i + (lane & 15), Tile::n0(wave) / 2 + 8 * j + (lane >> 4) * 4, acc[i][j],
                      acc[i][j + 1]);
        });
    }
};

template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool DIRECT, bool GRAD, bool ERF>
__global__ __launch_bounds__(64 * WM * WN) void seg_gated(GatedArgs a) {
    using Tile = GatedTile<T, BM, BN, WM, WN, STAGES, DIRECT, GRAD, ERF>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const GatedPlace p = gated_place<BM, BN / 2>(a, lane);
    if (p.rows > 0) Tile::run(a, p, (lds_char *)lds_mem, wave, lane);
}

// The same for float, in bf16 parts; a tile with a sum that is not finite is
// computed again with float products.
template <int BM, int BN, bool WHOLE, bool GRAD, bool ERF>
__global__ __launch_bounds__(kRowSplitThreads, 3) void seg_gated_split(GatedArgs a) {
    using Tile = SplitTile<BM, BN, WHOLE>;
    using Plain = GatedTile<float, 64, 64, 2, 2, 2, false, GRAD, ERF>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds > Plain::kLds ? Tile::kLds : Plain::kLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const GatedPlace p = gated_place<BM, BN / 2>(a, lane);
    if (p.rows == 0) return;
    f32x4 acc[Tile::MT][Tile::NT] = {};
    if (!Tile::run(acc, (int)a.K, lds, threadIdx.x, [&](int r) { return gated_row<float>(a, p, r); },
                   [&](int c) { return gated_pair<float>(a, p, c); })) {
        for (int r = 0; r < p.rows; r += 64)
            for (int c = 0; c < BN / 2 && p.n0 + c < a.M; c += 32) {
                const GatedPlace q{p.s, p.row0 + r, p.n0 + c, min(64, p.rows - r)};
                __syncthreads();
                Plain::run(a, q, lds, wave, lane);
            }
        return;
    }
    gated_store<float, BM, BN / 2, kRowSplitThreads, GRAD, ERF>(a, p, lds, [&](auto f) {
#pragma unroll
        for (int i = 0; i < Tile::MT; ++i)
#pragma unroll
            for (int j = 0; j < Tile::NT; j += 2)
                f(Tile::m0(wave) + 16 * i + (lane & 15), Tile::n0(wave) / 2 + 8 * j + (lane >> 4) * 4, acc[i][j],
                  acc[i][j + 1]);
    });
}

// Many rows per segment: AH * 128 rows x 128 outputs per workgroup, in phases.
// The halves of the tile's columns are G's rows and U's.
template <typename T, int AH, bool GRAD, bool ERF>
__global__ __launch_bounds__(kPhaseThreads) void seg_gated_many(GatedArgs a) {
    using Tile = PhaseTile<T, AH>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[kPhaseLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const GatedPlace p = gated_place<AH * kHalf, kHalf>(a, lane);
    if (p.rows == 0) return;
    f32x4 acc[2][2][4][2] = {};
    Tile::run(acc, p.rows, (int)a.K, lds, wave, lane, [&](int r) { return gated_row<T>(a, p, r); },
              [&](int c) { return gated_weight<T>(a, p, c & (kHalf - 1), c >> 7); });
    gated_store<T, AH * kHalf, kHalf, kPhaseThreads, GRAD, ERF>(a, p, lds, [&](auto f) {
#pragma unroll
        for (int h = 0; h < AH; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    f(phase_row(h, i, wave) + (lane & 15), phase_col(0, j, wave) + (lane >> 4) * 4, acc[h][0][i][j],
                      acc[h][1][i][j]);
    });
}

// Few rows per segment: 16 rows x 8 NT outputs per workgroup, the contraction
// split over its waves.
template <typename T, int NT, int NW, int STAGES, bool DIRECT, bool GRAD, bool ERF>
__global__ __launch_bounds__(64 * NW) void seg_gated_few(GatedArgs a) {
    using Tile = FewTile<T, NT, NW, STAGES, DIRECT>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = xcd_tile(a.slots * a.ntiles);
    if (id >= a.slots * a.ntiles) return;
    GatedPlace p;
    const int64_t slot = id / a.ntiles;
    p.n0 = (id - slot * a.ntiles) * (8 * NT);
    p.s = tight_segment(a.offsets, a.S, 4, slot, lane);
    p.row0 = a.offsets[p.s] + ((slot - tight_key(a.offsets, p.s, 4)) << 4);
    const int64_t end = min(a.offsets[p.s + 1], a.N);
    if (p.row0 >= end || p.row0 < 0) return;
    p.rows = (int)min((int64_t)16, end - p.row0);
    Tile::run((int)a.K, lds, wave, lane, [&](int r) { return gated_row<T>(a, p, r); },
              [&](int c) { return gated_pair<T>(a, p, c); });
    T *out = reinterpret_cast<T *>(a.out);
    const int r = lane & 15;
    const int64_t row = p.row0 + r;
    for (int j = wave; j < NT / 2; j += NW) {
        f32x4 g = Tile::sum(lds, 2 * j, lane), u = Tile::sum(lds, 2 * j + 1, lane);
        if (r >= p.rows) continue;
        const int64_t n = p.n0 + 16 * j + (lane >> 4) * 4;
        if constexpr (GRAD) {
            gated_slope<ERF>(g, u, load_four<T>(reinterpret_cast<const T *>(a.grad) + row * a.M, n, a.M), a);
            store_four<T>(out + row * 2 * a.M, n, a.M, g);
            store_four<T>(out + row * 2 * a.M + a.M, n, a.M, u);
        } else {
            store_four<T>(out + row * a.M, n, a.M, gated_value<ERF>(g, u, a));
        }
    }
}

// Slots of BM rows and tiles of `outputs`.
bool gated_grid(GatedArgs &a, int lg, int64_t outputs, dim3 &grid) {
    a.slots = tight_slots(a.N, a.S, lg);
    a.ntiles = (a.M + outputs - 1) / outputs;
    return a.slots <= INT64_MAX / a.ntiles && tile_grid(a.slots * a.ntiles, grid);
}

template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool DIRECT, bool GRAD, bool ERF>
int gated_launch(GatedArgs a, hipStream_t st) {
    dim3 grid;
    if (!gated_grid(a, __builtin_ctz(BM), BN / 2, grid)) return SEGRED_ERR_UNSUPPORTED;
    timed_launch_ggl(true, (seg_gated<T, BM, BN, WM, WN, STAGES, DIRECT, GRAD, ERF>), grid, dim3(64 * WM * WN), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}
template <int BM, int BN, bool GRAD, bool ERF>
int gated_split_launch(GatedArgs a, hipStream_t st) {
    dim3 grid;
    if (!gated_grid(a, __builtin_ctz(BM), BN / 2, grid)) return SEGRED_ERR_UNSUPPORTED;
    if (a.K % 8 == 0) timed_launch_ggl(true, (seg_gated_split<BM, BN, true, GRAD, ERF>), grid, dim3(kRowSplitThreads), 0, st, a);
    else timed_launch_ggl(true, (seg_gated_split<BM, BN, false, GRAD, ERF>), grid, dim3(kRowSplitThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}
template <typename T, int AH, bool GRAD, bool ERF>
int gated_many_launch(GatedArgs a, hipStream_t st) {
    dim3 grid;
    if (!gated_grid(a, AH == 2 ? 8 : 7, kHalf, grid)) return SEGRED_ERR_UNSUPPORTED;
    timed_launch_ggl(true, (seg_gated_many<T, AH, GRAD, ERF>), grid, dim3(kPhaseThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}
template <typename T, int NT, int NW, int STAGES, bool DIRECT, bool GRAD, bool ERF>
int gated_few_launch(GatedArgs a, hipStream_t st) {
    dim3 grid;
    if (!gated_grid(a, 4, 8 * NT, grid)) return SEGRED_ERR_UNSUPPORTED;
    timed_launch_ggl(true, (seg_gated_few<T, NT, NW, STAGES, DIRECT, GRAD, ERF>), grid, dim3(64 * NW), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

// The kernel for a 16-bit call whose rows are whole units.  Measured times in us
// (bfloat16, mean rows per segment given, uneven, weights from HBM; forward, the
// gradient adds about the same to all):
//
//   segments, k, m      64, 2048, 1024               8, 1024, 2560   8, 512, 2560   1, 4096, 4096
//   mean rows           1    8   64  128  512         256   2048     1024   2048    128   1024  4096
//   256 x 128          75  159  154  164  337          59    196       84    127     58     89   222
//   128 x 128          70  151  141  169  376          42    228       82    148     56     65   262
//   128 x 64           77  152  146  190  406          44    217       68    128     52     72   274
//   64 x 32            70  115  172  223  578          60    310       96    195     25    120   435
//   32 x 64            62  120  174  237  674          69    389      129    247     27    161   532
//   few                77  115  406  767 2883         297   2267      646   1299     77    566  2258
//
// The rule is the least of tile_time().
int gated_kind(const GatedArgs &a, bool grad) {
    constexpr double kMore[] = {11, 4.7, 4.3, 2};  // us more of a round for the gradient
    auto time = [&](int i) {
        const TileCost &g = kTileCosts[i];
        // half a tile more per segment for its end
        const double slots = a.S == 1 ? (double)((a.N + g.rows - 1) / g.rows) : (double)a.N / g.rows + 0.5 * a.S;
        return tile_time(g, grad ? kMore[i] : 0, a.K, slots * ((2 * a.M + g.columns - 1) / g.columns), a.S == 1);
    };
    int best = 0;
    for (int i = 1; i < 4; ++i)
        if (time(i) < time(best)) best = i;
    return best;
}

// Float: segred_matmul's rule with 2 m outputs.  Times in us (forward):
//
//   segments, k, m      8, 1024, 512                       64, 1024, 512                1, 2048, 2048
//   mean rows           1    8   16   24   64  128  512    1    8   16   24   64  128   1    8   24  128  512
//   few                11   11   11   19   28   44  141   55   60   65   88  162  305  16   16   17   44  150
//   32 x 128           27   27   27   27   28   44  108   66   78   75   89  123  207  49   50   50   52   86
//   16 x 128, any      29   28   27   28   35   47  127   66   70   75   98  138  241  55   52   52   50  113
//   64 x 128 in parts  40   40   40   40   40   40   70   67   76   77   75   99  132  76   76   76   75   76
//
// (8 segments, 128 x 128: all within 8 to 10 us.)  From 9 to 63 rows a segment the first would
// be faster than the second where workgroups are few.
constexpr int64_t kFewRows = 8, kFewGroups = 192, kSplitRows = 24, kSplitTiles = 224;
template <typename T, bool GRAD, bool ERF>
int gated_dispatch(const GatedArgs &a, bool direct, hipStream_t st) {
    const int64_t mean = a.N / a.S;
    if constexpr (sizeof(T) == 4) {
        const int64_t tiles = (a.N / 64 + a.S / 2) * ((2 * a.M + 127) / 128);
        if (direct && mean <= kFewRows) return gated_few_launch<T, 4, 4, 3, true, GRAD, ERF>(a, st);
        if (direct && (mean <= kSplitRows || tiles < kSplitTiles))
            return gated_launch<T, 32, 128, 1, 4, 3, true, GRAD, ERF>(a, st);
        if (mean <= kSplitRows) return gated_launch<T, 16, 128, 1, 4, 2, false, GRAD, ERF>(a, st);
        return gated_split_launch<64, 128, GRAD, ERF>(a, st);
    } else {
        // waves that split the contraction where there are few workgroups (one
        // segment of 16 rows, 4,096 x 4,096: 15 us against 23 of 64 x 32; of 4,095 x 4,095 68
        // against 75 of 16 x 64, but 8 of 12 rows, 1,021 x 2,551, 53 against 39)
        const bool few = mean <= 2 * kFewRows && a.S * ((a.M + 31) / 32) <= kFewGroups;
        if (!direct && few) return gated_few_launch<T, 4, 4, 3, false, GRAD, ERF>(a, st);
        if (!direct && mean <= 2 * kFewRows) return gated_launch<T, 16, 128, 1, 4, 2, false, GRAD, ERF>(a, st);
        if (!direct) return gated_launch<T, 64, 128, 2, 2, 2, false, GRAD, ERF>(a, st);
        if (few) return gated_few_launch<T, 4, 4, 3, true, GRAD, ERF>(a, st);
        if (mean <= 2) return gated_launch<T, 32, 128, 1, 4, 3, true, GRAD, ERF>(a, st);
        switch (gated_kind(a, GRAD)) {
        case 0: return gated_many_launch<T, 2, GRAD, ERF>(a, st);
        case 1: return gated_many_launch<T, 1, GRAD, ERF>(a, st);
        case 2: return gated_launch<T, 128, 128, 2, 4, 2, true, GRAD, ERF>(a, st);
        default: return gated_launch<T, 64, 64, 2, 2, 3, true, GRAD, ERF>(a, st);
        }
    }
}

template <bool GRAD, bool ERF>
int gated_typed(const GatedArgs &a, int32_t dtype, bool direct, hipStream_t st) {
    switch (dtype) {
    case SEGRED_BF16: return gated_dispatch<__bf16, GRAD, ERF>(a, direct, st);
    case SEGRED_F16: return gated_dispatch<_Float16, GRAD, ERF>(a, direct, st);
    default: return gated_dispatch<float, GRAD, ERF>(a, direct, st);
    }
}

int gated_call(bool is_grad, const void *grad, const void *values, int32_t dtype, int64_t k, const int64_t *rows,
               int64_t value_rows, const void *weights, int64_t m, int32_t activation, const int64_t *offsets,
               int64_t num_segments, int64_t num_rows, void *out, hipStream_t stream) {
    const int64_t e = float_size(dtype);
    if (dtype < SEGRED_U32 || dtype > SEGRED_F16) return SEGRED_ERR_INVALID_ARGUMENT;
    if (activation < SEGRED_SILU || activation > SEGRED_RELU) return SEGRED_ERR_INVALID_ARGUMENT;
    if (k < 1 || m < 1 || value_rows < 0 || num_segments < 0 || num_rows < 0) return SEGRED_ERR_INVALID_ARGUMENT;
    if (!rows && value_rows < num_rows) return SEGRED_ERR_INVALID_ARGUMENT;
    if (num_segments > 0 && num_rows > 0 &&
        ((value_rows > 0 && !values) || !weights || !offsets || !out || (is_grad && !grad)))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (e == 0 || k > kMaxWidth || m > kMaxWidth / 2) return SEGRED_ERR_UNSUPPORTED;
    if (!aligned(values, e) || !aligned(weights, e) || !aligned(out, e) || !aligned(grad, e) || !aligned(offsets, 8) ||
        !aligned(rows, 8))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (too_large(value_rows, k, 4) || too_large(num_rows, m, 8) || too_large(num_segments, k * m, 8))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (num_segments == 0 || num_rows == 0) return SEGRED_OK;

    GatedArgs a{};
    a.values = static_cast<const char *>(values);
    a.rows = rows;
    a.value_rows = value_rows;
    a.weights = static_cast<const char *>(weights);
    a.offsets = offsets;
    a.S = num_segments;
    a.N = num_rows;
    a.K = k;
    a.M = m;
    a.grad = static_cast<const char *>(grad);
    a.out = out;
    // 0.5 (1 + tanh y) = 1 / (1 + exp(-2 y)), y = sqrt(2 / pi) (x + 0.044715 x^3)
    a.c1 = activation == SEGRED_GELU_TANH ? 1.5957691216057308f : 1.f;
    a.c2 = activation == SEGRED_GELU_TANH ? 0.071354816272600248f : 0.f;
    a.relu = activation == SEGRED_RELU;
    const bool direct = (k * e) % 16 == 0 && aligned(values, 16) && aligned(weights, 16);
    if (activation == SEGRED_GELU)
        return is_grad ? gated_typed<true, true>(a, dtype, direct, stream) : gated_typed<false, true>(a, dtype, direct, stream);
    return is_grad ? gated_typed<true, false>(a, dtype, direct, stream) : gated_typed<false, false>(a, dtype, direct, stream);
}

}  // namespace segred

using namespace segred;

extern "C" int segred_gated(const void *values, int32_t dtype, int64_t k, const int64_t *rows, int64_t value_rows,
                            const void *weights, int64_t m, int32_t activation, const int64_t *offsets,
                            int64_t num_segments, int64_t num_rows, void *out, hipStream_t stream) {
    return gated_call(false, nullptr, values, dtype, k, rows, value_rows, weights, m, activation, offsets, num_segments,
                      num_rows, out, stream);
}

extern "C" int segred_gated_grad(const void *grad, const void *values, int32_t dtype, int64_t k, const int64_t *rows,
                                 int64_t value_rows, const void *weights, int64_t m, int32_t activation,
                                 const int64_t *offsets, int64_t num_segments, int64_t num_rows, void *out,
                                 hipStream_t stream) {
    return gated_call(true, grad, values, dtype, k, rows, value_rows, weights, m, activation, offsets, num_segments,
                      num_rows, out, stream);
}
