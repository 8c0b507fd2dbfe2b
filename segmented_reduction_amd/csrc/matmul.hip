// matmul.hip -- the matrix product of each segment's rows with weights of its
// own: out[r] = values[r] W[s] for the rows r of segment s.
#include <algorithm>

#include "internal.hpp"
#include "tile.hpp"

namespace segred {

struct MatmulArgs {
    const char *values;
    const int64_t *rows;  // row of `values` behind each row, or null
    int64_t value_rows;
    const char *weights;
    const int64_t *offsets;
    int64_t S, N, K, M;
    int64_t slots, ntiles;
    void *out;
    int vec;  // rows of `out` hold whole 16-byte units on 16-byte boundaries
};

// A tile of one segment: rows row0 .. row0 + rows - 1, columns from n0.
struct MatmulPlace {
    int64_t s, row0, n0;
    int rows;  // 0: nothing to do
};
template <int BM, int BN>
__device__ __forceinline__ MatmulPlace matmul_place(const MatmulArgs &a, int lane) {
    constexpr int kLg = __builtin_ctz(BM);
    MatmulPlace p{0, 0, 0, 0};
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

// Start of the values row behind tile row r, or null for a row of zeros.
__device__ __forceinline__ const char *matmul_row(const MatmulArgs &a, const MatmulPlace &p, int r, int64_t row_bytes) {
    if (r >= p.rows) return nullptr;
    int64_t v = p.row0 + r;
    if (a.rows) v = a.rows[v];
    return v >= 0 && v < a.value_rows ? a.values + v * row_bytes : nullptr;
}

// Stores a wave's neighbouring blocks; 16-bit ones through LDS, which the
// workgroup's waves have finished reading when they meet here.
template <typename T, int BM, int BN, int THREADS, int MT, int NT>
__device__ __forceinline__ void matmul_store(const MatmulArgs &a, const MatmulPlace &p, const f32x4 (&acc)[MT][NT],
                                             lds_char *lds, int m_w, int n_w, int lane) {
    T *out = reinterpret_cast<T *>(a.out) + p.row0 * a.M;
    if constexpr (sizeof(T) == 2) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                tile_put<T, BN>(lds, m_w + 16 * i + (lane & 15), n_w + 16 * j + (lane >> 4) * 4, acc[i][j]);
        __syncthreads();
        tile_out<T, BM, BN, THREADS>(lds, out, p.rows, p.n0, a.M, a.vec != 0);
    } else {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = m_w + 16 * i + (lane & 15);
            if (r < p.rows)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    store_quad<T>(out + r * a.M, p.n0 + n_w + 16 * j + (lane >> 4) * 4, a.M, acc[i][j], a.vec != 0);
        }
    }
}

template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool B_COL, bool DIRECT>
struct MatmulTile {
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    using AStage = RowStage<T, BM, kThreads, DIRECT>;
    using BRow = RowStage<T, BN, kThreads, DIRECT>;
    using BCol = ColStage<T, BN, kThreads, DIRECT>;
    static constexpr int kABytes = AStage::kBytes;
    static constexpr int kStageBytes = kABytes + (B_COL ? BCol::kBytes : BRow::kBytes);
    static constexpr int kLoads = AStage::kLoads + (B_COL ? BCol::kLoads : BRow::kLoads);
    static constexpr int kLds = STAGES * kStageBytes;
    static_assert(DIRECT || STAGES == 2, "units that pass through registers use two buffers");

    static __device__ __forceinline__ void run(const MatmulArgs &a, const MatmulPlace &p, lds_char *lds, int wave, int lane) {
        AStage sa;
        const int K = (int)a.K;
        const int64_t n0 = p.n0;
        sa.init(wave, lane, K, [&](int r) { return matmul_row(a, p, r, a.K * (int64_t)sizeof(T)); });
        const char *w = a.weights + p.s * a.K * a.M * (int64_t)sizeof(T);
        BRow sbr;
        BCol sbc;
        uint64_t wp[BCol::kLoads];
        int wleft[BCol::kLoads];
        if constexpr (B_COL) {
#pragma unroll
            for (int i = 0; i < BCol::kLoads; ++i) {
                const int64_t n = n0 + BCol::col(i, wave, lane);
                wp[i] = (uint64_t)(w + (BCol::row(i, wave, lane) * a.M + n) * (int64_t)sizeof(T));
                wleft[i] = (int)(a.M - n);
            }
        } else {
            sbr.init(wave, lane, K, [&](int r) -> const char * {
                return n0 + r < a.M ? w + (n0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
            });
        }
        auto issue = [&](int t, lds_char *buf) {
            const int k0 = t * kStep<T>;
            sa.issue(buf, wave, k0);
            if constexpr (B_COL) {
                const uint64_t step = (uint64_t)k0 * a.M * sizeof(T);
                sbc.issue(
                    buf + kABytes, wave, [&](int i) { return wp[i] + step; },
                    [&](int i) { return k0 + BCol::row(i, wave, lane) < K ? wleft[i] : 0; });
            } else {
                sbr.issue(buf + kABytes, wave, k0);
            }
        };
        auto commit = [&](lds_char *buf) {
            sa.commit(buf, wave, lane);
            if constexpr (B_COL) sbc.commit(buf + kABytes, wave, lane);
            else sbr.commit(buf + kABytes, wave, lane);
        };

        f32x4 acc[MT][NT] = {};
        const int m_w = wave / WN * (MT * 16), n_w = wave % WN * (NT * 16);
        const int steps = (K + kStep<T> - 1) / kStep<T>;
        auto products = [&](const lds_char *buf) {
            step_products<T, MT, NT, false, BM, B_COL, BN>(acc, buf, buf + kABytes, m_w, n_w, lane);
        };
        if constexpr (DIRECT) {
#pragma unroll
            for (int t = 0; t < STAGES - 1; ++t) issue(t, lds + t * kStageBytes);
            int cur = 0, fill = STAGES - 1;
            for (int t = 0; t < steps; ++t) {
                wait_and_meet<(STAGES - 2) * kLoads>();
                issue(t + STAGES - 1, lds + fill * kStageBytes);
                products(lds + cur * kStageBytes);
                cur = cur + 1 == STAGES ? 0 : cur + 1;
                fill = fill + 1 == STAGES ? 0 : fill + 1;
            }
            // the last loads write zeros into LDS; they must land before it is given away
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
            issue(0, lds);
            commit(lds);
            for (int t = 0; t < steps; ++t) {
                __syncthreads();
                if (t + 1 < steps) issue(t + 1, lds);
                products(lds + (t & 1) * kStageBytes);
                if (t + 1 < steps) commit(lds + ((t + 1) & 1) * kStageBytes);
            }
        }
        matmul_store<T, BM, BN, kThreads>(a, p, acc, lds, m_w, n_w, lane);
    }
};

// One BM x BN tile of one segment per workgroup.
template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool B_COL, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN) void seg_matmul(MatmulArgs a) {
    using Tile = MatmulTile<T, BM, BN, WM, WN, STAGES, B_COL, DIRECT>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const MatmulPlace p = matmul_place<BM, BN>(a, lane);
    if (p.rows > 0) Tile::run(a, p, (lds_char *)lds_mem, wave, lane);
}

// The same for float, in bf16 parts; a tile with a sum that is not finite is
// computed again with float products.  (Three workgroups a CU: 8,192 rows in 8
// segments, 1,024 x 1,024, take 122 us against 137 with the two that the
// registers of transposed weights would allow otherwise.)
constexpr int kSplitThreads = 256;
template <int BM, int BN, bool B_COL, bool WHOLE>
__global__ __launch_bounds__(kSplitThreads, 3) void seg_matmul_split(MatmulArgs a) {
    using Plain = MatmulTile<float, 64, 64, 2, 2, 2, B_COL, false>;
    using SA = SplitStage<BM, kSplitThreads, false, WHOLE>;
    using SB = SplitStage<BN, kSplitThreads, B_COL, WHOLE>;
    constexpr int MT = BM / 32, NT = BN / 32, kSplitLds = 3 * (SA::kPlane + SB::kPlane);
    __shared__ __attribute__((aligned(1024))) char lds_mem[kSplitLds > Plain::kLds ? kSplitLds : Plain::kLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const MatmulPlace p = matmul_place<BM, BN>(a, lane);
    if (p.rows == 0) return;

    const int K = (int)a.K, M = (int)a.M;
    SA sa;
    SB sb;
    uint64_t ap[SA::kParts], bp[SB::kParts];
    int aleft[SA::kParts], bleft[SB::kParts];
#pragma unroll
    for (int i = 0; i < SA::kParts; ++i) {
        const char *q = matmul_row(a, p, SA::row(i, tid), a.K * 4);
        ap[i] = (uint64_t)(q + SA::at(i, tid) * 4);
        aleft[i] = q ? K - SA::at(i, tid) : 0;
    }
    const char *w = a.weights + p.s * a.K * a.M * 4;
#pragma unroll
    for (int i = 0; i < SB::kParts; ++i) {
        const int64_t r = SB::row(i, tid), c = SB::at(i, tid);
        if constexpr (B_COL) {
            bp[i] = (uint64_t)(w + (r * a.M + p.n0 + c) * 4);
            bleft[i] = (int)(a.M - p.n0 - c);
        } else {
            bp[i] = (uint64_t)(w + ((p.n0 + r) * a.K + c) * 4);
            bleft[i] = p.n0 + r < a.M ? K - (int)c : 0;
        }
    }
    f32x4 acc[MT][NT] = {};
    const int m_w = wave / 2 * (BM / 2), n_w = wave % 2 * (BN / 2);
    split_steps(
        (K + kSplitK - 1) / kSplitK,
        [&](int64_t t) {
            const int k0 = (int)t * kSplitK;
            sa.issue([&](int i) { return ap[i] + (uint64_t)k0 * 4; }, [&](int i) { return aleft[i] - k0; });
            if constexpr (B_COL)
                sb.issue([&](int i) { return bp[i] + (uint64_t)k0 * M * 4; },
                         [&](int i) { return k0 + SB::row(i, tid) < K ? bleft[i] : 0; });
            else
                sb.issue([&](int i) { return bp[i] + (uint64_t)k0 * 4; }, [&](int i) { return bleft[i] - k0; });
        },
        [&] {
            sa.commit(lds, tid);
            sb.commit(lds + 3 * SA::kPlane, tid);
        },
        [&] { split_step<MT, NT, false, BM, B_COL, BN>(acc, lds, lds + 3 * SA::kPlane, m_w, n_w, lane); });
    if (__syncthreads_or(any_not_finite(acc))) {
        for (int r = 0; r < p.rows; r += 64)
            for (int c = 0; c < BN && p.n0 + c < a.M; c += 64) {
                const MatmulPlace q{p.s, p.row0 + r, p.n0 + c, min(64, p.rows - r)};
                __syncthreads();
                Plain::run(a, q, lds, wave, lane);
            }
        return;
    }
    matmul_store<float, BM, BN, kSplitThreads>(a, p, acc, lds, m_w, n_w, lane);
}

template <int BM, int BN>
int matmul_split_launch(MatmulArgs a, bool b_col, hipStream_t st) {
    a.slots = tight_slots(a.N, a.S, __builtin_ctz(BM));
    a.ntiles = (a.M + BN - 1) / BN;
    dim3 grid;
    if (a.slots > INT64_MAX / a.ntiles || !tile_grid(a.slots * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    const bool whole = a.K % 8 == 0 && (!b_col || a.M % 8 == 0);
    if (b_col && whole) timed_launch_ggl(true, (seg_matmul_split<BM, BN, true, true>), grid, dim3(kSplitThreads), 0, st, a);
    else if (b_col) timed_launch_ggl(true, (seg_matmul_split<BM, BN, true, false>), grid, dim3(kSplitThreads), 0, st, a);
    else if (whole) timed_launch_ggl(true, (seg_matmul_split<BM, BN, false, true>), grid, dim3(kSplitThreads), 0, st, a);
    else timed_launch_ggl(true, (seg_matmul_split<BM, BN, false, false>), grid, dim3(kSplitThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

// Many rows per segment: AH * 128 rows x 256 columns per workgroup, in phases.
// A tile of at most 128 rows walks the steps of one half only.
template <typename T, int AH, bool B_COL>
__global__ __launch_bounds__(kPhaseThreads) void seg_matmul_many(MatmulArgs a) {
    using AStage = RowStage<T, kHalf, kPhaseThreads, true>;
    using BRow = RowStage<T, kHalf, kPhaseThreads, true>;
    using BCol = ColStage<T, kHalf, kPhaseThreads, true>;
    constexpr int kLg = AH == 2 ? 8 : 7;
    __shared__ __attribute__((aligned(1024))) char lds_mem[kPhaseLds];
    lds_char *lds = (lds_char *)lds_mem;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = xcd_tile(a.slots * a.ntiles);
    if (id >= a.slots * a.ntiles) return;
    const TilePlace at = tile_place(id, a.slots, a.ntiles);
    const int64_t slot = at.m;
    const int64_t n0 = at.n * (2 * kHalf);
    const int64_t s = tight_segment(a.offsets, a.S, kLg, slot, lane);
    const int64_t row0 = a.offsets[s] + ((slot - tight_key(a.offsets, s, kLg)) << kLg);
    const int64_t end = min(a.offsets[s + 1], a.N);
    if (row0 >= end || row0 < 0) return;
    const int rows = (int)min((int64_t)(AH * kHalf), end - row0), K = (int)a.K;

    AStage sa[AH];
#pragma unroll
    for (int h = 0; h < AH; ++h)
        sa[h].init(wave, lane, K, [&](int r) -> const char * {
            r += h * kHalf;
            if (r >= rows) return nullptr;
            int64_t v = row0 + r;
            if (a.rows) v = a.rows[v];
            if (v < 0 || v >= a.value_rows) return nullptr;
            return a.values + v * a.K * (int64_t)sizeof(T);
        });
    const char *w = a.weights + s * a.K * a.M * (int64_t)sizeof(T);
    BRow sbr[2];
    BCol sbc;
    uint64_t wp[2][BCol::kLoads];
    int wleft[2][BCol::kLoads];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (B_COL) {
#pragma unroll
            for (int i = 0; i < BCol::kLoads; ++i) {
                const int64_t n = n0 + h * kHalf + BCol::col(i, wave, lane);
                wp[h][i] = (uint64_t)(w + (BCol::row(i, wave, lane) * a.M + n) * (int64_t)sizeof(T));
                wleft[h][i] = (int)(a.M - n);
            }
        } else {
            sbr[h].init(wave, lane, K, [&](int r) -> const char * {
                const int64_t n = n0 + h * kHalf + r;
                return n < a.M ? w + n * a.K * (int64_t)sizeof(T) : nullptr;
            });
        }
    }
    f32x4 acc[2][2][4][2] = {};
    auto fetch_a = [&](int h, int t, lds_char *place) { sa[h].issue(place, wave, t * kStep<T>); };
    auto fetch_b = [&](int h, int t, lds_char *place) {
        const int k0 = t * kStep<T>;
        if constexpr (B_COL) {
            const uint64_t step = (uint64_t)k0 * a.M * sizeof(T);
            sbc.issue(
                place, wave, [&](int i) { return wp[h][i] + step; },
                [&](int i) { return k0 + BCol::row(i, wave, lane) < K ? wleft[h][i] : 0; });
        } else {
            sbr[h].issue(place, wave, k0);
        }
    };
    auto products = [](f32x4 (&c)[4][2], const u32x4 (&x)[2][4], const u32x4 (&y)[2][2]) { quadrant<T>(c, x, y); };
    const int steps = (K + kStep<T> - 1) / kStep<T>;
    if (AH == 2 && rows > kHalf)
        phase_steps<T, AH, B_COL>(acc, lds, steps, wave, lane, fetch_a, fetch_b, products);
    else
        phase_steps<T, 1, B_COL>(acc, lds, steps, wave, lane, fetch_a, fetch_b, products);

    __syncthreads();
    constexpr int BN = 2 * kHalf;
#pragma unroll
    for (int p = 0; p < AH; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    tile_put<T, BN>(lds, phase_row(p, i, wave) + (lane & 15), phase_col(q, j, wave) + (lane >> 4) * 4,
                                    acc[p][q][i][j]);
    __syncthreads();
    tile_out<T, AH * kHalf, BN, kPhaseThreads>(lds, reinterpret_cast<T *>(a.out) + row0 * a.M, rows, n0, a.M, a.vec != 0);
}

template <typename T, int AH>
int matmul_many_launch(MatmulArgs a, bool b_col, hipStream_t st) {
    a.slots = tight_slots(a.N, a.S, AH == 2 ? 8 : 7);
    a.ntiles = (a.M + 2 * kHalf - 1) / (2 * kHalf);
    dim3 grid;
    if (a.slots > INT64_MAX / a.ntiles || !tile_grid(a.slots * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    if constexpr (AH == 1)
        if (b_col) {
            timed_launch_ggl(true, (seg_matmul_many<T, 1, true>), grid, dim3(kPhaseThreads), 0, st, a);
            return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
        }
    timed_launch_ggl(true, (seg_matmul_many<T, AH, false>), grid, dim3(kPhaseThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

// Few rows per segment: 16 rows x 16 NT columns per workgroup, the
// contraction split over its NW waves.
template <typename T, int NT, int NW, int STAGES, bool B_COL>
__global__ __launch_bounds__(64 * NW) void seg_matmul_few(MatmulArgs a) {
    using AStage = RowStage<T, 16, 64, true>;
    using BRow = RowStage<T, 16 * NT, 64, true>;
    using BCol = ColStage<T, 16 * NT, 64, true>;
    constexpr int kABytes = AStage::kBytes;
    constexpr int kStageBytes = kABytes + (B_COL ? BCol::kBytes : BRow::kBytes);
    constexpr int kLoads = AStage::kLoads + (B_COL ? BCol::kLoads : BRow::kLoads);
    __shared__ __attribute__((aligned(1024))) char lds_mem[NW * STAGES * kStageBytes];
    lds_char *lds = (lds_char *)lds_mem;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = xcd_tile(a.slots * a.ntiles);
    if (id >= a.slots * a.ntiles) return;
    const int64_t slot = id / a.ntiles, n0 = (id - slot * a.ntiles) * (16 * NT);
    const int64_t s = tight_segment(a.offsets, a.S, 4, slot, lane);
    const int64_t row0 = a.offsets[s] + ((slot - tight_key(a.offsets, s, 4)) << 4);
    const int64_t end = min(a.offsets[s + 1], a.N);
    if (row0 >= end || row0 < 0) return;
    const int rows = (int)min((int64_t)16, end - row0);
    const int K = (int)a.K;

    AStage sa;
    sa.init(0, lane, K, [&](int r) -> const char * {
        if (r >= rows) return nullptr;
        int64_t v = row0 + r;
        if (a.rows) v = a.rows[v];
        if (v < 0 || v >= a.value_rows) return nullptr;
        return a.values + v * a.K * (int64_t)sizeof(T);
    });
    const char *w = a.weights + s * a.K * a.M * (int64_t)sizeof(T);
    BRow sbr;
    BCol sbc;
    uint64_t wp[BCol::kLoads];
    int wleft[BCol::kLoads];
    if constexpr (B_COL) {
#pragma unroll
        for (int i = 0; i < BCol::kLoads; ++i) {
            const int64_t n = n0 + BCol::col(i, 0, lane);
            wp[i] = (uint64_t)(w + (BCol::row(i, 0, lane) * a.M + n) * (int64_t)sizeof(T));
            wleft[i] = (int)(a.M - n);
        }
    } else {
        sbr.init(0, lane, K, [&](int r) -> const char * {
            return n0 + r < a.M ? w + (n0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
        });
    }
    f32x4 acc[1][NT] = {};
    const int steps = (K + kStep<T> - 1) / kStep<T>;
    wave_steps<STAGES, true, kLoads, kStageBytes>(
        lds + wave * STAGES * kStageBytes, wave * steps / NW, (wave + 1) * steps / NW,
        [&](int t, bool live, lds_char *buf) {
            const int k0 = live ? t * kStep<T> : K;
            sa.issue(buf, 0, k0);
            if constexpr (B_COL) {
                const uint64_t step = (uint64_t)k0 * a.M * sizeof(T);
                sbc.issue(
                    buf + kABytes, 0, [&](int i) { return wp[i] + step; },
                    [&](int i) { return k0 + BCol::row(i, 0, lane) < K ? wleft[i] : 0; });
            } else {
                sbr.issue(buf + kABytes, 0, k0);
            }
        },
        [](lds_char *) {},
        [&](int, const lds_char *buf) {
            step_products<T, 1, NT, false, 16, B_COL, 16 * NT>(acc, buf, buf + kABytes, 0, 0, lane);
        },
        [] {});
    T *out = reinterpret_cast<T *>(a.out);
    join_waves<NW, 1, NT>(lds, acc, wave, lane, [&](int r, int c, f32x4 sum) {
        if (r < rows) store_quad<T>(out + (row0 + r) * a.M, n0 + c, a.M, sum, a.vec != 0);
    });
}

template <typename T, int NT, int NW, int STAGES>
int matmul_few_launch(MatmulArgs a, bool b_col, hipStream_t st) {
    a.slots = tight_slots(a.N, a.S, 4);
    a.ntiles = (a.M + 16 * NT - 1) / (16 * NT);
    dim3 grid;
    if (a.slots > INT64_MAX / a.ntiles || !tile_grid(a.slots * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    if (b_col) timed_launch_ggl(true, (seg_matmul_few<T, NT, NW, STAGES, true>), grid, dim3(64 * NW), 0, st, a);
    else timed_launch_ggl(true, (seg_matmul_few<T, NT, NW, STAGES, false>), grid, dim3(64 * NW), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool DIRECT>
int matmul_launch(MatmulArgs a, bool b_col, hipStream_t st) {
    a.slots = tight_slots(a.N, a.S, __builtin_ctz(BM));
    a.ntiles = (a.M + BN - 1) / BN;
    dim3 grid;
    if (a.slots > INT64_MAX / a.ntiles || !tile_grid(a.slots * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    constexpr int kThreads = 64 * WM * WN;
    if (b_col)
        timed_launch_ggl(true, (seg_matmul<T, BM, BN, WM, WN, STAGES, true, DIRECT>), grid, dim3(kThreads), 0, st, a);
    else
        timed_launch_ggl(true, (seg_matmul<T, BM, BN, WM, WN, STAGES, false, DIRECT>), grid, dim3(kThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

// The kernel for a call, by its mean rows per segment and the number of tiles.
// Times in us of bfloat16 products of 64 segments, 2,048 x 2,048, whose mean
// rows are given (uneven; weights from HBM; "row" is a transposed weight):
//
//   mean          4    16    32    64    96   128   256   512
//   few         104   141   220   384                           row
//   64 x 128    140   130   133   151   169   188   287   436   row
//   256 x 256   130   150   150   148   156   164   218   310   row
//   128 x 256   151   143   140   143   161   164   225   358   row
//   few         100   142   200   350                           col
//   64 x 128    106   108   116   141   163   183   262   444   col
//   128 x 256   126   120   118   122   155   160   230   387   col
//
// and with few tiles (8 segments, 2,048 x 1,024):
//
//   mean          8    16    64   256   512  1024
//   few           9    10    22    56               row
//   64 x 64      12    12    13    23    34    58   row
//   64 x 128     20    21    21    23    32    52   row
//   256 x 256    31    31    31    43    45    49   row
//   few          10    11    23    59               col
//   64 x 64      16    15    16    27    36    62   col
//   64 x 128     20    20    21    25    34    55   col
//   128 x 256    36    36    36    38    41    78   col
//
// float (64 segments, 2,048 x 2,048; "row" and "col" are near each other),
// the last line in bf16 parts:
//
//   mean          4    16    32    64   256   512
//   few         187   243
//   32 x 64     209   242   322   470  1412  2629
//   64 x 128    239   242   272   371   952  1728
//
// and with few tiles (8 segments, 2,048 x 1,024): 32 x 64 takes 46 us at 64 rows
// and 124 at 256, 64 x 128 83 and 106.
constexpr int64_t kFewRows = 8, kManyRows = 64, kManyTiles = 1536, kFewTiles = 512;
constexpr int64_t kSplitRows = 24, kSplitTiles = 224;
template <typename T>
int matmul_dispatch(const MatmulArgs &a, bool b_col, bool direct, hipStream_t st) {
    const int64_t mean = a.N / a.S;
    // 64 x 128 tiles, half a tile more per segment for its end
    const int64_t tiles = (a.N / 64 + a.S / 2) * ((a.M + 127) / 128);
    if constexpr (sizeof(T) == 4) {
        if (direct && mean <= kFewRows) return matmul_few_launch<T, 4, 4, 3>(a, b_col, st);
        if (direct && (mean <= kSplitRows || tiles < kSplitTiles))
            return matmul_launch<T, 32, 64, 1, 4, 4, true>(a, b_col, st);
        if (mean <= kSplitRows) return matmul_launch<T, 16, 128, 1, 4, 2, false>(a, b_col, st);
        return matmul_split_launch<64, 128>(a, b_col, st);
    } else {
        if (!direct && mean <= 2 * kFewRows) return matmul_launch<T, 16, 128, 1, 4, 2, false>(a, b_col, st);
        if (!direct) return matmul_launch<T, 64, 128, 2, 2, 2, false>(a, b_col, st);
        const bool few_tiles = (a.N / 64 + a.S / 2) * ((a.M + 63) / 64) <= kFewTiles;  // of 64 x 64
        if (mean <= (few_tiles ? 2 * kFewRows : kFewRows)) return matmul_few_launch<T, 4, 4, 3>(a, b_col, st);
        if (a.K >= 256 && a.M > 128 && tiles >= kManyTiles && mean >= kManyRows) {
            // a tile of 256 rows takes about 7/4 of one of 128; whole rounds of 256 CUs
            const int64_t nt = (a.M + 255) / 256;
            const int64_t one = ((a.N / 128 + a.S / 2) * nt + 255) / 256, two = ((a.N / 256 + a.S / 2) * nt + 255) / 256;
            if (b_col || 4 * one < 7 * two) return matmul_many_launch<T, 1>(a, b_col, st);
            return matmul_many_launch<T, 2>(a, b_col, st);
        }
        if (few_tiles) return matmul_launch<T, 64, 64, 2, 2, 3, true>(a, b_col, st);
        return matmul_launch<T, 64, 128, 2, 2, 2, true>(a, b_col, st);
    }
}

}  // namespace segred

using namespace segred;

extern "C" int segred_matmul(const void *values, int32_t dtype, int64_t k, const int64_t *rows, int64_t value_rows,
                             const void *weights, int32_t transpose, int64_t m, const int64_t *offsets,
                             int64_t num_segments, int64_t num_rows, void *out, hipStream_t stream) {
    const int64_t e = float_size(dtype);
    if (dtype < SEGRED_U32 || dtype > SEGRED_F16) return SEGRED_ERR_INVALID_ARGUMENT;
    if (k < 1 || m < 1 || value_rows < 0 || num_segments < 0 || num_rows < 0) return SEGRED_ERR_INVALID_ARGUMENT;
    if (!rows && value_rows < num_rows) return SEGRED_ERR_INVALID_ARGUMENT;
    if (num_segments > 0 && num_rows > 0 && ((value_rows > 0 && !values) || !weights || !offsets || !out))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (e == 0 || k > kMaxWidth || m > kMaxWidth) return SEGRED_ERR_UNSUPPORTED;
    if (!aligned(values, e) || !aligned(weights, e) || !aligned(out, e) || !aligned(offsets, 8) || !aligned(rows, 8))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (too_large(value_rows, k, 4) || too_large(num_rows, m, 4) || too_large(num_segments, k * m, 4))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (num_segments == 0 || num_rows == 0) return SEGRED_OK;

    MatmulArgs a{};
    a.values = static_cast<const char *>(values);
    a.rows = rows;
    a.value_rows = value_rows;
    a.weights = static_cast<const char *>(weights);
    a.offsets = offsets;
    a.S = num_segments;
    a.N = num_rows;
    a.K = k;
    a.M = m;
    a.out = out;
    a.vec = ((m * e) % 16 == 0 && aligned(out, 16)) ? 1 : 0;
    const int64_t along = transpose ? k : m;  // the weights' contiguous axis
    const bool direct = (k * e) % 16 == 0 && (along * e) % 16 == 0 && aligned(values, 16) && aligned(weights, 16);
    switch (dtype) {
    case SEGRED_BF16: return matmul_dispatch<__bf16>(a, !transpose, direct, stream);
    case SEGRED_F16: return matmul_dispatch<_Float16>(a, !transpose, direct, stream);
    default: return matmul_dispatch<float>(a, !transpose, direct, stream);
    }
}
