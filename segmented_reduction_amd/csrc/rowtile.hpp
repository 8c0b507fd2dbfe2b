// rowtile.hpp -- tiles of x W^T whose sums stay in registers for an epilogue of
// the caller's: gated projections and the softmax cross entropy.
//
// Both operands run along the contraction in memory (row form, tile.hpp).  The
// caller names their rows: arow(r) and brow(c) give the start of tile row r's
// and tile column c's operand row, or null for a row of zeros.
#pragma once

#include <cmath>

#include "internal.hpp"
#include "tile.hpp"

namespace segred {

// A BM x BN tile of WM x WN waves: acc[i][j] are the wave's neighbouring 16 x 16
// blocks.  Afterwards all LDS has been read and written.
template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool DIRECT>
struct RowTile {
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    using AStage = RowStage<T, BM, kThreads, DIRECT>;
    using BStage = RowStage<T, BN, kThreads, DIRECT>;
    static constexpr int kStageBytes = AStage::kBytes + BStage::kBytes;
    static constexpr int kLds = STAGES * kStageBytes;
    static_assert(DIRECT || STAGES == 2, "units that pass through registers use two buffers");
    // Row and column of block (0, 0) of a wave.
    static __device__ __forceinline__ int m0(int wave) { return wave / WN * (MT * 16); }
    static __device__ __forceinline__ int n0(int wave) { return wave % WN * (NT * 16); }

    template <typename FA, typename FB>
    static __device__ __forceinline__ void run(f32x4 (&acc)[MT][NT], int K, lds_char *lds, int wave, int lane, FA arow,
                                               FB brow) {
        constexpr int kLoads = AStage::kLoads + BStage::kLoads;
        AStage sa;
        BStage sb;
        sa.init(wave, lane, K, arow);
        sb.init(wave, lane, K, brow);
        auto issue = [&](int t, lds_char *buf) {
            sa.issue(buf, wave, t * kStep<T>);
            sb.issue(buf + AStage::kBytes, wave, t * kStep<T>);
        };
        auto commit = [&](lds_char *buf) {
            sa.commit(buf, wave, lane);
            sb.commit(buf + AStage::kBytes, wave, lane);
        };
        auto products = [&](const lds_char *buf) {
            step_products<T, MT, NT, false, BM, false, BN>(acc, buf, buf + AStage::kBytes, m0(wave), n0(wave), lane);
        };
        // Float products are added up 128 k at a time, so that a long sum's rounding
        // grows with the root of the pieces and not of all its terms (k = 2,048: 5e-7 of
        // a gated result against 1.2e-6).  (8 segments of 100 rows, 1,024 x 512: 27.3 us against
        // 25.9.  Where bf16 parts fall back on this tile the second sums are 3 to 5 spilled registers
        // on the way there: 40,000 rows, 96 x 130, 30.7 us against 30.3.)
        f32x4 total[sizeof(T) == 4 ? MT : 1][sizeof(T) == 4 ? NT : 1] = {};
        auto settle = [&](bool now) {
            if constexpr (sizeof(T) == 4) {
                if (!now) return;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        total[i][j] += acc[i][j];
                        acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                    }
            }
        };
        const int steps = (K + kStep<T> - 1) / kStep<T>;
        if constexpr (DIRECT) {
#pragma unroll
            for (int t = 0; t < STAGES - 1; ++t) issue(t, lds + t * kStageBytes);
            int cur = 0, fill = STAGES - 1;
            for (int t = 0; t < steps; ++t) {
                wait_and_meet<(STAGES - 2) * kLoads>();
                issue(t + STAGES - 1, lds + fill * kStageBytes);
                products(lds + cur * kStageBytes);
                settle((t & 3) == 3);
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
                settle((t & 3) == 3);
                if (t + 1 < steps) commit(lds + ((t + 1) & 1) * kStageBytes);
            }
        }
        if constexpr (sizeof(T) == 4)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] += total[i][j];
        __syncthreads();
    }
};

// AH * 128 rows x 256 columns in phases, 16-bit types, rows of whole 16-byte
// units.  acc[a][b] are the quadrants; brow's column c of half h is h * 128 + c.
// A tile of at most 128 rows walks the steps of one half only.
template <typename T, int AH>
struct PhaseTile {
    using Stage = RowStage<T, kHalf, kPhaseThreads, true>;

    template <typename FA, typename FB>
    static __device__ __forceinline__ void run(f32x4 (&acc)[2][2][4][2], int rows, int K, lds_char *lds, int wave,
                                               int lane, FA arow, FB brow) {
        Stage sa[AH], sb[2];
#pragma unroll
        for (int h = 0; h < AH; ++h) sa[h].init(wave, lane, K, [&](int r) { return arow(h * kHalf + r); });
#pragma unroll
        for (int h = 0; h < 2; ++h) sb[h].init(wave, lane, K, [&](int c) { return brow(h * kHalf + c); });
        auto fetch_a = [&](int h, int t, lds_char *place) { sa[h].issue(place, wave, t * kStep<T>); };
        auto fetch_b = [&](int h, int t, lds_char *place) { sb[h].issue(place, wave, t * kStep<T>); };
        auto products = [](f32x4 (&c)[4][2], const u32x4 (&x)[2][4], const u32x4 (&y)[2][2]) { quadrant<T>(c, x, y); };
        const int steps = (K + kStep<T> - 1) / kStep<T>;
        if (AH == 2 && rows > kHalf)
            phase_steps<T, AH, false>(acc, lds, steps, wave, lane, fetch_a, fetch_b, products);
        else
            phase_steps<T, 1, false>(acc, lds, steps, wave, lane, fetch_a, fetch_b, products);
        __syncthreads();
    }
};

// Float in three bf16 parts, BM x BN by four waves, 2 by 2.  False where a sum is
// not finite: then the caller has the tile computed again by RowTile<float, ...>.
constexpr int kRowSplitThreads = 256;
template <int BM, int BN, bool WHOLE>
struct SplitTile {
    using Stage = SplitStage<BM, kRowSplitThreads, false, WHOLE>;
    using BStage = SplitStage<BN, kRowSplitThreads, false, WHOLE>;
    static constexpr int MT = BM / 32, NT = BN / 32;
    static constexpr int kLds = Stage::kLds + BStage::kLds;
    static __device__ __forceinline__ int m0(int wave) { return wave / 2 * (BM / 2); }
    static __device__ __forceinline__ int n0(int wave) { return wave % 2 * (BN / 2); }

    template <typename FA, typename FB>
    static __device__ __forceinline__ bool run(f32x4 (&acc)[MT][NT], int K, lds_char *lds, int tid, FA arow, FB brow) {
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        Stage sa;
        BStage sb;
        uint64_t ap[Stage::kParts], bp[BStage::kParts];
        int aleft[Stage::kParts], bleft[BStage::kParts];
#pragma unroll
        for (int i = 0; i < Stage::kParts; ++i) {
            const char *q = arow(Stage::row(i, tid));
            ap[i] = (uint64_t)(q + Stage::at(i, tid) * 4);
            aleft[i] = q ? K - Stage::at(i, tid) : 0;
        }
#pragma unroll
        for (int i = 0; i < BStage::kParts; ++i) {
            const char *q = brow(BStage::row(i, tid));
            bp[i] = (uint64_t)(q + BStage::at(i, tid) * 4);
            bleft[i] = q ? K - BStage::at(i, tid) : 0;
        }
        split_steps(
            (K + kSplitK - 1) / kSplitK,
            [&](int64_t t) {
                const int k0 = (int)t * kSplitK;
                sa.issue([&](int i) { return ap[i] + (uint64_t)k0 * 4; }, [&](int i) { return aleft[i] - k0; });
                sb.issue([&](int i) { return bp[i] + (uint64_t)k0 * 4; }, [&](int i) { return bleft[i] - k0; });
            },
            [&] {
                sa.commit(lds, tid);
                sb.commit(lds + Stage::kLds, tid);
            },
            [&] { split_step<MT, NT, false, BM, false, BN>(acc, lds, lds + Stage::kLds, m0(wave), n0(wave), lane); });
        return !__syncthreads_or(any_not_finite(acc));
    }
};

// 16 rows x 16 NT columns, the contraction split over NW waves.  Each quad of four
// columns of all NT blocks belongs to one thread afterwards: out(block j, row, column
// in the block, sum), j uniform in a wave.  DIRECT: rows of whole units, through LDS.
// Otherwise (16-bit types) a lane loads its units of the operands, at any place, as the
// matrix units take them, a step ahead (units that straddle words are slow, so only for
// calls of few workgroups).
template <typename T, int NT, int NW, int STAGES, bool DIRECT = true>
struct FewTile {
    using AStage = RowStage<T, 16, 64, true>;
    using BStage = RowStage<T, 16 * NT, 64, true>;
    static constexpr int kThreads = 64 * NW;
    static constexpr int kStageBytes = AStage::kBytes + BStage::kBytes;
    static constexpr int kSums = NW * NT * 1024, kLds = DIRECT ? NW * STAGES * kStageBytes : kSums + 1024;

    template <typename FA, typename FB>
    static __device__ __forceinline__ void any_steps(f32x4 (&acc)[NT], int K, int wave, int lane, FA arow, FB brow) {
        static_assert(sizeof(T) == 2, "16-bit types");
        uint64_t p[NT + 1];
        int left[NT + 1];  // <= 0: a row of zeros
#pragma unroll
        for (int j = 0; j <= NT; ++j) {
            const char *row = j < NT ? brow(16 * j + (lane & 15)) : arow(lane & 15);
            p[j] = row ? (uint64_t)row + (lane >> 4) * 16 : (uint64_t)zero_unit();
            left[j] = row ? K - (lane >> 4) * kUnit<T> : 0;
        }
        u32x4 next[2][NT + 1], cur[2][NT + 1];
        // steps of 64 elements: whole ones without a bound, the last with one
        const int whole = K / 64, t1 = (wave + 1) * whole / NW;
        auto products = [&] {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[j] = mma<T>(cur[h][j], cur[h][NT], acc[j]);
        };
        auto fetch = [&](int t) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j <= NT; ++j) next[h][j] = load_whole<T>(p[j] + (left[j] > 0 ? t * 128 + h * 64 : 0));
        };
        auto take = [&] {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j <= NT; ++j) cur[h][j] = next[h][j];
        };
        int t = wave * whole / NW;
        if (t < t1) fetch(t);
        for (; t < t1; ++t) {
            take();
            if (t + 1 < t1) fetch(t + 1);
            products();
        }
        if (wave == NW - 1 && whole * 64 < K) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j <= NT; ++j)
                    cur[h][j] = load_unit<T>(p[j] + (left[j] > 0 ? whole * 128 + h * 64 : 0), left[j] - whole * 64 - h * 32);
            products();
        }
    }

    // Leaves the waves' sums in LDS, each NT KiB: quad `lane` of block j of wave w
    // at (w * NT + j) * 1024 + lane * 16.
    template <typename FA, typename FB>
    static __device__ __forceinline__ void run(int K, lds_char *lds, int wave, int lane, FA arow, FB brow) {
        f32x4 acc[1][NT] = {};
        if constexpr (DIRECT) steps(acc, K, lds, wave, lane, arow, brow);
        else any_steps(acc[0], K, wave, lane, arow, brow);
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<__attribute__((address_space(3))) f32x4 *>(lds + (wave * NT + j) * 1024 + lane * 16) =
                acc[0][j];
        __syncthreads();
    }
    template <typename FA, typename FB>
    static __device__ __forceinline__ void steps(f32x4 (&acc)[1][NT], int K, lds_char *lds, int wave, int lane, FA arow,
                                                 FB brow) {
        AStage sa;
        BStage sb;
        sa.init(0, lane, K, arow);
        sb.init(0, lane, K, brow);
        const int steps = (K + kStep<T> - 1) / kStep<T>;
        wave_steps<STAGES, true, AStage::kLoads + BStage::kLoads, kStageBytes>(
            lds + wave * STAGES * kStageBytes, wave * steps / NW, (wave + 1) * steps / NW,
            [&](int t, bool live, lds_char *buf) {
                const int k0 = live ? t * kStep<T> : K;
                sa.issue(buf, 0, k0);
                sb.issue(buf + AStage::kBytes, 0, k0);
            },
            [](lds_char *) {},
            [&](int, const lds_char *buf) {
                step_products<T, 1, NT, false, 16, false, 16 * NT>(acc, buf, buf + AStage::kBytes, 0, 0, lane);
            },
            [] {});
        __syncthreads();
    }
    // The sum of quad `lane` of block j, added in wave order.
    static __device__ __forceinline__ f32x4 sum(const lds_char *lds, int j, int lane) {
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w)
            s += *reinterpret_cast<const __attribute__((address_space(3))) f32x4 *>(lds + (w * NT + j) * 1024 + lane * 16);
        return s;
    }
};

// ---------------------------------------------------------- tiles and memory

// Four neighbouring elements from column n of a row of `width`, at any element
// boundary (one access; elements behind the row's end are left alone).
template <typename T> struct QuadOf;
template <> struct QuadOf<float> { typedef f32x4 __attribute__((aligned(4))) any; typedef f32x4 type; };
template <> struct QuadOf<__bf16> { typedef bf16x4 __attribute__((aligned(2))) any; typedef bf16x4 type; };
template <> struct QuadOf<_Float16> { typedef f16x4 __attribute__((aligned(2))) any; typedef f16x4 type; };
template <typename T>
__device__ __forceinline__ f32x4 load_four(const T *row, int64_t n, int64_t width) {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
    if (n + 4 <= width) {
        const typename QuadOf<T>::type q = *(__attribute__((address_space(1))) const typename QuadOf<T>::any *)(row + n);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = (float)q[j];
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (n + j < width) c[j] = (float)row[n + j];
    }
    return c;
}
template <typename T>
__device__ __forceinline__ void store_four(T *row, int64_t n, int64_t width, f32x4 c) {
    if (n + 4 <= width) {
        typename QuadOf<T>::type q;
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = (T)c[j];
        *(__attribute__((address_space(1))) typename QuadOf<T>::any *)(row + n) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (n + j < width) row[n + j] = (T)c[j];
    }
}

// A tile of 16-bit elements, first `rows` rows and the columns below `limit`,
// from rows of `width` elements into the places of tile_put; zeros elsewhere.
template <typename T, int BM, int BN, int THREADS>
__device__ __forceinline__ void tile_in(lds_char *lds, const T *from, int rows, int64_t n0, int64_t width) {
    constexpr int kUnits = BN / 8;
#pragma unroll 4
    for (int i = threadIdx.x; i < BM * kUnits; i += THREADS) {
        const int r = i / kUnits, u = i % kUnits;
        const int64_t n = n0 + u * 8;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (r < rows && n < width) v = load_unit<T>((uint64_t)(from + r * width + n), (int)min(width - n, (int64_t)8));
        *reinterpret_cast<__attribute__((address_space(3))) u32x4 *>(lds + tile_unit<T, BN>(r, u)) = v;
    }
}
template <typename T, int BN>
__device__ __forceinline__ f32x4 tile_get(const lds_char *lds, int r, int c) {
    typedef __attribute__((ext_vector_type(4))) T T4;
    const T4 q = *reinterpret_cast<const __attribute__((address_space(3))) T4 *>(lds + tile_unit<T, BN>(r, c >> 3) + (c & 4) * 2);
    return f32x4{(float)q[0], (float)q[1], (float)q[2], (float)q[3]};
}
// Writes the first `rows` rows of the tile to out, whose rows are `stride`
// elements apart, the columns below `limit`.
template <typename T, int BM, int BN, int THREADS>
__device__ __forceinline__ void tile_write(const lds_char *lds, T *out, int rows, int64_t n0, int64_t limit,
                                           int64_t stride) {
    typedef u32x4 __attribute__((aligned(2))) unit2;
    constexpr int kUnits = BN / 8;
#pragma unroll 4
    for (int i = threadIdx.x; i < BM * kUnits; i += THREADS) {
        const int r = i / kUnits, u = i % kUnits;
        const int64_t n = n0 + u * 8;
        if (r >= rows || n >= limit) continue;
        union {
            u32x4 v;
            T e[8];
        } x;
        x.v = *reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>(lds + tile_unit<T, BN>(r, u));
        T *to = out + r * stride + n;
        if (n + 8 <= limit) {
            *(__attribute__((address_space(1))) unit2 *)to = x.v;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n + e < limit) to[e] = x.e[e];
        }
    }
}

// Turns a tile of 16-bit elements in LDS: BM rows of BN in the places of
// tile_put become BN rows of BM.  Every thread holds its share in registers
// between two barriers; 16 lanes read 4 x 16 elements transposed at a time.
template <typename T, int BM, int BN, int THREADS>
__device__ __forceinline__ void tile_turn(lds_char *lds, int wave, int lane) {
    constexpr int kUnits = BM / 8 * BN / THREADS;  // of 8 elements, per thread
    static_assert(kUnits >= 1 && BM / 8 * BN % THREADS == 0 && BN % 16 == 0, "whole units");
    const int group = wave * 4 + (lane >> 4), l = lane & 15;
    union {
        s16x4 h[2];
        u32x4 v;
    } x[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int at = i * (THREADS / 16) + group, ru = at % (BM / 8), cb = at / (BM / 8);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = ru * 8 + h * 4 + (l >> 2), c = cb * 16 + (l & 3) * 4;
            x[i].h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)(lds + tile_unit<T, BN>(r, c >> 3) + (c & 4) * 2));
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int at = i * (THREADS / 16) + group, ru = at % (BM / 8), cb = at / (BM / 8);
        *reinterpret_cast<__attribute__((address_space(3))) u32x4 *>(lds + tile_unit<T, BM>(cb * 16 + l, ru)) = x[i].v;
    }
    __syncthreads();
}

// ---------------------------------------------------------- which tile to take
//
// A kernel's time is its rounds over the CUs, each an overhead (loads until the
// first product, the epilogue) and a part that grows with k; small tiles have less
// of the one and more of the other.  The constants are fitted to measured times
// (gated.hip and loss.hip have tables of these).
struct TileCost {
    int rows, columns, each;    // of a tile (columns: rows of the weights); tiles that a CU holds
    double fixed, alone, full;  // us of a round; per 1,024 of k: with one tile on the CU, with `each`
};
constexpr TileCost kTileCosts[] = {{256, 256, 1, 13, 24.8, 24.8},
                                   {128, 256, 1, 6, 15.7, 15.7},
                                   {128, 128, 2, 2.5, 12, 18.3},
                                   {64, 64, 3, 2.9, 5, 9}};
// us of `tiles` tiles, where a round takes `more` us more; EXACT: so many there are
// for certain (uneven segments: the last round is seldom full, and tiles that just
// fit one round do not always).
inline double tile_time(const TileCost &g, double more, int64_t k, double tiles, bool exact) {
    const double kk = (double)k / 1024, fixed = g.fixed + more, whole = fixed + kk * g.full;
    auto part = [&](int n) {  // a round of n tiles a CU
        return fixed + kk * (g.each > 1 ? g.alone + (g.full - g.alone) * (n - 1) / (g.each - 1) : g.full);
    };
    const double load = tiles / 256, x = load / g.each;
    if (x <= 0.92) return part((int)std::ceil(load));
    if (exact) {
        const int64_t n = (int64_t)std::ceil(load);
        return (double)(n / g.each) * whole + (n % g.each ? part((int)(n % g.each)) : 0);
    }
    return whole * (x <= 1 ? 1.35 : x < 2 ? 2 : x + 0.4);
}

}  // namespace segred
