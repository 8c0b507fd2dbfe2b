// adapter.hip -- a projection that all rows share with a low-rank adapter per
// segment beside it: out[r] = x[r] W + scale_a (x[r] A_a) B_a, a the adapter
// of r's segment.
//
// Two kernels.  adapter_low computes u = scale (x A) per segment, 32 ranks a
// workgroup, the contraction split over its waves.  adapter_main computes
// x W over tiles of rows that may span many segments and goes on, in the same
// accumulators, with one step per adapter met in the tile: u's rows of that
// adapter (zeros for the others) times B_a.  So x and W are read once, out is
// written once, and each adapter costs a few steps.
//
// u is kept in more bits than the inputs have: for 16-bit inputs as the sum of
// two bf16 (2^-17 relative), stored as [hi 32 | lo 32] per 32 ranks, so that
// one step multiplies both halves by the same 32 ranks of B.  float16 B is
// split the same way, because u may leave float16's range.
#include <algorithm>
#include <type_traits>

#include "internal.hpp"
#include "tile.hpp"

namespace segred {

struct AdapterArgs {
    const char *values;   // [N, K]
    const char *weights;  // [M, K] (row form) or [K, M] (col form)
    const char *first;    // [L, R, K] or [L, K, R]
    const char *second;   // [L, M, R2] or [L, R, M]
    const int64_t *offsets, *which;
    const float *scale;   // [L] or null
    int64_t S, N, K, M, L, R;
    int64_t R2;           // ranks between rows of `second`: R, or more where it is a copy
    const char *copy_from;  // the caller's second factor, where `second` is a copy of it
    int copy_rows;          // rows of it per workgroup
    int64_t slots, mtiles, ntiles, blocks;  // blocks: ceil(R / 32)
    char *u;              // [N, blocks * 128 bytes]
    int32_t *ids;         // [N] adapter of each row, -1: none
    char *low;            // [N, R] or null
    int low_f32;          // of float, else of the inputs' type
    char *out;
    int vec;
};

constexpr int kRankBlock = 32;

// Rows of the second factor that do not hold whole 16-byte units are copied,
// with zeros behind them, for the adapters that some segment has: by the
// workgroups of its first segment, kCopyRows rows each, or as many as have at
// most kCopyPart elements (at least one row, of up to 2^24): indexes inside a
// workgroup's part have 32 bits.
constexpr int64_t kCopyRows = 512, kCopyPart = int64_t(1) << 24;
template <typename T>
__device__ __forceinline__ void copy_second(const AdapterArgs &a, int64_t wg, int threads) {
    const int64_t per = (a.M + a.copy_rows - 1) / a.copy_rows, s = wg / per, m0 = (wg - s * per) * a.copy_rows;
    const int64_t adapter = a.which[s];
    if (adapter < 0 || adapter >= a.L) return;
    const int lane = threadIdx.x & 63;
    for (int64_t q = 0; q < s; q += 64)
        if (ballot(q + lane < s && a.which[q + lane] == adapter) != 0) return;
    const int R = (int)a.R, R2 = (int)a.R2, rows = (int)min((int64_t)a.copy_rows, a.M - m0);
    const T *from = reinterpret_cast<const T *>(a.copy_from) + (adapter * a.M + m0) * R;
    T *to = reinterpret_cast<T *>(const_cast<char *>(a.second)) + (adapter * a.M + m0) * R2;
    for (int i = threadIdx.x; i < rows * R2; i += threads) {
        const int r = i / R2, c = i - r * R2;
        to[i] = c < R ? from[r * R + c] : (T)0.f;
    }
}

template <typename T, int MT, int NW, int STAGES, bool B_COL, bool DIRECT>
__global__ __launch_bounds__(64 * NW) void adapter_low(AdapterArgs a) {
    constexpr int BM = 16 * MT, BN = kRankBlock, NT = 2;
    constexpr int kLg = __builtin_ctz(BM);
    using AStage = RowStage<T, BM, 64, DIRECT>;
    using BRow = RowStage<T, BN, 64, DIRECT>;
    using BCol = ColStage<T, BN, 64, DIRECT>;
    constexpr int kABytes = AStage::kBytes;
    constexpr int kStageBytes = kABytes + (B_COL ? BCol::kBytes : BRow::kBytes);
    constexpr int kLoads = AStage::kLoads + (B_COL ? BCol::kLoads : BRow::kLoads);
    __shared__ __attribute__((aligned(1024))) char lds_mem[NW * STAGES * kStageBytes];
    lds_char *lds = (lds_char *)lds_mem;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t launch = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (launch >= a.slots * a.blocks) {
        if (a.copy_from && launch < a.slots * a.blocks + a.S * ((a.M + a.copy_rows - 1) / a.copy_rows))
            copy_second<T>(a, launch - a.slots * a.blocks, 64 * NW);
        return;
    }
    const int64_t id = xcd_tile(a.slots * a.blocks);
    const int64_t slot = id / a.blocks, block = id - slot * a.blocks;
    const int r0 = (int)block * kRankBlock;
    const int64_t s = tight_segment(a.offsets, a.S, kLg, slot, lane);
    const int64_t row0 = a.offsets[s] + ((slot - tight_key(a.offsets, s, kLg)) << kLg);
    const int64_t end = min(a.offsets[s + 1], a.N);
    if (row0 >= end || row0 < 0) return;
    const int rows = (int)min((int64_t)BM, end - row0);
    const int64_t adapter = a.which[s];
    const bool has = adapter >= 0 && adapter < a.L;
    if (block == 0)
        for (int r = threadIdx.x; r < rows; r += 64 * NW) a.ids[row0 + r] = has ? (int32_t)adapter : -1;
    const int K = (int)a.K, R = (int)a.R;
    if (!has) {
        if (a.low)
            for (int i = threadIdx.x; i < rows * kRankBlock; i += 64 * NW) {
                const int64_t at = (row0 + i / kRankBlock) * R + r0 + i % kRankBlock;
                if (r0 + i % kRankBlock >= R) continue;
                if (a.low_f32) reinterpret_cast<float *>(a.low)[at] = 0.f;
                else reinterpret_cast<T *>(a.low)[at] = (T)0.f;
            }
        return;
    }

    AStage sa;
    sa.init(0, lane, K, [&](int r) -> const char * {
        return r < rows ? a.values + (row0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
    });
    const char *w = a.first + adapter * a.K * a.R * (int64_t)sizeof(T);
    BRow sbr;
    BCol sbc;
    uint64_t wp[BCol::kLoads];
    int wleft[BCol::kLoads];
    if constexpr (B_COL) {
#pragma unroll
        for (int i = 0; i < BCol::kLoads; ++i) {
            const int n = r0 + BCol::col(i, 0, lane);
            wp[i] = (uint64_t)(w + (BCol::row(i, 0, lane) * a.R + n) * (int64_t)sizeof(T));
            wleft[i] = R - n;
        }
    } else {
        sbr.init(0, lane, K, [&](int r) -> const char * {
            return r0 + r < R ? w + (r0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
        });
    }
    f32x4 acc[MT][NT] = {};
    const int steps = (K + kStep<T> - 1) / kStep<T>;
    wave_steps<STAGES, DIRECT, kLoads, kStageBytes>(
        lds + wave * STAGES * kStageBytes, wave * steps / NW, (wave + 1) * steps / NW,
        [&](int t, bool live, lds_char *buf) {
            const int k0 = live ? t * kStep<T> : K;
            sa.issue(buf, 0, k0);
            if constexpr (B_COL) {
                const uint64_t step = (uint64_t)k0 * a.R * sizeof(T);
                sbc.issue(
                    buf + kABytes, 0, [&](int i) { return wp[i] + step; },
                    [&](int i) { return k0 + BCol::row(i, 0, lane) < K ? wleft[i] : 0; });
            } else {
                sbr.issue(buf + kABytes, 0, k0);
            }
        },
        [&](lds_char *buf) {
            sa.commit(buf, 0, lane);
            if constexpr (B_COL) sbc.commit(buf + kABytes, 0, lane);
            else sbr.commit(buf + kABytes, 0, lane);
        },
        [&](int, const lds_char *buf) {
            step_products<T, MT, NT, false, BM, B_COL, BN>(acc, buf, buf + kABytes, 0, 0, lane);
        },
        [] {});
    const float scale = a.scale ? a.scale[adapter] : 1.f;
    join_waves<NW, MT, NT>(lds, acc, wave, lane, [&](int r, int c, f32x4 sum) {
        if (r >= rows) return;
        sum *= scale;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r0 + c + j >= R) sum[j] = 0.f;  // not an infinite row's 0 * inf
        char *u = a.u + ((row0 + r) * a.blocks + block) * 128;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<f32x4 *>(u + c * 4) = sum;
        } else {
            bf16x4 hi, lo;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // a float above the largest bf16 would round to an infinity
                constexpr float kMost = 0x1.fep127f;
                hi[j] = (__bf16)(sum[j] * 0.f == 0.f ? fminf(fmaxf(sum[j], -kMost), kMost) : sum[j]);
                const float rest = sum[j] - (float)hi[j];  // NaN beside an infinity
                lo[j] = (__bf16)(rest == rest ? rest : 0.f);
            }
            *reinterpret_cast<bf16x4 *>(u + c * 2) = hi;
            *reinterpret_cast<bf16x4 *>(u + 64 + c * 2) = lo;
        }
        if (a.low && a.low_f32)
            store_quad<float>(reinterpret_cast<float *>(a.low) + (row0 + r) * R, r0 + c, R, sum, false);
        else if (a.low)
            store_quad<T>(reinterpret_cast<T *>(a.low) + (row0 + r) * R, r0 + c, R, sum, false);
    });
}

// The steps of an output tile after those of x W: rows of u against the
// adapters met in the tile.
template <typename T, int BM, int BN, int THREADS, bool B_COL, bool DIRECT>
struct AdapterSteps {
    using AS = RowStage<T, BM, THREADS, DIRECT>;
    using BR = RowStage<T, BN, THREADS, DIRECT>;
    using BC = ColStage<T, BN, THREADS, DIRECT>;
    uint64_t up[AS::kLoads];
    int rid[AS::kLoads];

    __device__ __forceinline__ void init(const AdapterArgs &a, const int *s_ids, int64_t row0, int wave, int lane) {
        const int unit = (lane & 7) ^ (lane >> 3);
#pragma unroll
        for (int i = 0; i < AS::kLoads; ++i) {
            const int r = AS::group(i, wave) * 8 + (lane >> 3);
            rid[i] = s_ids[r];
            up[i] = (uint64_t)(a.u + (row0 + r) * a.blocks * 128 + unit * 16);
        }
    }
    __device__ __forceinline__ void issue(AS &sa, BR &sbr, BC &sbc, const AdapterArgs &a, lds_char *buf, int adapter,
                                          int block, int64_t n0, int wave, int lane) {
        const uint64_t zeros = (uint64_t)zero_unit();
#pragma unroll
        for (int i = 0; i < AS::kLoads; ++i) {
            const bool mine = rid[i] == adapter;
            const uint64_t q = up[i] + (uint64_t)block * 128;
            if constexpr (DIRECT) load_to_lds(mine ? q : zeros, buf + AS::group(i, wave) * 1024);
            else sa.v[i] = load_unit<T>(q, mine ? kUnit<T> : 0);
        }
        lds_char *bb = buf + AS::kBytes;
        const char *w = a.second + (int64_t)adapter * a.M * a.R2 * (int64_t)sizeof(T);
        const int R = (int)a.R, M = (int)a.M;
        constexpr int kMask = kRankBlock - 1;
        if constexpr (B_COL) {
            auto rank = [&](int i) { return block * kRankBlock + (BC::row(i, wave, lane) & kMask); };
            sbc.issue(
                bb, wave,
                [&](int i) { return (uint64_t)(w + (rank(i) * a.M + n0 + BC::col(i, wave, lane)) * (int64_t)sizeof(T)); },
                [&](int i) { return rank(i) < R ? M - (int)n0 - BC::col(i, wave, lane) : 0; });
        } else {
            const int rank = block * kRankBlock + ((((lane & 7) ^ (lane >> 3)) * kUnit<T>) & kMask);
#pragma unroll
            for (int i = 0; i < BR::kLoads; ++i) {
                const int64_t n = n0 + BR::group(i, wave) * 8 + (lane >> 3);
                const uint64_t q = (uint64_t)(w + (n * a.R2 + rank) * (int64_t)sizeof(T));
                const int left = n < a.M ? R - rank : 0;
                if constexpr (DIRECT) load_to_lds(left > 0 ? q : zeros, bb + BR::group(i, wave) * 1024);
                else sbr.v[i] = load_unit<T>(q, left);
            }
        }
    }
};

// Products of an adapter step: bf16 halves of u against B's two bf16 halves.
template <int MT, int NT, bool B_COL, int BW>
__device__ __forceinline__ void split_products(f32x4 (&acc)[MT][NT], const lds_char *la, const lds_char *lb, int m0,
                                               int n0, int lane) {
    bf16x8 hi[NT], lo[NT];
    u32x4 b[1][NT];
    if constexpr (B_COL) col_frags<_Float16, BW>(b, lb, n0, lane);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if constexpr (!B_COL) b[0][j] = row_frag(lb, n0 + 16 * j, 0, lane);
        const f16x8 h = __builtin_bit_cast(f16x8, b[0][j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            hi[j][e] = (__bf16)(float)h[e];
            lo[j][e] = (__bf16)((float)h[e] - (float)hi[j][e]);
        }
    }
    u32x4 u[2][MT];
    row_frags(u, la, m0, lane);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const bf16x8 a = __builtin_bit_cast(bf16x8, u[ks][i]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi[j], a, acc[i][j], 0, 0, 0);
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo[j], a, acc[i][j], 0, 0, 0);
            }
        }
}

// The products of an adapter's step with all rows of a tile, added where a row
// has that adapter: elsewhere u is zero, but an infinity or a NaN of the
// adapter would make something of it.  A lane holds columns of the rows
// m0 + 16 i + lane % 16.
template <typename T, int MT, int NT, bool B_COL, int BM, int BW>
__device__ __forceinline__ void adapter_products(f32x4 (&acc)[MT][NT], const lds_char *la, const lds_char *lb, int m0,
                                                 int n0, int lane, const int *s_ids, int adapter) {
    f32x4 part[MT][NT] = {};
    if constexpr (__is_same(T, _Float16)) split_products<MT, NT, B_COL, BW>(part, la, lb, m0, n0, lane);
    else step_products<T, MT, NT, false, BM, B_COL, BW>(part, la, lb, m0, n0, lane);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const bool mine = s_ids[m0 + 16 * i + (lane & 15)] == adapter;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] += mine ? part[i][j][e] : 0.f;
    }
}

// Fills s_ids (adapter of each tile row, -1: none) and s_list (the adapters
// met, in row order); returns their number.  All threads must call it.
template <int BM, int THREADS>
__device__ __forceinline__ int tile_adapters(const AdapterArgs &a, int64_t row0, int rows, int *s_ids, int *s_list,
                                             int *s_count) {
    const int tid = threadIdx.x;
    for (int r = tid; r < BM; r += THREADS) {
        const int id = r < rows ? a.ids[row0 + r] : -1;
        s_ids[r] = id < a.L ? id : -1;
    }
    if (tid == 0) *s_count = 0;
    __syncthreads();
    if (tid < 64) {  // one wave walks the rows, 64 at a time
        int n = 0;
        for (int b = 0; b < BM; b += 64) {
            const int id = b + tid < BM ? s_ids[b + tid] : -1;
            bool first = id >= 0;
            for (int q = 0; q < n; ++q) first = first && s_list[q] != id;
            const int most = BM - b < 64 ? BM - b : 64;
            for (int q = 0; q < most - 1; ++q) first = first && (q >= tid || __builtin_amdgcn_readlane(id, q) != id);
            const uint64_t m = ballot(first);
            if (first) s_list[n + popc64(m & ((uint64_t(1) << tid) - 1))] = id;
            wave_lds_sync();
            n += popc64(m);
        }
        if (tid == 0) *s_count = n;
    }
    __syncthreads();
    return *s_count;
}

// A tile of the output; s_ids and s_list as tile_adapters leaves them.
template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool B_COL, bool DIRECT>
struct AdapterTile {
    static_assert(DIRECT || STAGES == 2, "units that pass through registers use two buffers");
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    using Steps = AdapterSteps<T, BM, BN, kThreads, B_COL, DIRECT>;
    using AStage = typename Steps::AS;
    using BRow = typename Steps::BR;
    using BCol = typename Steps::BC;
    static constexpr int kABytes = AStage::kBytes;
    static constexpr int kStageBytes = kABytes + (B_COL ? BCol::kBytes : BRow::kBytes);
    static constexpr int kLoads = AStage::kLoads + (B_COL ? BCol::kLoads : BRow::kLoads);
    static constexpr int kLds = STAGES * kStageBytes;

    static __device__ __forceinline__ void run(const AdapterArgs &a, int64_t row0, int rows, int64_t n0, int met,
                                               const int *s_ids, const int *s_list, lds_char *lds, int wave, int lane) {
        const int K = (int)a.K;
        AStage sa;
        sa.init(wave, lane, K, [&](int r) -> const char * {
            return r < rows ? a.values + (row0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
        });
        BRow sbr;
        BCol sbc;
        uint64_t wp[BCol::kLoads];
        int wleft[BCol::kLoads];
        if constexpr (B_COL) {
#pragma unroll
            for (int i = 0; i < BCol::kLoads; ++i) {
                const int64_t n = n0 + BCol::col(i, wave, lane);
                wp[i] = (uint64_t)(a.weights + (BCol::row(i, wave, lane) * a.M + n) * (int64_t)sizeof(T));
                wleft[i] = (int)(a.M - n);
            }
        } else {
            sbr.init(wave, lane, K, [&](int r) -> const char * {
                return n0 + r < a.M ? a.weights + (n0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
            });
        }
        Steps extra;
        extra.init(a, s_ids, row0, wave, lane);
        const int base = (K + kStep<T> - 1) / kStep<T>, blocks = (int)a.blocks;
        const int steps = base + met * blocks;
        auto issue = [&](int t, lds_char *buf) {
            if (t < base || t >= steps) {  // past the last step: zeros, as past the contraction
                const int k0 = min(t, base) * kStep<T>;
                sa.issue(buf, wave, k0);
                if constexpr (B_COL) {
                    const uint64_t step = (uint64_t)k0 * a.M * sizeof(T);
                    sbc.issue(
                        buf + kABytes, wave, [&](int i) { return wp[i] + step; },
                        [&](int i) { return k0 + BCol::row(i, wave, lane) < K ? wleft[i] : 0; });
                } else {
                    sbr.issue(buf + kABytes, wave, k0);
                }
            } else {
                const int e = (t - base) / blocks;
                extra.issue(sa, sbr, sbc, a, buf, __builtin_amdgcn_readfirstlane(s_list[e]), (t - base) - e * blocks, n0,
                            wave, lane);
            }
        };
        auto commit = [&](lds_char *buf) {
            sa.commit(buf, wave, lane);
            if constexpr (B_COL) sbc.commit(buf + kABytes, wave, lane);
            else sbr.commit(buf + kABytes, wave, lane);
        };

        f32x4 acc[MT][NT] = {};
        const int m_w = wave / WN * (MT * 16), n_w = wave % WN * (NT * 16);
        auto products = [&](int t, const lds_char *buf, auto extra) {
            if constexpr (decltype(extra)::value)
                adapter_products<T, MT, NT, B_COL, BM, BN>(acc, buf, buf + kABytes, m_w, n_w, lane, s_ids,
                                                           s_list[(t - base) / blocks]);
            else
                step_products<T, MT, NT, false, BM, B_COL, BN>(acc, buf, buf + kABytes, m_w, n_w, lane);
        };
        if constexpr (DIRECT) {
#pragma unroll
            for (int t = 0; t < STAGES - 1; ++t) issue(t, lds + t * kStageBytes);
            int cur = 0, fill = STAGES - 1;
            auto step = [&](int t, auto extra) {
                wait_and_meet<(STAGES - 2) * kLoads>();
                issue(t + STAGES - 1, lds + fill * kStageBytes);
                products(t, lds + cur * kStageBytes, extra);
                cur = cur + 1 == STAGES ? 0 : cur + 1;
                fill = fill + 1 == STAGES ? 0 : fill + 1;
            };
            for (int t = 0; t < base; ++t) step(t, std::false_type{});
            for (int t = base; t < steps; ++t) step(t, std::true_type{});
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the zeros past the last step
        } else {
            issue(0, lds);
            commit(lds);
            auto step = [&](int t, auto extra) {
                __syncthreads();
                if (t + 1 < steps) issue(t + 1, lds);
                products(t, lds + (t & 1) * kStageBytes, extra);
                if (t + 1 < steps) commit(lds + ((t + 1) & 1) * kStageBytes);
            };
            for (int t = 0; t < base; ++t) step(t, std::false_type{});
            for (int t = base; t < steps; ++t) step(t, std::true_type{});
        }

        T *out = reinterpret_cast<T *>(a.out) + row0 * a.M;
        if constexpr (sizeof(T) == 2) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    tile_put<T, BN>(lds, m_w + 16 * i + (lane & 15), n_w + 16 * j + (lane >> 4) * 4, acc[i][j]);
            __syncthreads();
            tile_out<T, BM, BN, kThreads>(lds, out, rows, n0, a.M, a.vec != 0);
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int r = m_w + 16 * i + (lane & 15);
                if (r < rows)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        store_quad<T>(out + r * a.M, n0 + n_w + 16 * j + (lane >> 4) * 4, a.M, acc[i][j], a.vec != 0);
            }
        }
    }
};

// The output tile of a workgroup.
struct AdapterPlace {
    int64_t row0, n0;
    int rows;  // 0: nothing to do
};
__device__ __forceinline__ AdapterPlace adapter_place(const AdapterArgs &a, int bm, int bn) {
    AdapterPlace p{0, 0, 0};
    const int64_t total = a.mtiles * a.ntiles, id = xcd_tile(total);
    if (id >= total) return p;
    const TilePlace at = tile_place(id, a.mtiles, a.ntiles);
    p.row0 = a.offsets[0] + at.m * bm;
    p.n0 = at.n * bn;
    const int64_t end = min(a.offsets[a.S], a.N);
    if (p.row0 >= 0 && p.row0 < end) p.rows = (int)min((int64_t)bm, end - p.row0);
    return p;
}

template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool B_COL, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN) void adapter_main(AdapterArgs a) {
    using Tile = AdapterTile<T, BM, BN, WM, WN, STAGES, B_COL, DIRECT>;
    // one array: beside a second the compiler's reads of LDS wait for all loads
    // into it, also for those of later steps
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds + (2 * BM + 1) * sizeof(int)];
    int *s_ids = reinterpret_cast<int *>(lds_mem + Tile::kLds), *s_list = s_ids + BM, *s_count = s_list + BM;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const AdapterPlace p = adapter_place(a, BM, BN);
    if (p.rows == 0) return;
    const int met = tile_adapters<BM, Tile::kThreads>(a, p.row0, p.rows, s_ids, s_list, s_count);
    Tile::run(a, p.row0, p.rows, p.n0, met, s_ids, s_list, (lds_char *)lds_mem, wave, lane);
}

// The same for float, in bf16 parts; a tile with a sum that is not finite is
// computed again with float products.
constexpr int kSplitThreads = 256;
template <int BN, bool B_COL, bool WHOLE>
__global__ __launch_bounds__(kSplitThreads, 3) void adapter_main_split(AdapterArgs a) {
    constexpr int BM = 64;
    static_assert(kSplitK == kRankBlock, "a step is a block of ranks");
    using Plain = AdapterTile<float, BM, 64, 2, 2, 2, B_COL, false>;
    using SA = SplitStage<BM, kSplitThreads, false, WHOLE>;
    using SB = SplitStage<BN, kSplitThreads, B_COL, WHOLE>;
    constexpr int MT = BM / 32, NT = BN / 32, kSplitLds = 3 * (SA::kPlane + SB::kPlane);
    constexpr int kLds = kSplitLds > Plain::kLds ? kSplitLds : Plain::kLds;
    __shared__ __attribute__((aligned(1024))) char lds_mem[kLds + (2 * BM + 1) * sizeof(int)];
    int *s_ids = reinterpret_cast<int *>(lds_mem + kLds), *s_list = s_ids + BM, *s_count = s_list + BM;
    lds_char *lds = (lds_char *)lds_mem;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const AdapterPlace p = adapter_place(a, BM, BN);
    if (p.rows == 0) return;
    const int met = tile_adapters<BM, kSplitThreads>(a, p.row0, p.rows, s_ids, s_list, s_count);

    const int K = (int)a.K, M = (int)a.M, R = (int)a.R;
    SA sa;
    SB sb;
    uint64_t ap[SA::kParts], bp[SB::kParts];
    int aleft[SA::kParts], bleft[SB::kParts];
#pragma unroll
    for (int i = 0; i < SA::kParts; ++i) {
        const int r = SA::row(i, tid), c = SA::at(i, tid);
        ap[i] = (uint64_t)(a.values + ((p.row0 + r) * a.K + c) * 4);
        aleft[i] = r < p.rows ? K - c : 0;
    }
#pragma unroll
    for (int i = 0; i < SB::kParts; ++i) {
        const int64_t r = SB::row(i, tid), c = SB::at(i, tid);
        if constexpr (B_COL) {
            bp[i] = (uint64_t)(a.weights + (r * a.M + p.n0 + c) * 4);
            bleft[i] = (int)(a.M - p.n0 - c);
        } else {
            bp[i] = (uint64_t)(a.weights + ((p.n0 + r) * a.K + c) * 4);
            bleft[i] = p.n0 + r < a.M ? K - (int)c : 0;
        }
    }
    const int base = (K + kSplitK - 1) / kSplitK, blocks = (int)a.blocks;
    f32x4 acc[MT][NT] = {};
    const int m_w = wave / 2 * (BM / 2), n_w = wave % 2 * (BN / 2);
    split_steps(
        base + met * blocks,
        [&](int64_t step) {
            const int t = (int)step;
            if (t < base) {
                const int k0 = t * kSplitK;
                sa.issue([&](int i) { return ap[i] + (uint64_t)k0 * 4; }, [&](int i) { return aleft[i] - k0; });
                if constexpr (B_COL)
                    sb.issue([&](int i) { return bp[i] + (uint64_t)k0 * M * 4; },
                             [&](int i) { return k0 + SB::row(i, tid) < K ? bleft[i] : 0; });
                else
                    sb.issue([&](int i) { return bp[i] + (uint64_t)k0 * 4; }, [&](int i) { return bleft[i] - k0; });
                return;
            }
            const int e = (t - base) / blocks, rank = ((t - base) - e * blocks) * kRankBlock;
            const int adapter = __builtin_amdgcn_readfirstlane(s_list[e]);
            const char *w = a.second + (int64_t)adapter * a.M * a.R2 * 4;
            sa.issue(
                [&](int i) {
                    return (uint64_t)(a.u + (p.row0 + SA::row(i, tid)) * a.blocks * 128 + (rank + SA::at(i, tid)) * 4);
                },
                [&](int i) { return s_ids[SA::row(i, tid)] == adapter ? 8 : 0; });
            if constexpr (B_COL)
                sb.template issue<false>(
                    [&](int i) { return (uint64_t)(w + ((rank + SB::row(i, tid)) * a.M + p.n0 + SB::at(i, tid)) * 4); },
                    [&](int i) { return rank + SB::row(i, tid) < R ? (int)(a.M - p.n0) - SB::at(i, tid) : 0; });
            else
                sb.template issue<false>(
                    [&](int i) { return (uint64_t)(w + ((p.n0 + SB::row(i, tid)) * a.R2 + rank + SB::at(i, tid)) * 4); },
                    [&](int i) { return p.n0 + SB::row(i, tid) < a.M ? R - rank - SB::at(i, tid) : 0; });
        },
        [&] {
            sa.commit(lds, tid);
            sb.commit(lds + 3 * SA::kPlane, tid);
        },
        [&] { split_step<MT, NT, false, BM, B_COL, BN>(acc, lds, lds + 3 * SA::kPlane, m_w, n_w, lane); });
    if (__syncthreads_or(any_not_finite(acc))) {
        for (int c = 0; c < BN && p.n0 + c < a.M; c += 64) {
            __syncthreads();
            Plain::run(a, p.row0, p.rows, p.n0 + c, met, s_ids, s_list, lds, wave, lane);
        }
        return;
    }
    float *out = reinterpret_cast<float *>(a.out) + p.row0 * a.M;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int r = m_w + 16 * i + (lane & 15);
        if (r < p.rows)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                store_quad<float>(out + r * a.M, p.n0 + n_w + 16 * j + (lane >> 4) * 4, a.M, acc[i][j], a.vec != 0);
    }
}

// Four columns from n of a row's adapter part, u B, in float32.
template <typename T, bool B_COL>
__device__ __forceinline__ f32x4 adapter_quad(const AdapterArgs &a, int64_t row, int adapter, int64_t n) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    const int R = (int)a.R, columns = (int)min((int64_t)4, a.M - n);
    if (adapter < 0 || adapter >= a.L || columns <= 0) return sum;
    constexpr int U = kUnit<T>;
    const char *u = a.u + row * a.blocks * 128;
    const T *b = reinterpret_cast<const T *>(a.second) + (int64_t)adapter * a.M * a.R2;
    for (int r0 = 0; r0 < R; r0 += U) {
        const char *p = u + r0 / kRankBlock * 128 + r0 % kRankBlock * (128 / kRankBlock) / (sizeof(T) == 2 ? 2 : 1);
        float x[U];  // zeros past the rank
        if constexpr (sizeof(T) == 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
            for (int e = 0; e < U; ++e) x[e] = v[e];
        } else {
            const bf16x8 hi = *reinterpret_cast<const bf16x8 *>(p), lo = *reinterpret_cast<const bf16x8 *>(p + 64);
#pragma unroll
            for (int e = 0; e < U; ++e) x[e] = (float)hi[e] + (float)lo[e];
        }
        union Units {
            u32x4 v;
            T e[U];
        };
        if constexpr (B_COL) {
#pragma unroll
            for (int e = 0; e < U; ++e) {
                if (r0 + e >= R) continue;
                Units w;
                w.v = load_unit<T>((uint64_t)(b + (int64_t)(r0 + e) * a.M + n), columns);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] = fmaf(x[e], (float)w.e[j], sum[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= columns) continue;
                Units w;
                w.v = load_unit<T>((uint64_t)(b + (n + j) * a.R2 + r0), R - r0);
#pragma unroll
                for (int e = 0; e < U; ++e) sum[j] = fmaf(x[e], (float)w.e[e], sum[j]);
            }
        }
    }
    return sum;
}

// Few rows: 16 MT rows x 16 columns per workgroup, whose waves split the
// contraction of x W.  The adapters' part, for which every row may have an
// adapter of its own, is added per element instead of in steps: 64 rows with 64
// adapters of rank 16 beside 4,096 x 4,096 took 18 us in steps.
template <typename T, int MT, int NW, int STAGES, bool B_COL>
__global__ __launch_bounds__(64 * NW) void adapter_main_few(AdapterArgs a) {
    static_assert(MT <= NW, "a quad of columns per thread");
    constexpr int BM = 16 * MT, BN = 16;
    using AStage = RowStage<T, BM, 64, true>;
    using BRow = RowStage<T, BN, 64, true>;
    using BCol = ColStage<T, BN, 64, true>;
    constexpr int kABytes = AStage::kBytes;
    constexpr int kStageBytes = kABytes + (B_COL ? BCol::kBytes : BRow::kBytes);
    constexpr int kLoads = AStage::kLoads + (B_COL ? BCol::kLoads : BRow::kLoads);
    __shared__ __attribute__((aligned(1024))) char lds_mem[NW * STAGES * kStageBytes];
    lds_char *lds = (lds_char *)lds_mem;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = xcd_tile(a.mtiles * a.ntiles);
    if (id >= a.mtiles * a.ntiles) return;
    const int64_t n0 = id / a.mtiles * BN;  // row tiles of the same columns of W together
    const int64_t row0 = a.offsets[0] + id % a.mtiles * BM;
    const int64_t end = min(a.offsets[a.S], a.N);
    if (row0 >= end || row0 < 0) return;
    const int rows = (int)min((int64_t)BM, end - row0), K = (int)a.K;

    AStage sa;
    sa.init(0, lane, K, [&](int r) -> const char * {
        return r < rows ? a.values + (row0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
    });
    BRow sbr;
    BCol sbc;
    uint64_t wp[BCol::kLoads];
    int wleft[BCol::kLoads];
    if constexpr (B_COL) {
#pragma unroll
        for (int i = 0; i < BCol::kLoads; ++i) {
            const int64_t n = n0 + BCol::col(i, 0, lane);
            wp[i] = (uint64_t)(a.weights + (BCol::row(i, 0, lane) * a.M + n) * (int64_t)sizeof(T));
            wleft[i] = (int)(a.M - n);
        }
    } else {
        sbr.init(0, lane, K, [&](int r) -> const char * {
            return n0 + r < a.M ? a.weights + (n0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
        });
    }
    f32x4 acc[MT][1] = {}, extra = {0.f, 0.f, 0.f, 0.f};
    const int steps = (K + kStep<T> - 1) / kStep<T>;
    wave_steps<STAGES, true, kLoads, kStageBytes>(
        lds + wave * STAGES * kStageBytes, wave * steps / NW, (wave + 1) * steps / NW,
        [&](int t, bool live, lds_char *buf) {
            const int k0 = live ? t * kStep<T> : steps * kStep<T>;
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
            step_products<T, MT, 1, false, BM, B_COL, BN>(acc, buf, buf + kABytes, 0, 0, lane);
        },
        [&] {
            // this thread's quad in join_waves()
            const int r = wave * 16 + (lane & 15);
            if (wave < MT && r < rows)
                extra = adapter_quad<T, B_COL>(a, row0 + r, a.ids[row0 + r], n0 + (lane >> 4) * 4);
        });
    T *out = reinterpret_cast<T *>(a.out);
    join_waves<NW, MT, 1>(lds, acc, wave, lane, [&](int r, int c, f32x4 sum) {
        if (r < rows) store_quad<T>(out + (row0 + r) * a.M, n0 + c, a.M, sum + extra, a.vec != 0);
    });
}

template <typename T, int MT, int NW, int STAGES>
int adapter_few_launch(AdapterArgs a, bool b_col, hipStream_t st) {
    a.mtiles = (a.N + 16 * MT - 1) / (16 * MT);
    a.ntiles = (a.M + 15) / 16;
    dim3 grid;
    if (!tile_grid(a.mtiles * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    if (b_col) timed_launch_ggl(true, (adapter_main_few<T, MT, NW, STAGES, true>), grid, dim3(64 * NW), 0, st, a);
    else timed_launch_ggl(true, (adapter_main_few<T, MT, NW, STAGES, false>), grid, dim3(64 * NW), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

// Many rows: AH * 128 rows x 256 columns per workgroup, in phases (16-bit
// types, whole units).
template <typename T, int AH, bool B_COL>
__global__ __launch_bounds__(kPhaseThreads) void adapter_main_many(AdapterArgs a) {
    using AStage = RowStage<T, kHalf, kPhaseThreads, true>;
    using BRow = RowStage<T, kHalf, kPhaseThreads, true>;
    using BCol = ColStage<T, kHalf, kPhaseThreads, true>;
    constexpr int BM = AH * kHalf;
    // one array: beside a second (__syncthreads_or has one) the compiler's reads
    // of LDS wait for all loads into it, also for those of later steps
    __shared__ __attribute__((aligned(1024))) char lds_mem[kPhaseLds + (2 * BM + 1) * sizeof(int)];
    int *s_ids = reinterpret_cast<int *>(lds_mem + kPhaseLds), *s_list = s_ids + BM, *s_count = s_list + BM;
    lds_char *lds = (lds_char *)lds_mem;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t total = a.mtiles * a.ntiles;
    const int64_t id = xcd_tile(total);
    if (id >= total) return;
    const TilePlace at = tile_place(id, a.mtiles, a.ntiles);
    const int64_t row0 = a.offsets[0] + at.m * BM;
    const int64_t n0 = at.n * (2 * kHalf);
    const int64_t end = min(a.offsets[a.S], a.N);
    if (row0 >= end || row0 < 0) return;
    const int rows = (int)min((int64_t)BM, end - row0);
    const int K = (int)a.K, R = (int)a.R;
    const int met = tile_adapters<BM, kPhaseThreads>(a, row0, rows, s_ids, s_list, s_count);

    AStage sa[AH];
#pragma unroll
    for (int h = 0; h < AH; ++h)
        sa[h].init(wave, lane, K, [&](int r) -> const char * {
            r += h * kHalf;
            return r < rows ? a.values + (row0 + r) * a.K * (int64_t)sizeof(T) : nullptr;
        });
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
                wp[h][i] = (uint64_t)(a.weights + (BCol::row(i, wave, lane) * a.M + n) * (int64_t)sizeof(T));
                wleft[h][i] = (int)(a.M - n);
            }
        } else {
            sbr[h].init(wave, lane, K, [&](int r) -> const char * {
                const int64_t n = n0 + h * kHalf + r;
                return n < a.M ? a.weights + n * a.K * (int64_t)sizeof(T) : nullptr;
            });
        }
    }
    f32x4 acc[2][2][4][2] = {};
    phase_steps<T, AH, B_COL>(
        acc, lds, (K + kStep<T> - 1) / kStep<T>, wave, lane,
        [&](int h, int t, lds_char *place) { sa[h].issue(place, wave, t * kStep<T>); },
        [&](int h, int t, lds_char *place) {
            const int k0 = t * kStep<T>;
            if constexpr (B_COL) {
                const uint64_t step = (uint64_t)k0 * a.M * sizeof(T);
                sbc.issue(
                    place, wave, [&](int i) { return wp[h][i] + step; },
                    [&](int i) { return k0 + BCol::row(i, wave, lane) < K ? wleft[h][i] : 0; });
            } else {
                sbr[h].issue(place, wave, k0);
            }
        },
        [](f32x4 (&c)[4][2], const u32x4 (&x)[2][4], const u32x4 (&y)[2][2]) { quadrant<T>(c, x, y); });
    __syncthreads();

    // the adapters met in the tile, 32 ranks a step
    const int blocks = (int)a.blocks, extra = met * blocks;
    const int unit = (lane & 7) ^ (lane >> 3);
    auto adapter_of = [&](int t, int &block) {
        const int e = t / blocks;
        block = t - e * blocks;
        return __builtin_amdgcn_readfirstlane(s_list[e]);
    };
    auto fetch_u = [&](int h, int t, lds_char *place) {
        int block = 0;
        const int adapter = t < extra ? adapter_of(t, block) : -2;  // past the last step: zeros
#pragma unroll
        for (int i = 0; i < AStage::kLoads; ++i) {
            const int g = AStage::group(i, wave), r = h * kHalf + g * 8 + (lane >> 3);
            const uint64_t q = (uint64_t)(a.u + ((row0 + r) * a.blocks + block) * 128 + unit * 16);
            load_to_lds(s_ids[r] == adapter ? q : (uint64_t)zero_unit(), place + g * 1024);
        }
    };
    auto fetch_second = [&](int h, int t, lds_char *place) {
        int block = 0;
        const int adapter = t < extra ? adapter_of(t, block) : -1;
        const int have = adapter >= 0 ? R - block * kRankBlock : 0;  // ranks of this step
        const char *w = a.second + ((int64_t)max(adapter, 0) * a.M * a.R2) * (int64_t)sizeof(T);
        constexpr int kMask = kRankBlock - 1;
        if constexpr (B_COL) {
            auto rank = [&](int i) { return BCol::row(i, wave, lane) & kMask; };
            auto col = [&](int i) { return n0 + h * kHalf + BCol::col(i, wave, lane); };
            sbc.issue(
                place, wave,
                [&](int i) { return (uint64_t)(w + ((block * kRankBlock + rank(i)) * a.M + col(i)) * (int64_t)sizeof(T)); },
                [&](int i) { return rank(i) < have ? (int)(a.M - col(i)) : 0; });
        } else {
            const int rank = (unit * kUnit<T>) & kMask;
#pragma unroll
            for (int i = 0; i < BRow::kLoads; ++i) {
                const int g = BRow::group(i, wave);
                const int64_t n = n0 + h * kHalf + g * 8 + (lane >> 3);
                const uint64_t q = (uint64_t)(w + (n * a.R2 + block * kRankBlock + rank) * (int64_t)sizeof(T));
                load_to_lds(n < a.M && rank < have ? q : (uint64_t)zero_unit(), place + g * 1024);
            }
        }
    };
    auto products = [&](f32x4 (&c)[4][2], const u32x4 (&x)[2][4], const u32x4 (&y)[2][2]) {
        if constexpr (__is_same(T, _Float16)) {
            // bf16 halves of u against the two bf16 that a float16 is the sum
            // of; y[1] holds the same ranks again, so wait for it here
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f16x8 h = __builtin_bit_cast(f16x8, y[0][j]);
                bf16x8 hi, lo;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    hi[e] = (__bf16)(float)h[e];
                    lo[e] = (__bf16)((float)h[e] - (float)hi[e]);
                }
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bf16x8 v = __builtin_bit_cast(bf16x8, x[ks][i]);
                        c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, v, c[i][j], 0, 0, 0);
                        c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, v, c[i][j], 0, 0, 0);
                    }
            }
        } else {
            quadrant<T>(c, x, y);
        }
    };
    if (extra > 0) {
        phase_steps<T, AH, B_COL>(acc, lds, extra, wave, lane, fetch_u, fetch_second, products);
        // Where rows differ in their adapter, an infinity or a NaN of one has
        // reached the rows of others, and the tile is computed again in those of
        // 64 x 128, which keep parts of their own.  (Such parts do not fit the
        // registers here; looking for these values in every step took 5% of a
        // call.)  6,000 rows of 12 requests beside 4,096 x 2,048, rank 64: 130 us,
        // and 380 where one of eight adapters is NaN.
        bool mixed = met > 1;
        for (int r = lane; r < rows; r += 64) mixed = mixed || s_ids[r] < 0;
        float bad = 0.f;
#pragma unroll
        for (int p = 0; p < AH; ++p)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) bad = not_finite(acc[p][q][i][j], bad);
        if (ballot(mixed) != 0 && bad != 0.f) *s_count = -1;
    }

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
    tile_out<T, BM, BN, kPhaseThreads>(lds, reinterpret_cast<T *>(a.out) + row0 * a.M, rows, n0, a.M, a.vec != 0);
    if (*s_count < 0) {
        using Again = AdapterTile<T, 64, 128, 2, 4, 3, B_COL, true>;
        static_assert(Again::kThreads == kPhaseThreads && Again::kLds <= kPhaseLds, "the same workgroup and LDS");
#pragma unroll 1
        for (int r = 0; r < rows; r += 64)
#pragma unroll 1
            for (int c = 0; c < BN && n0 + c < a.M; c += 128) {
                __syncthreads();
                Again::run(a, row0 + r, min(64, rows - r), n0 + c, met, s_ids + r, s_list, lds, wave, lane);
            }
    }
}

template <typename T, int AH>
int adapter_many_launch(AdapterArgs a, bool b_col, hipStream_t st) {
    a.mtiles = (a.N + AH * kHalf - 1) / (AH * kHalf);
    a.ntiles = (a.M + 2 * kHalf - 1) / (2 * kHalf);
    dim3 grid;
    if (!tile_grid(a.mtiles * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    if constexpr (AH == 1)
        if (b_col) {
            timed_launch_ggl(true, (adapter_main_many<T, 1, true>), grid, dim3(kPhaseThreads), 0, st, a);
            return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
        }
    timed_launch_ggl(true, (adapter_main_many<T, AH, false>), grid, dim3(kPhaseThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

template <typename T, int BM, int BN, int WM, int WN, int STAGES, bool DIRECT>
int adapter_main_launch(AdapterArgs a, bool b_col, hipStream_t st) {
    a.mtiles = (a.N + BM - 1) / BM;
    a.ntiles = (a.M + BN - 1) / BN;
    dim3 grid;
    if (!tile_grid(a.mtiles * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    constexpr int kThreads = 64 * WM * WN;
    if (b_col) timed_launch_ggl(true, (adapter_main<T, BM, BN, WM, WN, STAGES, true, DIRECT>), grid, dim3(kThreads), 0, st, a);
    else timed_launch_ggl(true, (adapter_main<T, BM, BN, WM, WN, STAGES, false, DIRECT>), grid, dim3(kThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

int adapter_split_launch(AdapterArgs a, bool b_col, hipStream_t st) {
    constexpr int BN = 128;
    a.mtiles = (a.N + 63) / 64;
    a.ntiles = (a.M + BN - 1) / BN;
    dim3 grid;
    if (!tile_grid(a.mtiles * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    const bool whole = a.K % 8 == 0 && (!b_col || a.M % 8 == 0);
    if (b_col && whole) timed_launch_ggl(true, (adapter_main_split<BN, true, true>), grid, dim3(kSplitThreads), 0, st, a);
    else if (b_col) timed_launch_ggl(true, (adapter_main_split<BN, true, false>), grid, dim3(kSplitThreads), 0, st, a);
    else if (whole) timed_launch_ggl(true, (adapter_main_split<BN, false, true>), grid, dim3(kSplitThreads), 0, st, a);
    else timed_launch_ggl(true, (adapter_main_split<BN, false, false>), grid, dim3(kSplitThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

template <typename T, int MT, bool DIRECT>
int adapter_low_launch(AdapterArgs a, bool b_col, hipStream_t st) {
    constexpr int NW = DIRECT ? 4 : 8, STAGES = DIRECT ? 3 : 2;
    a.slots = tight_slots(a.N, a.S, __builtin_ctz(16 * MT));
    dim3 grid;
    const int64_t copies = a.copy_from ? a.S * ((a.M + a.copy_rows - 1) / a.copy_rows) : 0;
    if (!tile_grid(a.slots * a.blocks + copies, grid)) return SEGRED_ERR_UNSUPPORTED;
    if (b_col) timed_launch_ggl(false, (adapter_low<T, MT, NW, STAGES, true, DIRECT>), grid, dim3(64 * NW), 0, st, a);
    else timed_launch_ggl(false, (adapter_low<T, MT, NW, STAGES, false, DIRECT>), grid, dim3(64 * NW), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

constexpr int64_t kAdapterSplit = 320;  // tiles of 64 x 128
constexpr int64_t kAdapterTall = 128;  // tiles of 64 rows
constexpr int64_t kAdapterFew = 128;  // rows up to which waves split the contraction
template <typename T>
int adapter_dispatch(const AdapterArgs &a, bool b_col, bool low_direct, bool main_direct, hipStream_t st) {
    // x A^T in tiles of 16 rows and 32 ranks, of 64 rows where there are ranks
    // for two tiles and enough of them.  bfloat16 beside 4,096 x 256, times of
    // 16 and of 64: 45 us and 48 for 6,000 rows of rank 16; of rank 64, 41 and
    // 43 for 2,048 rows, 48 and 45 for 4,096, 55 and 49 for 6,000.  (Tiles of 16
    // rows by 4 waves, of which a CU holds two; with 8 waves the latter take 60,
    // and calls of 1 to 128 rows the same within 0.8 us.)
    const bool tall = sizeof(T) == 2 && a.blocks > 1 && (a.N / 64 + a.S / 2) * a.blocks >= kAdapterTall;
    int rc;
    if (!low_direct) rc = adapter_low_launch<T, 1, false>(a, b_col, st);
    else if (tall) rc = adapter_low_launch<T, sizeof(T) == 2 ? 4 : 1, true>(a, b_col, st);
    else rc = adapter_low_launch<T, 1, true>(a, b_col, st);
    if (rc != SEGRED_OK) return rc;
    // Up to 128 rows waves split the contraction, in blocks of 16 to 64 rows by as
    // many waves as there is LDS for.  Times in us, every row an adapter of 32, of
    // blocks x waves x stages against tiles of 64 x 64:
    //
    //   rows                                16     32     48     64    128    129
    //   bfloat16, 4,096 x 4,096, rank 16
    //     1x4x4, 1x8x4                17.2/16.9  19/22
    //     2x4x4, 2x8x3                18.3/17.4 18.4/17.9  27/25  27/25
    //     3x4x4, 3x8x2                19.6/18.4 19.8/19.2 20.1/19.8  30/27  40/38  40/37
    //     4x4x3, 4x8x2                20.8/18.8 21.2/19.6 21.1/20.3 20.6/21.1 30.8/30.9 42/39
    //     64 x 64                       44.9   55.7   55.7   55.9   56.2   56.5
    //   the same, transposed
    //     4x4x3, 4x8x2                30.6/28.9 30.1/29.4 31.3/30.7 33.7/31.9 54/50  69/65
    //     64 x 64                       49.5   61.4   61.0   61.1   61.4   61.5
    //   float, 2,048 x 2,048, rank 16
    //     1x4x4, 1x8x4                21.3/19.5 21.4/19.8
    //     4x4x3, 4x8x2                29.1/27.7 29.0/27.5 29.0/27.8 28.5/27.8 29.7/28.6 46/43
    //     64 x 64                       78.4   95.4   95.9   95.5   94.8   95.2
    if (main_direct && a.N <= kAdapterFew) {
        if (a.N <= 16) return adapter_few_launch<T, 1, 8, 4>(a, b_col, st);
        if (a.N <= 32) return adapter_few_launch<T, 2, 8, 3>(a, b_col, st);
        if (a.N <= 48) return adapter_few_launch<T, 3, 4, 4>(a, b_col, st);
        return adapter_few_launch<T, 4, 4, 3>(a, b_col, st);
    }
    // float in bf16 parts from 320 tiles of 64 x 128 on: beside 2,048 x 2,048, 105
    // us against 97 for 1,024 rows (256 tiles), 131 against 177 for 2,048, 424
    // against 625 for 8,192; beside 515 x 1,030, 51 against 48 for 1,024 (144) and
    // 83 against 100 for 4,096 (576)
    if constexpr (sizeof(T) == 4)
        if ((a.N + 63) / 64 * ((a.M + 127) / 128) >= kAdapterSplit) return adapter_split_launch(a, b_col, st);
    if (!main_direct) return adapter_main_launch<T, 64, 64, 2, 2, 2, false>(a, b_col, st);
    if constexpr (sizeof(T) == 2) {
        // tiles of 128 x 256 in phases where there is one for every second CU
        // (bfloat16, 2,048 x 2,048: 1,024 rows take 44 us in phases against 33
        // in 64 x 64, 4,096 rows 55 against 91); 256 rows where that saves a
        // round of 256 CUs, such a tile taking about 7/4 of one of 128
        const int64_t nt = (a.M + 255) / 256, t1 = (a.N + 127) / 128 * nt, t2 = (a.N + 255) / 256 * nt;
        if (a.M >= 256 && t1 >= 128) {
            if (b_col || 4 * ((t1 + 255) / 256) < 7 * ((t2 + 255) / 256)) return adapter_many_launch<T, 1>(a, b_col, st);
            return adapter_many_launch<T, 2>(a, b_col, st);
        }
    }
    return adapter_main_launch<T, 64, 64, 2, 2, 3, true>(a, b_col, st);
}

// Working memory: the rows' adapters, the low-rank rows, and a copy of the
// second factor with whole units where its rows hold none.
struct AdapterSpace {
    size_t ids, low, copy;
    int64_t ranks;  // between rows of the copy
};
AdapterSpace adapter_space(int64_t e, int64_t m, int64_t adapters, int64_t rank, int64_t rows) {
    auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
    AdapterSpace s{};
    s.ids = up((size_t)rows * 4);
    s.low = up((size_t)rows * ((rank + kRankBlock - 1) / kRankBlock) * 128);
    s.ranks = (rank * e + 15) / 16 * 16 / e;
    s.copy = (rank * e) % 16 == 0 ? 0 : (size_t)(adapters * m * s.ranks * e);
    return s;
}

}  // namespace segred

using namespace segred;

extern "C" int64_t segred_adapter_workspace(int32_t dtype, int64_t m, int64_t adapters, int64_t rank, int64_t num_rows) {
    const int64_t e = float_size(dtype);
    if (e == 0 || m < 1 || adapters < 0 || rank < 1 || num_rows < 1 || m > kMaxWidth || rank > kMaxWidth ||
        adapters > INT32_MAX || num_rows > (int64_t(1) << 40) || too_large(num_rows, rank + 64, 4) ||
        too_large(adapters, m * (rank + 8), 4))
        return 0;
    const AdapterSpace s = adapter_space(e, m, adapters, rank, num_rows);
    return (int64_t)(s.ids + s.low + s.copy);
}

extern "C" int segred_adapter(const void *values, int32_t dtype, int64_t k, const void *weights, int64_t m,
                              const int64_t *offsets, const int64_t *which, int64_t num_segments, int64_t num_rows,
                              const void *down, const void *up, const float *scale, int64_t adapters, int64_t rank,
                              int32_t transpose, void *out, void *low, void *workspace, int64_t workspace_bytes,
                              hipStream_t stream) {
    return segred_adapter_mixed(values, dtype, k, weights, m, offsets, which, num_segments, num_rows, down, up, scale,
                                adapters, rank, transpose, out, low, dtype, workspace, workspace_bytes, stream);
}

extern "C" int segred_adapter_mixed(const void *values, int32_t dtype, int64_t k, const void *weights, int64_t m,
                                    const int64_t *offsets, const int64_t *which, int64_t num_segments,
                                    int64_t num_rows, const void *down, const void *up, const float *scale,
                                    int64_t adapters, int64_t rank, int32_t transpose, void *out, void *low,
                                    int32_t low_dtype, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    const int64_t e = float_size(dtype);
    if (dtype < SEGRED_U32 || dtype > SEGRED_F16) return SEGRED_ERR_INVALID_ARGUMENT;
    if (low_dtype != dtype && low_dtype != SEGRED_F32) return SEGRED_ERR_INVALID_ARGUMENT;
    if (k < 1 || m < 1 || rank < 1 || adapters < 0 || num_segments < 0 || num_rows < 0) return SEGRED_ERR_INVALID_ARGUMENT;
    const bool some = num_segments > 0 && num_rows > 0;
    if (some && (!values || !weights || !offsets || !which || !out || (adapters > 0 && (!down || !up))))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (e == 0 || k > kMaxWidth || m > kMaxWidth || rank > kMaxWidth || adapters > INT32_MAX || num_rows > (int64_t(1) << 40))
        return SEGRED_ERR_UNSUPPORTED;
    if (!aligned(values, e) || !aligned(weights, e) || !aligned(out, e) || !aligned(down, e) || !aligned(up, e) ||
        !aligned(low, float_size(low_dtype)) || !aligned(scale, 4) || !aligned(offsets, 8) || !aligned(which, 8) || !aligned(workspace, 16))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (too_large(num_rows, k, 4) || too_large(num_rows, m, 4) || too_large(num_rows, rank, 4) ||
        too_large(num_rows, rank + 64, 4) || too_large(adapters, k * rank, 4) || too_large(adapters, m * (rank + 8), 4))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (!some) return SEGRED_OK;
    const int64_t need = segred_adapter_workspace(dtype, m, adapters, rank, num_rows);
    if (!workspace || workspace_bytes < need) return SEGRED_ERR_INVALID_ARGUMENT;

    AdapterArgs a{};
    a.values = static_cast<const char *>(values);
    a.weights = static_cast<const char *>(weights);
    // forward: down is [L, R, K] and up [L, M, R]; transposed, from [N, M] to
    // [N, K]: up is the first factor, [L, M, R], and down the second
    a.first = static_cast<const char *>(transpose ? up : down);
    a.second = static_cast<const char *>(transpose ? down : up);
    a.offsets = offsets;
    a.which = which;
    a.scale = scale;
    a.S = num_segments;
    a.N = num_rows;
    a.K = transpose ? m : k;
    a.M = transpose ? k : m;
    a.L = adapters;
    a.R = rank;
    a.blocks = (rank + kRankBlock - 1) / kRankBlock;
    a.ids = static_cast<int32_t *>(workspace);
    const AdapterSpace space = adapter_space(e, m, adapters, rank, num_rows);
    a.u = static_cast<char *>(workspace) + space.ids;
    a.R2 = rank;
    if (!transpose && space.copy > 0 && num_rows > kAdapterFew) {
        a.copy_from = a.second;
        a.second = a.u + space.low;
        a.R2 = space.ranks;
        a.copy_rows = (int)std::max<int64_t>(1, std::min(kCopyRows, kCopyPart / a.R2));
    }
    a.low = static_cast<char *>(low);
    a.low_f32 = low_dtype == SEGRED_F32;
    a.out = static_cast<char *>(out);
    a.vec = ((a.M * e) % 16 == 0 && aligned(out, 16)) ? 1 : 0;
    auto units = [&](const void *p, int64_t width) { return (width * e) % 16 == 0 && aligned(p, 16); };
    const bool x = units(values, a.K);
    const bool low_direct = x && units(a.first, transpose ? rank : k);
    const bool main_direct = x && units(weights, k) && (num_rows <= kAdapterFew || units(a.second, transpose ? k : a.R2));
    switch (dtype) {
    case SEGRED_BF16: return adapter_dispatch<__bf16>(a, transpose != 0, low_direct, main_direct, stream);
    case SEGRED_F16: return adapter_dispatch<_Float16>(a, transpose != 0, low_direct, main_direct, stream);
    default: return adapter_dispatch<float>(a, transpose != 0, low_direct, main_direct, stream);
    }
}
