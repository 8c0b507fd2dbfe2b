// outer.hip -- the sum of outer products of each segment's rows:
// out[s] = sum over the rows r of segment s of left[r]^T right[r], the
// gradient of the weights of a product over segments.
#include <algorithm>
#include <type_traits>

#include "internal.hpp"
#include "outer.hpp"
#include "tile.hpp"

namespace segred {

constexpr int64_t kWhole = int64_t(1) << 62;  // more rows than there are

struct OuterArgs {
    const char *left, *right;
    const int64_t *left_rows, *right_rows;  // source rows, or null
    int64_t left_count, right_count;
    const int64_t *offsets;
    int64_t S, N, K, M;
    int64_t slots, mtiles, ntiles;
    int64_t step;   // a slot is this many rows of a segment, or the whole segment (kWhole)
    void *out;      // T or float [S, K, M]
    float *partial;  // [slots, K, M], when a segment may have more than one slot
    int out_f32, vec;
    int64_t width;       // elements from one row of `left` to the next, K or more
    const float *scale;  // what the sums are multiplied by, or null
};

// What a workgroup computes: a tile of one slot's sum.
struct OuterPlace {
    int64_t s, slot, row0, rows, m0, n0;
    bool work;  // false: nothing to store
};

// A tile's work grows with its segment's rows, so where every segment is one
// slot, up to 64 long ones are taken longest first and the longest tiles do not
// begin last (bfloat16, 8,192 rows in 8 uneven segments of 2,560 x 1,024: 98 ->
// 75 us; 16,384 in 32 segments of 1,024 x 1,024 whose lengths fall as i^-0.8: 117
// -> 100; 64 segments of about the same length lose 4%).
// Up to 16 segments are spread over all XCDs (workgroups are dealt to these in
// turn), each with one contiguous range of the segment's tiles; more are dealt
// to the XCDs forth and back, whole, so that the rows of a segment are read into
// one L2 only.  Short segments are left in their order: finding the rank takes
// about half a microsecond.
constexpr int kRanked = 64, kSpread = 16, kRankedRows = 256;
__host__ __device__ inline bool outer_ranked(const OuterArgs &a) {
    return a.step == kWhole && a.S <= kRanked && a.N >= a.S * kRankedRows;
}
__device__ __forceinline__ OuterPlace outer_place(const OuterArgs &a, int bm, int bn, int lane) {
    OuterPlace o{};
    const int64_t per = a.mtiles * a.ntiles;
    int64_t tile, piece = 0;
    if (outer_ranked(a)) {
        const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
        int64_t rank;
        if (a.S <= kSpread) {
            rank = id / per;
            const int64_t in = id - rank * per, q = per >> 3, r = per & 7, x = in & 7;
            tile = x * q + (x < r ? x : r) + (in >> 3);
        } else {
            const int64_t x = id & 7, i = id >> 3, turn = i / per;
            rank = turn * 8 + (turn & 1 ? 7 - x : x);
            tile = i - turn * per;
        }
        if (rank >= a.S) return o;
        // length (cut off at 2^25) and lane in one word, all different
        const int64_t len = lane < a.S ? a.offsets[lane + 1] - a.offsets[lane] : -1;
        const uint32_t word = len < 0 ? 63u - lane : (uint32_t)min(len, (int64_t)(1 << 25) - 1) << 6 | (63u - lane);
        int above = 0;
        for (int i = 0; i < (int)a.S; ++i) above += (uint32_t)__builtin_amdgcn_readlane((int)word, i) > word ? 1 : 0;
        o.s = __builtin_ctzll(ballot(lane < a.S && above == (int)rank));
        o.slot = o.s;
    } else {
        const int64_t total = a.slots * per, id = xcd_tile(total);
        if (id >= total) return o;
        o.slot = id / per;
        tile = id - o.slot * per;
        if (a.step == kWhole) {
            o.s = o.slot;
        } else {
            o.s = slot_segment(a.S, o.slot, lane, [&](int64_t s) { return slot_key(a.offsets, s, a.step); });
            piece = o.slot - slot_key(a.offsets, o.s, a.step);
        }
    }
    const TilePlace p = tile_place(tile, a.mtiles, a.ntiles);
    o.m0 = p.m * bm;
    o.n0 = p.n * bn;
    o.row0 = a.offsets[o.s] + piece * (a.step == kWhole ? 0 : a.step);
    const int64_t end = min(a.offsets[o.s + 1], a.N);
    o.rows = o.row0 < 0 ? 0 : max((int64_t)0, min(a.step, end - o.row0));
    o.work = o.rows > 0 || (piece == 0 && !a.partial);
    return o;
}
// Workgroups of that order.
int64_t outer_tiles(const OuterArgs &a) {
    const int64_t per = a.mtiles * a.ntiles;
    return (outer_ranked(a) && a.S > kSpread ? (a.S + 7) / 8 * 8 : a.slots) * per;
}

// Four sums of row r from column n: a partial one of the slot, or the result.
template <typename T>
__device__ __forceinline__ void outer_store(const OuterArgs &a, int64_t s, int64_t slot, int64_t r, int64_t n, f32x4 c) {
    if (a.scale && !a.partial) c *= *a.scale;
    if (a.partial)
        store_quad<float>(a.partial + (slot * a.K + r) * a.M, n, a.M, c, a.vec != 0);
    else if (a.out_f32)
        store_quad<float>(static_cast<float *>(a.out) + (s * a.K + r) * a.M, n, a.M, c, a.vec != 0);
    else
        store_quad<T>(static_cast<T *>(a.out) + (s * a.K + r) * a.M, n, a.M, c, a.vec != 0);
}

// A thread's N units per step of one operand.  row(i) is unit i's row in a step;
// the address of a row that is not gathered moves on from step to step (two
// thirds of the instructions of a step of 128 x 128 were addresses before).
template <int N>
struct OuterSide {
    const int64_t *index;  // of the slot's first row, or null
    uint64_t count, bytes, step_bytes;
    uint64_t p[N];  // gathered: in row 0
    int64_t v[N];   // gathered rows of the next step

    // byte(i): unit i's place in a row; `step`: rows of a step.
    template <typename R, typename B>
    __device__ __forceinline__ void init(const OuterPlace &at, const int64_t *rows, int64_t row_count, const char *base,
                                         int64_t row_bytes, int step, R row, B byte) {
        index = rows ? rows + at.row0 : nullptr;
        count = (uint64_t)row_count;
        bytes = (uint64_t)(uint32_t)row_bytes;
        step_bytes = bytes * step;
#pragma unroll
        for (int i = 0; i < N; ++i)
            p[i] = (uint64_t)(base + byte(i)) + (rows ? 0 : (uint64_t)(at.row0 + row(i)) * bytes);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0;
    }
    // Starts the loads of the gathered rows of the step at row k0 with `left`
    // rows, if it has any.  Behind the last they read that one again: in
    // branches each load would be waited for by itself.
    template <typename R>
    __device__ __forceinline__ void ask(int64_t k0, int left, R row) {
        if (!index || left <= 0) return;
        const int64_t *from = index + k0;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = from[(uint32_t)min(row(i), left - 1)];
    }
    // Takes note that they have come: of both sides before either issues, and on
    // every path, or the compiler waits again where it uses their registers,
    // and then for all that has been issued by then.
    __device__ __forceinline__ void settle() {
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
    }
    // issue(src, ok) for the step that was asked for, or the one after the last.
    template <typename R, typename F>
    __device__ __forceinline__ void step(int left, R row, F issue) {
        if (index) {
            issue([&](int i) { return p[i] + (uint64_t)v[i] * bytes; },
                  [&](int i) { return row(i) < left && (uint64_t)v[i] < count; });
        } else {
            issue([&](int i) { return p[i]; }, [&](int i) { return row(i) < left; });
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] += step_bytes;
        }
    }
};

// Stores a wave's neighbouring blocks.
template <typename T, int MT, int NT>
__device__ __forceinline__ void outer_blocks(const OuterArgs &a, const OuterPlace &at, const f32x4 (&acc)[MT][NT],
                                             int m_w, int n_w, int lane) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t r = at.m0 + m_w + 16 * i + (lane & 15);
        if (r >= a.K) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            outer_store<T>(a, at.s, at.slot, r, at.n0 + n_w + 16 * j + (lane >> 4) * 4, acc[i][j]);
    }
}

// L and Q: the operands' types in memory, where they are not T.
template <typename T, int BM, int BN, int WM, int WN, bool DIRECT, typename L = T, typename Q = T>
struct OuterTile {
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    using SA = ColStage<T, BM, kThreads, DIRECT, L>;
    using SB = ColStage<T, BN, kThreads, DIRECT, Q>;
    static constexpr int kStageBytes = SA::kBytes + SB::kBytes;
    static constexpr int kLds = 2 * kStageBytes;

    // O: the type of a result that is not float.
    template <typename O = T>
    static __device__ __forceinline__ void run(const OuterArgs &a, const OuterPlace &at, lds_char *lds, int wave, int lane) {
        const int64_t m0 = at.m0, n0 = at.n0, lb = a.width * (int64_t)sizeof(L), rb = a.M * (int64_t)sizeof(Q);
        SA sa;
        SB sb;
        OuterSide<SA::kLoads> left;
        OuterSide<SB::kLoads> right;
        auto lrow = [&](int i) { return SA::row(i, wave, lane); };
        auto rrow = [&](int i) { return SB::row(i, wave, lane); };
        auto lcol = [&](int i) { return (int)(a.K - m0) - SA::col(i, wave, lane); };
        auto rcol = [&](int i) { return (int)(a.M - n0) - SB::col(i, wave, lane); };
        left.init(at, a.left_rows, a.left_count, a.left, lb, kStep<T>, lrow,
                  [&](int i) { return (m0 + SA::col(i, wave, lane)) * (int64_t)sizeof(L); });
        right.init(at, a.right_rows, a.right_count, a.right, rb, kStep<T>, rrow,
                   [&](int i) { return (n0 + SB::col(i, wave, lane)) * (int64_t)sizeof(Q); });
        auto rows_of = [&](int64_t t) { return (int)max(min(at.rows - t * kStep<T>, (int64_t)kStep<T>), (int64_t)0); };
        auto ask = [&](int64_t t) {
            left.ask(t * kStep<T>, rows_of(t), lrow);
            right.ask(t * kStep<T>, rows_of(t), rrow);
        };
        auto issue = [&](int64_t t, lds_char *buf) {
            left.settle();
            right.settle();
            left.step(rows_of(t), lrow, [&](auto src, auto ok) {
                sa.issue(buf, wave, src, [&](int i) { return ok(i) ? lcol(i) : 0; });
            });
            right.step(rows_of(t), rrow, [&](auto src, auto ok) {
                sb.issue(buf + SA::kBytes, wave, src, [&](int i) { return ok(i) ? rcol(i) : 0; });
            });
        };
        auto commit = [&](lds_char *buf) {
            sa.commit(buf, wave, lane);
            sb.commit(buf + SA::kBytes, wave, lane);
        };

        f32x4 acc[MT][NT] = {};
        const int m_w = wave / WN * (MT * 16), n_w = wave % WN * (NT * 16);
        const int64_t steps = (at.rows + kStep<T> - 1) / kStep<T>;
        if (steps > 0) {
            ask(0);
            issue(0, lds);
            ask(1);
            commit(lds);
        }
        for (int64_t t = 0; t < steps; ++t) {
            wait_and_meet<0>();
            lds_char *next = lds + ((t + 1) & 1) * kStageBytes;
            if (t + 1 < steps) {
                issue(t + 1, next);
                ask(t + 2);
            }
            const lds_char *buf = lds + (t & 1) * kStageBytes;
            step_products<T, MT, NT, true, BM, true, BN>(acc, buf, buf + SA::kBytes, m_w, n_w, lane);
            if (t + 1 < steps) commit(next);
        }
        outer_blocks<O, MT, NT>(a, at, acc, m_w, n_w, lane);
    }
};

template <typename T, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN) void seg_outer(OuterArgs a) {
    using Tile = OuterTile<T, BM, BN, WM, WN, DIRECT>;
    __shared__ __attribute__((aligned(1024))) char lds_mem[Tile::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const OuterPlace at = outer_place(a, BM, BN, lane);
    if (at.work) Tile::run(a, at, (lds_char *)lds_mem, wave, lane);
}

// The same for float, in bf16 parts; a tile with a sum that is not finite is
// computed again with float products.
// (Three workgroups a CU: 300,000 rows in 5 segments, 64 x 96 each, take 57 us
// against 76 with the two that the registers would allow otherwise.)
// L, Q: types of the operands; where one is of 16 bits it is not rounded
// again, and a result that is not float has its type, O.
constexpr int kSplitThreads = 256;
template <int BM, int BN, bool WHOLE, typename L, typename Q>
__global__ __launch_bounds__(kSplitThreads, 3) void seg_outer_split(OuterArgs a) {
    typedef std::conditional_t<sizeof(L) == 2, L, Q> O;
    using Plain = OuterTile<float, 64, 64, 2, 2, false, L, Q>;
    using SA = SplitStage<BM, kSplitThreads, true, WHOLE, L>;
    using SB = SplitStage<BN, kSplitThreads, true, WHOLE, Q>;
    constexpr int MT = BM / 32, NT = BN / 32, kSplitLds = SA::kLds + SB::kLds;
    __shared__ __attribute__((aligned(1024))) char lds_mem[kSplitLds > Plain::kLds ? kSplitLds : Plain::kLds];
    lds_char *lds = (lds_char *)lds_mem;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const OuterPlace at = outer_place(a, BM, BN, lane);
    if (!at.work) return;

    SA sa;
    SB sb;
    OuterSide<SA::kParts> left;
    OuterSide<SB::kParts> right;
    auto lrow = [&](int i) { return SA::row(i, tid); };
    auto rrow = [&](int i) { return SB::row(i, tid); };
    auto lcol = [&](int i) { return (int)(a.K - at.m0) - SA::at(i, tid); };
    auto rcol = [&](int i) { return (int)(a.M - at.n0) - SB::at(i, tid); };
    left.init(at, a.left_rows, a.left_count, a.left, a.width * (int64_t)sizeof(L), kSplitK, lrow,
              [&](int i) { return (at.m0 + SA::at(i, tid)) * (int64_t)sizeof(L); });
    right.init(at, a.right_rows, a.right_count, a.right, a.M * (int64_t)sizeof(Q), kSplitK, rrow,
               [&](int i) { return (at.n0 + SB::at(i, tid)) * (int64_t)sizeof(Q); });
    auto rows_of = [&](int64_t t) { return (int)max(min(at.rows - t * kSplitK, (int64_t)kSplitK), (int64_t)0); };
    auto ask = [&](int64_t t) {
        left.ask(t * kSplitK, rows_of(t), lrow);
        right.ask(t * kSplitK, rows_of(t), rrow);
    };
    f32x4 acc[MT][NT] = {};
    const int m_w = wave / 2 * (BM / 2), n_w = wave % 2 * (BN / 2);
    ask(0);
    split_steps(
        (at.rows + kSplitK - 1) / kSplitK,
        [&](int64_t t) {
            left.settle();
            right.settle();
            left.step(rows_of(t), lrow, [&](auto src, auto ok) {
                sa.issue(src, [&](int i) { return ok(i) ? lcol(i) : 0; });
            });
            right.step(rows_of(t), rrow, [&](auto src, auto ok) {
                sb.issue(src, [&](int i) { return ok(i) ? rcol(i) : 0; });
            });
            ask(t + 1);
        },
        [&] {
            sa.commit(lds, tid);
            sb.commit(lds + SA::kLds, tid);
        },
        [&] { split_step<MT, NT, true, BM, true, BN, kPlanes<L>, kPlanes<Q>>(acc, lds, lds + SA::kLds, m_w, n_w, lane); });
    if (__syncthreads_or(any_not_finite(acc))) {
        OuterPlace q = at;
        for (int r = 0; r < BM && at.m0 + r < a.K; r += 64)
            for (int c = 0; c < BN && at.n0 + c < a.M; c += 64) {
                q.m0 = at.m0 + r;
                q.n0 = at.n0 + c;
                __syncthreads();
                Plain::template run<O>(a, q, lds, wave, lane);
            }
        return;
    }
    outer_blocks<O, MT, NT>(a, at, acc, m_w, n_w, lane);
}

// Adds the slots of each segment and rounds once.  PARTS threads share a cell:
// thread p adds the slots p, p + PARTS, ... in that order, then the parts are
// added in order, so that few cells with many slots still read with many
// threads.  (300,000 rows in 5 segments, 64 x 96 each, about 60 slots a
// segment: 33 us with one part; 100 segments of 256 x 256 with about two slots
// each: 49 us with one, 133 us with 8.)
constexpr int kJoinThreads = 256, kJoinParts = 8;
template <typename T, int PARTS>
__global__ __launch_bounds__(kJoinThreads) void outer_join(OuterArgs a) {
    constexpr int kCells = kJoinThreads / PARTS;
    __shared__ float s_part[PARTS][kCells];
    const int64_t cells = a.K * a.M;
    const int part = threadIdx.x / kCells, cell = threadIdx.x % kCells;
    const int64_t i = (int64_t)blockIdx.x * kCells + cell;
    float sum = 0.f;
    if (i < a.S * cells) {
        const int64_t s = i / cells, c = i - s * cells;
        const int64_t begin = a.offsets[s], len = min(a.offsets[s + 1], a.N) - begin;
        const int64_t n = begin < 0 || len <= 0 ? 0 : (len - 1) / a.step + 1;
        const float *p = a.partial + slot_key(a.offsets, s, a.step) * cells + c;
#pragma unroll 4
        for (int64_t j = part; j < n; j += PARTS) sum += p[j * cells];
    }
    if constexpr (PARTS > 1) {
        s_part[part][cell] = sum;
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int q = 1; q < PARTS; ++q) sum += s_part[q][cell];
    }
    if (a.scale) sum *= *a.scale;
    if (i < a.S * cells) {
        if (a.out_f32) static_cast<float *>(a.out)[i] = sum;
        else static_cast<T *>(a.out)[i] = (T)sum;
    }
}

// Tile and rows of a slot.  Where the segments' tiles of 128 x 128 would give
// every CU one, or there is a segment for every CU, a slot is a whole segment
// (in tiles of that size for 16-bit types, of 64 x 128 in bf16 parts).  Else the
// tiles are 64 x 64, or 64 x 128 where the left side has no more than 64 columns
// and the right side more (the mirrored case, 96 x 64, reads its right side
// twice: there is no tile of 128 x 64), and the segments are cut into slots of at
// least kSlotRows rows, as many as the device holds workgroups at a time (3 of
// 64 x 128 or 4 of 64 x 64 a CU).
struct OuterPlan {
    bool small;  // 64 x 64, or
    bool wide;   // 64 x 128
    int64_t step;
};
constexpr int64_t kCus = 256, kSlotRows = 256;
OuterPlan outer_plan(int64_t k, int64_t m, int64_t S, int64_t N) {
    auto tiles = [&](int64_t bm, int64_t bn) { return ((k + bm - 1) / bm) * ((m + bn - 1) / bn); };
    OuterPlan p{false, false, kWhole};
    if (S >= kCus || S * tiles(128, 128) >= kCus) return p;
    p.small = true;
    p.wide = k <= 64 && m > 64;
    if (N <= kSlotRows) return p;
    const int64_t per = tiles(64, p.wide ? 128 : 64), room = std::max<int64_t>(1, kCus * (p.wide ? 3 : 4) / per);
    const int64_t rows = N / std::max<int64_t>(1, room - S) + 1;
    p.step = std::max<int64_t>(kSlotRows, (rows + 63) / 64 * 64);
    return p;
}

// Adds the slots, where there are several.
template <typename T>
int outer_finish(const OuterArgs &a, hipStream_t st) {
    if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    if (!a.partial) return SEGRED_OK;
    const bool shared = a.slots >= kJoinParts * a.S;
    const int64_t cells = shared ? kJoinThreads / kJoinParts : kJoinThreads;
    const unsigned wgs = (unsigned)((a.S * a.K * a.M + cells - 1) / cells);
    if (shared) timed_launch_ggl(false, (outer_join<T, kJoinParts>), dim3(wgs), dim3(kJoinThreads), 0, st, a);
    else timed_launch_ggl(false, (outer_join<T, 1>), dim3(wgs), dim3(kJoinThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

template <typename T, int BM, int BN, int WM, int WN>
int outer_launch(OuterArgs a, bool direct, hipStream_t st) {
    a.mtiles = (a.K + BM - 1) / BM;
    a.ntiles = (a.M + BN - 1) / BN;
    dim3 grid;
    if (!tile_grid(outer_tiles(a), grid)) return SEGRED_ERR_UNSUPPORTED;
    constexpr int kThreads = 64 * WM * WN;
    if (direct)
        timed_launch_ggl(true, (seg_outer<T, BM, BN, WM, WN, true>), grid, dim3(kThreads), 0, st, a);
    else
        timed_launch_ggl(true, (seg_outer<T, BM, BN, WM, WN, false>), grid, dim3(kThreads), 0, st, a);
    return outer_finish<T>(a, st);
}

template <typename L, typename Q, int BM, int BN>
int outer_split_launch(OuterArgs a, hipStream_t st) {
    a.mtiles = (a.K + BM - 1) / BM;
    a.ntiles = (a.M + BN - 1) / BN;
    dim3 grid;
    if (!tile_grid(outer_tiles(a), grid)) return SEGRED_ERR_UNSUPPORTED;
    if (a.width % 8 == 0 && a.M % 8 == 0)
        timed_launch_ggl(true, (seg_outer_split<BM, BN, true, L, Q>), grid, dim3(kSplitThreads), 0, st, a);
    else
        timed_launch_ggl(true, (seg_outer_split<BM, BN, false, L, Q>), grid, dim3(kSplitThreads), 0, st, a);
    return outer_finish<std::conditional_t<sizeof(L) == 2, L, Q>>(a, st);
}

template <typename L, typename Q>
int outer_split_dispatch(const OuterArgs &a, const OuterPlan &p, hipStream_t st) {
    if (p.small && !p.wide) return outer_split_launch<L, Q, 64, 64>(a, st);
    return outer_split_launch<L, Q, 64, 128>(a, st);
}

template <typename T>
int outer_dispatch(const OuterArgs &a, const OuterPlan &p, bool direct, hipStream_t st) {
    if constexpr (sizeof(T) == 4) {
        return outer_split_dispatch<T, T>(a, p, st);
    } else {
        if (p.wide) return outer_launch<T, 64, 128, 2, 2>(a, direct, st);
        if (p.small) return outer_launch<T, 64, 64, 2, 2>(a, direct, st);
        return outer_launch<T, 128, 128, 2, 2>(a, direct, st);
    }
}

int outer_scaled(const void *left, int64_t width, int64_t vc, const void *right, const int64_t *right_rows, int64_t n,
                 int64_t m, int32_t dtype, const int64_t *offsets, void *out, int32_t out_dtype, const float *scale,
                 void *workspace, hipStream_t stream) {
    const int64_t e = float_size(dtype), oe = float_size(out_dtype);
    OuterArgs a{};
    a.left = static_cast<const char *>(left);
    a.right = static_cast<const char *>(right);
    a.right_rows = right_rows;
    a.left_count = a.right_count = n;
    a.offsets = offsets;
    a.S = 1;
    a.N = n;
    a.K = vc;
    a.width = width;
    a.M = m;
    const OuterPlan plan = outer_plan(vc, m, 1, n);
    a.step = plan.step;
    a.slots = n / a.step + 1;
    a.out = out;
    a.out_f32 = out_dtype == SEGRED_F32;
    a.partial = plan.step == kWhole ? nullptr : static_cast<float *>(workspace);
    a.scale = scale;
    a.vec = (m % 4 == 0 && aligned(out, 4 * oe)) ? 1 : 0;
    const bool direct = (width * e) % 16 == 0 && (m * e) % 16 == 0 && aligned(left, 16) && aligned(right, 16);
    switch (dtype) {
    case SEGRED_BF16: return outer_dispatch<__bf16>(a, plan, direct, stream);
    case SEGRED_F16: return outer_dispatch<_Float16>(a, plan, direct, stream);
    default: return outer_dispatch<float>(a, plan, direct, stream);
    }
}

}  // namespace segred

using namespace segred;

extern "C" int64_t segred_outer_workspace(int64_t k, int64_t m, int64_t num_segments, int64_t num_rows) {
    if (k < 1 || m < 1 || num_segments < 1 || num_rows < 0 || k > kMaxWidth || m > kMaxWidth) return 0;
    if (too_large(num_segments, k * m, 4)) return 0;
    const int64_t step = outer_plan(k, m, num_segments, num_rows).step;
    return step == kWhole ? 0 : (num_rows / step + num_segments) * k * m * 4;
}

extern "C" int segred_outer(const void *left, const int64_t *left_rows, int64_t left_count, int64_t k,
                            const void *right, const int64_t *right_rows, int64_t right_count, int64_t m,
                            int32_t dtype, const int64_t *offsets, int64_t num_segments, int64_t num_rows, void *out,
                            int32_t out_dtype, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    return segred_outer_mixed(left, dtype, left_rows, left_count, k, right, dtype, right_rows, right_count, m, offsets,
                              num_segments, num_rows, out, out_dtype, workspace, workspace_bytes, stream);
}

extern "C" int segred_outer_mixed(const void *left, int32_t left_dtype, const int64_t *left_rows, int64_t left_count,
                                  int64_t k, const void *right, int32_t right_dtype, const int64_t *right_rows,
                                  int64_t right_count, int64_t m, const int64_t *offsets, int64_t num_segments,
                                  int64_t num_rows, void *out, int32_t out_dtype, void *workspace,
                                  int64_t workspace_bytes, hipStream_t stream) {
    const int64_t le = float_size(left_dtype), re = float_size(right_dtype);
    for (int32_t dtype : {left_dtype, right_dtype})
        if (dtype < SEGRED_U32 || dtype > SEGRED_F16) return SEGRED_ERR_INVALID_ARGUMENT;
    if (k < 1 || m < 1 || left_count < 0 || right_count < 0 || num_segments < 0 || num_rows < 0)
        return SEGRED_ERR_INVALID_ARGUMENT;
    if ((!left_rows && left_count < num_rows) || (!right_rows && right_count < num_rows)) return SEGRED_ERR_INVALID_ARGUMENT;
    if (num_segments > 0 && (!offsets || !out || (num_rows > 0 && ((left_count > 0 && !left) || (right_count > 0 && !right)))))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (le == 0 || re == 0 || k > kMaxWidth || m > kMaxWidth) return SEGRED_ERR_UNSUPPORTED;
    if (left_dtype != right_dtype && left_dtype != SEGRED_F32 && right_dtype != SEGRED_F32) return SEGRED_ERR_UNSUPPORTED;
    if (out_dtype != left_dtype && out_dtype != right_dtype && out_dtype != SEGRED_F32) return SEGRED_ERR_INVALID_ARGUMENT;
    const int64_t oe = float_size(out_dtype);
    if (!aligned(left, le) || !aligned(right, re) || !aligned(out, oe) || !aligned(offsets, 8) || !aligned(left_rows, 8) ||
        !aligned(right_rows, 8) || !aligned(workspace, 16))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (too_large(left_count, k, 4) || too_large(right_count, m, 4) || too_large(num_segments, k * m, 4))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (num_segments == 0) return SEGRED_OK;
    const int64_t need = segred_outer_workspace(k, m, num_segments, num_rows);
    if (need > 0 && (!workspace || workspace_bytes < need)) return SEGRED_ERR_INVALID_ARGUMENT;

    OuterArgs a{};
    a.left = static_cast<const char *>(left);
    a.right = static_cast<const char *>(right);
    a.left_rows = left_rows;
    a.right_rows = right_rows;
    a.left_count = left_count;
    a.right_count = right_count;
    a.offsets = offsets;
    a.S = num_segments;
    a.N = num_rows;
    a.K = a.width = k;
    a.M = m;
    const OuterPlan plan = outer_plan(k, m, num_segments, num_rows);
    a.step = plan.step;
    a.slots = num_rows / a.step + num_segments;
    a.out = out;
    a.out_f32 = out_dtype == SEGRED_F32;
    a.partial = need > 0 ? static_cast<float *>(workspace) : nullptr;
    a.vec = (m % 4 == 0 && aligned(out, 4 * oe)) ? 1 : 0;
    const bool direct = (k * le) % 16 == 0 && (m * re) % 16 == 0 && aligned(left, 16) && aligned(right, 16);
    if (left_dtype != right_dtype) {
        if (left_dtype == SEGRED_BF16) return outer_split_dispatch<__bf16, float>(a, plan, stream);
        if (left_dtype == SEGRED_F16) return outer_split_dispatch<_Float16, float>(a, plan, stream);
        if (right_dtype == SEGRED_BF16) return outer_split_dispatch<float, __bf16>(a, plan, stream);
        return outer_split_dispatch<float, _Float16>(a, plan, stream);
    }
    switch (left_dtype) {
    case SEGRED_BF16: return outer_dispatch<__bf16>(a, plan, direct, stream);
    case SEGRED_F16: return outer_dispatch<_Float16>(a, plan, direct, stream);
    default: return outer_dispatch<float>(a, plan, direct, stream);
    }
}
