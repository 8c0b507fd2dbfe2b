// outer.hip -- the sum of outer products of each segment's rows:
// out[s] = sum over the rows r of segment s of left[r]^T right[r], the
// gradient of the weights of a product over segments.
#include <algorithm>

#include "internal.hpp"
#include "tile.hpp"

namespace segred {

struct OuterArgs {
    const char *left, *right;
    const int64_t *left_rows, *right_rows;  // source rows, or null
    int64_t left_count, right_count;
    const int64_t *offsets;
    int64_t S, N, K, M;
    int64_t slots, mtiles, ntiles;
    int lg;         // a slot is 2^lg rows of a segment
    void *out;      // T or float [S, K, M]
    float *partial;  // [slots, K, M], when a segment may have more than one slot
    int out_f32, vec;
};

template <typename T, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN) void seg_outer(OuterArgs a) {
    constexpr int kThreads = 64 * WM * WN;
    constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    using SA = ColStage<T, BM, kThreads, DIRECT>;
    using SB = ColStage<T, BN, kThreads, DIRECT>;
    constexpr int kStageBytes = SA::kBytes + SB::kBytes;
    __shared__ __attribute__((aligned(1024))) char lds_mem[2 * kStageBytes];
    lds_char *lds = (lds_char *)lds_mem;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t total = a.slots * a.mtiles * a.ntiles;
    const int64_t id = xcd_tile(total);
    if (id >= total) return;
    const int64_t slot = id / (a.mtiles * a.ntiles), tile = id - slot * a.mtiles * a.ntiles;
    const int64_t m0 = tile / a.ntiles * BM, n0 = tile % a.ntiles * BN;

    const int64_t s = slot_segment(a.offsets, a.S, a.lg, slot, lane);
    const int64_t piece = slot - slot_key(a.offsets, s, a.lg);
    const int64_t row0 = a.offsets[s] + (piece << a.lg);
    const int64_t end = min(a.offsets[s + 1], a.N);
    const int64_t rows = row0 < 0 ? 0 : max((int64_t)0, min(int64_t(1) << a.lg, end - row0));
    if (rows == 0 && (piece > 0 || a.partial)) return;

    SA sa;
    SB sb;
    int64_t ia[SA::kLoads], ib[SB::kLoads];  // source row of the next step's units, -1: none
    auto fetch = [&](int64_t k0) {
#pragma unroll
        for (int i = 0; i < SA::kLoads; ++i) {
            const int64_t r = k0 + SA::row(i, wave, lane);
            ia[i] = r < rows ? (a.left_rows ? a.left_rows[row0 + r] : row0 + r) : -1;
        }
#pragma unroll
        for (int i = 0; i < SB::kLoads; ++i) {
            const int64_t r = k0 + SB::row(i, wave, lane);
            ib[i] = r < rows ? (a.right_rows ? a.right_rows[row0 + r] : row0 + r) : -1;
        }
    };
    auto issue = [&](lds_char *buf) {
        sa.issue(
            buf, wave,
            [&](int i) { return (uint64_t)(a.left + (ia[i] * a.K + m0 + SA::col(i, wave, lane)) * (int64_t)sizeof(T)); },
            [&](int i) { return ia[i] >= 0 && ia[i] < a.left_count ? (int)(a.K - m0) - SA::col(i, wave, lane) : 0; });
        sb.issue(
            buf + SA::kBytes, wave,
            [&](int i) { return (uint64_t)(a.right + (ib[i] * a.M + n0 + SB::col(i, wave, lane)) * (int64_t)sizeof(T)); },
            [&](int i) { return ib[i] >= 0 && ib[i] < a.right_count ? (int)(a.M - n0) - SB::col(i, wave, lane) : 0; });
    };
    auto commit = [&](lds_char *buf) {
        sa.commit(buf, wave, lane);
        sb.commit(buf + SA::kBytes, wave, lane);
    };

    f32x4 acc[MT][NT] = {};
    const int m_w = wave / WN * (MT * 16), n_w = wave % WN * (NT * 16);
    const int64_t steps = (rows + kStep<T> - 1) / kStep<T>;
    if (steps > 0) {
        fetch(0);
        issue(lds);
        fetch(kStep<T>);
        commit(lds);
        for (int64_t t = 0; t < steps; ++t) {
            wait_and_meet<0>();
            lds_char *next = lds + ((t + 1) & 1) * kStageBytes;
            if (t + 1 < steps) {
                issue(next);
                fetch((t + 2) * kStep<T>);
            }
            const lds_char *buf = lds + (t & 1) * kStageBytes;
            step_products<T, MT, NT, true, BM, true, BN>(acc, buf, buf + SA::kBytes, m_w, n_w, lane);
            if (t + 1 < steps) commit(next);
        }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t r = m0 + m_w + 16 * i + (lane & 15);
        if (r >= a.K) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int64_t n = n0 + n_w + 16 * j + (lane >> 4) * 4;
            if (a.partial)
                store_quad<float>(a.partial + (slot * a.K + r) * a.M, n, a.M, acc[i][j], a.vec != 0);
            else if (a.out_f32)
                store_quad<float>(static_cast<float *>(a.out) + (s * a.K + r) * a.M, n, a.M, acc[i][j], a.vec != 0);
            else
                store_quad<T>(static_cast<T *>(a.out) + (s * a.K + r) * a.M, n, a.M, acc[i][j], a.vec != 0);
        }
    }
}

// Sums the slots of each segment in slot order and rounds once.
constexpr int kJoinThreads = 256;
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void outer_join(OuterArgs a) {
    const int64_t cells = a.K * a.M;
    const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
    if (i >= a.S * cells) return;
    const int64_t s = i / cells, c = i - s * cells;
    const int64_t begin = a.offsets[s], len = min(a.offsets[s + 1], a.N) - begin;
    const int64_t n = begin < 0 || len <= 0 ? 0 : ((len - 1) >> a.lg) + 1;
    const float *p = a.partial + slot_key(a.offsets, s, a.lg) * cells + c;
    float sum = 0.f;
    for (int64_t j = 0; j < n; ++j) sum += p[j * cells];
    if (a.out_f32) static_cast<float *>(a.out)[i] = sum;
    else static_cast<T *>(a.out)[i] = (T)sum;
}

// Rows of a slot: a whole segment where the tiles of all segments fill the
// device; else enough pieces that they do.
constexpr int64_t kOuterTiles = 512;
constexpr int kOuterTile = 128;
int outer_lg(int64_t k, int64_t m, int64_t S, int64_t N) {
    const int64_t per = ((k + kOuterTile - 1) / kOuterTile) * ((m + kOuterTile - 1) / kOuterTile);
    if (S * per >= kOuterTiles || N <= 512) return 62;
    const int64_t want = std::max<int64_t>(512, N * per / kOuterTiles);
    int lg = 9;
    while ((int64_t(1) << lg) < want) ++lg;
    return lg;
}

template <typename T, int BM, int BN, int WM, int WN>
int outer_launch(OuterArgs a, bool direct, hipStream_t st) {
    a.mtiles = (a.K + BM - 1) / BM;
    a.ntiles = (a.M + BN - 1) / BN;
    dim3 grid;
    if (!tile_grid(a.slots * a.mtiles * a.ntiles, grid)) return SEGRED_ERR_UNSUPPORTED;
    constexpr int kThreads = 64 * WM * WN;
    if (direct)
        timed_launch_ggl(true, (seg_outer<T, BM, BN, WM, WN, true>), grid, dim3(kThreads), 0, st, a);
    else
        timed_launch_ggl(true, (seg_outer<T, BM, BN, WM, WN, false>), grid, dim3(kThreads), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    if (a.partial) {
        const int64_t wgs = (a.S * a.K * a.M + kJoinThreads - 1) / kJoinThreads;
        timed_launch_ggl(false, outer_join<T>, dim3((unsigned)wgs), dim3(kJoinThreads), 0, st, a);
        if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    }
    return SEGRED_OK;
}

template <typename T>
int outer_dispatch(const OuterArgs &a, bool direct, hipStream_t st) {
    return outer_launch<T, 128, 128, 2, 2>(a, direct, st);
}

}  // namespace segred

using namespace segred;

extern "C" int64_t segred_outer_workspace(int64_t k, int64_t m, int64_t num_segments, int64_t num_rows) {
    if (k < 1 || m < 1 || num_segments < 1 || num_rows < 0 || k > kMaxWidth || m > kMaxWidth) return 0;
    if (too_large(num_segments, k * m, 4)) return 0;
    const int lg = outer_lg(k, m, num_segments, num_rows);
    if (lg == 62) return 0;
    return ((num_rows >> lg) + num_segments) * k * m * 4;
}

extern "C" int segred_outer(const void *left, const int64_t *left_rows, int64_t left_count, int64_t k,
                            const void *right, const int64_t *right_rows, int64_t right_count, int64_t m,
                            int32_t dtype, const int64_t *offsets, int64_t num_segments, int64_t num_rows, void *out,
                            int32_t out_dtype, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    const int64_t e = float_size(dtype);
    if (dtype < SEGRED_U32 || dtype > SEGRED_F16) return SEGRED_ERR_INVALID_ARGUMENT;
    if (k < 1 || m < 1 || left_count < 0 || right_count < 0 || num_segments < 0 || num_rows < 0)
        return SEGRED_ERR_INVALID_ARGUMENT;
    if ((!left_rows && left_count < num_rows) || (!right_rows && right_count < num_rows)) return SEGRED_ERR_INVALID_ARGUMENT;
    if (num_segments > 0 && (!offsets || !out || (num_rows > 0 && (!left || !right)))) return SEGRED_ERR_INVALID_ARGUMENT;
    if (e == 0 || k > kMaxWidth || m > kMaxWidth) return SEGRED_ERR_UNSUPPORTED;
    if (out_dtype != dtype && out_dtype != SEGRED_F32) return SEGRED_ERR_INVALID_ARGUMENT;
    const int64_t oe = float_size(out_dtype);
    if (!aligned(left, e) || !aligned(right, e) || !aligned(out, oe) || !aligned(offsets, 8) || !aligned(left_rows, 8) ||
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
    a.K = k;
    a.M = m;
    a.lg = outer_lg(k, m, num_segments, num_rows);
    a.slots = (num_rows >> a.lg) + num_segments;
    a.out = out;
    a.out_f32 = out_dtype == SEGRED_F32;
    a.partial = need > 0 ? static_cast<float *>(workspace) : nullptr;
    a.vec = (m % 4 == 0 && aligned(out, 4 * oe)) ? 1 : 0;
    const bool direct = (k * e) % 16 == 0 && (m * e) % 16 == 0 && aligned(left, 16) && aligned(right, 16);
    switch (dtype) {
    case SEGRED_BF16: return outer_dispatch<__bf16>(a, direct, stream);
    case SEGRED_F16: return outer_dispatch<_Float16>(a, direct, stream);
    default: return outer_dispatch<float>(a, direct, stream);
    }
}
