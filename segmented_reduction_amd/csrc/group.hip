// group.hip -- rows grouped by an index: a stable counting sort of the entries
// by the group they name, the place of each entry in it, and the offsets of
// the groups.  No atomics: entries are ranked among the 64 lanes of a wave by
// ballots, waves by their place in the tile and tiles by a scan, so that the
// result is the one stable order.
#include <algorithm>

#include "internal.hpp"
#include "scan.hpp"
#include "wave.hpp"

namespace segred {

// The entries of one digit pass.  The first pass reads the index itself, the
// later ones the (key, entry) pairs the pass before wrote.
struct GroupArgs {
    const int64_t *index;
    const uint32_t *keys_in, *entries_in;  // later passes
    uint32_t *keys_out, *entries_out;      // all but the last pass (keys_out also then, for the bounds)
    int64_t *order, *position, *offsets;   // last pass
    uint32_t *hist;                        // [digits][tiles]
    uint32_t *totals;                      // [digits]
    uint32_t rows, dim, tiles, fanout;
    int shift, bits;
    int first, last;
};

constexpr int kGroupThreads = 256;
constexpr int kGroupWaves = kGroupThreads / 64;
constexpr int kGroupSteps = 16;  // entries per lane
constexpr int kGroupTile = kGroupThreads * kGroupSteps;
constexpr int kGroupMaxBits = 10;

__device__ __forceinline__ uint32_t group_key(int64_t v, uint32_t dim) {
    return v >= 0 && v < (int64_t)dim ? (uint32_t)v : dim;  // entries of no group go behind the last one
}

// Lanes of the wave whose digit equals this lane's.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits, bool valid) {
    uint64_t m = ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const bool set = (digit >> b) & 1;
        const uint64_t with = ballot(set);
        m &= set ? with : ~with;
    }
    return m;
}

// Exclusive offsets of `digits` totals into s_base (all threads of the group).
template <int THREADS>
__device__ __forceinline__ void digit_bases(const uint32_t *totals, int digits, uint32_t *s_base, int64_t *s_tmp) {
    constexpr int kPer = (1 << kGroupMaxBits) / THREADS > 0 ? (1 << kGroupMaxBits) / THREADS : 1;
    uint32_t v[kPer];
    uint32_t sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = threadIdx.x * kPer + j;
        v[j] = d < digits ? totals[d] : 0u;
        sum += v[j];
    }
    int64_t total;
    uint32_t base = (uint32_t)(block_inclusive_scan<THREADS, false>((int64_t)sum, s_tmp, total) - sum);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = threadIdx.x * kPer + j;
        if (d < digits) s_base[d] = base;
        base += v[j];
    }
    __syncthreads();
}

// Entries of each digit in each tile.
__global__ __launch_bounds__(kGroupThreads) void group_count(GroupArgs a) {
    extern __shared__ uint32_t s_count[];  // [waves][digits]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int digits = 1 << a.bits;
    for (int i = threadIdx.x; i < kGroupWaves * digits; i += kGroupThreads) s_count[i] = 0;
    __syncthreads();
    uint32_t *mine = s_count + wave * digits;
    const uint32_t first = blockIdx.x * kGroupTile + wave * 64 * kGroupSteps;
    uint32_t key[kGroupSteps];
#pragma unroll
    for (int i = 0; i < kGroupSteps; ++i) {
        const uint32_t e = first + i * 64 + lane;
        key[i] = e < a.rows ? (a.first ? group_key(a.index[e], a.dim) : a.keys_in[e]) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kGroupSteps; ++i) {
        const bool valid = first + i * 64 + lane < a.rows;
        const uint32_t d = (key[i] >> a.shift) & (digits - 1);
        const uint64_t same = same_digit(d, a.bits, valid);
        if (valid && (same & ((uint64_t(1) << lane) - 1)) == 0) mine[d] += popc64(same);
        wave_lds_sync();
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kGroupThreads) {
        uint32_t n = 0;
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) n += s_count[w * digits + d];
        a.hist[(size_t)d * a.tiles + blockIdx.x] = n;
    }
}

// Exclusive scan over the tiles of each digit (one workgroup per digit).
__global__ __launch_bounds__(kGroupThreads) void group_scan(GroupArgs a) {
    __shared__ int64_t s_tmp[2 * kGroupWaves];
    constexpr int kPer = 4;
    uint32_t *row = a.hist + (size_t)blockIdx.x * a.tiles;
    uint32_t running = 0;
    for (uint32_t b = 0; b < a.tiles; b += kGroupThreads * kPer) {
        uint32_t v[kPer], sum = 0;
        const uint32_t t = b + threadIdx.x * kPer;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            v[j] = t + j < a.tiles ? row[t + j] : 0u;
            sum += v[j];
        }
        int64_t total;
        uint32_t base = running + (uint32_t)(block_inclusive_scan<kGroupThreads, false>((int64_t)sum, s_tmp, total) - sum);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (t + j < a.tiles) row[t + j] = base;
            base += v[j];
        }
        running += (uint32_t)total;
    }
    if (threadIdx.x == 0) a.totals[blockIdx.x] = running;
}

// Moves each entry to its place in this pass's order.
__global__ __launch_bounds__(kGroupThreads) void group_place(GroupArgs a) {
    extern __shared__ uint32_t s_count[];  // [waves][digits], then [digits] bases
    __shared__ int64_t s_tmp[2 * kGroupWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int digits = 1 << a.bits;
    uint32_t *s_base = s_count + kGroupWaves * digits;
    for (int i = threadIdx.x; i < kGroupWaves * digits; i += kGroupThreads) s_count[i] = 0;
    digit_bases<kGroupThreads>(a.totals, digits, s_base, s_tmp);
    uint32_t *mine = s_count + wave * digits;
    const uint32_t first = blockIdx.x * kGroupTile + wave * 64 * kGroupSteps;
    uint32_t key[kGroupSteps], rank[kGroupSteps];
#pragma unroll
    for (int i = 0; i < kGroupSteps; ++i) {
        const uint32_t e = first + i * 64 + lane;
        key[i] = e < a.rows ? (a.first ? group_key(a.index[e], a.dim) : a.keys_in[e]) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kGroupSteps; ++i) {
        const bool valid = first + i * 64 + lane < a.rows;
        const uint32_t d = (key[i] >> a.shift) & (digits - 1);
        const uint64_t same = same_digit(d, a.bits, valid);
        const uint32_t before = popc64(same & ((uint64_t(1) << lane) - 1));
        const uint32_t seen = mine[d];
        rank[i] = seen + before;
        wave_lds_sync();
        if (valid && before == 0) mine[d] = seen + popc64(same);
        wave_lds_sync();
    }
    __syncthreads();
    // counts -> first place of each (wave, digit)
    for (int d = threadIdx.x; d < digits; d += kGroupThreads) {
        uint32_t at = s_base[d] + a.hist[(size_t)d * a.tiles + blockIdx.x];
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) {
            const uint32_t n = s_count[w * digits + d];
            s_count[w * digits + d] = at;
            at += n;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGroupSteps; ++i) {
        const uint32_t e = first + i * 64 + lane;
        if (e >= a.rows) continue;
        const uint32_t to = mine[(key[i] >> a.shift) & (digits - 1)] + rank[i];
        const uint32_t entry = a.first ? e : a.entries_in[e];
        if (a.last) {
            a.order[to] = a.fanout > 1 ? entry / a.fanout : entry;
            a.position[entry] = key[i] < a.dim ? (int64_t)to : -1;
            if (a.keys_out) a.keys_out[to] = key[i];
        } else {
            a.keys_out[to] = key[i];
            a.entries_out[to] = entry;
        }
    }
    if (a.last && a.first && blockIdx.x == 0)  // one pass: the digits are the groups
        for (uint32_t d = threadIdx.x; d <= a.dim; d += kGroupThreads) a.offsets[d] = s_base[d];
}

// offsets[s] = the first place whose key is not below s (several passes).
__global__ __launch_bounds__(kGroupThreads) void group_bounds(const uint32_t *keys, uint32_t rows, uint32_t dim,
                                                              int64_t *offsets) {
    const uint64_t s = (uint64_t)blockIdx.x * kGroupThreads + threadIdx.x;
    if (s > dim) return;
    uint32_t lo = 0, hi = rows;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < s) lo = mid + 1;
        else hi = mid;
    }
    offsets[s] = lo;
}

// Few entries and few groups: one workgroup, one launch.  Each wave counts
// its stretch, the counts are scanned over (digit, wave), and a second walk
// over the stretch places the entries.
constexpr int kGroupSmallRows = 8192;
constexpr int kGroupSmallDim = 1023;
template <int THREADS>
__global__ __launch_bounds__(THREADS) void group_small(GroupArgs a) {
    constexpr int kWaves = THREADS / 64;
    extern __shared__ uint32_t s_count[];  // [waves][digits], [digits] totals, [digits] bases
    __shared__ int64_t s_tmp[2 * kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int digits = (int)a.dim + 1;
    uint32_t *s_total = s_count + kWaves * digits, *s_base = s_total + digits;
    for (int i = threadIdx.x; i < kWaves * digits; i += THREADS) s_count[i] = 0;
    __syncthreads();
    uint32_t *mine = s_count + wave * digits;
    const uint32_t steps = (a.rows + THREADS - 1) / THREADS;
    const uint32_t first = wave * 64 * steps;
    for (uint32_t i = 0; i < steps; ++i) {
        const uint32_t e = first + i * 64 + lane;
        const bool valid = e < a.rows;
        const uint32_t d = valid ? group_key(a.index[e], a.dim) : 0u;
        const uint64_t same = same_digit(d, a.bits, valid);
        if (valid && (same & ((uint64_t(1) << lane) - 1)) == 0) mine[d] += popc64(same);
        wave_lds_sync();
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += THREADS) {
        uint32_t n = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) n += s_count[w * digits + d];
        s_total[d] = n;
    }
    __syncthreads();
    digit_bases<THREADS>(s_total, digits, s_base, s_tmp);
    for (int d = threadIdx.x; d < digits; d += THREADS) {
        uint32_t at = s_base[d];
        a.offsets[d] = at;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const uint32_t n = s_count[w * digits + d];
            s_count[w * digits + d] = at;
            at += n;
        }
    }
    __syncthreads();
    for (uint32_t i = 0; i < steps; ++i) {
        const uint32_t e = first + i * 64 + lane;
        const bool valid = e < a.rows;
        const uint32_t d = valid ? group_key(a.index[e], a.dim) : 0u;
        const uint64_t same = same_digit(d, a.bits, valid);
        const uint32_t before = popc64(same & ((uint64_t(1) << lane) - 1));
        const uint32_t at = mine[d];
        wave_lds_sync();
        if (valid) {
            if (before == 0) mine[d] = at + popc64(same);
            a.order[at + before] = a.fanout > 1 ? e / a.fanout : e;
            a.position[e] = d < a.dim ? (int64_t)(at + before) : -1;
        }
        wave_lds_sync();
    }
}

struct GroupPlan {
    bool small;
    int passes, bits;
    int64_t tiles;
    size_t hist, totals, pairs, bytes;  // bytes of each part
};

GroupPlan group_plan(int64_t rows, int64_t dim) {
    GroupPlan p{};
    int bits = 1;
    while ((dim >> bits) != 0) ++bits;  // keys 0 .. dim
    p.passes = (bits + kGroupMaxBits - 1) / kGroupMaxBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.small = rows <= kGroupSmallRows && dim <= kGroupSmallDim;
    if (p.small) return p;
    p.tiles = (rows + kGroupTile - 1) / kGroupTile;
    auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
    p.hist = up((size_t)p.tiles * 4 << p.bits);
    p.totals = up(size_t(4) << p.bits);
    p.pairs = p.passes > 1 ? up((size_t)rows * 4) : 0;
    p.bytes = p.hist + p.totals + 4 * p.pairs;
    return p;
}

// Groups without an entry: every offset is 0.
__global__ __launch_bounds__(kGroupThreads) void group_none(int64_t *offsets, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * kGroupThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kGroupThreads)
        offsets[i] = 0;
}

}  // namespace segred

using namespace segred;

extern "C" int64_t segred_group_workspace(int64_t rows, int64_t dim_size) {
    if (rows < 1 || dim_size < 0 || rows > INT32_MAX || dim_size > INT32_MAX - 1) return 0;
    return (int64_t)group_plan(rows, dim_size).bytes;
}

extern "C" int segred_group(const int64_t *index, int64_t rows, int64_t fanout, int64_t dim_size, int64_t *order,
                            int64_t *position, int64_t *offsets, void *workspace, int64_t workspace_bytes,
                            hipStream_t stream) {
    if (rows < 0 || fanout < 1 || dim_size < 0 || !offsets) return SEGRED_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!index || !order || !position)) return SEGRED_ERR_INVALID_ARGUMENT;
    if (!aligned(index, 8) || !aligned(order, 8) || !aligned(position, 8) || !aligned(offsets, 8) || !aligned(workspace, 16))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (rows > INT32_MAX || dim_size > INT32_MAX - 1 || fanout > INT32_MAX) return SEGRED_ERR_UNSUPPORTED;
    if (rows == 0) {
        const unsigned grid = (unsigned)std::min<int64_t>((dim_size + kGroupThreads) / kGroupThreads, 4096);
        timed_launch_ggl(false, group_none, dim3(grid), dim3(kGroupThreads), 0, stream, offsets, dim_size + 1);
        return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
    }
    const GroupPlan p = group_plan(rows, dim_size);
    if (p.bytes > 0 && (!workspace || workspace_bytes < (int64_t)p.bytes)) return SEGRED_ERR_INVALID_ARGUMENT;

    GroupArgs a{};
    a.index = index;
    a.order = order;
    a.position = position;
    a.offsets = offsets;
    a.rows = (uint32_t)rows;
    a.dim = (uint32_t)dim_size;
    a.fanout = (uint32_t)fanout;
    a.bits = p.bits;
    if (p.small) {
        const unsigned digits = a.dim + 1;
        if (rows <= 1024)
            timed_launch_ggl(true, group_small<256>, dim3(1), dim3(256), (4 + 2) * digits * 4, stream, a);
        else
            timed_launch_ggl(true, group_small<1024>, dim3(1), dim3(1024), (16 + 2) * digits * 4, stream, a);
        return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
    }
    char *w = static_cast<char *>(workspace);
    a.hist = reinterpret_cast<uint32_t *>(w);
    a.totals = reinterpret_cast<uint32_t *>(w + p.hist);
    a.tiles = (uint32_t)p.tiles;
    uint32_t *pair[2][2];
    for (int i = 0; i < 4; ++i) pair[i >> 1][i & 1] = reinterpret_cast<uint32_t *>(w + p.hist + p.totals + i * p.pairs);
    const unsigned digits = 1u << p.bits;
    for (int pass = 0; pass < p.passes; ++pass) {
        a.shift = pass * p.bits;
        a.first = pass == 0;
        a.last = pass == p.passes - 1;
        a.keys_in = pair[(pass + 1) & 1][0];
        a.entries_in = pair[(pass + 1) & 1][1];
        a.keys_out = p.passes > 1 ? pair[pass & 1][0] : nullptr;
        a.entries_out = pair[pass & 1][1];
        timed_launch_ggl(true, group_count, dim3((unsigned)p.tiles), dim3(kGroupThreads), kGroupWaves * digits * 4, stream, a);
        timed_launch_ggl(false, group_scan, dim3(digits), dim3(kGroupThreads), 0, stream, a);
        timed_launch_ggl(true, group_place, dim3((unsigned)p.tiles), dim3(kGroupThreads), (kGroupWaves + 1) * digits * 4,
                         stream, a);
        if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    }
    if (p.passes > 1) {
        const unsigned grid = (unsigned)(((int64_t)dim_size + kGroupThreads) / kGroupThreads);
        timed_launch_ggl(false, group_bounds, dim3(grid), dim3(kGroupThreads), 0, stream, (const uint32_t *)a.keys_out,
                         a.rows, a.dim, offsets);
        if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    }
    return SEGRED_OK;
}
