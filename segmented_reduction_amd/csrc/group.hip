// group.hip -- rows grouped by an index: a stable counting sort of the entries
// by the group they name, the place of each entry in it, and the offsets of
// the groups.  No atomics: entries are ranked among the 64 lanes of a wave by
// ballots, waves by their place in the tile and tiles by a scan, so that the
// result is the one stable order.
//
// The index is sorted by digits of up to 11 bits, the lowest first: per pass a
// count of each tile's digits, a scan of those counts over the tiles, and the
// move.  A tile is put in order in LDS before it is written, so that its writes
// are runs, and consecutive tiles go to one XCD, whose L2 joins the ends of
// their runs.  An entry's place after two passes is read through the places of
// the first (both written in order, and read along as many fronts as there are
// digits) instead of being scattered: 4 million entries of 250,000 groups take
// 93 us, and took 304 with scattered places and unordered tiles.  Their 98 MB of
// input and output would take 21.  What bounds a move (21 us) is the work per
// entry in the vector units (the lanes of its digit, its rank, three passages
// through LDS); the places (24 us) are bound by the cache, which serves
// each of the scattered reads with a line of its own.
#include <algorithm>
#include <type_traits>

#include "internal.hpp"
#include "tile.hpp"
#include "wave.hpp"

namespace segred {

// One digit pass.  The first reads the index itself, the later ones the
// (key, entry) pairs the pass before wrote.
struct GroupArgs {
    const int64_t *index;
    const uint32_t *keys_in, *entries_in;  // later passes
    uint32_t *keys_out, *entries_out;      // entries: all but the last pass
    int64_t *order;                        // last pass
    int64_t *position;                     // last pass, where there is one or there are more than two
    uint32_t *where;                       // place of each input of this pass (two passes)
    int64_t *offsets;                      // where there is one pass
    uint32_t *hist;                        // [tiles][digits] where few, else [digits][tiles]
    uint32_t *totals;                      // [digits]
    uint32_t rows, dim, tiles, fanout;
    int shift, bits;
    int first, last;
    int few;  // few tiles: group_place adds up their counts itself
};

constexpr int kGroupThreads = 512;
constexpr int kGroupWaves = kGroupThreads / 64;
// Entries per lane of a tile, 1,024 or 4,096 entries in all (tiles of 256 lanes
// and 16 entries each: 108 us for 4 million entries of 100,000 groups instead
// of 90).  Short ones up to 262,144 entries, so that there are tiles for more
// CUs: 33 us against 41 there for 100,000 groups and 16 against 18 for 500, but
// 1,048,576 entries of 1,000 groups take 29 against 23.  Where tiles and digits
// are few a workgroup adds up the counts of the tiles before its own, which
// saves the launch of the scan: 32,768 entries of 64 groups take 13 us so and
// 17 with it; but of 2,000 groups 25 against 18.
constexpr int kGroupShort = 2, kGroupLong = 8;
constexpr int64_t kGroupShortRows = 262144, kGroupFewTiles = 64, kGroupFewCounts = 32768;
constexpr int kGroupMaxBits = 11;
// Entries per lane where places are read through two passes (4 million entries
// of 250,000 groups: 4 are 4 us faster than 1, 8 no faster).
constexpr int kGroupEach = 4;
constexpr uint32_t kNoPlace = 0xffffffffu;

__device__ __forceinline__ uint32_t group_key(int64_t v, uint32_t dim) {
    return v >= 0 && v < (int64_t)dim ? (uint32_t)v : dim;  // entries of no group go behind the last one
}

// Lanes of the wave whose digit of BITS bits equals this lane's.
template <int BITS>
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool valid) {
    const uint64_t m = ballot(valid);
    uint32_t lo = (uint32_t)m, hi = (uint32_t)(m >> 32);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
        const uint32_t set = (uint32_t)((int32_t)(digit << (31 - b)) >> 31);  // all ones where the bit is 1
        const uint64_t with = ballot(set != 0);
        // m & ~(with ^ set), one instruction
        lo = __builtin_amdgcn_bitop3_b32(lo, (uint32_t)with, set, 0x90);
        hi = __builtin_amdgcn_bitop3_b32(hi, (uint32_t)(with >> 32), set, 0x90);
    }
    return (uint64_t)hi << 32 | lo;
}

// Keys of the wave's entries first, first + 64 ...: all loads are under way
// before the first is waited for, so entries behind the last read that one.
template <int STEPS>
__device__ __forceinline__ void load_keys(const GroupArgs &a, uint32_t first, uint32_t (&key)[STEPS]) {
    if (a.first) {
        int64_t v[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) v[i] = a.index[min(first + i * 64, a.rows - 1)];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) key[i] = group_key(v[i], a.dim);
    } else {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) key[i] = a.keys_in[min(first + i * 64, a.rows - 1)];
    }
}

// Sum of v over the threads before this one (all threads of the group), and
// over all of them.  s_tmp holds an entry per wave, free again after the next
// barrier.
template <int THREADS>
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t *s_tmp, uint32_t &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t x = v;
    x += dpp32<kDppRowShr1>(0, x);
    x += dpp32<kDppRowShr2>(0, x);
    x += dpp32<kDppRowShr4>(0, x);
    x += dpp32<kDppRowShr8>(0, x);
    x += dpp32<kDppRowBcast15, 0xA>(0, x);
    x += dpp32<kDppRowBcast31, 0xC>(0, x);
    if (lane == 63) s_tmp[wave] = x;
    __syncthreads();
    uint32_t before = x - v;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        const uint32_t n = s_tmp[w];
        before += w < wave ? n : 0u;
        total += n;
    }
    return before;
}

// Exclusive offsets of `digits` totals, at most MAX, into s_base (all threads
// of the group).  `totals` may be s_base itself.
template <int THREADS, int MAX>
__device__ __forceinline__ void digit_bases(const uint32_t *totals, int digits, uint32_t *s_base, uint32_t *s_tmp) {
    constexpr int kPer = MAX / THREADS > 0 ? MAX / THREADS : 1;
    uint32_t v[kPer];
    uint32_t sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = threadIdx.x * kPer + j;
        v[j] = d < digits ? totals[d] : 0u;
        sum += v[j];
    }
    uint32_t total;
    uint32_t base = sum_before<THREADS>(sum, s_tmp, total);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = threadIdx.x * kPer + j;
        if (d < digits) s_base[d] = base;
        base += v[j];
    }
    __syncthreads();
}

// Entries of each digit in each tile.
template <int BITS, int STEPS>
__global__ __launch_bounds__(kGroupThreads) void group_count(GroupArgs a) {
    extern __shared__ uint32_t s_count[];  // [waves][digits]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int digits = 1 << BITS, kTile = kGroupThreads * STEPS;
    for (int i = threadIdx.x; i < kGroupWaves * digits; i += kGroupThreads) s_count[i] = 0;
    __syncthreads();
    uint32_t *mine = s_count + wave * digits;
    const uint32_t tile = (uint32_t)xcd_tile(a.tiles);
    const uint32_t first = tile * kTile + wave * 64 * STEPS;
    uint32_t key[STEPS];
    load_keys<STEPS>(a, first + lane, key);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const bool valid = first + i * 64 + lane < a.rows;
        const uint32_t d = (key[i] >> a.shift) & (digits - 1);
        const uint64_t same = same_digit<BITS>(d, valid);
        if (valid && (same & ((uint64_t(1) << lane) - 1)) == 0) mine[d] += popc64(same);
        wave_lds_sync();
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kGroupThreads) {
        uint32_t n = 0;
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) n += s_count[w * digits + d];
        a.hist[a.few ? (size_t)tile * digits + d : (size_t)d * a.tiles + tile] = n;
    }
}

// Exclusive scan over the tiles of each digit (one workgroup per digit).
__global__ __launch_bounds__(kGroupThreads) void group_scan(GroupArgs a) {
    __shared__ uint32_t s_tmp[kGroupWaves];
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
        uint32_t total;
        uint32_t base = running + sum_before<kGroupThreads>(sum, s_tmp, total);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (t + j < a.tiles) row[t + j] = base;
            base += v[j];
        }
        running += total;
        __syncthreads();
    }
    if (threadIdx.x == 0) a.totals[blockIdx.x] = running;
}

// Moves each entry to its place in this pass's order.  Counts within a tile have
// 16 bits, and keys and entries pass through the same part of LDS one after the
// other, so that a CU holds four workgroups of 512 digits (its 32 waves).
template <int BITS, int STEPS>
__global__ __launch_bounds__(kGroupThreads) void group_place(GroupArgs a) {
    extern __shared__ uint32_t s_base[];  // [digits] bases, [digits] places, [tile] keys or entries, [waves][digits] counts
    __shared__ uint32_t s_tmp[kGroupWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int digits = 1 << BITS, kTile = kGroupThreads * STEPS;
    static_assert(kTile < 65536, "the counts of a tile have 16 bits");
    uint32_t *s_place = s_base + digits, *s_item = s_place + digits;
    uint16_t *s_count = reinterpret_cast<uint16_t *>(s_item + kTile);
    for (int i = threadIdx.x; i < kGroupWaves * digits / 2; i += kGroupThreads)
        reinterpret_cast<uint32_t *>(s_count)[i] = 0;
    const uint32_t tile = (uint32_t)xcd_tile(a.tiles);
    if (a.few) {
        for (int d = threadIdx.x; d < digits; d += kGroupThreads) {
            uint32_t before = 0, n = 0;
#pragma unroll 8
            for (uint32_t t = 0; t < a.tiles; ++t) {
                const uint32_t c = a.hist[(size_t)t * digits + d];
                before += t < tile ? c : 0u;
                n += c;
            }
            s_base[d] = n;
            s_place[d] = before;  // until the digits of this tile are known
            if (a.last && tile == 0) a.totals[d] = n;
        }
        __syncthreads();
        digit_bases<kGroupThreads, digits>(s_base, digits, s_base, s_tmp);
    } else {
        digit_bases<kGroupThreads, digits>(a.totals, digits, s_base, s_tmp);
    }
    if (a.offsets && tile == 0)  // one pass: the digits are the groups
        for (uint32_t d = threadIdx.x; d <= a.dim; d += kGroupThreads) a.offsets[d] = s_base[d];
    uint16_t *mine = s_count + wave * digits;
    const uint32_t begin = tile * kTile, first = begin + wave * 64 * STEPS;
    const int have = (int)min((uint32_t)kTile, a.rows - begin);
    uint32_t key[STEPS], entry[STEPS], rank[STEPS];
    load_keys<STEPS>(a, first + lane, key);
    if (a.first) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) entry[i] = first + i * 64 + lane;
    } else {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) entry[i] = a.entries_in[min(first + i * 64 + lane, a.rows - 1)];
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const bool valid = first + i * 64 + lane < a.rows;
        const uint32_t d = (key[i] >> a.shift) & (digits - 1);
        const uint64_t same = same_digit<BITS>(d, valid);
        const uint32_t before = popc64(same & ((uint64_t(1) << lane) - 1));
        const uint32_t seen = mine[d];
        rank[i] = seen + before;
        wave_lds_sync();
        if (valid && before == 0) mine[d] = (uint16_t)(seen + popc64(same));
        wave_lds_sync();
    }
    __syncthreads();
    // digit totals of the tile, and each wave's place among them
    for (int d = threadIdx.x; d < digits; d += kGroupThreads) {
        uint32_t n = 0;
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) {
            const uint32_t c = s_count[w * digits + d];
            s_count[w * digits + d] = (uint16_t)n;
            n += c;
        }
        s_base[d] += a.few ? s_place[d] : a.hist[(size_t)d * a.tiles + tile];
        s_place[d] = n;
    }
    __syncthreads();
    digit_bases<kGroupThreads, digits>(s_place, digits, s_place, s_tmp);
    // s_base: what turns a place in the tile into one in the order
    for (int d = threadIdx.x; d < digits; d += kGroupThreads) s_base[d] -= s_place[d];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const uint32_t e = first + i * 64 + lane;
        if (e >= a.rows) continue;
        const uint32_t d = (key[i] >> a.shift) & (digits - 1);
        const uint32_t at = s_place[d] + mine[d] + rank[i];
        rank[i] = at;
        s_item[at] = key[i];
        const uint32_t to = s_base[d] + at;
        if (a.where) a.where[e] = a.last && key[i] >= a.dim ? kNoPlace : to;
        else if (a.first && a.last) a.position[e] = key[i] < a.dim ? (int64_t)to : -1;
    }
    __syncthreads();
    uint32_t to[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int at = i * kGroupThreads + threadIdx.x;
        if (at >= have) continue;
        key[i] = s_item[at];
        to[i] = s_base[(key[i] >> a.shift) & (digits - 1)] + at;
        if (a.keys_out) a.keys_out[to[i]] = key[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (first + i * 64 + lane < a.rows) s_item[rank[i]] = entry[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int at = i * kGroupThreads + threadIdx.x;
        if (at >= have) continue;
        const uint32_t from = s_item[at];
        if (a.last) {
            a.order[to[i]] = a.fanout > 1 ? from / a.fanout : from;
            if (!a.where && !a.first) a.position[from] = key[i] < a.dim ? (int64_t)to[i] : -1;
        } else {
            a.entries_out[to[i]] = from;
        }
    }
}

// After several passes: offsets[s] = the first place whose key is not below s,
// looked for among the entries of s's last digit; and after two, the places of
// the entries through those of both passes.
__global__ __launch_bounds__(kGroupThreads) void group_bounds(GroupArgs a, const uint32_t *where, int64_t *offsets,
                                                              int64_t *position, uint32_t place_wgs) {
    if (blockIdx.x < place_wgs) {
        const uint32_t first = (uint32_t)xcd_tile(place_wgs) * kGroupThreads * kGroupEach + threadIdx.x;
        uint32_t at[kGroupEach], to[kGroupEach];
#pragma unroll
        for (int i = 0; i < kGroupEach; ++i) {
            const uint32_t e = first + i * kGroupThreads;
            at[i] = e < a.rows ? where[e] : 0;
        }
#pragma unroll
        for (int i = 0; i < kGroupEach; ++i) to[i] = a.where[at[i]];
#pragma unroll
        for (int i = 0; i < kGroupEach; ++i) {
            const uint32_t e = first + i * kGroupThreads;
            if (e < a.rows) position[e] = to[i] == kNoPlace ? -1 : (int64_t)to[i];
        }
        return;
    }
    __shared__ uint32_t s_base[(1 << kGroupMaxBits) + 1];
    __shared__ uint32_t s_tmp[kGroupWaves];
    const int digits = 1 << a.bits;
    digit_bases<kGroupThreads, 1 << kGroupMaxBits>(a.totals, digits, s_base, s_tmp);
    if (threadIdx.x == 0) s_base[digits] = a.rows;
    __syncthreads();
    const uint64_t s = (uint64_t)(blockIdx.x - place_wgs) * kGroupThreads + threadIdx.x;
    if (s > a.dim) return;
    const uint32_t d = (uint32_t)(s >> a.shift);
    uint32_t lo = s_base[d], hi = s_base[d + 1];
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (a.keys_out[mid] < s) lo = mid + 1;
        else hi = mid;
    }
    offsets[s] = lo;
}

// Few entries and few groups: one workgroup, one launch (8,192 entries of 256
// groups take 14 us so and 13 in tiles).  Each wave counts
// its stretch, the counts are scanned over (digit, wave), and a second walk
// over the stretch places the entries.
constexpr int kGroupSmallRows = 4096;
constexpr int kGroupSmallDim = 2047;
template <int THREADS, int BITS>
__global__ __launch_bounds__(THREADS) void group_small(GroupArgs a) {
    constexpr int kWaves = THREADS / 64;
    extern __shared__ uint32_t s_count[];  // [waves][digits], [digits] totals, [digits] bases
    __shared__ uint32_t s_tmp[kWaves];
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
        const uint64_t same = same_digit<BITS>(d, valid);
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
    digit_bases<THREADS, 1 << BITS>(s_total, digits, s_base, s_tmp);
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
        const uint64_t same = same_digit<BITS>(d, valid);
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

// Calls f with the number of bits as a constant.
template <int B = 1, typename F>
void for_bits(int bits, F f) {
    if (bits == B) f(std::integral_constant<int, B>{});
    else if constexpr (B < kGroupMaxBits) for_bits<B + 1>(bits, f);
}

struct GroupPlan {
    bool small;
    int passes, bits, steps;
    int64_t tiles;
    size_t hist, totals, pairs, bytes;  // bytes of each part (pairs: of one array of a pass)
};

GroupPlan group_plan(int64_t rows, int64_t dim) {
    GroupPlan p{};
    int bits = 1;
    while ((dim >> bits) != 0) ++bits;  // keys 0 .. dim
    p.passes = (bits + kGroupMaxBits - 1) / kGroupMaxBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.small = rows <= kGroupSmallRows && dim <= kGroupSmallDim;
    if (p.small) return p;
    p.steps = rows <= kGroupShortRows ? kGroupShort : kGroupLong;
    p.tiles = (rows + kGroupThreads * p.steps - 1) / (kGroupThreads * p.steps);
    auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
    p.hist = up((size_t)p.tiles * 4 << p.bits);
    p.totals = up(size_t(4) << p.bits);
    // two passes: (key, entry) after the first, keys after the second, the
    // places of both; more: (key, entry) twice, in turn
    p.pairs = p.passes > 1 ? up((size_t)rows * 4) : 0;
    p.bytes = p.hist + p.totals + (p.passes == 2 ? 5 : 4) * p.pairs;
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
    a.rows = (uint32_t)rows;
    a.dim = (uint32_t)dim_size;
    a.fanout = (uint32_t)fanout;
    a.bits = p.bits;
    if (p.small) {
        a.position = position;
        a.offsets = offsets;
        const unsigned digits = a.dim + 1;
        for_bits(p.bits, [&](auto bits) {
            constexpr int kBits = decltype(bits)::value;
            if (rows <= 1024)
                timed_launch_ggl(true, (group_small<256, kBits>), dim3(1), dim3(256), (4 + 2) * digits * 4, stream, a);
            else
                timed_launch_ggl(true, (group_small<1024, kBits>), dim3(1), dim3(1024), (16 + 2) * digits * 4, stream, a);
        });
        return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
    }
    char *w = static_cast<char *>(workspace);
    a.hist = reinterpret_cast<uint32_t *>(w);
    a.totals = reinterpret_cast<uint32_t *>(w + p.hist);
    a.tiles = (uint32_t)p.tiles;
    a.few = p.tiles <= kGroupFewTiles && p.tiles << p.bits <= kGroupFewCounts;
    auto array = [&](int i) { return reinterpret_cast<uint32_t *>(w + p.hist + p.totals + i * p.pairs); };
    const unsigned digits = 1u << p.bits;
    const size_t count_lds = kGroupWaves * digits * 4;
    const size_t place_lds = kGroupWaves * digits * 2 + 2 * digits * 4 + kGroupThreads * p.steps * 4;
    a.position = position;
    for (int pass = 0; pass < p.passes; ++pass) {
        a.shift = pass * p.bits;
        a.first = pass == 0;
        a.last = pass == p.passes - 1;
        a.offsets = p.passes == 1 ? offsets : nullptr;
        if (p.passes == 2) {
            a.keys_in = array(0);
            a.entries_in = array(1);
            a.keys_out = array(pass == 0 ? 0 : 2);
            a.entries_out = array(1);
            a.where = array(3 + pass);
        } else if (p.passes > 2) {
            a.keys_in = array(pass & 1 ? 0 : 2);
            a.entries_in = array(pass & 1 ? 1 : 3);
            a.keys_out = array(pass & 1 ? 2 : 0);
            a.entries_out = array(pass & 1 ? 3 : 1);
        }
        for_bits(p.bits, [&](auto bits) {
            constexpr int kBits = decltype(bits)::value;
            const bool small_tile = p.steps == kGroupShort;
            const dim3 grid((unsigned)p.tiles), block(kGroupThreads);
            if (small_tile) timed_launch_ggl(true, (group_count<kBits, kGroupShort>), grid, block, (unsigned)count_lds, stream, a);
            else timed_launch_ggl(true, (group_count<kBits, kGroupLong>), grid, block, (unsigned)count_lds, stream, a);
            if (!a.few) timed_launch_ggl(false, group_scan, dim3(digits), block, 0, stream, a);
            if (small_tile) timed_launch_ggl(true, (group_place<kBits, kGroupShort>), grid, block, (unsigned)place_lds, stream, a);
            else timed_launch_ggl(true, (group_place<kBits, kGroupLong>), grid, block, (unsigned)place_lds, stream, a);
        });
        if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    }
    if (p.passes > 1) {
        const uint32_t bounds = (uint32_t)((dim_size + kGroupThreads) / kGroupThreads);
        const uint32_t places = p.passes == 2 ? (a.rows + kGroupThreads * kGroupEach - 1) / (kGroupThreads * kGroupEach) : 0;
        timed_launch_ggl(false, group_bounds, dim3(bounds + places), dim3(kGroupThreads), 0, stream, a,
                         (const uint32_t *)array(3), offsets, position, places);
        if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    }
    return SEGRED_OK;
}
