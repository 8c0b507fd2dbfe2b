// norm.hip -- layer norm (and the norm by the root mean square) of rows, and
// its gradient with the sums of the weight's and the bias's over the rows.
//
// With m the mean of a row (0 without centering), r = 1 / sqrt(mean((x - m)^2) +
// eps) and u = (x - m) r,
//   out = u w + b
//   dx  = r (gw - mean(gw) - u mean(gw u)), gw = g w   (mean(gw) only if centered)
//   dw  = sum over rows of g u, db = sum over rows of g.
// A row's mean is no part of the result, so errors in proportion to it must not be one
// either: a row is taken around a number near its mean, the shift (its first element +
// the mean of the differences from it, so that a constant row gives zeros exactly), and
// the sums of x - shift and of its squares then give what the shift misses the mean by,
// and the squares around the mean.
// Both directions move their rows once and are bound by memory: a row is held
// in registers (up to 16,384 elements; the gradient of float32 rows above 8,192 spills
// 36 to 49 of a lane's 256), the statistics are found there in two
// passes (shift, then sums around it), and the gradient finds them again
// instead of reading them.  (16,384 x 4,096 bfloat16 forward 50 us, 5.3 TB/s; 16,384 x
// 2,048 forward 26 and gradient 39 + 5 for the join of the workgroups' sums, 5.3 TB/s.)
#include <algorithm>
#include <cmath>

#include "internal.hpp"
#include "tile.hpp"

namespace segred {

struct NormArgs {
    const char *grad, *values;  // grad: the gradient call's
    const void *weight, *bias;  // null: ones, zeros
    int weight_f32;             // else of the values' type
    int64_t N;
    int K, center;
    float eps;
    char *out;       // or the gradient of the values
    void *grad_weight, *grad_bias;  // null: not asked for
    float *partial;  // [blocks][2][K]; null: one workgroup has the whole sums
    int64_t blocks;
};

// Column of unit u of a row's lane `l` of L.
template <typename T, int L>
__device__ __forceinline__ int norm_col(int u, int l) { return (u * L + l) * kUnit<T>; }

// The first min(n, unit) elements of a unit at any element boundary.
template <typename T>
__device__ __forceinline__ void store_unit(char *to, const float (&c)[kUnit<T>], int n) {
    typedef u32x4 __attribute__((aligned(2))) unit2;
    typedef u32x4 __attribute__((aligned(4))) unit4;
    union {
        u32x4 v;
        T e[kUnit<T>];
    } x;
#pragma unroll
    for (int e = 0; e < kUnit<T>; ++e) x.e[e] = (T)c[e];
    if (n >= kUnit<T>) {
        if constexpr (sizeof(T) == 2) *(__attribute__((address_space(1))) unit2 *)to = x.v;
        else *(__attribute__((address_space(1))) unit4 *)to = x.v;
    } else {
#pragma unroll
        for (int e = 0; e < kUnit<T>; ++e)
            if (e < n) reinterpret_cast<T *>(to)[e] = x.e[e];
    }
}

// Unit u of a row that begins at `row` (0: no row), zeros behind its end.  WHOLE:
// rows hold whole units, so that each is there or not.
template <typename T, int L, bool WHOLE>
__device__ __forceinline__ u32x4 norm_load(uint64_t row, int u, int l, int K) {
    const int c = norm_col<T, L>(u, l);
    const uint64_t at = row + (uint64_t)c * sizeof(T);
    if constexpr (WHOLE) return load_whole<T>(row != 0 && c < K ? at : (uint64_t)zero_unit());
    else return load_unit<T>(at, row != 0 ? K - c : 0);
}
template <typename T, int L, bool WHOLE>
__device__ __forceinline__ void norm_store(uint64_t row, int u, int l, int K, const float (&y)[kUnit<T>]) {
    const int c = norm_col<T, L>(u, l);
    if (c < K) store_unit<T>((char *)(row + (uint64_t)c * sizeof(T)), y, WHOLE ? kUnit<T> : K - c);
}

template <typename T>
__device__ __forceinline__ float param(const void *p, int f32, int c) {
    return f32 ? static_cast<const float *>(p)[c] : (float)static_cast<const T *>(p)[c];
}
// Those of a unit's columns, `left` of which exist; the others, and all without
// a parameter, are `none`.
template <typename T>
__device__ __forceinline__ void param_unit(float (&to)[kUnit<T>], const void *p, int f32, int c, int left, float none) {
    constexpr int N = kUnit<T>;
    if (!p) {
#pragma unroll
        for (int e = 0; e < N; ++e) to[e] = none;
    } else if (f32 || sizeof(T) == 4) {
        u32x4 v[N / 4];
#pragma unroll
        for (int q = 0; q < N / 4; ++q) v[q] = load_unit<float>((uint64_t)p + (uint64_t)c * 4 + q * 16, left - 4 * q);
#pragma unroll
        for (int e = 0; e < N; ++e) to[e] = __uint_as_float(v[e / 4][e % 4]);
    } else {
        const u32x4 v = load_unit<T>((uint64_t)p + (uint64_t)c * sizeof(T), left);
#pragma unroll
        for (int e = 0; e < N; ++e) to[e] = element<T>(v, e);
    }
}
template <typename T>
__device__ __forceinline__ void put_param(void *p, int f32, int64_t c, float v) {
    if (f32) static_cast<float *>(p)[c] = v;
    else static_cast<T *>(p)[c] = (T)v;
}

// Sums over the lanes of a row that are in other waves too: Q values a wave
// meet in LDS, two places in turn, so that one barrier a row is enough.
template <int L, int Q>
struct RowJoin {
    static constexpr int kWaves = (L > 256 ? L : 256) / 64, kRowWaves = L > 64 ? L / 64 : 1;
    float (*s)[kWaves][Q];  // [2][waves][Q]
    int turn = 0;
    // The values of the row's waves, there until the call after the next.
    __device__ __forceinline__ const float (*meet(const float (&v)[Q], int wave, int lane))[Q] {
        float (*p)[Q] = s[turn];
        turn ^= 1;
        if (lane == 0)
#pragma unroll
            for (int q = 0; q < Q; ++q) p[wave][q] = v[q];
        __syncthreads();
        return p + wave / kRowWaves * kRowWaves;
    }
};

// The first element of a row, or of the wave's part of it, from its lane 0 of LW.
template <int LW>
__device__ __forceinline__ float norm_first(float v) {
    static_assert(LW == 64 || LW == 16, "a wave, or a row of its lanes");
    if constexpr (LW == 64) return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
    return dpp_take<kDppRowFirst>(v);
}

// Elements of a row that wave `part` of its L lanes holds.
template <typename T, int L, int U>
__device__ __forceinline__ int norm_part(int part, int K) {
    int n = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) n += max(0, min(64 * kUnit<T>, K - norm_col<T, L>(u, part * 64)));
    return n;
}

// A number near the mean of a row (or part) of n elements, where 1 / n = per: `first`, its
// first element, + the mean of the differences from that, so that it is `first` itself
// where all are equal.  Of 16-bit elements (2,048 at most a wave) such a row's sum is exact, and
// the differences' is found from it; float elements are subtracted one by one.
template <typename T, int L, int U, bool WHOLE, typename F>
__device__ __forceinline__ float norm_shift(float first, float n, float per, int l, int K, F x) {
    constexpr int N = kUnit<T>, LW = L > 64 ? 64 : L;
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int left = K - norm_col<T, L>(u, l);
        const float m = left > 0 ? first : 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) sum += sizeof(T) == 2 ? x(u, e) : x(u, e) - (WHOLE || e < left ? m : 0.f);
    }
    sum = lanes_sum<LW>(sum);
    if constexpr (sizeof(T) == 2) sum = fmaf(-n, first, sum);
    return fmaf(sum, per, first);
}

// The mean of a row from its parts, each with a shift and the sum of its elements'
// differences from it, as the first part's shift and what the mean is above that.
struct NormParts {
    float base, mean;
};
template <typename T, int L, int U, int UNROLL, typename P>
__device__ __forceinline__ NormParts norm_join_parts(P p, int K, float per) {
    NormParts t{p[0][0], p[0][1]};
#pragma unroll UNROLL
    for (int q = 1; q < L / 64; ++q) t.mean += fmaf((float)norm_part<T, L, U>(q, K), p[q][0] - t.base, p[q][1]);
    t.mean *= per;
    return t;
}

// L lanes hold a row, E elements each.  A workgroup walks rows with its weight
// and bias in registers; the next row is on its way while one is worked on.
template <int L> constexpr int kNormThreads = L > 256 ? L : 256;

// What a lane of these kernels goes through: rows `first`, `first` + stride, ..., one
// per L lanes, as addresses; a row past the last has address 0.
template <int L>
struct NormWalk {
    int64_t row, step;
    uint64_t row_bytes;
    __device__ __forceinline__ NormWalk(int64_t rows_each, int K, int element) {
        int at = threadIdx.x / L;
        if constexpr (L >= 64) at = __builtin_amdgcn_readfirstlane(at);
        row = (int64_t)blockIdx.x * rows_each + at;
        step = (int64_t)gridDim.x * rows_each;
        row_bytes = (uint64_t)K * element;
    }
    __device__ __forceinline__ uint64_t of(const void *base, int64_t r, int64_t rows) const {
        return r < rows ? (uint64_t)base + (uint64_t)r * row_bytes : 0;
    }
};

template <typename T, int L, int E, bool WHOLE>
__global__ __launch_bounds__(kNormThreads<L>) void norm_rows(NormArgs a) {
    constexpr int kRows = kNormThreads<L> / L, N = kUnit<T>, U = E / N, W = L > 64 ? L / 64 : 1;
    constexpr int LW = L > 64 ? 64 : L;  // lanes of a row in one wave
    __shared__ float s_join[2][kNormThreads<L> / 64][3];
    const int l = threadIdx.x % L, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), K = a.K;
    const int part = wave % W;
    RowJoin<L, 3> join{s_join};
    const float per = 1.f / (float)K;
    float w[U][N], b[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = norm_col<T, L>(u, l);
        param_unit<T>(w[u], a.weight, a.weight_f32, c, K - c, 1.f);
        param_unit<T>(b[u], a.bias, a.weight_f32, c, K - c, 0.f);
    }
    const float count = W > 1 ? (float)norm_part<T, L, U>(part, K) : (float)K;
    const float own = 1.f / fmaxf(count, 1.f);

    NormWalk<L> at(kRows, K, sizeof(T));
    u32x4 next[U];
    auto fetch = [&](int64_t r) {
        const uint64_t from = at.of(a.values, r, a.N);
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = norm_load<T, L, WHOLE>(from, u, l, K);
    };
    fetch(at.row);
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.N; first += at.step, at.row += at.step) {
        float x[U][N], shift = 0.f, over = 0.f, m2 = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < N; ++e) x[u][e] = element<T>(next[u], e);
        fetch(at.row + at.step);
        if (a.center) {
            shift = norm_shift<T, L, U, WHOLE>(norm_first<LW>(x[0][0]), count, W > 1 ? own : per, l, K,
                                               [&](int u, int e) { return x[u][e]; });
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int left = K - norm_col<T, L>(u, l);
            const float m = left > 0 ? shift : 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                x[u][e] -= WHOLE || e < left ? m : 0.f;
                over += x[u][e];
                m2 = fmaf(x[u][e], x[u][e], m2);
            }
        }
        m2 = lanes_sum<LW>(m2);
        over = a.center ? lanes_sum<LW>(over) : 0.f;
        float rest = -over * per;  // the shift less the mean
        if constexpr (W > 1) {
            // the parts' sums around shifts of their own, joined
            const float v[3] = {shift, over, m2};
            const auto p = join.meet(v, wave, lane);
            const NormParts t = norm_join_parts<T, L, U, W>(p, K, per);
            m2 = 0.f;
#pragma unroll
            for (int q = 0; q < W; ++q) {
                const float d = p[q][0] - t.base - t.mean;
                m2 += fmaf(d, fmaf((float)norm_part<T, L, U>(q, K), d, 2.f * p[q][1]), p[q][2]);
            }
            rest = shift - t.base - t.mean;
        } else {
            m2 = fmaf(over, rest, m2);
        }
        const float r = 1.f / sqrtf(fmaf(m2, per, a.eps));
        rest *= r;
        const uint64_t to = at.of(a.out, at.row, a.N);
        if (to != 0)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float y[N];
#pragma unroll
                for (int e = 0; e < N; ++e) y[e] = fmaf(fmaf(x[u][e], r, rest), w[u][e], b[u][e]);
                norm_store<T, L, WHOLE>(to, u, l, K, y);
            }
    }
}

// The gradient.  A workgroup walks rows as above and adds up g u and g of its
// columns in registers; at the end its parts go to `partial`.  One exchange a
// row between waves: besides the shift, the sum and the squares, sum gw and the sum
// of gw (x - shift of this wave's part), which is corrected for the row's mean.
template <typename T, int L, int E, bool WHOLE>
__global__ __launch_bounds__(kNormThreads<L>) void norm_grad_rows(NormArgs a) {
    constexpr int kThreads = kNormThreads<L>, kRows = kThreads / L, N = kUnit<T>, U = E / N, W = L > 64 ? L / 64 : 1;
    constexpr int LW = L > 64 ? 64 : L;
    // Eight parts one at a time, except beside bfloat16 rows of whole units: the 40 numbers at
    // once do not fit the registers with a row's sums (k = 16,384, us at once / one at a time:
    // float32 105 / 86, float16 89 / 68, bfloat16 62 / 67; the forward call, which has none of
    // these sums, 25 / 31).
    constexpr int kTurn = W > 4 && !(WHOLE && __is_same(T, __bf16)) ? 1 : W;
    __shared__ float s_join[2][kThreads / 64][5];
    __shared__ float s_sums[kRows > 1 ? 2 * L * E : 1];
    const int l = threadIdx.x % L, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), K = a.K;
    const int part = wave % W;
    RowJoin<L, 5> join{s_join};
    const float per = 1.f / (float)K;
    float w[U][N], dw[U][N], db[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = norm_col<T, L>(u, l);
        param_unit<T>(w[u], a.weight, a.weight_f32, c, K - c, 1.f);
#pragma unroll
        for (int e = 0; e < N; ++e) dw[u][e] = db[u][e] = 0.f;
    }
    const float count = W > 1 ? (float)norm_part<T, L, U>(part, K) : (float)K;
    const float own = 1.f / fmaxf(count, 1.f);

    NormWalk<L> at(kRows, K, sizeof(T));
    u32x4 next_x[U], next_g[U];
    auto fetch = [&](int64_t r) {
        const uint64_t from_x = at.of(a.values, r, a.N), from_g = at.of(a.grad, r, a.N);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            next_x[u] = norm_load<T, L, WHOLE>(from_x, u, l, K);
            next_g[u] = norm_load<T, L, WHOLE>(from_g, u, l, K);
        }
    };
    fetch(at.row);
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.N; first += at.step, at.row += at.step) {
        u32x4 x[U], g[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = next_x[u];
            g[u] = next_g[u];
        }
        fetch(at.row + at.step);
        float shift = 0.f, over = 0.f, m2 = 0.f, c1 = 0.f, c2 = 0.f;
        if (a.center) {
            shift = norm_shift<T, L, U, WHOLE>(norm_first<LW>(element<T>(x[0], 0)), count, W > 1 ? own : per, l, K,
                                               [&](int u, int e) { return element<T>(x[u], e); });
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int left = K - norm_col<T, L>(u, l);
            const float m = left > 0 ? shift : 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = element<T>(x[u], e) - (WHOLE || e < left ? m : 0.f);
                const float gw = element<T>(g[u], e) * w[u][e];
                over += d;
                m2 = fmaf(d, d, m2);
                c1 += gw;
                c2 = fmaf(gw, d, c2);
            }
        }
        m2 = lanes_sum<LW>(m2);
        c1 = lanes_sum<LW>(c1);
        c2 = lanes_sum<LW>(c2);
        over = a.center ? lanes_sum<LW>(over) : 0.f;
        float rest = -over * per;  // the shift less the mean
        if constexpr (W > 1) {
            const float v[5] = {shift, over, m2, c1, c2};
            const auto p = join.meet(v, wave, lane);
            const NormParts t = norm_join_parts<T, L, U, kTurn>(p, K, per);
            m2 = c1 = c2 = 0.f;
#pragma unroll kTurn
            for (int q = 0; q < W; ++q) {
                const float d = p[q][0] - t.base - t.mean;
                m2 += fmaf(d, fmaf((float)norm_part<T, L, U>(q, K), d, 2.f * p[q][1]), p[q][2]);
                c1 += p[q][3];
                c2 += fmaf(p[q][3], d, p[q][4]);
            }
            rest = shift - t.base - t.mean;
        } else {
            m2 = fmaf(over, rest, m2);
            c2 = fmaf(c1, rest, c2);
        }
        const float r = 1.f / sqrtf(fmaf(m2, per, a.eps));
        const float along = c2 * r * per * r;               // mean(gw u) r
        const float level = a.center ? c1 * per * r : 0.f;  // mean(gw) r
        rest *= r;
        const uint64_t to = at.of(a.out, at.row, a.N);
        if (to != 0)  // past the last row g is 0, but r may be infinite
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float y[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float unit = fmaf(element<T>(x[u], e) - shift, r, rest), ge = element<T>(g[u], e);
                    y[e] = fmaf(ge * r, w[u][e], -fmaf(unit, along, level));
                    dw[u][e] = fmaf(ge, unit, dw[u][e]);
                    db[u][e] += ge;
                }
                norm_store<T, L, WHOLE>(to, u, l, K, y);
            }
    }
    if (!a.grad_weight && !a.grad_bias) return;

    // The rows of a wave, then of the workgroup, in order.
    if constexpr (LW < 64) {
#pragma unroll
        for (int i = 0; i < E; ++i)
            for (int s = 32; s >= LW; s >>= 1) {
                dw[i / N][i % N] += lane_get(dw[i / N][i % N], lane ^ s);
                db[i / N][i % N] += lane_get(db[i / N][i % N], lane ^ s);
            }
    }
    if constexpr (kRows > 1) {
        for (int v = 0; v < kThreads / 64 / W; ++v) {
            if (wave / W == v && lane < LW)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    float *p = s_sums + i * L + l, *q = p + L * E;
                    *p = v ? *p + dw[i / N][i % N] : dw[i / N][i % N];
                    *q = v ? *q + db[i / N][i % N] : db[i / N][i % N];
                }
            __syncthreads();
        }
        if (wave >= W || lane >= LW) return;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            dw[i / N][i % N] = s_sums[i * L + l];
            db[i / N][i % N] = s_sums[(E + i) * L + l];
        }
    }
    float *to = a.partial ? a.partial + (int64_t)blockIdx.x * 2 * K : nullptr;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = norm_col<T, L>(i / N, l) + i % N;
        if (c >= K) continue;
        if (to) {
            to[c] = dw[i / N][i % N];
            to[K + c] = db[i / N][i % N];
        } else {  // the only workgroup
            if (a.grad_weight) put_param<T>(a.grad_weight, a.weight_f32, c, dw[i / N][i % N]);
            if (a.grad_bias) put_param<T>(a.grad_bias, a.weight_f32, c, db[i / N][i % N]);
        }
    }
}

// Rows too long for registers: read again for each pass (from L2, mostly).
constexpr int kLongThreads = 512, kLongWaves = kLongThreads / 64;
__device__ __forceinline__ float long_sum(float v, float *s, int wave, int lane) {
    v = lanes_sum<64>(v);
    __syncthreads();
    if (lane == 0) s[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int q = 0; q < kLongWaves; ++q) v += s[q];
    return v;
}

template <typename T, bool GRAD>
__global__ __launch_bounds__(kLongThreads) void norm_long(NormArgs a) {
    __shared__ float s[kLongWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, K = a.K;
    const float per = 1.f / (float)K;
    float *part = GRAD && a.partial ? a.partial + (int64_t)blockIdx.x * 2 * K : nullptr;
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const T *x = reinterpret_cast<const T *>(a.values) + row * K;
        const T *g = reinterpret_cast<const T *>(a.grad) + row * K;
        T *out = reinterpret_cast<T *>(a.out) + row * K;
        float shift = 0.f, over = 0.f, m2 = 0.f, c1 = 0.f, c2 = 0.f;
        if (a.center) {
            const float first = (float)x[0];
            float sum = 0.f;
            for (int c = threadIdx.x; c < K; c += kLongThreads) sum += (float)x[c] - first;
            shift = fmaf(long_sum(sum, s, wave, lane), per, first);
        }
        for (int c = threadIdx.x; c < K; c += kLongThreads) {
            const float d = (float)x[c] - shift;
            over += d;
            m2 = fmaf(d, d, m2);
            if constexpr (GRAD) {
                const float gw = (float)g[c] * (a.weight ? param<T>(a.weight, a.weight_f32, c) : 1.f);
                c1 += gw;
                c2 = fmaf(gw, d, c2);
            }
        }
        over = a.center ? long_sum(over, s, wave, lane) : 0.f;
        const float rest = -over * per;
        m2 = fmaf(over, rest, long_sum(m2, s, wave, lane));
        const float r = 1.f / sqrtf(fmaf(m2, per, a.eps));
        if constexpr (GRAD) {
            c1 = long_sum(c1, s, wave, lane);
            const float level = a.center ? c1 * per : 0.f;
            const float along = fmaf(c1, rest, long_sum(c2, s, wave, lane)) * r * per;
            for (int c = threadIdx.x; c < K; c += kLongThreads) {
                const float unit = fmaf((float)x[c] - shift, r, rest * r), ge = (float)g[c];
                const float w = a.weight ? param<T>(a.weight, a.weight_f32, c) : 1.f;
                out[c] = (T)(r * (fmaf(ge, w, -level) - unit * along));
                if (part) {
                    part[c] = row == (int64_t)blockIdx.x ? ge * unit : fmaf(ge, unit, part[c]);
                    part[K + c] = row == (int64_t)blockIdx.x ? ge : part[K + c] + ge;
                }
            }
        } else {
            for (int c = threadIdx.x; c < K; c += kLongThreads) {
                const float w = a.weight ? param<T>(a.weight, a.weight_f32, c) : 1.f;
                out[c] = (T)fmaf(fmaf((float)x[c] - shift, r, rest * r), w, a.bias ? param<T>(a.bias, a.weight_f32, c) : 0.f);
            }
        }
    }
}

// Adds the workgroups' parts: 16 threads share a column, thread p takes parts
// p, p + 16, ... in that order, and these sums are added in order.
constexpr int kNormJoinCols = 64, kNormJoinParts = 16;
template <typename T>
__global__ __launch_bounds__(kNormJoinCols *kNormJoinParts) void norm_join(NormArgs a) {
    __shared__ float s_part[kNormJoinParts][kNormJoinCols];
    const int col = threadIdx.x % kNormJoinCols, part = threadIdx.x / kNormJoinCols;
    const int64_t c = (int64_t)blockIdx.x * kNormJoinCols + col, width = 2 * (int64_t)a.K;
    float sum = 0.f;
    if (c < width)
#pragma unroll 16
        for (int64_t p = part; p < a.blocks; p += kNormJoinParts) sum += a.partial[p * width + c];
    s_part[part][col] = sum;
    __syncthreads();
    if (part > 0 || c >= width) return;
#pragma unroll
    for (int q = 1; q < kNormJoinParts; ++q) sum += s_part[q][col];
    if (c < a.K) {
        if (a.grad_weight) put_param<T>(a.grad_weight, a.weight_f32, c, sum);
    } else if (a.grad_bias) {
        put_param<T>(a.grad_bias, a.weight_f32, c - a.K, sum);
    }
}

// Lanes and elements per lane of a row.  Few waves per row, so that fewer wait for
// each other, as long as the gradient's sums fit the registers.  33.5M bfloat16
// elements, forward / gradient in us (a copy of them takes 26):
//
//   k       512       1024      2048      4096      8192      16384
//           25 / 45   24 / 42   26 / 46   26 / 56   28 / 60   29 / 64   as below
//                     30 / 64   24 / 49                                 128 lanes (8, 16 each)
//                               29 / 65   43 / 83   30 / 77             twice the lanes, half the elements
//
// and of 16.8M float32 with k = 2,048 the gradient 43 by 128 lanes, 47 by 64.  The chosen
// ones once more, with the sums around a shift and parameters in float32 (of float32 16.8M):
//
//   k            512       1024      2048      4096      8192      16384     96        333
//   bfloat16     23 / 43   23 / 40   23 / 44   23 / 48   24 / 51   25 / 62   25 / 49   37 / 146
//   float16      23 / 44   23 / 41   22 / 44   23 / 47   24 / 51   25 / 68   24 / 49   38 / 145
//   float32      22 / 39   22 / 38   22 / 39   22 / 43   23 / 43   25 / 86   22 / 38   23 / 45
//
// (with sums around a rounded mean, whose errors grow with it, 22 / 44 of 96 and 34 / 144 of
// 333 bfloat16 elements; wide rows are not slower).  Held to 128 registers and so 4 waves a SIMD
// the gradient of 1,024 bfloat16 elements took 40.6 us, left alone 40.4.
struct NormShape {
    int lanes, elements;  // lanes 0: too long for registers
};
NormShape norm_shape(int64_t k, bool grad, bool wide) {
    if (k <= 128) return {16, 8};
    if (k <= 512) return {64, 8};
    if (k <= 1024) return {64, 16};
    if (k <= 2048) return grad && !wide ? NormShape{64, 32} : NormShape{128, 16};
    if (k <= 4096) return {256, 16};
    if (k <= 8192) return {256, 32};
    if (k <= 16384) return {512, 32};
    return {0, 0};
}

// Workgroups of a call, by its sizes alone, so that sums do not depend on the
// device: as many as it holds at a time (more read the parameters more often: k =
// 4,096 in 1,024 workgroups 24 us, in 4,096 27), and for the gradient fewer where
// their parts are long (k = 8,192 in 256 60 us, in 512 63; k = 512 in 512 50, in
// 768 46).  One workgroup takes the gradient of as many rows as it has in two rounds and
// leaves the sums itself (8 rows of 512: 4.8 us, 10.2 with the host's side, against 5.9 and
// 14.3 with the join; in four rounds 6.2 and 10.2, but rows of 8,192 16 and 14).
int64_t norm_blocks(const NormShape &s, int64_t rows, bool grad) {
    const int64_t row = (int64_t)s.lanes * s.elements;
    int64_t most = s.lanes == 0 ? 512 : s.lanes <= 128 ? 2048 : s.lanes == 256 ? 1024 : 512;
    if (grad) most = s.lanes == 0 || row > 4096 ? 256 : row <= 512 ? 768 : 512;
    const int64_t each = s.lanes > 0 && s.lanes < 256 ? 256 / s.lanes : 1;
    if (grad && s.lanes > 0 && rows <= 2 * each) return 1;
    return std::min(most, (rows + each - 1) / each);
}

// Bytes of the workgroups' sums.
int64_t norm_room(int64_t k, int64_t rows, bool wide) {
    const NormShape s = norm_shape(k, true, wide);
    const int64_t blocks = norm_blocks(s, rows, true);
    return blocks == 1 && s.lanes > 0 ? 0 : blocks * 2 * k * 4;
}

template <typename T, bool GRAD, int L, int E, bool WHOLE>
void norm_start_as(const NormArgs &a, hipStream_t st) {
    if constexpr (GRAD)
        timed_launch_ggl(true, (norm_grad_rows<T, L, E, WHOLE>), dim3((unsigned)a.blocks), dim3(kNormThreads<L>), 0, st, a);
    else
        timed_launch_ggl(true, (norm_rows<T, L, E, WHOLE>), dim3((unsigned)a.blocks), dim3(kNormThreads<L>), 0, st, a);
}
template <typename T, bool GRAD, int L, int E>
void norm_start(const NormArgs &a, hipStream_t st) {
    if (a.K % kUnit<T> == 0) norm_start_as<T, GRAD, L, E, true>(a, st);
    else norm_start_as<T, GRAD, L, E, false>(a, st);
}

template <typename T, bool GRAD>
int norm_dispatch(NormArgs a, hipStream_t st) {
    if (a.N > 0) {
        const NormShape s = norm_shape(a.K, GRAD, sizeof(T) == 4);
        const int row = s.lanes * s.elements;
        constexpr bool kMiddle = GRAD && sizeof(T) == 2;
        a.blocks = norm_blocks(s, a.N, GRAD);
        if (s.lanes == 0) timed_launch_ggl(true, (norm_long<T, GRAD>), dim3((unsigned)a.blocks), dim3(kLongThreads), 0, st, a);
        else if (s.lanes == 16) norm_start<T, GRAD, 16, 8>(a, st);
        else if (s.lanes == 64 && s.elements == 8) norm_start<T, GRAD, 64, 8>(a, st);
        else if (s.lanes == 64 && s.elements == 16) norm_start<T, GRAD, 64, 16>(a, st);
        else if (row == 2048) norm_start<T, GRAD, kMiddle ? 64 : 128, kMiddle ? 32 : 16>(a, st);
        else if (s.lanes == 256 && s.elements == 16) norm_start<T, GRAD, 256, 16>(a, st);
        else if (s.lanes == 256) norm_start<T, GRAD, 256, 32>(a, st);
        else norm_start<T, GRAD, 512, 32>(a, st);
        if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    }
    if (GRAD && (a.grad_weight || a.grad_bias) && (a.partial || a.N == 0)) {
        const int64_t wgs = (2 * (int64_t)a.K + kNormJoinCols - 1) / kNormJoinCols;
        timed_launch_ggl(false, (norm_join<T>), dim3((unsigned)wgs), dim3(kNormJoinCols * kNormJoinParts), 0, st, a);
        if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    }
    return SEGRED_OK;
}

template <bool GRAD>
int norm_typed(const NormArgs &a, int32_t dtype, hipStream_t st) {
    switch (dtype) {
    case SEGRED_BF16: return norm_dispatch<__bf16, GRAD>(a, st);
    case SEGRED_F16: return norm_dispatch<_Float16, GRAD>(a, st);
    default: return norm_dispatch<float, GRAD>(a, st);
    }
}

// What both calls ask of the arguments that they share.
int norm_check(const void *values, int32_t dtype, int64_t k, int64_t rows, const void *weight, const void *bias,
               int32_t weight_dtype, float eps, const void *out) {
    const int64_t e = float_size(dtype);
    if (dtype < SEGRED_U32 || dtype > SEGRED_F16 || k < 1 || rows < 0) return SEGRED_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0.f) || std::isinf(eps) || (rows > 0 && (!values || !out))) return SEGRED_ERR_INVALID_ARGUMENT;
    if (e == 0 || k > kMaxWidth) return SEGRED_ERR_UNSUPPORTED;
    if (weight_dtype != dtype && weight_dtype != SEGRED_F32) return SEGRED_ERR_INVALID_ARGUMENT;
    const int64_t we = float_size(weight_dtype);
    if (!aligned(values, e) || !aligned(out, e) || !aligned(weight, we) || !aligned(bias, we) || too_large(rows, k, 4))
        return SEGRED_ERR_INVALID_ARGUMENT;
    return SEGRED_OK;
}

}  // namespace segred

using namespace segred;

extern "C" int segred_norm(const void *values, int32_t dtype, int64_t k, int64_t rows, const void *weight,
                           const void *bias, int32_t weight_dtype, float eps, int32_t center, void *out,
                           hipStream_t stream) {
    const int rc = norm_check(values, dtype, k, rows, weight, bias, weight_dtype, eps, out);
    if (rc != SEGRED_OK || rows == 0) return rc;
    NormArgs a{};
    a.values = static_cast<const char *>(values);
    a.weight = weight;
    a.bias = bias;
    a.weight_f32 = weight_dtype == SEGRED_F32;
    a.N = rows;
    a.K = (int)k;
    a.center = center != 0;
    a.eps = eps;
    a.out = static_cast<char *>(out);
    return norm_typed<false>(a, dtype, stream);
}

extern "C" int64_t segred_norm_grad_workspace(int64_t k, int64_t rows) {
    if (k < 1 || rows < 1 || k > kMaxWidth) return 0;
    return std::max(norm_room(k, rows, false), norm_room(k, rows, true));
}

extern "C" int segred_norm_grad(const void *grad, const void *values, int32_t dtype, int64_t k, int64_t rows,
                                const void *weight, int32_t weight_dtype, float eps, int32_t center, void *grad_values,
                                void *grad_weight, void *grad_bias, void *workspace, int64_t workspace_bytes,
                                hipStream_t stream) {
    const int rc = norm_check(values, dtype, k, rows, weight, nullptr, weight_dtype, eps, grad_values);
    if (rc != SEGRED_OK) return rc;
    const int64_t e = float_size(dtype), we = float_size(weight_dtype);
    if ((rows > 0 && !grad) || !aligned(grad, e) || !aligned(grad_weight, we) || !aligned(grad_bias, we) ||
        !aligned(workspace, 16))
        return SEGRED_ERR_INVALID_ARGUMENT;
    const bool sums = grad_weight || grad_bias;
    const int64_t need = sums ? segred_norm_grad_workspace(k, rows) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return SEGRED_ERR_INVALID_ARGUMENT;
    NormArgs a{};
    a.grad = static_cast<const char *>(grad);
    a.values = static_cast<const char *>(values);
    a.weight = weight;
    a.weight_f32 = weight_dtype == SEGRED_F32;
    a.N = rows;
    a.K = (int)k;
    a.center = center != 0;
    a.eps = eps;
    a.out = static_cast<char *>(grad_values);
    a.grad_weight = grad_weight;
    a.grad_bias = grad_bias;
    a.partial = sums && rows > 0 && norm_room(k, rows, dtype == SEGRED_F32) > 0 ? static_cast<float *>(workspace) : nullptr;
    return norm_typed<true>(a, dtype, stream);
}
