// norm.hip -- layer norm (and the norm by the root mean square) of rows, and
// its gradient with the sums of the weight's and the bias's over the rows.
//
// With m the mean of a row (0 without centering), r = 1 / sqrt(mean((x - m)^2) +
// eps) and u = (x - m) r,
//   out = u w + b
//   dx  = r (gw - mean(gw) - u mean(gw u)), gw = g w   (mean(gw) only if centered)
//   dw  = sum over rows of g u, db = sum over rows of g.
// Both directions move their rows once and are bound by memory: a row is held
// in registers (up to 16,384 elements), the statistics are found there in two
// passes (mean, then squares around it), and the gradient finds them again
// instead of reading them.
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
    float *partial;  // [blocks][2][K]
    int64_t blocks;
};

template <typename T>
__device__ __forceinline__ float element(u32x4 v, int e) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(v[e]);
    else if constexpr (__is_same(T, __bf16)) return __uint_as_float(e & 1 ? v[e >> 1] & 0xffff0000u : v[e >> 1] << 16);
    else return (float)__builtin_bit_cast(f16x8, v)[e];
}

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

template <typename T>
__device__ __forceinline__ float param(const void *p, int f32, int c) {
    return f32 ? static_cast<const float *>(p)[c] : (float)static_cast<const T *>(p)[c];
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
    static constexpr int kWaves = L / 64;
    float (*s)[kWaves > 1 ? kWaves : 1][Q];  // [2][waves][Q]
    int turn = 0;
    // all(w, q): value q of wave w, valid until the call after the next.
    __device__ __forceinline__ const float (*meet(const float (&v)[Q], int wave, int lane))[Q] {
        float (*p)[Q] = s[turn];
        turn ^= 1;
        if (lane == 0)
#pragma unroll
            for (int q = 0; q < Q; ++q) p[wave][q] = v[q];
        __syncthreads();
        return p;
    }
};

// L lanes hold a row, E elements each.  A workgroup walks rows with its weight
// and bias in registers; the next row is on its way while one is worked on.
template <int L> constexpr int kNormThreads = L > 256 ? L : 256;

template <typename T, int L, int E>
__global__ __launch_bounds__(kNormThreads<L>) void norm_rows(NormArgs a) {
    constexpr int kThreads = kNormThreads<L>, kRows = kThreads / L, U = E / kUnit<T>, W = L > 64 ? L / 64 : 1;
    constexpr int LW = L > 64 ? 64 : L;  // lanes of a row in one wave
    __shared__ float s_join[2][W][2];
    const int l = threadIdx.x % L, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, K = a.K;
    RowJoin<L, 2> join{s_join};
    const int64_t row_bytes = (int64_t)K * sizeof(T), stride = (int64_t)gridDim.x * kRows;
    const float per = 1.f / (float)K;
    float w[E], b[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = norm_col<T, L>(i / kUnit<T>, l) + i % kUnit<T>;
        w[i] = c < K && a.weight ? param<T>(a.weight, a.weight_f32, c) : 1.f;
        b[i] = c < K && a.bias ? param<T>(a.bias, a.weight_f32, c) : 0.f;
    }
    // elements of this wave's part of a row
    int mine = 0;
    if constexpr (W > 1)
        for (int u = 0; u < U; ++u) mine += max(0, min(64 * kUnit<T>, K - norm_col<T, L>(u, wave * 64)));

    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / L;
    u32x4 next[U];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = norm_col<T, L>(u, l);
            next[u] = load_unit<T>((uint64_t)(a.values + r * row_bytes) + c * sizeof(T), r < a.N ? K - c : 0);
        }
    };
    fetch(row);
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.N; first += stride, row += stride) {
        float x[E];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = element<T>(next[i / kUnit<T>], i % kUnit<T>);
        fetch(row + stride);
        float mean = 0.f, m2 = 0.f;
        if (a.center) {
#pragma unroll
            for (int i = 0; i < E; ++i) sum += x[i];
            sum = lanes_sum<LW>(sum);
            mean = W > 1 ? (mine > 0 ? sum / (float)mine : 0.f) : sum * per;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = norm_col<T, L>(i / kUnit<T>, l) + i % kUnit<T>;
            const float d = c < K ? x[i] - mean : 0.f;
            m2 = fmaf(d, d, m2);
        }
        m2 = lanes_sum<LW>(m2);
        if constexpr (W > 1) {
            // the parts' means and squares around them, joined
            const float v[2] = {sum, m2};
            const auto p = join.meet(v, wave, lane);
            m2 = 0.f;
            if (a.center) {
                mean = 0.f;
#pragma unroll
                for (int q = 0; q < W; ++q) mean += p[q][0];
                mean *= per;
            }
#pragma unroll
            for (int q = 0; q < W; ++q) {
                int n = 0;
#pragma unroll
                for (int u = 0; u < U; ++u) n += max(0, min(64 * kUnit<T>, K - norm_col<T, L>(u, q * 64)));
                const float d = a.center && n > 0 ? p[q][0] / (float)n - mean : 0.f;
                m2 += fmaf((float)n * d, d, p[q][1]);
            }
        }
        const float r = 1.f / sqrtf(fmaf(m2, per, a.eps));
        if (row < a.N)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = norm_col<T, L>(u, l);
                float y[kUnit<T>];
#pragma unroll
                for (int e = 0; e < kUnit<T>; ++e) {
                    const int i = u * kUnit<T> + e;
                    y[e] = fmaf((x[i] - mean) * r, w[i], b[i]);
                }
                if (c < K) store_unit<T>(a.out + row * row_bytes + c * (int64_t)sizeof(T), y, K - c);
            }
    }
}

// The gradient.  A workgroup walks rows as above and adds up g u and g of its
// columns in registers; at the end its parts go to `partial`.  One exchange a
// row between waves: besides the mean and the squares, sum gw and the sum of
// gw (x - mean of this wave's part), which is corrected for the row's mean.
template <typename T, int L, int E>
__global__ __launch_bounds__(kNormThreads<L>) void norm_grad_rows(NormArgs a) {
    constexpr int kThreads = kNormThreads<L>, kRows = kThreads / L, U = E / kUnit<T>, W = L > 64 ? L / 64 : 1;
    constexpr int LW = L > 64 ? 64 : L;
    __shared__ float s_join[2][W][4];
    __shared__ float s_sums[kRows > 1 ? 2 * LW * E : 1];
    const int l = threadIdx.x % L, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, K = a.K;
    RowJoin<L, 4> join{s_join};
    const int64_t row_bytes = (int64_t)K * sizeof(T), stride = (int64_t)gridDim.x * kRows;
    const float per = 1.f / (float)K;
    float w[E], dw[E], db[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = norm_col<T, L>(i / kUnit<T>, l) + i % kUnit<T>;
        w[i] = c < K ? (a.weight ? param<T>(a.weight, a.weight_f32, c) : 1.f) : 0.f;
        dw[i] = db[i] = 0.f;
    }
    int mine = 0;
    if constexpr (W > 1)
        for (int u = 0; u < U; ++u) mine += max(0, min(64 * kUnit<T>, K - norm_col<T, L>(u, wave * 64)));

    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / L;
    u32x4 next_x[U], next_g[U];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = norm_col<T, L>(u, l), n = r < a.N ? K - c : 0;
            const uint64_t at = (uint64_t)(r * row_bytes) + c * sizeof(T);
            next_x[u] = load_unit<T>((uint64_t)a.values + at, n);
            next_g[u] = load_unit<T>((uint64_t)a.grad + at, n);
        }
    };
    fetch(row);
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.N; first += stride, row += stride) {
        u32x4 x[U], g[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = next_x[u];
            g[u] = next_g[u];
        }
        fetch(row + stride);
        float sum = 0.f, mean = 0.f, m2 = 0.f, c1 = 0.f, c2 = 0.f;
        if (a.center) {
#pragma unroll
            for (int i = 0; i < E; ++i) sum += element<T>(x[i / kUnit<T>], i % kUnit<T>);
            sum = lanes_sum<LW>(sum);
            mean = W > 1 ? (mine > 0 ? sum / (float)mine : 0.f) : sum * per;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = norm_col<T, L>(i / kUnit<T>, l) + i % kUnit<T>;
            const float d = c < K ? element<T>(x[i / kUnit<T>], i % kUnit<T>) - mean : 0.f;
            const float gw = element<T>(g[i / kUnit<T>], i % kUnit<T>) * w[i];
            m2 = fmaf(d, d, m2);
            c1 += gw;
            c2 = fmaf(gw, d, c2);
        }
        m2 = lanes_sum<LW>(m2);
        c1 = lanes_sum<LW>(c1);
        c2 = lanes_sum<LW>(c2);
        if constexpr (W > 1) {
            const float v[4] = {sum, m2, c1, c2};
            const auto p = join.meet(v, wave, lane);
            m2 = c1 = c2 = 0.f;
            if (a.center) {
                mean = 0.f;
#pragma unroll
                for (int q = 0; q < W; ++q) mean += p[q][0];
                mean *= per;
            }
#pragma unroll
            for (int q = 0; q < W; ++q) {
                int n = 0;
#pragma unroll
                for (int u = 0; u < U; ++u) n += max(0, min(64 * kUnit<T>, K - norm_col<T, L>(u, q * 64)));
                const float d = a.center && n > 0 ? p[q][0] / (float)n - mean : 0.f;
                m2 += fmaf((float)n * d, d, p[q][1]);
                c1 += p[q][2];
                c2 += fmaf(p[q][2], d, p[q][3]);
            }
        }
        const float r = 1.f / sqrtf(fmaf(m2, per, a.eps));
        const float along = c2 * r * per;  // mean(gw u)
        const float level = a.center ? c1 * per : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = norm_col<T, L>(u, l);
            float y[kUnit<T>];
#pragma unroll
            for (int e = 0; e < kUnit<T>; ++e) {
                const int i = u * kUnit<T> + e;
                const float unit = (element<T>(x[u], e) - mean) * r, ge = element<T>(g[u], e);
                y[e] = r * (fmaf(ge, w[i], -level) - unit * along);
                // a row past the last has g = 0, but r of it may be infinite
                if (row < a.N) dw[i] = fmaf(ge, unit, dw[i]);
                db[i] += ge;
            }
            if (row < a.N && c < K) store_unit<T>(a.out + row * row_bytes + c * (int64_t)sizeof(T), y, K - c);
        }
    }
    if (!a.partial) return;

    // The rows of a wave, then of the workgroup, in order.
    if constexpr (LW < 64) {
#pragma unroll
        for (int i = 0; i < E; ++i)
            for (int s = 32; s >= LW; s >>= 1) {
                dw[i] += lane_get(dw[i], lane ^ s);
                db[i] += lane_get(db[i], lane ^ s);
            }
    }
    if constexpr (kRows > 1) {
        for (int v = 0; v < kThreads / 64; ++v) {
            if (wave == v && lane < LW)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    float *p = s_sums + i * LW + lane, *q = p + LW * E;
                    *p = v ? *p + dw[i] : dw[i];
                    *q = v ? *q + db[i] : db[i];
                }
            __syncthreads();
        }
        if (wave > 0 || lane >= LW) return;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            dw[i] = s_sums[i * LW + lane];
            db[i] = s_sums[(E + i) * LW + lane];
        }
    }
    float *to = a.partial + (int64_t)blockIdx.x * 2 * K;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = norm_col<T, L>(i / kUnit<T>, l) + i % kUnit<T>;
        if (c < K) {
            to[c] = dw[i];
            to[K + c] = db[i];
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
        float mean = 0.f, m2 = 0.f, c1 = 0.f, c2 = 0.f;
        if (a.center) {
            for (int c = threadIdx.x; c < K; c += kLongThreads) mean += (float)x[c];
            mean = long_sum(mean, s, wave, lane) * per;
        }
        for (int c = threadIdx.x; c < K; c += kLongThreads) {
            const float d = (float)x[c] - mean;
            m2 = fmaf(d, d, m2);
            if constexpr (GRAD) {
                const float gw = (float)g[c] * (a.weight ? param<T>(a.weight, a.weight_f32, c) : 1.f);
                c1 += gw;
                c2 = fmaf(gw, d, c2);
            }
        }
        const float r = 1.f / sqrtf(fmaf(long_sum(m2, s, wave, lane), per, a.eps));
        if constexpr (GRAD) {
            const float level = a.center ? long_sum(c1, s, wave, lane) * per : 0.f;
            const float along = long_sum(c2, s, wave, lane) * r * per;
            for (int c = threadIdx.x; c < K; c += kLongThreads) {
                const float unit = ((float)x[c] - mean) * r, ge = (float)g[c];
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
                out[c] = (T)fmaf(((float)x[c] - mean) * r, w, a.bias ? param<T>(a.bias, a.weight_f32, c) : 0.f);
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
#pragma unroll 4
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

// Lanes and elements per lane of a row.
struct NormShape {
    int lanes, elements;  // lanes 0: too long for registers
};
NormShape norm_shape(int64_t k) {
    if (k <= 128) return {16, 8};
    if (k <= 512) return {64, 8};
    if (k <= 1024) return {64, 16};
    if (k <= 2048) return {64, 32};
    if (k <= 4096) return {256, 16};
    if (k <= 8192) return {256, 32};
    if (k <= 16384) return {512, 32};
    return {0, 0};
}

// Workgroups of a call: by rows alone, so that sums do not depend on the device.
constexpr int64_t kNormBlocks = 2048, kNormGradBlocks = 512;
int64_t norm_blocks(int64_t k, int64_t rows, int64_t most) {
    const NormShape s = norm_shape(k);
    const int64_t each = s.lanes > 0 && s.lanes < 256 ? 256 / s.lanes : 1;
    return std::min(most, (rows + each - 1) / each);
}

template <typename T, bool GRAD, int L, int E>
void norm_start(const NormArgs &a, hipStream_t st) {
    if constexpr (GRAD)
        timed_launch_ggl(true, (norm_grad_rows<T, L, E>), dim3((unsigned)a.blocks), dim3(kNormThreads<L>), 0, st, a);
    else
        timed_launch_ggl(true, (norm_rows<T, L, E>), dim3((unsigned)a.blocks), dim3(kNormThreads<L>), 0, st, a);
}

template <typename T, bool GRAD>
int norm_dispatch(const NormArgs &a, hipStream_t st) {
    if (a.N > 0) {
        const NormShape s = norm_shape(a.K);
        if (s.lanes == 0) timed_launch_ggl(true, (norm_long<T, GRAD>), dim3((unsigned)a.blocks), dim3(kLongThreads), 0, st, a);
        else if (s.lanes == 16) norm_start<T, GRAD, 16, 8>(a, st);
        else if (s.lanes == 64 && s.elements == 8) norm_start<T, GRAD, 64, 8>(a, st);
        else if (s.lanes == 64 && s.elements == 16) norm_start<T, GRAD, 64, 16>(a, st);
        else if (s.lanes == 64) norm_start<T, GRAD, 64, 32>(a, st);
        else if (s.lanes == 256 && s.elements == 16) norm_start<T, GRAD, 256, 16>(a, st);
        else if (s.lanes == 256) norm_start<T, GRAD, 256, 32>(a, st);
        else norm_start<T, GRAD, 512, 32>(a, st);
        if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    }
    if (GRAD && (a.grad_weight || a.grad_bias)) {
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
    a.blocks = norm_blocks(k, rows, kNormBlocks);
    return norm_typed<false>(a, dtype, stream);
}

extern "C" int64_t segred_norm_grad_workspace(int64_t k, int64_t rows) {
    if (k < 1 || rows < 1 || k > kMaxWidth) return 0;
    return norm_blocks(k, rows, kNormGradBlocks) * 2 * k * 4;
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
    a.partial = need > 0 ? static_cast<float *>(workspace) : nullptr;
    a.blocks = norm_blocks(k, rows, kNormGradBlocks);
    return norm_typed<true>(a, dtype, stream);
}
