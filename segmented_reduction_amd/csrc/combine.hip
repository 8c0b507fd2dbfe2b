// combine.hip -- the rows a token was sent to, joined by its weights:
// out[t] = sum over j of weights[t, j] values[position[t, j]], and the
// gradient of that with respect to the rows and the weights.
#include <algorithm>

#include "internal.hpp"
#include "tile.hpp"

namespace segred {

struct CombineArgs {
    const char *values;       // [rows, M]
    const char *grad;         // [tokens, M] (gradient call)
    const int64_t *position;  // [tokens, fanout]
    const float *weights;     // [tokens, fanout]
    int64_t rows, tokens, fanout, M, units;
    char *out;                // [tokens, M], or the gradient of values [rows, M]
    float *grad_weights;      // [tokens, fanout]
    int64_t blocks;           // blocks of kJoin entries of a token (gradient call)
    const int64_t *order, *offsets;  // entries by the row they name (gradient call, rows named more than once)
};

constexpr int kCombineThreads = 256;
constexpr int kJoin = 4;  // entries of a token handled together

// One unit of 16 bytes (or one element where rows are not whole units).
template <typename T, bool VEC>
struct Unit {
    static constexpr int kN = VEC ? kUnit<T> : 1;
    T v[kN];
    __device__ __forceinline__ void load(const char *p) {
        if constexpr (VEC) *reinterpret_cast<u32x4 *>(v) = *reinterpret_cast<const u32x4 *>(p);
        else v[0] = *reinterpret_cast<const T *>(p);
    }
    __device__ __forceinline__ void store(char *p) const {
        if constexpr (VEC) *reinterpret_cast<u32x4 *>(p) = *reinterpret_cast<const u32x4 *>(v);
        else *reinterpret_cast<T *>(p) = v[0];
    }
};

// One unit of one output row per thread.
template <typename T, bool VEC>
__global__ __launch_bounds__(kCombineThreads) void combine_rows(CombineArgs a) {
    using U = Unit<T, VEC>;
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kCombineThreads + threadIdx.x;
    if (i >= a.tokens * a.units) return;
    const int64_t t = i / a.units, c = (i - t * a.units) * U::kN;
    float acc[U::kN] = {};
    for (int64_t j0 = 0; j0 < a.fanout; j0 += kJoin) {
        U u[kJoin];
        float w[kJoin];
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            const int64_t p = j0 + j < a.fanout ? a.position[t * a.fanout + j0 + j] : -1;
            const bool there = p >= 0 && p < a.rows;
            w[j] = there ? a.weights[t * a.fanout + j0 + j] : 0.f;
            u[j] = U{};
            if (there) u[j].load(a.values + (p * a.M + c) * (int64_t)sizeof(T));
        }
#pragma unroll
        for (int j = 0; j < kJoin; ++j)
#pragma unroll
            for (int e = 0; e < U::kN; ++e) acc[e] = fmaf(w[j], (float)u[j].v[e], acc[e]);
    }
    U o;
#pragma unroll
    for (int e = 0; e < U::kN; ++e) o.v[e] = (T)acc[e];
    o.store(a.out + (t * a.M + c) * (int64_t)sizeof(T));
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += lane_get(x, lane_id() ^ o);
    return x;
}

// One wave per token and kJoin of its entries: the token's gradient row is
// read once for them.
template <typename T, bool VEC>
__global__ __launch_bounds__(kCombineThreads) void combine_grads(CombineArgs a) {
    using U = Unit<T, VEC>;
    const int lane = threadIdx.x & 63;
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kCombineThreads / 64) + (threadIdx.x >> 6);
    if (i >= a.tokens * a.blocks) return;
    const int64_t t = i / a.blocks, j0 = (i - t * a.blocks) * kJoin;
    int64_t p[kJoin];
    float w[kJoin], dot[kJoin] = {};
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
        p[j] = j0 + j < a.fanout ? a.position[t * a.fanout + j0 + j] : -1;
        if (p[j] >= a.rows) p[j] = -1;
        w[j] = p[j] >= 0 ? a.weights[t * a.fanout + j0 + j] : 0.f;
    }
    for (int64_t c = (int64_t)lane * U::kN; c < a.M; c += 64 * U::kN) {
        U g, y[kJoin];
        g.load(a.grad + (t * a.M + c) * (int64_t)sizeof(T));
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            y[j] = U{};
            if (p[j] >= 0) y[j].load(a.values + (p[j] * a.M + c) * (int64_t)sizeof(T));
        }
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            if (p[j] < 0) continue;
            U o;
#pragma unroll
            for (int e = 0; e < U::kN; ++e) {
                dot[j] = fmaf((float)g.v[e], (float)y[j].v[e], dot[j]);
                o.v[e] = (T)(w[j] * (float)g.v[e]);
            }
            if (!a.offsets) o.store(a.out + (p[j] * a.M + c) * (int64_t)sizeof(T));
        }
    }
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
        const float d = wave_sum(dot[j]);
        if (lane == 0 && j0 + j < a.fanout) a.grad_weights[t * a.fanout + j0 + j] = p[j] >= 0 ? d : 0.f;
    }
}

// Rows that several entries may name: one unit of one row per thread, which
// adds the entries' gradients in their order, so that no two threads write a
// row.  The entries come sorted by row, kJoin of them are under way at a time.
template <typename T, bool VEC>
__global__ __launch_bounds__(kCombineThreads) void combine_row_grads(CombineArgs a) {
    using U = Unit<T, VEC>;
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kCombineThreads + threadIdx.x;
    if (i >= a.rows * a.units) return;
    const int64_t p = i / a.units, c = (i - p * a.units) * U::kN, end = a.offsets[p + 1];
    float acc[U::kN] = {};
    for (int64_t q0 = a.offsets[p]; q0 < end; q0 += kJoin) {
        int64_t e[kJoin];
        U g[kJoin];
        float w[kJoin];
#pragma unroll
        for (int j = 0; j < kJoin; ++j) e[j] = a.order[min(q0 + j, end - 1)];
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            w[j] = a.weights[e[j]];
            g[j].load(a.grad + (e[j] / a.fanout * a.M + c) * (int64_t)sizeof(T));
        }
#pragma unroll
        for (int j = 0; j < kJoin; ++j)
#pragma unroll
            for (int n = 0; n < U::kN; ++n)
                if (q0 + j < end) acc[n] = fmaf(w[j], (float)g[j].v[n], acc[n]);
    }
    U o;
#pragma unroll
    for (int n = 0; n < U::kN; ++n) o.v[n] = (T)acc[n];
    o.store(a.out + (p * a.M + c) * (int64_t)sizeof(T));
}

template <typename T>
int combine_launch(CombineArgs a, bool grads, bool vec, hipStream_t st) {
    a.units = vec ? a.M / kUnit<T> : a.M;
    a.blocks = (a.fanout + kJoin - 1) / kJoin;
    const int64_t per = grads ? kCombineThreads / 64 : kCombineThreads;
    const int64_t items = grads ? a.tokens * a.blocks : a.tokens * a.units;
    dim3 grid;
    if (!tile_grid((items + per - 1) / per, grid)) return SEGRED_ERR_UNSUPPORTED;
    if (grads && vec) timed_launch_ggl(true, (combine_grads<T, true>), grid, dim3(kCombineThreads), 0, st, a);
    else if (grads) timed_launch_ggl(true, (combine_grads<T, false>), grid, dim3(kCombineThreads), 0, st, a);
    else if (vec) timed_launch_ggl(true, (combine_rows<T, true>), grid, dim3(kCombineThreads), 0, st, a);
    else timed_launch_ggl(true, (combine_rows<T, false>), grid, dim3(kCombineThreads), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SEGRED_ERR_HIP;
    if (!a.offsets) return SEGRED_OK;
    if (!tile_grid((a.rows * a.units + kCombineThreads - 1) / kCombineThreads, grid)) return SEGRED_ERR_UNSUPPORTED;
    if (vec) timed_launch_ggl(true, (combine_row_grads<T, true>), grid, dim3(kCombineThreads), 0, st, a);
    else timed_launch_ggl(true, (combine_row_grads<T, false>), grid, dim3(kCombineThreads), 0, st, a);
    return hipGetLastError() == hipSuccess ? SEGRED_OK : SEGRED_ERR_HIP;
}

int combine_call(const CombineArgs &a, int32_t dtype, bool grads, hipStream_t st) {
    const int64_t e = float_size(dtype);
    const bool vec = (a.M * e) % 16 == 0 && aligned(a.values, 16) && aligned(a.out, 16) && aligned(a.grad, 16);
    switch (dtype) {
    case SEGRED_BF16: return combine_launch<__bf16>(a, grads, vec, st);
    case SEGRED_F16: return combine_launch<_Float16>(a, grads, vec, st);
    default: return combine_launch<float>(a, grads, vec, st);
    }
}

// The checks that both calls share.
int combine_check(const void *values, int32_t dtype, int64_t m, int64_t rows, const int64_t *position,
                  const float *weights, int64_t tokens, int64_t fanout, const void *out) {
    const int64_t e = float_size(dtype);
    if (dtype < SEGRED_U32 || dtype > SEGRED_F16) return SEGRED_ERR_INVALID_ARGUMENT;
    if (m < 1 || rows < 0 || tokens < 0 || fanout < 0) return SEGRED_ERR_INVALID_ARGUMENT;
    if ((rows > 0 && !values) || (tokens > 0 && fanout > 0 && (!position || !weights))) return SEGRED_ERR_INVALID_ARGUMENT;
    if (e == 0) return SEGRED_ERR_UNSUPPORTED;
    if (!aligned(values, e) || !aligned(out, e) || !aligned(position, 8) || !aligned(weights, 4))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (too_large(rows, m, 4) || too_large(tokens, m, 4) || too_large(tokens, fanout, 8)) return SEGRED_ERR_INVALID_ARGUMENT;
    return SEGRED_OK;
}

// The entries sorted by row, and what sorts them.
struct CombineSpace {
    size_t entries, offsets, group;  // bytes of each part; entries: of one array
};
CombineSpace combine_space(int64_t entries, int64_t rows) {
    auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
    return {up((size_t)entries * 8), up(((size_t)rows + 1) * 8), (size_t)segred_group_workspace(entries, rows)};
}
// Sizes that segred_group takes (the counts are not negative).
bool combine_sortable(int64_t rows, int64_t tokens, int64_t fanout) {
    return rows < INT32_MAX && !too_large(tokens, fanout, 8) && tokens * fanout <= INT32_MAX;
}

}  // namespace segred

using namespace segred;

extern "C" int segred_combine(const void *values, int32_t dtype, int64_t m, int64_t rows, const int64_t *position,
                              const float *weights, int64_t tokens, int64_t fanout, void *out, hipStream_t stream) {
    const int rc = combine_check(values, dtype, m, rows, position, weights, tokens, fanout, out);
    if (rc != SEGRED_OK) return rc;
    if (tokens == 0) return SEGRED_OK;
    if (!out) return SEGRED_ERR_INVALID_ARGUMENT;
    CombineArgs a{};
    a.values = static_cast<const char *>(values);
    a.position = position;
    a.weights = weights;
    a.rows = rows;
    a.tokens = tokens;
    a.fanout = fanout;
    a.M = m;
    a.out = static_cast<char *>(out);
    return combine_call(a, dtype, false, stream);
}

extern "C" int segred_combine_grad(const void *grad, const void *values, int32_t dtype, int64_t m, int64_t rows,
                                   const int64_t *position, const float *weights, int64_t tokens, int64_t fanout,
                                   void *grad_values, float *grad_weights, hipStream_t stream) {
    const int rc = combine_check(values, dtype, m, rows, position, weights, tokens, fanout, grad_values);
    if (rc != SEGRED_OK) return rc;
    if (!aligned(grad, float_size(dtype)) || !aligned(grad_weights, 4)) return SEGRED_ERR_INVALID_ARGUMENT;
    if (tokens == 0 || fanout == 0) return SEGRED_OK;
    if (!grad || !grad_weights || (rows > 0 && !grad_values)) return SEGRED_ERR_INVALID_ARGUMENT;
    CombineArgs a{};
    a.values = static_cast<const char *>(values);
    a.grad = static_cast<const char *>(grad);
    a.position = position;
    a.weights = weights;
    a.rows = rows;
    a.tokens = tokens;
    a.fanout = fanout;
    a.M = m;
    a.out = static_cast<char *>(grad_values);
    a.grad_weights = grad_weights;
    return combine_call(a, dtype, true, stream);
}

extern "C" int64_t segred_combine_grad_repeated_workspace(int64_t rows, int64_t tokens, int64_t fanout) {
    if (rows < 1 || tokens < 1 || fanout < 1 || !combine_sortable(rows, tokens, fanout)) return 0;
    const CombineSpace s = combine_space(tokens * fanout, rows);
    return (int64_t)(2 * s.entries + s.offsets + s.group);
}

extern "C" int segred_combine_grad_repeated(const void *grad, const void *values, int32_t dtype, int64_t m, int64_t rows,
                                            const int64_t *position, const float *weights, int64_t tokens,
                                            int64_t fanout, void *grad_values, float *grad_weights, void *workspace,
                                            int64_t workspace_bytes, hipStream_t stream) {
    int rc = combine_check(values, dtype, m, rows, position, weights, tokens, fanout, grad_values);
    if (rc != SEGRED_OK) return rc;
    if (!aligned(grad, float_size(dtype)) || !aligned(grad_weights, 4) || !aligned(workspace, 16))
        return SEGRED_ERR_INVALID_ARGUMENT;
    if (!combine_sortable(rows, tokens, fanout)) return SEGRED_ERR_UNSUPPORTED;
    const bool some = tokens > 0 && fanout > 0;
    if ((some && (!grad || !grad_weights)) || (rows > 0 && !grad_values)) return SEGRED_ERR_INVALID_ARGUMENT;
    const int64_t need = segred_combine_grad_repeated_workspace(rows, tokens, fanout);
    if (need > 0 && (!workspace || workspace_bytes < need)) return SEGRED_ERR_INVALID_ARGUMENT;
    CombineArgs a{};
    a.values = static_cast<const char *>(values);
    a.grad = static_cast<const char *>(grad);
    a.position = position;
    a.weights = weights;
    a.rows = rows;
    a.tokens = tokens;
    a.fanout = fanout;
    a.M = m;
    a.out = static_cast<char *>(grad_values);
    a.grad_weights = grad_weights;
    if (!some) {  // the sum over no entries: segred_combine of `rows` tokens without an entry
        if (rows == 0) return SEGRED_OK;
        a.tokens = rows;
        a.fanout = 0;
        return combine_call(a, dtype, false, stream);
    }
    if (rows > 0) {
        const CombineSpace s = combine_space(tokens * fanout, rows);
        char *w = static_cast<char *>(workspace);
        int64_t *order = reinterpret_cast<int64_t *>(w), *place = reinterpret_cast<int64_t *>(w + s.entries);
        int64_t *offsets = reinterpret_cast<int64_t *>(w + 2 * s.entries);
        rc = segred_group(position, tokens * fanout, 1, rows, order, place, offsets, w + 2 * s.entries + s.offsets,
                          (int64_t)s.group, stream);
        if (rc != SEGRED_OK) return rc;
        a.order = order;
        a.offsets = offsets;
    }
    return combine_call(a, dtype, true, stream);
}
