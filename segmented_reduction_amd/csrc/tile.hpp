// tile.hpp -- matrix-core tiles shared by the products over segments: how an
// operand tile lies in LDS, how it gets there, and how the waves multiply it.
//
// A workgroup computes a BM x BN tile of out = A B with a contraction axis k
// that it walks in steps of kStep<T> elements (128 bytes).  One step of an
// operand is staged in LDS in one of two forms:
//
//   row form   the operand's rows run along k in memory (x, and weights
//              applied transposed): LDS row r holds the 128 bytes of row r.
//              The 16-byte unit u of a row lies at place u ^ (r & 7), so that
//              the 16 lanes of a fragment read, which ask for the same unit
//              of 16 consecutive rows, spread over all banks.
//   col form   the operand's rows run across k (weights applied from the
//              right, both operands of a sum of outer products): LDS row k
//              holds the W elements of step row k.  Blocks of 16 elements lie
//              at place block ^ col_swizzle(k), for the same reason.
//
// Fragments follow v_mfma_f32_16x16x32_{bf16,f16} (a lane holds 8 consecutive
// k of one row) and v_mfma_f32_16x16x4_f32 (one k; four of them are fed from
// one 16-byte unit, so k is visited in another order, the same for both
// operands).  A 16-bit fragment in col form is read with
// ds_read_b64_tr_b16, which transposes 4 x 16 elements among 16 lanes.
//
// The first MFMA operand is B's fragment and the second A's, so that a lane
// ends up with four consecutive columns of one output row and stores them as
// one unit.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wave.hpp"

namespace segred {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(1))) const void global_void;

template <typename T> constexpr int kStep = 128 / (int)sizeof(T);  // k elements of one step
template <typename T> constexpr int kUnit = 16 / (int)sizeof(T);   // elements of a 16-byte unit

// What a load beyond the operand's edge reads instead.
__device__ const u32x4 kZeros[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};

__device__ __forceinline__ const char *zero_unit() { return reinterpret_cast<const char *>(&kZeros[0]); }

// 16 bytes per lane from global memory to LDS at `dst` + 16 * lane (dst is
// wave-uniform), without passing through registers.
__device__ __forceinline__ void load_to_lds(uint64_t src, lds_char *dst) {
    __builtin_amdgcn_global_load_lds((global_void *)src, (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

// 16 bytes at any element boundary.  (As global memory: a flat load would also
// be waited for by every LDS read behind it.)
template <typename T>
__device__ __forceinline__ u32x4 load_whole(uint64_t addr) {
    typedef u32x4 __attribute__((aligned(2))) unit2;
    typedef u32x4 __attribute__((aligned(4))) unit4;
    if constexpr (sizeof(T) == 2) return *(__attribute__((address_space(1))) const unit2 *)addr;
    return *(__attribute__((address_space(1))) const unit4 *)addr;
}

// Up to `n` leading elements of a 16-byte unit at any element boundary; the
// others are zero and not touched (n <= 0: nothing is read).
template <typename T>
__device__ __forceinline__ u32x4 load_unit(uint64_t addr, int n) {
    typedef __attribute__((address_space(1))) const uint32_t global_u32;
    typedef __attribute__((address_space(1))) const uint16_t global_u16;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (n >= kUnit<T>) {
        v = load_whole<T>(addr);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < n) v[j] = ((global_u32 *)addr)[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = 2 * j < n ? ((global_u16 *)addr)[2 * j] : 0u;
            const uint32_t hi = 2 * j + 1 < n ? ((global_u16 *)addr)[2 * j + 1] : 0u;
            v[j] = lo | hi << 16;
        }
    }
    return v;
}

// The same of four neighbouring elements of type S as floats, for T = float.
template <typename T, typename S>
__device__ __forceinline__ u32x4 load_as(uint64_t addr, int n) {
    if constexpr (__is_same(T, S)) {
        return load_unit<T>(addr, n);
    } else {
        static_assert(sizeof(T) == 4 && sizeof(S) == 2, "16-bit elements as floats");
        u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n) v[j] = __float_as_uint((float)((__attribute__((address_space(1))) const S *)addr)[j]);
        return v;
    }
}

// ---------------------------------------------------------------- staging
//
// A stage object belongs to one thread and moves that thread's units of one
// operand.  DIRECT: global_load_lds, for operands whose rows start on 16-byte
// boundaries and hold whole units.  Otherwise the units pass through
// registers (`v`) and commit() writes them after the step's products.

// Row form: ROWS x 128 bytes, 8 rows per wave and load.
template <typename T, int ROWS, int THREADS, bool DIRECT>
struct RowStage {
    static constexpr int kWaves = THREADS / 64;
    static constexpr int kLoads = (ROWS / 8 + kWaves - 1) / kWaves;
    static constexpr int kBytes = ROWS * 128;
    uint64_t p[kLoads];  // address of this lane's unit of the row's first step
    int left[kLoads];    // elements of the row from there on; <= 0: a row of zeros
    u32x4 v[DIRECT ? 1 : kLoads];

    // Row group of load i.  With fewer groups than waves the surplus waves
    // fetch a group again (the same bytes to the same place), so that every
    // wave has the same number of loads in flight.
    static __device__ __forceinline__ int group(int i, int wave) { return (i * kWaves + wave) % (ROWS / 8); }

    // row_ptr(r): start of tile row r, or null for a row of zeros.
    template <typename F>
    __device__ __forceinline__ void init(int wave, int lane, int K, F row_ptr) {
        const int unit = ((lane & 7) ^ (lane >> 3)) * kUnit<T>;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const char *q = row_ptr(group(i, wave) * 8 + (lane >> 3));
            p[i] = (uint64_t)q + (uint64_t)unit * sizeof(T);
            left[i] = q ? K - unit : 0;
        }
    }
    // The step that starts at element k0 of each row.
    __device__ __forceinline__ void issue(lds_char *lds, int wave, int k0) {
        const uint64_t zeros = (uint64_t)zero_unit();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint64_t q = p[i] + (uint64_t)k0 * sizeof(T);
            if constexpr (DIRECT) {
                load_to_lds(k0 < left[i] ? q : zeros, lds + group(i, wave) * 1024);
            } else {
                v[i] = load_unit<T>(q, left[i] - k0);
            }
        }
    }
    __device__ __forceinline__ void commit(lds_char *lds, int wave, int lane) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                *reinterpret_cast<__attribute__((address_space(3))) u32x4 *>(lds + group(i, wave) * 1024 + lane * 16) = v[i];
        }
    }
};

// Swizzle of the 16-element blocks of LDS row k in col form.
template <typename T, int W>
__device__ __forceinline__ int col_swizzle(int k) {
    constexpr int kMask = (W / 16 < 8 ? W / 16 : 8) - 1;
    static_assert((W / 16 & (W / 16 - 1)) == 0, "power of two blocks");
    if constexpr (sizeof(T) == 2) return ((k & 3) | ((k >> 3) & 1) << 2) & kMask;
    return ((k >> 2) & 3) & kMask;
}

// Col form: kStep<T> rows of W elements.  S: their type in memory, where that
// is another (not DIRECT).
template <typename T, int W, int THREADS, bool DIRECT, typename S = T>
struct ColStage {
    static_assert(!DIRECT || __is_same(T, S), "direct loads convert nothing");
    static constexpr int kWaves = THREADS / 64;
    static constexpr int kUnits = W / kUnit<T>;                         // per LDS row
    static constexpr int kGroups = kStep<T> * W * (int)sizeof(T) / 1024;  // wave loads of a step
    static constexpr int kLoads = (kGroups + kWaves - 1) / kWaves;
    static constexpr int kBytes = kStep<T> * W * (int)sizeof(T);
    static constexpr int kSub = 16 / kUnit<T>;  // units of a block
    u32x4 v[DIRECT ? 1 : kLoads];

    static __device__ __forceinline__ int group(int i, int wave) { return (i * kWaves + wave) % kGroups; }
    // Step row and element column of load i of this lane.
    static __device__ __forceinline__ int row(int i, int wave, int lane) {
        return (group(i, wave) * 64 + lane) / kUnits;
    }
    static __device__ __forceinline__ int col(int i, int wave, int lane) {
        const int place = (group(i, wave) * 64 + lane) % kUnits;
        const int block = (place / kSub) ^ col_swizzle<T, W>(row(i, wave, lane));
        return (block * kSub + place % kSub) * kUnit<T>;
    }
    // src(i): address of load i's unit; left(i): how many elements of its row
    // exist from there on (<= 0: none, zeros instead).
    template <typename F, typename G>
    __device__ __forceinline__ void issue(lds_char *lds, int wave, F src, G left) {
        const uint64_t zeros = (uint64_t)zero_unit();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if constexpr (DIRECT) load_to_lds(left(i) > 0 ? src(i) : zeros, lds + group(i, wave) * 1024);
            else v[i] = load_as<T, S>(src(i), left(i));
        }
    }
    __device__ __forceinline__ void commit(lds_char *lds, int wave, int lane) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                *reinterpret_cast<__attribute__((address_space(3))) u32x4 *>(lds + group(i, wave) * 1024 + lane * 16) = v[i];
        }
    }
};

// --------------------------------------------------------------- fragments

// 8 k of one row (or 4 for float): k = 32 * ks + 8 * (lane / 16) + 0..7
// (16 * ks + 4 * (lane / 16) + 0..3), row = r0 + lane % 16.
__device__ __forceinline__ u32x4 row_frag(const lds_char *lds, int r0, int ks, int lane) {
    const int off = (r0 + (lane & 15)) * 128 + (((ks * 4 + (lane >> 4)) ^ (lane & 7)) << 4);
    return *reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>(lds + off);
}

template <typename T, int W>
__device__ __forceinline__ u32x4 col_frag(const lds_char *lds, int c0, int ks, int lane) {
    constexpr int kRow = W * (int)sizeof(T);
    if constexpr (sizeof(T) == 2) {
        union {
            s16x4 h[2];
            u32x4 v;
        } f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = ks * 32 + (lane >> 4) * 8 + h * 4 + ((lane & 15) >> 2);
            const int off = k * kRow + (((c0 >> 4) ^ col_swizzle<T, W>(k)) << 5) + (lane & 3) * 8;
            f.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)(const_cast<lds_char *>(lds) + off));
        }
        return f.v;
    } else {
        u32x4 f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = ks * 16 + (lane >> 4) * 4 + j;
            const int off = k * kRow + (((c0 >> 4) ^ col_swizzle<T, W>(k)) << 6) + (lane & 15) * 4;
            f[j] = *reinterpret_cast<const __attribute__((address_space(3))) uint32_t *>(lds + off);
        }
        return f;
    }
}

// Fragments of N blocks next to each other, of both k halves of a step.
template <int N>
__device__ __forceinline__ void row_frags(u32x4 (&f)[2][N], const lds_char *lds, int r0, int lane) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < N; ++i) f[ks][i] = row_frag(lds, r0 + 16 * i, ks, lane);
}

// The same in col form (KS = 1: of the first k half alone).  The transposing
// reads of the 16-bit types and the wait for them are one piece of assembly:
// before its own the compiler waits for all loads into LDS, also for those of
// later steps (8 segments of 64 rows, 2,048 x 1,024, in 64 x 64 tiles: 23.5 us
// instead of 14; of 1,024 rows, 2,560 x 1,024: 79 instead of 73).
template <typename T, int W, int N, int KS>
__device__ __forceinline__ void col_frags(u32x4 (&f)[KS][N], const lds_char *lds, int c0, int lane) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < N; ++i) f[ks][i] = col_frag<T, W>(lds, c0 + 16 * i, ks, lane);
    } else {
        constexpr int kRow = W * (int)sizeof(T);
        const int k = (lane >> 4) * 8 + ((lane & 15) >> 2);
        auto at = [&](int i) {  // the same swizzle for k + 4 and k + 32
            return (uint32_t)(uintptr_t)(lds + k * kRow + ((((c0 >> 4) + i) ^ col_swizzle<T, W>(k)) << 5) + (lane & 3) * 8);
        };
        union Frag {
            s16x4 h[2];
            u32x4 v;
        };
#define SEGRED_TR(D, A, O) "ds_read_b64_tr_b16 %" #D ", %" #A " offset:%" #O "\n\t"
#pragma unroll
        for (int i = 0; i + 1 < N; i += 2) {
            const uint32_t p = at(i), q = at(i + 1);
            Frag x[KS], y[KS];
            if constexpr (KS == 2)
                asm volatile(SEGRED_TR(0, 8, 10) SEGRED_TR(1, 8, 11) SEGRED_TR(4, 9, 10) SEGRED_TR(5, 9, 11)
                             SEGRED_TR(2, 8, 12) SEGRED_TR(3, 8, 13) SEGRED_TR(6, 9, 12) SEGRED_TR(7, 9, 13)
                             "s_waitcnt lgkmcnt(0)"
                             : "=&v"(x[0].h[0]), "=&v"(x[0].h[1]), "=&v"(x[1].h[0]), "=&v"(x[1].h[1]),
                               "=&v"(y[0].h[0]), "=&v"(y[0].h[1]), "=&v"(y[1].h[0]), "=&v"(y[1].h[1])
                             : "v"(p), "v"(q), "n"(0), "n"(4 * kRow), "n"(32 * kRow), "n"(36 * kRow)
                             : "memory");
            else
                asm volatile(SEGRED_TR(0, 4, 6) SEGRED_TR(1, 4, 7) SEGRED_TR(2, 5, 6) SEGRED_TR(3, 5, 7)
                             "s_waitcnt lgkmcnt(0)"
                             : "=&v"(x[0].h[0]), "=&v"(x[0].h[1]), "=&v"(y[0].h[0]), "=&v"(y[0].h[1])
                             : "v"(p), "v"(q), "n"(0), "n"(4 * kRow)
                             : "memory");
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                f[ks][i] = x[ks].v;
                f[ks][i + 1] = y[ks].v;
            }
        }
        if constexpr (N % 2 == 1) {
            const uint32_t p = at(N - 1);
            Frag x[KS];
            if constexpr (KS == 2)
                asm volatile(SEGRED_TR(0, 4, 5) SEGRED_TR(1, 4, 6) SEGRED_TR(2, 4, 7) SEGRED_TR(3, 4, 8)
                             "s_waitcnt lgkmcnt(0)"
                             : "=&v"(x[0].h[0]), "=&v"(x[0].h[1]), "=&v"(x[1].h[0]), "=&v"(x[1].h[1])
                             : "v"(p), "n"(0), "n"(4 * kRow), "n"(32 * kRow), "n"(36 * kRow)
                             : "memory");
            else
                asm volatile(SEGRED_TR(0, 2, 3) SEGRED_TR(1, 2, 4)
                             "s_waitcnt lgkmcnt(0)"
                             : "=&v"(x[0].h[0]), "=&v"(x[0].h[1])
                             : "v"(p), "n"(0), "n"(4 * kRow)
                             : "memory");
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) f[ks][N - 1] = x[ks].v;
        }
#undef SEGRED_TR
    }
}

template <typename T>
__device__ __forceinline__ f32x4 mma(u32x4 b, u32x4 a, f32x4 c) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[j]), __uint_as_float(a[j]), c, 0, 0, 0);
        return c;
    } else if constexpr (__is_same(T, __bf16)) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
    }
}

// One step of a wave's MT x NT neighbouring blocks of 16 x 16: rows from m0,
// columns from n0 of the workgroup's tile.
template <typename T, int MT, int NT, bool A_COL, int AW, bool B_COL, int BW>
__device__ __forceinline__ void step_products(f32x4 (&acc)[MT][NT], const lds_char *la, const lds_char *lb, int m0,
                                              int n0, int lane) {
    u32x4 a[2][MT], b[2][NT];
    if constexpr (A_COL) col_frags<T, AW>(a, la, m0, lane);
    else row_frags(a, la, m0, lane);
    if constexpr (B_COL) col_frags<T, BW>(b, lb, n0, lane);
    else row_frags(b, lb, n0, lane);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = mma<T>(b[ks][j], a[ks][i], acc[i][j]);
}

// ------------------------------------------------------------------- waits

// Waits until at most N of this wave's loads are in flight and meets the
// other waves.  (A workgroup fence would wait for all of them.)
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The launch grid of `total` tiles and the tile index of a workgroup.  A
// dimension of the grid may not pass 2^32 threads, so long grids are folded.
constexpr int64_t kGridFold = int64_t(1) << 20;
inline bool tile_grid(int64_t total, dim3 &grid) {
    const int64_t y = (total + kGridFold - 1) / kGridFold;
    if (y > 65535) return false;
    grid = dim3((unsigned)(y > 1 ? kGridFold : total), (unsigned)y);
    return true;
}

// ------------------------------------------------------- float in three bf16
//
// v_mfma_f32_16x16x4_f32 runs at a sixteenth of the 16-bit rate, so a float
// product is made of 16-bit ones: x = h + m + l exactly, h the leading 8 bits
// of x (cut off), m and l the remainders rounded to bf16, and
//   x y = h h' + (h m' + m h') + (h l' + m m' + l h') + ...
// with what is left out (m l', l m', l l') below 2^-22 |x y|, about the
// rounding of a product to float.  Six products at 16 times the rate.  bf16 has
// float's exponents, but the matrix cores take parts below 2^-126 for zero, so
// that values below 2^-102 lose bits (less than 2^-125 each).
//
// An infinity has no such parts (h is infinite, m and l are NaN), and of a
// product that leaves float's range l h' may be an infinity of the wrong sign
// beside that of h h', since l has either sign.  Either way the sum is not
// finite: a tile with such a sum is computed again with float products, so that
// infinities and NaN come out as float arithmetic gives them.
//
// A step is 32 k.  It passes through registers, is split on its way into LDS
// and lies there as three planes in the forms of the 16-bit types (row form
// with rows of 64 bytes: unit u of row r at place u ^ (r >> 2 & 3)).
constexpr int kSplitK = 32;

struct Split {
    u32x4 h, m, l;
};
// Splits eight floats.
__device__ __forceinline__ Split split_unit(u32x4 a, u32x4 b) {
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    Split s;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t x0 = j < 2 ? a[2 * j] : b[2 * j - 4], x1 = j < 2 ? a[2 * j + 1] : b[2 * j - 3];
        const uint32_t t0 = x0 & 0xffff0000u, t1 = x1 & 0xffff0000u;
        const float r0 = __uint_as_float(x0) - __uint_as_float(t0), r1 = __uint_as_float(x1) - __uint_as_float(t1);
        const uint32_t m = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{r0, r1}), bf16x2));
        const float q0 = r0 - __uint_as_float(m << 16), q1 = r1 - __uint_as_float(m & 0xffff0000u);
        s.h[j] = __builtin_amdgcn_perm(t1, t0, 0x07060302u);
        s.m[j] = m;
        s.l[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{q0, q1}), bf16x2));
    }
    return s;
}

// A 16-bit operand beside a float one has fewer parts: a bf16 is its own h, a
// float16 (11 bits) is h + m.
template <typename S> constexpr int kPlanes = sizeof(S) == 4 ? 3 : __is_same(S, __bf16) ? 1 : 2;

// h and m of eight 16-bit values (h alone for bf16).
template <typename S>
__device__ __forceinline__ Split split_short(u32x4 a) {
    const u32x4 none = {0u, 0u, 0u, 0u};
    if constexpr (__is_same(S, __bf16)) {
        return {a, none, none};
    } else {
        const f16x8 x = __builtin_bit_cast(f16x8, a);
        bf16x8 h, m;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = (float)x[j], t = __uint_as_float(__float_as_uint(f) & 0xffff0000u);
            h[j] = (__bf16)t;
            m[j] = (__bf16)(f - t);
        }
        return {__builtin_bit_cast(u32x4, h), __builtin_bit_cast(u32x4, m), none};
    }
}

// NaN where a value of c is infinite or NaN, else z.
__device__ __forceinline__ float not_finite(f32x4 c, float z) {
#pragma unroll
    for (int j = 0; j < 4; ++j) z = fmaf(c[j], 0.f, z);
    return z;
}
template <int MT, int NT>
__device__ __forceinline__ bool any_not_finite(const f32x4 (&acc)[MT][NT]) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) z = not_finite(acc[i][j], z);
    return z != 0.f;
}

// One operand's step in registers: W rows (or columns) of 32 k, eight
// neighbouring values of type S at a time.  COL: W neighbours of one k, else 32
// k of one row.  WHOLE: rows hold whole parts, so that each is there or not.
template <int W, int THREADS, bool COL, bool WHOLE, typename S = float>
struct SplitStage {
    static constexpr int kParts = W * 4 / THREADS;  // of eight values, per thread
    static constexpr int kPlane = W * 64;           // bytes
    static constexpr int kLds = kPlanes<S> * kPlane;
    static_assert(kParts >= 1 && W * 4 % THREADS == 0, "whole parts");
    u32x4 v[kParts][sizeof(S) / 2];

    // Row (k if COL) and first element inside it of part i.
    static __device__ __forceinline__ int row(int i, int tid) { return (i * THREADS + tid) / (COL ? W / 8 : 4); }
    static __device__ __forceinline__ int at(int i, int tid) { return (i * THREADS + tid) % (COL ? W / 8 : 4) * 8; }
    // src(i): address of part i; left(i): values of its row from there on.
    template <bool EIGHT = WHOLE, typename F, typename G>
    __device__ __forceinline__ void issue(F src, G left) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            if constexpr (sizeof(S) == 2) {
                if constexpr (EIGHT) v[i][0] = load_whole<S>(left(i) > 0 ? src(i) : (uint64_t)zero_unit());
                else v[i][0] = load_unit<S>(src(i), left(i));
            } else if constexpr (EIGHT) {
                const uint64_t q = left(i) > 0 ? src(i) : (uint64_t)zero_unit();
                v[i][0] = load_whole<float>(q);
                v[i][1] = load_whole<float>(q + 16);
            } else {
                v[i][0] = load_unit<float>(src(i), left(i));
                v[i][1] = load_unit<float>(src(i) + 16, left(i) - 4);
            }
        }
    }
    __device__ __forceinline__ void commit(lds_char *lds, int tid) const {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int r = row(i, tid), c = at(i, tid);
            int off;
            if constexpr (COL) off = r * W * 2 + (((c >> 4) ^ col_swizzle<__bf16, W>(r)) << 5) + (c & 8) * 2;
            else off = r * 64 + (((c >> 3) ^ ((r >> 2) & 3)) << 4);
            Split s;
            if constexpr (sizeof(S) == 4) s = split_unit(v[i][0], v[i][1]);
            else s = split_short<S>(v[i][0]);
            typedef __attribute__((address_space(3))) u32x4 lds_unit;
            *reinterpret_cast<lds_unit *>(lds + off) = s.h;
            if constexpr (kPlanes<S> > 1) *reinterpret_cast<lds_unit *>(lds + kPlane + off) = s.m;
            if constexpr (kPlanes<S> > 2) *reinterpret_cast<lds_unit *>(lds + 2 * kPlane + off) = s.l;
        }
    }
};

template <bool COL, int W>
__device__ __forceinline__ u32x4 split_frag(const lds_char *plane, int r0, int lane) {
    if constexpr (COL) return col_frag<__bf16, W>(plane, r0, 0, lane);
    const int off = (r0 + (lane & 15)) * 64 + (((lane >> 4) ^ ((lane >> 2) & 3)) << 4);
    return *reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>(plane + off);
}

// One step of a wave's MT x NT neighbouring blocks, the small terms first.  PA
// and PB: parts of either operand.
template <int MT, int NT, bool A_COL, int AW, bool B_COL, int BW, int PA = 3, int PB = 3>
__device__ __forceinline__ void split_step(f32x4 (&acc)[MT][NT], const lds_char *la, const lds_char *lb, int m0, int n0,
                                           int lane) {
    u32x4 a[PA][MT];
#pragma unroll
    for (int p = 0; p < PA; ++p)
#pragma unroll
        for (int i = 0; i < MT; ++i) a[p][i] = split_frag<A_COL, AW>(la + p * AW * 64, m0 + 16 * i, lane);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        u32x4 b[PB];
#pragma unroll
        for (int p = 0; p < PB; ++p) b[p] = split_frag<B_COL, BW>(lb + p * BW * 64, n0 + 16 * j, lane);
#pragma unroll
        for (int q = 0; q < 6; ++q) {
            constexpr int kA[6] = {2, 1, 0, 1, 0, 0}, kB[6] = {0, 1, 2, 0, 1, 0};
            if (kA[q] >= PA || kB[q] >= PB) continue;
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i][j] = mma<__bf16>(b[kB[q]], a[kA[q]][i], acc[i][j]);
        }
    }
}

// Walks the steps of a tile: issue(t) loads into registers, commit() writes
// them, products() multiplies.  One buffer; a second workgroup on the CU works
// through the waits.
template <typename I, typename C, typename P>
__device__ __forceinline__ void split_steps(int64_t steps, I issue, C commit, P products) {
    if (steps > 0) issue(0);
    for (int64_t t = 0; t < steps; ++t) {
        commit();
        __syncthreads();
        if (t + 1 < steps) issue(t + 1);
        products();
        __syncthreads();
    }
}

// ------------------------------------------------------------- in phases
//
// The large tiles of the 16-bit types: 256 columns by AH * 128 rows, 8 waves,
// 2 by 4.  Each operand's step is cut into halves of 128 rows (columns), and a
// wave owns 64 x 32 of each quadrant.  A step takes one phase per quadrant, in
// an order that changes one half at a time; a phase first moves data
// (fragments of the half that changes, from LDS; a half of a later step, from
// memory into a place that has been read) and then multiplies.  Waves 4..7,
// which share the SIMDs with waves 0..3, run one barrier behind, so that on
// each SIMD one wave multiplies while the other moves data.
//
//   AH = 2     reads    fetches    multiplies      places: two steps
//     0        A0(t)    A1(t+1)    A0 B0
//     1        B1(t)    B0(t+2)    A0 B1
//     2        A1(t)    A0(t+2)    A1 B1
//     3        B0(t+1)  B1(t+2)    A1 B0
//
//   AH = 1     reads           fetches            multiplies   three steps
//     0        A0(t)           A0(t+2)            A0 B0
//     1        B1(t), B0(t+1)  B1(t+2), B0(t+3)   A0 B1
//
// A half is read one phase after every wave has waited for it; the loads
// issued since (2 per half and thread) may be in flight.  A half's place is
// filled again two phases after it was read, when the wave that reads last has
// multiplied what it read.  The loads past the last step fetch zeros.
constexpr int kHalf = 128;
constexpr int kPhaseThreads = 512;
constexpr int kHalfBytes = kHalf * 128;
constexpr int kPhaseLds = 9 * kHalfBytes;  // two steps of A0 A1 B0 B1, or three of A0 B0 B1

// The products of a phase: c += a b over the step's two k halves.
template <typename T>
__device__ __forceinline__ void quadrant(f32x4 (&c)[4][2], const u32x4 (&a)[2][4], const u32x4 (&b)[2][2]) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) c[i][j] = mma<T>(b[ks][j], a[ks][i], c[i][j]);
}

// fetch_a(h, t, place) and fetch_b(h, t, place) start half h of step t (two
// loads per thread; zeros past the last step); products(c, a, b) are a
// phase's.  acc[a][b] are the quadrants.
template <typename T, int AH, bool B_COL, typename FA, typename FB, typename P>
__device__ __forceinline__ void phase_steps(f32x4 (&acc)[2][2][4][2], lds_char *lds, int steps, int wave, int lane,
                                            FA fetch_a, FB fetch_b, P products) {
    static_assert(sizeof(T) == 2, "16-bit types");
    const int ma = (wave >> 2) * 64, nb = (wave & 3) * 32;
    u32x4 a[2][4], b0[2][2], b1[2][2];
    auto read_a = [&](const lds_char *p) { row_frags(a, p, ma, lane); };
    auto read_b = [&](u32x4 (&b)[2][2], const lds_char *p) {
        if constexpr (B_COL) col_frags<T, kHalf>(b, p, nb, lane);
        else row_frags(b, p, nb, lane);
    };
    auto multiply = [&](f32x4 (&c)[4][2], const u32x4 (&b)[2][2]) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        products(c, a, b);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
#define SEGRED_MEET(N)                                                      \
    __builtin_amdgcn_sched_barrier(0);                                      \
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");

    if constexpr (AH == 2) {
        auto place_a = [&](int h, int t) { return lds + ((t & 1) * 4 + h) * kHalfBytes; };
        auto place_b = [&](int h, int t) { return lds + ((t & 1) * 4 + 2 + h) * kHalfBytes; };
        u32x4 b0_next[2][2];
        fetch_b(0, 0, place_b(0, 0));
        fetch_a(0, 0, place_a(0, 0));
        fetch_b(1, 0, place_b(1, 0));
        fetch_a(1, 0, place_a(1, 0));
        fetch_b(0, 1, place_b(0, 1));
        fetch_a(0, 1, place_a(0, 1));
        fetch_b(1, 1, place_b(1, 1));
        wait_and_meet<10>();
        read_b(b0, place_b(0, 0));
        wait_and_meet<10>();
        if (wave >= 4) asm volatile("s_barrier" ::: "memory");
        for (int t = 0; t < steps; ++t) {
            read_a(place_a(0, t));
            fetch_a(1, t + 1, place_a(1, t + 1));
            SEGRED_MEET(10)
            multiply(acc[0][0], b0);

            read_b(b1, place_b(1, t));
            fetch_b(0, t + 2, place_b(0, t));
            SEGRED_MEET(10)
            multiply(acc[0][1], b1);

            read_a(place_a(1, t));
            fetch_a(0, t + 2, place_a(0, t));
            SEGRED_MEET(10)
            multiply(acc[1][1], b1);

            read_b(b0_next, place_b(0, t + 1));
            fetch_b(1, t + 2, place_b(1, t));
            SEGRED_MEET(10)
            multiply(acc[1][0], b0);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int j = 0; j < 2; ++j) b0[ks][j] = b0_next[ks][j];
        }
    } else {
        constexpr int kStepBytes = 3 * kHalfBytes;  // A0 B0 B1
        fetch_b(0, 0, lds + kHalfBytes);
        fetch_a(0, 0, lds);
        fetch_b(1, 0, lds + 2 * kHalfBytes);
        fetch_b(0, 1, lds + kStepBytes + kHalfBytes);
        fetch_a(0, 1, lds + kStepBytes);
        fetch_b(1, 1, lds + kStepBytes + 2 * kHalfBytes);
        fetch_b(0, 2, lds + 2 * kStepBytes + kHalfBytes);
        wait_and_meet<10>();
        read_b(b0, lds + kHalfBytes);
        wait_and_meet<10>();
        if (wave >= 4) asm volatile("s_barrier" ::: "memory");
        lds_char *now = lds, *next = lds + kStepBytes, *after = lds + 2 * kStepBytes;
        for (int t = 0; t < steps; ++t) {
            read_a(now);
            fetch_a(0, t + 2, after);
            SEGRED_MEET(8)
            multiply(acc[0][0], b0);

            read_b(b0, next + kHalfBytes);  // before b1, whose arrival then implies b0's
            read_b(b1, now + 2 * kHalfBytes);
            fetch_b(1, t + 2, after + 2 * kHalfBytes);
            fetch_b(0, t + 3, now + kHalfBytes);
            SEGRED_MEET(10)
            multiply(acc[0][1], b1);
            lds_char *const first = now;
            now = next;
            next = after;
            after = first;
        }
    }
#undef SEGRED_MEET
    if (wave < 4) asm volatile("s_barrier" ::: "memory");
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the zeros past the last step
}

// Row and column of quadrant (a, b)'s 16 x 16 block (i, j) in the tile.
__device__ __forceinline__ int phase_row(int a, int i, int wave) { return a * kHalf + (wave >> 2) * 64 + 16 * i; }
__device__ __forceinline__ int phase_col(int b, int j, int wave) { return b * kHalf + (wave & 3) * 32 + 16 * j; }

// ------------------------------------------------------------- wave's own
//
// With few rows a workgroup's waves split the contraction instead of the
// tile: each wave walks its steps [t0, t1) through LDS buffers of its own,
// without meeting the others, and the accumulators are added at the end.

// Waits until at most N of this wave's loads are in flight and its LDS reads
// are done.
template <int N>
__device__ __forceinline__ void wait_own() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// issue(t, live, buf): start step t (zeros where not live); commit(buf): write
// units held in registers; products(t, buf); meanwhile(): what can be done
// while the first steps arrive.
template <int STAGES, bool DIRECT, int LOADS, int BYTES, typename I, typename C, typename P, typename M>
__device__ __forceinline__ void wave_steps(lds_char *lds, int t0, int t1, I issue, C commit, P products, M meanwhile) {
    if constexpr (DIRECT) {
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) issue(t0 + i, t0 + i < t1, lds + i * BYTES);
        meanwhile();
        int cur = 0, fill = STAGES - 1;
        for (int t = t0; t < t1; ++t) {
            wait_own<(STAGES - 2) * LOADS>();
            issue(t + STAGES - 1, t + STAGES - 1 < t1, lds + fill * BYTES);
            products(t, lds + cur * BYTES);
            cur = cur + 1 == STAGES ? 0 : cur + 1;
            fill = fill + 1 == STAGES ? 0 : fill + 1;
        }
        wait_own<0>();  // the last loads write zeros into LDS
    } else {
        if (t0 < t1) {
            issue(t0, true, lds);
            commit(lds);
        }
        meanwhile();
        for (int t = t0; t < t1; ++t) {
            wave_lds_sync();
            if (t + 1 < t1) issue(t + 1, true, lds);
            products(t, lds + ((t - t0) & 1) * BYTES);
            wave_lds_sync();
            if (t + 1 < t1) commit(lds + ((t + 1 - t0) & 1) * BYTES);
        }
    }
}

// Adds the waves' accumulators in wave order and gives each quad of columns
// to one thread: out(row, column, sum).  `lds` is the workgroup's, at least
// NW * MT * NT KiB, and may be the step buffers.
template <int NW, int MT, int NT, typename F>
__device__ __forceinline__ void join_waves(lds_char *lds, const f32x4 (&acc)[MT][NT], int wave, int lane, F out) {
    typedef __attribute__((address_space(3))) f32x4 lds_quad;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<lds_quad *>(lds + ((wave * MT + i) * NT + j) * 1024 + lane * 16) = acc[i][j];
    __syncthreads();
    for (int q = wave * 64 + lane; q < MT * NT * 64; q += NW * 64) {
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w)
            sum += *reinterpret_cast<const lds_quad *>(lds + w * MT * NT * 1024 + q * 16);
        const int block = q >> 6, l = q & 63;
        out(block / NT * 16 + (l & 15), block % NT * 16 + (l >> 4) * 4, sum);
    }
}

// ------------------------------------------------------------------ output

// Four consecutive elements from column n of a row of `width` elements, each
// rounded to T once.  VEC: the row starts on a 4-element boundary and its
// width is a multiple of 4.
template <typename T>
__device__ __forceinline__ void store_quad(T *row, int64_t n, int64_t width, f32x4 c, bool vec) {
    if (vec) {
        if (n < width) {
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<f32x4 *>(row + n) = c;
            } else {
                typedef __attribute__((ext_vector_type(4))) T T4;
                T4 q;
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = (T)c[j];
                *reinterpret_cast<T4 *>(row + n) = q;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < width) row[n + j] = (T)c[j];
    }
}

// A tile of 16-bit results on its way out through LDS, so that its rows are
// written in whole stretches: stored from the lanes' quads, 32 bytes of a row at
// a time, the 256 x 256 tiles of 32,768 rows by 2,048 columns took 50 us of 350.
// The 16-byte unit u of row r lies at place u ^ (r & 7) * 2, which spreads the
// quads of 16 rows over the banks.
template <typename T, int BN>
__device__ __forceinline__ int tile_unit(int r, int u) {
    constexpr int kUnits = BN / 8;
    return r * BN * 2 + ((u ^ (((r & 7) << 1) & (kUnits - 1))) << 4);
}
template <typename T, int BN>
__device__ __forceinline__ void tile_put(lds_char *lds, int r, int c, f32x4 v) {
    static_assert(sizeof(T) == 2, "16-bit results");
    typedef __attribute__((ext_vector_type(4))) T T4;
    T4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = (T)v[j];
    *reinterpret_cast<__attribute__((address_space(3))) T4 *>(lds + tile_unit<T, BN>(r, c >> 3) + (c & 4) * 2) = q;
}
// Writes the first `rows` rows of the tile to out, whose rows have `width`
// elements of which the tile's begin at n0.  VEC: rows of whole units on
// 16-byte boundaries.
template <typename T, int BM, int BN, int THREADS>
__device__ __forceinline__ void tile_out(const lds_char *lds, T *out, int rows, int64_t n0, int64_t width, bool vec) {
    constexpr int kUnits = BN / 8;
#pragma unroll 4
    for (int i = threadIdx.x; i < BM * kUnits; i += THREADS) {
        const int r = i / kUnits, u = i % kUnits;
        const int64_t n = n0 + u * 8;
        if (r >= rows || n >= width) continue;
        union {
            u32x4 v;
            T e[8];
        } x;
        x.v = *reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>(lds + tile_unit<T, BN>(r, u));
        T *to = out + r * width + n;
        if (vec) {
            *reinterpret_cast<u32x4 *>(to) = x.v;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n + e < width) to[e] = x.e[e];
        }
    }
}

// ------------------------------------------------------------- tile places

// Workgroups are dealt to the 8 XCDs in turn; this maps the launch index to a
// tile index such that each XCD (with an L2 of its own) owns one contiguous
// range of tiles.
__device__ __forceinline__ int64_t xcd_tile(int64_t total) {
    const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (id >= total) return total;
    const int64_t q = total >> 3, r = total & 7, x = id & 7, i = id >> 3;
    return x * q + (x < r ? x : r) + i;
}

// Row tile and column tile of tile `id` of mt x nt: groups of 4 row tiles walk
// the column tiles together, so that the 32 tiles an XCD works on at a time
// share 4 row strips and 8 column strips.
struct TilePlace {
    int64_t m, n;
};
__device__ __forceinline__ TilePlace tile_place(int64_t id, int64_t mt, int64_t nt) {
    const int64_t group = id / (4 * nt), in = id - group * 4 * nt;
    const int64_t gm = min((int64_t)4, mt - group * 4);
    return {group * 4 + in % gm, in / gm};
}

// The rows of segment s are cut into slots of `step` rows from the segment's
// start.  Slot keys need no table: segment s owns the slots from
// key(s) = (offsets[s] - offsets[0]) / step + s up to key(s + 1), which are at
// least ceil(len / step) and at least one; what is over is empty.  There are
// (offsets[S] - offsets[0]) / step + S slots in all.
__device__ __forceinline__ int64_t slot_key(const int64_t *offsets, int64_t s, int64_t step) {
    return (offsets[s] - offsets[0]) / step + s;
}

// The same with fewer empty slots, for calls that need none for an empty
// segment, and for steps of 2^lg rows:
// key(s) = (offsets[s] - offsets[0] + s (2^lg - 1)) / 2^lg, which still grows
// by at least ceil(len / 2^lg).  tight_slots() of them in all.
__device__ __forceinline__ int64_t tight_key(const int64_t *offsets, int64_t s, int lg) {
    return (offsets[s] - offsets[0] + (s << lg) - s) >> lg;
}
inline int64_t tight_slots(int64_t rows, int64_t segments, int lg) { return (rows + (segments << lg) - segments) >> lg; }

// The segment of `slot`, found with 64 probes a round (every lane must call
// it): the last one whose key is not above it.
template <typename K>
__device__ __forceinline__ int64_t slot_segment(int64_t S, int64_t slot, int lane, K key) {
    int64_t lo = 0, hi = S;
    while (hi - lo > 1) {
        const int64_t d = (hi - lo + 63) >> 6;
        const int64_t s = lo + lane * d;
        bool below = false;
        if (s < hi) below = key(s) <= slot;
        const int n = popc64(ballot(below));
        lo += (n > 0 ? n - 1 : 0) * d;
        hi = hi < lo + d ? hi : lo + d;
    }
    return readfirst(lo);
}
__device__ __forceinline__ int64_t tight_segment(const int64_t *offsets, int64_t S, int lg, int64_t slot, int lane) {
    return slot_segment(S, slot, lane, [&](int64_t s) { return tight_key(offsets, s, lg); });
}

}  // namespace segred
