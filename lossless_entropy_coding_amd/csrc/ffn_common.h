// Device helpers and launch interfaces of the feed-forward operators
// (matrix products with a fused epilogue, layer norm).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ec.h"

namespace ec {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kE4m3Max = 448.0f;

// ------------------------------------------------------------- product launch

// One product D[i, j] = sum_c A[i, c] B[j, c] with an epilogue; i are rows of
// the output, j its contiguous columns, c the contraction:
//   forward      i = token,         j = output column, c = input column
//   grad input   i = token,         j = input column,  c = output column
//   grad weight  i = output column, j = input column,  c = token
// A(i, c) is at a + i * a_i + c * a_c (elements), B(j, c) likewise.
struct ProductArgs {
    const void *a, *b;
    uint64_t a_i, a_c, b_j, b_c, b_group;  // b_group: elements between experts' B (forward, grad input)
    uint32_t I, J, C;
    uint32_t op;                           // ec_linear_op
    uint32_t dtype;                        // EC_BF16 or EC_E4M3
    uint32_t groups;                       // 0: one product
    const int32_t *offsets;                // [groups + 1]: rows i (forward, grad input) or contraction c (grad weight)
    uint32_t *status;
    // epilogue
    uint32_t act, out_dtype, bias_dtype, x_scales, w_scales;
    const void *bias;
    const uint16_t *residual;
    uint64_t residual_stride;
    const float *x_scale, *w_scale, *out_scale;
    void *out;
    uint64_t out_stride, out_group;        // out_group: elements between experts' dw
    uint16_t *preact;                      // written (forward) or read (grad input)
    uint64_t preact_stride;
};

struct ColumnSumArgs {                     // db
    const uint16_t *dy;
    uint64_t dy_stride;
    uint32_t m, n, groups;
    const int32_t *offsets;
    float *db;
    float *partial;                        // [parts][groups or 1][n] when parts > 1
    uint32_t parts;
    uint32_t *status;
};

hipError_t launch_product(const ProductArgs &a, hipStream_t s);
hipError_t launch_column_sum(const ColumnSumArgs &a, hipStream_t s);

struct NormArgs {
    const void *x;
    uint64_t rows, x_stride;
    uint32_t cols, dtype, w_dtype, out_dtype;
    const void *weight, *bias;
    float eps;
    void *y;
    uint64_t y_stride;
    const float *out_scale;
    float *mean, *rstd;
};

struct NormGradArgs {
    const void *dy, *x, *weight, *dres;
    uint64_t rows, dy_stride, x_stride, dres_stride, dx_stride;
    uint32_t cols, dtype, w_dtype;
    const float *mean, *rstd;
    void *dx;
    float *dweight, *dbias;
    float *partial;                        // [parts][2][cols]
    uint32_t parts;
};

hipError_t launch_norm(const NormArgs &a, hipStream_t s);
uint32_t norm_grad_parts(uint64_t rows, uint64_t cols);
hipError_t launch_norm_grad(const NormGradArgs &a, hipStream_t s);

// ---------------------------------------------------------------- conversions

__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
    __bf16 b = (__bf16)v;                  // round to nearest, ties to even
    return __builtin_bit_cast(uint16_t, b);
}

__device__ __forceinline__ uint32_t f32_to_bf16x2(float lo, float hi) {
    bf16x2 b;
    b[0] = (__bf16)lo;
    b[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, b);
}

// The conversion makes NaN of what is beyond 448; e4m3 bytes here saturate
// (and NaN stays NaN), so values are clamped first.
__device__ __forceinline__ float e4m3_clamp(float v) {
    const float c = __builtin_amdgcn_fmed3f(v, -kE4m3Max, kE4m3Max);
    return v != v ? v : c;
}

__device__ __forceinline__ uint32_t f32_to_e4m3x4(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(a), e4m3_clamp(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(c), e4m3_clamp(d), r, true);
}

// ---------------------------------------------------------------- activations

// h(z) = Phi(-|z|) and e = exp(-z^2 / 2) with the rational approximation
// 7.1.26 of Abramowitz and Stegun (|error| of Phi <= 7.5e-8):
//   erfc(u) ~ (a1 t + ... + a5 t^5) exp(-u^2), t = 1 / (1 + p u), u = |z| / sqrt 2.
// The tail is the product itself, never 1 minus something near 1, so small
// values keep their relative accuracy.
__device__ __forceinline__ float normal_tail(float z, float *e) {
    const float u = __builtin_fabsf(z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(u, 0.3275911f * 0.70710678f, 1.0f));
    *e = __builtin_amdgcn_exp2f(z * z * -0.72134752f);
    float p = __builtin_fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
    p = __builtin_fmaf(t, p, 0.5f * 1.421413741f);
    p = __builtin_fmaf(t, p, 0.5f * -0.284496736f);
    p = __builtin_fmaf(t, p, 0.5f * 0.254829592f);
    return p * t * *e;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == EC_ACT_GELU) {
        float e;
        const float h = normal_tail(z, &e);
        return z * (z < 0.0f ? h : 1.0f - h);
    } else if constexpr (ACT == EC_ACT_SILU) {
        return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
    } else if constexpr (ACT == EC_ACT_RELU) {
        return z < 0.0f ? 0.0f : z;
    } else {
        return z;
    }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == EC_ACT_GELU) {
        float e;
        const float h = normal_tail(z, &e);
        return __builtin_fmaf(z * e, 0.39894228f, z < 0.0f ? h : 1.0f - h);
    } else if constexpr (ACT == EC_ACT_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
        return s * __builtin_fmaf(z, 1.0f - s, 1.0f);
    } else if constexpr (ACT == EC_ACT_RELU) {
        return z > 0.0f ? 1.0f : 0.0f;
    } else {
        return 1.0f;
    }
}

// ------------------------------------------------------------- ragged groups

// Row range of expert g: the running maximum of the offsets, clamped to
// [0, m], so that ranges never overlap whatever the offsets hold.  All 64
// lanes of a wave call it.
__device__ __forceinline__ void group_range(const int32_t *offsets, uint32_t m, uint32_t g, uint32_t *lo,
                                            uint32_t *hi) {
    const uint32_t lane = threadIdx.x & 63;
    int32_t before = 0;
    for (uint32_t i = lane; i <= g; i += 64) before = max(before, offsets[i]);
#pragma unroll
    for (int d = 32; d; d >>= 1) before = max(before, __shfl_xor(before, d));
    *lo = min((uint32_t)before, m);
    *hi = min((uint32_t)max(before, offsets[g + 1]), m);
}

struct RowTile {
    uint32_t row, end;     // rows [row, end) of the group, at most one tile
    uint32_t group;
    bool none, zero;       // past the last tile; rows of no group (written as zeros)
};

// Tile t of a grouped product, tiles of `tile` rows: the rows before the
// first offset, those of each group, and those after the last, cut into tiles
// in this order.  Tiles number at most ceil(m / tile) + groups + 2.  All 64
// lanes of a wave call it.
__device__ __forceinline__ RowTile find_row_tile(const int32_t *offsets, uint32_t groups, uint32_t m, uint32_t tile,
                                                 uint32_t t) {
    const uint32_t lane = threadIdx.x & 63;
    uint32_t edge = 0, tiles = 0;          // carried: end of the ranges so far, their tiles
    // range r = 0 .. groups + 1 ends at offset[r] (r <= groups) or m
    for (uint32_t base = 0; base < groups + 2; base += 64) {
        const uint32_t r = base + lane;
        uint32_t end = r <= groups ? (uint32_t)min(max(offsets[min(r, groups)], 0), (int32_t)m) : m;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {  // running maximum
            const uint32_t o = (uint32_t)__shfl_up((int)end, d);
            if (lane >= (uint32_t)d) end = max(end, o);
        }
        end = max(end, edge);
        uint32_t start = (uint32_t)__shfl_up((int)end, 1);
        if (lane == 0) start = edge;
        uint32_t n = r < groups + 2 ? (end - start + tile - 1) / tile : 0, sum = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = (uint32_t)__shfl_up((int)sum, d);
            if (lane >= (uint32_t)d) sum += o;
        }
        sum += tiles;
        const uint64_t hit = __ballot(sum > t);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            const uint32_t first = (uint32_t)__shfl((int)(sum - n), l);
            const uint32_t lo = (uint32_t)__shfl((int)start, l), hi = (uint32_t)__shfl((int)end, l);
            RowTile q;
            q.row = lo + (t - first) * tile;
            q.end = min(hi, q.row + tile);
            q.zero = base + l == 0 || base + l == groups + 1;
            q.group = q.zero ? 0 : base + l - 1;
            q.none = false;
            return q;
        }
        edge = (uint32_t)__shfl((int)end, 63);
        tiles = (uint32_t)__shfl((int)sum, 63);
    }
    RowTile q;
    q.none = true;
    q.zero = false;
    q.row = q.end = q.group = 0;
    return q;
}

// Whether the offsets are usable as they stand; one wave.
__device__ __forceinline__ void check_offsets(const int32_t *offsets, uint32_t groups, uint32_t m, uint32_t *status) {
    if (!status) return;
    bool bad = false;
    for (uint32_t i = threadIdx.x & 63; i <= groups; i += 64) {
        const int32_t v = offsets[i];
        bad |= v < 0 || (uint32_t)v > m || (i && v < offsets[i - 1]);
    }
    if (__ballot(bad) && (threadIdx.x & 63) == 0)
        __hip_atomic_fetch_or(status, EC_S_BAD_OFFSETS, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ------------------------------------------------------------------- epilogue

// Stores V consecutive values of output row i, columns j .. j + V - 1 (clipped
// to J), after the epilogue of `OP`.  `zero` rows get zeros.
template <int OP, int ACT, int V>
__device__ __forceinline__ void store_values(const ProductArgs &p, uint32_t g, uint32_t i, uint32_t j, const float *acc,
                                             bool zero) {
    float v[V], z[V];
    const uint32_t left = p.J > j ? p.J - j : 0;
    if (!left) return;
    const bool whole = left >= (uint32_t)V;
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = acc[q];
    if constexpr (OP == EC_LINEAR_FORWARD) {
        if (p.x_scale) {
            const float f = p.x_scale[p.x_scales > 1 ? i : 0];
#pragma unroll
            for (int q = 0; q < V; ++q) v[q] *= f;
        }
        if (p.w_scale) {
            const float *f = p.w_scale + (uint64_t)g * p.w_scales;
#pragma unroll
            for (int q = 0; q < V; ++q) v[q] *= p.w_scales > 1 ? f[min(j + q, p.J - 1)] : f[0];
        }
        if (p.bias) {
            const uint64_t at = (uint64_t)g * p.J + j;
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (q < (int)left)
                    v[q] += p.bias_dtype == EC_FP32 ? ((const float *)p.bias)[at + q]
                                                    : bf16_to_f32(((const uint16_t *)p.bias)[at + q]);
        }
#pragma unroll
        for (int q = 0; q < V; ++q) {
            z[q] = v[q];
            v[q] = act_value<ACT>(v[q]);
        }
        if (p.residual) {
            const uint16_t *r = p.residual + i * p.residual_stride + j;
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (q < (int)left) v[q] += bf16_to_f32(r[q]);
        }
        if (p.out_scale) {
            const float f = *p.out_scale;
#pragma unroll
            for (int q = 0; q < V; ++q) v[q] *= f;
        }
        if (p.preact) {
            uint16_t *o = p.preact + i * p.preact_stride + j;
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (q < (int)left) o[q] = zero ? 0 : f32_to_bf16(z[q]);
        }
    } else if constexpr (OP == EC_LINEAR_GRAD_INPUT) {
        if constexpr (ACT != EC_ACT_NONE) {
            const uint16_t *r = p.preact + i * p.preact_stride + j;
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (q < (int)left) v[q] *= act_slope<ACT>(bf16_to_f32(r[q]));
        }
    }
    if (zero) {
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] = 0.0f;
    }
    const uint64_t at = (OP == EC_LINEAR_GRAD_WEIGHT ? g * p.out_group : 0) + i * p.out_stride + j;
    (void)whole;
    if (p.out_dtype == EC_FP32) {
        float *o = (float *)p.out + at;
#pragma unroll
        for (int q = 0; q < V; ++q)
            if (q < (int)left) o[q] = v[q];
    } else if (p.out_dtype == EC_BF16) {
        uint16_t *o = (uint16_t *)p.out + at;
#pragma unroll
        for (int q = 0; q < V; ++q)
            if (q < (int)left) o[q] = f32_to_bf16(v[q]);
    } else {
        uint8_t *o = (uint8_t *)p.out + at;
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            const uint32_t u = f32_to_e4m3x4(v[q], v[q + 1], v[q + 2], v[q + 3]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (q + r < (int)left) o[q + r] = (uint8_t)(u >> (8 * r));
        }
    }
}

}  // namespace ec
