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
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kE4m3Max = 448.0f;

// ------------------------------------------------------------- product launch

// Products beside ec_linear_op's.
enum ProductOp : uint32_t {
    kOpGated = 3,       // forward, B's first J rows the gate, the next J what it is multiplied by
    kOpRowStats,        // forward, of each row of D the maximum and the sum of exponentials only
    kOpLogitGrad,       // forward, D turned into the gradient of the cross entropy
    kOpPieceInput,      // grad input over a piece of the contraction, added up in fp32
    kOpPieceWeight      // grad weight of a piece
};

constexpr bool contracts_a_rows(uint32_t op) { return op == EC_LINEAR_GRAD_WEIGHT || op == kOpPieceWeight; }
constexpr bool contracts_b_rows(uint32_t op) {
    return op == EC_LINEAR_GRAD_INPUT || op == kOpPieceInput || contracts_a_rows(op);
}
// Whether the number of rows (of the contraction, in grad weight) is found on the device.
constexpr bool counts_rows(uint32_t op) { return op >= kOpLogitGrad; }

// One product D[i, j] = sum_c A[i, c] B[j, c] with an epilogue; i are rows of
// the output, j its contiguous columns, c the contraction:
//   forward      i = token,         j = output column, c = input column
//   grad input   i = token,         j = input column,  c = output column
//   grad weight  i = output column, j = input column,  c = token
// A(i, c) is at a + i * a_i + c * a_c (elements), B(j, c) likewise.
struct ProductArgs {
    const void *a, *b;
    uint64_t a_i, a_c, b_j, b_c, b_group;  // b_group: elements between experts' B (forward, grad input)
    bool a_padded, b_padded;               // A's (B's) rows hold zeros up to a multiple of 16 bytes
    uint32_t I, J, C;
    uint32_t op;                           // ec_linear_op or ProductOp
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
    float *db;                             // grad weight: [groups][I] sums of A over the contraction, or null
    // the loss over columns j (kOpRowStats, and by piece the operators after it)
    const void *target;                    // kOpRowStats: [I] int32 or int64
    uint32_t target_bytes;
    float *hit;                            // kOpRowStats: [I] D at the target's column, where that exists
    float2 *stats;                         // kOpRowStats: [I][tiles_j] maximum, sum of exponentials from it
    const uint32_t *used;                  // rows that exist, of those the launch has room for
    const float2 *row;                     // kOpLogitGrad: [I] log of the sum of exponentials, gradient of the loss
    const int32_t *row_target;             // kOpLogitGrad: [I] the target's column
    uint32_t first;                        // kOpLogitGrad: the piece's first column
    const float *sum_in;                   // kOpPieceInput: [I, J] added to D, or null
    const uint32_t *kept;                  // kOpPieceInput: where D's rows go in out, or null
    // filled in by the plan
    uint32_t tiles_i, tiles_j, splits, blocks;
    float *partial;                        // [splits][tile][TI * TJ] when splits > 1
};

struct ColumnSumArgs {                     // db
    const uint16_t *dy;
    uint64_t dy_stride;
    uint32_t m, n, groups;
    const int32_t *offsets;
    float *db;
    uint32_t *status;
};

bool product_fits(const ProductArgs &a);            // whether some tile can address its rows
uint64_t product_workspace(const ProductArgs &a);
bool product_need(const ProductArgs &a, uint64_t *bytes);   // both, from one plan
bool product_sums_columns(const ProductArgs &a);    // whether the product can write db as well
hipError_t launch_product(ProductArgs a, void *workspace, hipStream_t s);
hipError_t launch_check_offsets(const int32_t *offsets, uint32_t groups, uint32_t m, uint32_t *status, hipStream_t s);
uint64_t column_sum_workspace(const ColumnSumArgs &a);
hipError_t launch_column_sum(const ColumnSumArgs &a, float *workspace, hipStream_t s);
hipError_t launch_copy_rows(const void *in, uint64_t stride, uint64_t rows, uint64_t cols, uint32_t dtype, void *out,
                            uint64_t pitch, hipStream_t s);

// The gated product's backward pass up to the products: dz = [dy rest act'(gate), dy act(gate)] from
// preact = [gate, rest] (n columns each), and the sums of dz's rows before their rounding.
struct GatedGradArgs {
    const uint16_t *dy, *preact;
    uint64_t dy_stride, preact_stride;
    uint32_t m, n, groups, act;
    const int32_t *offsets;
    uint32_t *status;
    uint16_t *dz;                          // [m, pitch], zeros in columns 2 n ..; rows of no group are left as they are
    uint64_t pitch;
    float *db;                             // [groups][2 n], or null
    uint32_t slab;                         // rows a workgroup takes
    float *partial;                        // [slabs + groups][2 n]
};

hipError_t launch_gated(ProductArgs a, void *workspace, hipStream_t s);
uint32_t gated_grad_slab(uint32_t m, uint32_t n);
bool gated_grad_fits(const GatedGradArgs &a);
uint64_t gated_grad_workspace(const GatedGradArgs &a);
hipError_t launch_gated_grad(const GatedGradArgs &a, hipStream_t s);

// Cross entropy over the products of x and w, forward and backward.
struct LossArgs {
    const void *x, *w;
    uint64_t x_stride, w_stride;
    uint32_t m, n, k;
    const void *target;
    uint32_t target_bytes;
    int64_t ignore;
    float *loss, *lse;                     // lse: read in the backward pass
    const float *dloss;
    uint32_t dlosses;                      // 1 or m
    void *dx;
    uint64_t dx_stride;
    void *dw;
    uint64_t dw_stride;
    uint32_t dw_dtype;
    uint32_t *status;
};

// The workspace's bytes, or false where sizes are too large; launches where the workspace given holds them.
bool loss_need(const LossArgs &a, uint64_t *bytes);
bool loss_grad_need(const LossArgs &a, uint64_t *bytes);
int run_loss(const LossArgs &a, void *workspace, uint64_t bytes, hipStream_t s);        // ec_error
int run_loss_grad(const LossArgs &a, void *workspace, uint64_t bytes, hipStream_t s);

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
uint32_t norm_grad_slices(uint64_t cols);              // workgroups that share a row
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

__device__ __forceinline__ bf16x8 e4m3_to_bf16x8(uint32_t lo, uint32_t hi) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
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

// Phi(-|z|) and e = exp(-z^2 / 2).  Phi(-a) = e g(a), where g(a) =
// e^(a^2/2) Phi(-a) falls slowly, as t P(t) with t = 1 / (1 + 0.3 a) and P of
// degree 7: fitted for the least largest relative error on 0 <= a <= 14
// (1.5e-7; 4.6e-7 with P in fp32).  The tail is a product, never 1 minus
// something near 1, so it keeps its relative accuracy down to where e leaves
// fp32's normal range (|z| > 13.2): (16 + 1.25 z^2) 2^-24, the second part
// from the rounding of e's exponent.
__device__ __forceinline__ float normal_tail(float z, float *e) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(z), 0.3f, 1.0f));
    *e = __builtin_amdgcn_exp2f(z * z * -0.72134752f);
    float p = __builtin_fmaf(t, 0.0356747657f, -0.157203048f);
    p = __builtin_fmaf(t, p, 0.206353441f);
    p = __builtin_fmaf(t, p, -0.053683579f);
    p = __builtin_fmaf(t, p, 0.128561586f);
    p = __builtin_fmaf(t, p, 0.0999135002f);
    p = __builtin_fmaf(t, p, 0.120753951f);
    p = __builtin_fmaf(t, p, 0.119629301f);
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

// ------------------------------------------------------ sums of exponentials

constexpr float kLog2E = 1.44269504f;

// (maximum, sum of exponentials from it) of two sets of values.  With no value
// above -inf in either the sum stays 0.
__device__ __forceinline__ float2 join_stats(float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x), from = top == -__builtin_inff() ? 0.0f : top;
    return float2{top, a.y * __builtin_amdgcn_exp2f((a.x - from) * kLog2E) +
                           b.y * __builtin_amdgcn_exp2f((b.x - from) * kLog2E)};
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

// A grouped product's rows fall into ranges: those before the first offset,
// those of each group, and those after the last.  Each range is cut into
// tiles of `tile` rows, in this order: at most m / tile + (ranges with rows)
// of them.
struct RowTile {
    uint32_t row, end;     // rows [row, end) of the group, at most one tile
    uint32_t group;
    bool zero;             // rows of no group (written as zeros)
};

// 64 of the ranges, one a lane: [start, end), and the tiles up to and with
// the lane's.  edge and tiles carry over from the ranges before.
__device__ __forceinline__ void scan_ranges(const int32_t *offsets, uint32_t groups, uint32_t m, uint32_t tile,
                                            uint32_t base, uint32_t edge, uint32_t tiles, uint32_t *start,
                                            uint32_t *end, uint32_t *n, uint32_t *sum) {
    const uint32_t lane = threadIdx.x & 63, r = base + lane;
    // range r = 0 .. groups + 1 ends at offset[r] (r <= groups) or m
    uint32_t e = r <= groups ? (uint32_t)min(max(offsets[r], 0), (int32_t)m) : m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {      // running maximum
        const uint32_t o = (uint32_t)__shfl_up((int)e, d);
        if (lane >= (uint32_t)d) e = max(e, o);
    }
    e = max(e, edge);
    uint32_t s = (uint32_t)__shfl_up((int)e, 1);
    if (lane == 0) s = edge;
    const uint32_t c = r < groups + 2 ? (e - s + tile - 1) / tile : 0;
    uint32_t t = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)t, d);
        if (lane >= (uint32_t)d) t += o;
    }
    *start = s;
    *end = e;
    *n = c;
    *sum = t + tiles;
}

// The number of row tiles; all 64 lanes of a wave call it.
__device__ __forceinline__ uint32_t count_row_tiles(const int32_t *offsets, uint32_t groups, uint32_t m,
                                                    uint32_t tile) {
    uint32_t edge = 0, tiles = 0, start, end, n, sum;
    for (uint32_t base = 0; base < groups + 2; base += 64) {
        scan_ranges(offsets, groups, m, tile, base, edge, tiles, &start, &end, &n, &sum);
        edge = (uint32_t)__shfl((int)end, 63);
        tiles = (uint32_t)__shfl((int)sum, 63);
    }
    return tiles;
}

// Row tile t (less than their number); all 64 lanes of a wave call it.
__device__ __forceinline__ RowTile find_row_tile(const int32_t *offsets, uint32_t groups, uint32_t m, uint32_t tile,
                                                 uint32_t t) {
    uint32_t edge = 0, tiles = 0, start, end, n, sum;
    RowTile q = {0, 0, 0, true};
    for (uint32_t base = 0; base < groups + 2; base += 64) {
        scan_ranges(offsets, groups, m, tile, base, edge, tiles, &start, &end, &n, &sum);
        const uint64_t hit = __ballot(sum > t);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            const uint32_t first = (uint32_t)__shfl((int)(sum - n), l);
            const uint32_t lo = (uint32_t)__shfl((int)start, l), hi = (uint32_t)__shfl((int)end, l);
            q.row = lo + (t - first) * tile;
            q.end = min(hi, q.row + tile);
            q.zero = base + l == 0 || base + l == groups + 1;
            q.group = q.zero ? 0 : base + l - 1;
            break;
        }
        edge = (uint32_t)__shfl((int)end, 63);
        tiles = (uint32_t)__shfl((int)sum, 63);
    }
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

// Vectors at any address that suits their elements.
struct __attribute__((packed, aligned(1))) AnyByteU32x4 { u32x4 v; };
struct __attribute__((packed, aligned(2))) AnyU32x4 { u32x4 v; };
struct __attribute__((packed, aligned(1))) AnyU32x2 { u32x2 v; };
struct __attribute__((packed, aligned(4))) AnyF32x4 { f32x4 v; };

// Eight values of bf16 or fp32 at p[at ..], of which `left` exist (the rest read as zero).
__device__ __forceinline__ void load8_bf16(const void *p, uint64_t at, uint32_t left, float *v) {
    const uint16_t *b = (const uint16_t *)p + at;
    if (left >= 8) {
        const u32x4 w = ((const AnyU32x4 *)b)->v;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = __uint_as_float(w[q] << 16);
            v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < (int)left ? bf16_to_f32(b[q]) : 0.0f;
    }
}

__device__ __forceinline__ void load8(const void *p, uint32_t dtype, uint64_t at, uint32_t left, float *v) {
    if (dtype == EC_BF16) {
        load8_bf16(p, at, left, v);
    } else if (left >= 8) {
        const AnyF32x4 *f = (const AnyF32x4 *)((const float *)p + at);
        const f32x4 a = f[0].v, b = f[1].v;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = a[q];
            v[q + 4] = b[q];
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < (int)left ? ((const float *)p)[at + q] : 0.0f;
    }
}

// Stores eight values as `dtype`, the first `left` of them.
__device__ __forceinline__ void store8(void *p, uint32_t dtype, uint64_t at, uint32_t left, const float *v) {
    if (dtype == EC_BF16) {
        uint16_t *o = (uint16_t *)p + at;
        u32x4 w;
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = f32_to_bf16x2(v[2 * q], v[2 * q + 1]);
        if (left >= 8)
            ((AnyU32x4 *)o)->v = w;
        else
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < (int)left) o[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
    } else if (dtype == EC_E4M3) {
        uint8_t *o = (uint8_t *)p + at;
        u32x2 w;
        w[0] = f32_to_e4m3x4(v[0], v[1], v[2], v[3]);
        w[1] = f32_to_e4m3x4(v[4], v[5], v[6], v[7]);
        if (left >= 8)
            ((AnyU32x2 *)o)->v = w;
        else
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < (int)left) o[q] = (uint8_t)(w[q >> 2] >> (8 * (q & 3)));
    } else {
        float *o = (float *)p + at;
        if (left >= 8) {
            ((AnyF32x4 *)o)[0].v = f32x4{v[0], v[1], v[2], v[3]};
            ((AnyF32x4 *)o)[1].v = f32x4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < (int)left) o[q] = v[q];
        }
    }
}

// What the epilogue of eight output columns needs besides the sums.
struct Columns {
    float w_scale[8], bias[8];
    uint32_t left;                         // columns that exist, of those from j on
};

template <int OP>
__device__ __forceinline__ Columns load_columns(const ProductArgs &p, uint32_t g, uint32_t j) {
    Columns c;
    c.left = p.J > j ? p.J - j : 0;
    if constexpr (OP == EC_LINEAR_FORWARD) {
        if (p.w_scale) {
            if (p.w_scales > 1) {
                load8(p.w_scale, EC_FP32, (uint64_t)g * p.w_scales + j, c.left, c.w_scale);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) c.w_scale[q] = p.w_scale[g];
            }
        }
        if (p.bias) load8(p.bias, p.bias_dtype, (uint64_t)g * p.J + j, c.left, c.bias);
    }
    return c;
}

// The residual (forward) or the activation's input (grad input) of eight columns of row i.
template <int OP>
__device__ __forceinline__ void load_side(const ProductArgs &p, uint32_t i, uint32_t j, uint32_t left, float *v) {
    if constexpr (OP == EC_LINEAR_FORWARD) {
        if (p.residual && left) load8_bf16(p.residual, i * p.residual_stride + j, left, v);
    } else if constexpr (OP == EC_LINEAR_GRAD_INPUT) {
        if (p.act != EC_ACT_NONE && left) load8_bf16(p.preact, i * p.preact_stride + j, left, v);
    }
}

// Finishes and stores eight sums of row i, columns j .. j + 7.  `zero` rows
// get zeros (their sums are zeros, and only the bias could make them others).
template <int OP, int ACT>
__device__ __forceinline__ void finish8(const ProductArgs &p, uint32_t g, uint32_t i, uint32_t j, float *v,
                                        const Columns &c, const float *side, float x_scale, float out_scale,
                                        bool zero) {
    if (!c.left) return;
    if constexpr (OP == EC_LINEAR_FORWARD) {
        if (p.x_scale) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= x_scale;
        }
        if (p.w_scale) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= c.w_scale[q];
        }
        if (p.bias) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += c.bias[q];
        }
        if (zero) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = 0.0f;
        }
        if (p.preact) store8(p.preact, EC_BF16, i * p.preact_stride + j, c.left, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = act_value<ACT>(v[q]);
        if (p.residual && !zero) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += side[q];
        }
        if (p.out_scale) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= out_scale;
        }
    } else if constexpr (OP == kOpPieceInput) {
        if (p.sum_in) {
            float before[8];
            load8(p.sum_in, EC_FP32, (uint64_t)i * p.J + j, c.left, before);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += before[q];
        }
        if (p.kept) i = p.kept[i];
    } else if constexpr (OP == EC_LINEAR_GRAD_INPUT) {
        if constexpr (ACT != EC_ACT_NONE) {
            if (!zero) {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= act_slope<ACT>(side[q]);
            }
        }
    }
    store8(p.out, p.out_dtype, (OP == EC_LINEAR_GRAD_WEIGHT ? g * p.out_group : 0) + i * p.out_stride + j, c.left, v);
}

}  // namespace ec
