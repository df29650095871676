// Matrix products with a fused epilogue, dense and grouped by expert.
#include "ffn_common.h"

namespace ec {
namespace {

// ------------------------------------------------------------ simple product
//
// Tiles of 64 x 64 outputs, four waves of 32 x 32 each (2 x 2 MFMA tiles of
// 16 x 16 x 32).  The factors' tiles go through registers into LDS element by
// element, bounds checked, so any stride and size is right; e4m3 values are
// exact in bf16.  The j side is the MFMA's first operand, so that a lane ends
// up with four consecutive columns of one row.
constexpr int kTile = 64, kDepth = 32, kPitch = kDepth + 8;

template <bool E4M3>
__device__ __forceinline__ __bf16 element(const void *p, uint64_t at) {
    if constexpr (E4M3)
        return (__bf16)__builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t *)p)[at], 0);
    else
        return ((const __bf16 *)p)[at];
}

template <int OP, int ACT, bool E4M3>
__global__ __launch_bounds__(256) void simple_product_kernel(ProductArgs p) {
    __shared__ __attribute__((aligned(16))) __bf16 ta[kTile * kPitch], tb[kTile * kPitch];
    uint32_t g = 0, i0 = blockIdx.y * kTile, i1 = min(p.I, i0 + kTile), c0 = 0, c1 = p.C;
    bool zero = false;
    if (p.groups) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 64)
            check_offsets(p.offsets, p.groups, OP == EC_LINEAR_GRAD_WEIGHT ? p.C : p.I, p.status);
        if (OP == EC_LINEAR_GRAD_WEIGHT) {
            g = blockIdx.z;
            group_range(p.offsets, p.C, g, &c0, &c1);
        } else {
            const RowTile q = find_row_tile(p.offsets, p.groups, p.I, kTile, blockIdx.y);
            if (q.none) return;
            g = q.group;
            i0 = q.row;
            i1 = q.end;
            zero = q.zero;
            if (zero) c1 = 0;
        }
    }
    const uint32_t j0 = blockIdx.x * kTile;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
    f32x4 acc[2][2] = {};
    const uint64_t b_at = g * p.b_group;
    for (uint32_t c = c0; c < c1; c += kDepth) {
        __syncthreads();
        for (uint32_t q = threadIdx.x; q < kTile * kDepth; q += 256) {
            const uint32_t row = q / kDepth, col = q % kDepth;
            const bool in = c + col < c1;
            ta[row * kPitch + col] = in && i0 + row < i1
                                         ? element<E4M3>(p.a, (uint64_t)(i0 + row) * p.a_i + (uint64_t)(c + col) * p.a_c)
                                         : (__bf16)0.0f;
            tb[row * kPitch + col] = in && j0 + row < p.J
                                         ? element<E4M3>(p.b, b_at + (uint64_t)(j0 + row) * p.b_j +
                                                                  (uint64_t)(c + col) * p.b_c)
                                         : (__bf16)0.0f;
        }
        __syncthreads();
        bf16x8 fa[2], fb[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            fa[t] = *(const bf16x8 *)&ta[(wi + t * 16 + (lane & 15)) * kPitch + (lane >> 4) * 8];
            fb[t] = *(const bf16x8 *)&tb[(wj + t * 16 + (lane & 15)) * kPitch + (lane >> 4) * 8];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
                acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[y], fa[x], acc[x][y], 0, 0, 0);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint32_t i = i0 + wi + x * 16 + (lane & 15), j = j0 + wj + y * 16 + (lane >> 4) * 4;
            float v[4] = {acc[x][y][0], acc[x][y][1], acc[x][y][2], acc[x][y][3]};
            if (i < i1) store_values<OP, ACT, 4>(p, g, i, j, v, zero);
        }
}

// ---------------------------------------------------------------- column sums
//
// db[n] = sum of dy's rows; one thread per column, rows of the group in order.
__global__ __launch_bounds__(256) void column_sum_kernel(ColumnSumArgs p) {
    uint32_t lo = 0, hi = p.m;
    const uint32_t g = blockIdx.y;
    if (p.groups) group_range(p.offsets, p.m, g, &lo, &hi);
    const uint32_t n = blockIdx.x * 256 + threadIdx.x;
    if (n >= p.n) return;
    float s = 0.0f;
    for (uint32_t i = lo; i < hi; ++i) s += bf16_to_f32(p.dy[i * p.dy_stride + n]);
    p.db[(uint64_t)g * p.n + n] = s;
}

template <int OP, int ACT>
void launch_simple(const ProductArgs &a, dim3 grid, hipStream_t s) {
    if (OP == EC_LINEAR_FORWARD && a.dtype == EC_E4M3)
        simple_product_kernel<OP, ACT, true><<<grid, 256, 0, s>>>(a);
    else
        simple_product_kernel<OP, ACT, false><<<grid, 256, 0, s>>>(a);
}

template <int OP>
void launch_act(const ProductArgs &a, dim3 grid, hipStream_t s) {
    switch (a.act) {
        case EC_ACT_GELU: launch_simple<OP, EC_ACT_GELU>(a, grid, s); break;
        case EC_ACT_SILU: launch_simple<OP, EC_ACT_SILU>(a, grid, s); break;
        case EC_ACT_RELU: launch_simple<OP, EC_ACT_RELU>(a, grid, s); break;
        default: launch_simple<OP, EC_ACT_NONE>(a, grid, s);
    }
}

}  // namespace

hipError_t launch_product(const ProductArgs &a, hipStream_t s) {
    if (!a.I || !a.J) return hipSuccess;
    const bool ragged_rows = a.groups && a.op != EC_LINEAR_GRAD_WEIGHT;
    const uint64_t row_tiles = (a.I + (uint64_t)kTile - 1) / kTile + (ragged_rows ? a.groups + 2 : 0);
    if (row_tiles > 65535) return hipErrorInvalidValue;
    dim3 grid((a.J + kTile - 1) / kTile, (uint32_t)row_tiles, a.op == EC_LINEAR_GRAD_WEIGHT && a.groups ? a.groups : 1);
    if (a.op == EC_LINEAR_FORWARD)
        launch_act<EC_LINEAR_FORWARD>(a, grid, s);
    else if (a.op == EC_LINEAR_GRAD_INPUT)
        launch_act<EC_LINEAR_GRAD_INPUT>(a, grid, s);
    else
        launch_simple<EC_LINEAR_GRAD_WEIGHT, EC_ACT_NONE>(a, grid, s);
    return hipGetLastError();
}

hipError_t launch_column_sum(const ColumnSumArgs &a, hipStream_t s) {
    if (!a.n) return hipSuccess;
    column_sum_kernel<<<dim3((a.n + 255) / 256, a.groups ? a.groups : 1), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace ec
