// Layer norm, forward and backward.
#include "ffn_common.h"

namespace ec {
namespace {

template <bool F32>
__device__ __forceinline__ float load(const void *p, uint64_t at) {
    if constexpr (F32)
        return ((const float *)p)[at];
    else
        return bf16_to_f32(((const uint16_t *)p)[at]);
}

__device__ __forceinline__ float load_w(const void *p, uint32_t dtype, uint32_t c, float none) {
    if (!p) return none;
    return dtype == EC_FP32 ? ((const float *)p)[c] : bf16_to_f32(((const uint16_t *)p)[c]);
}

// Sum over the workgroup's 256 threads, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float *sh) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return sh[0] + sh[1] + sh[2] + sh[3];
}

// One workgroup a row; the row is read three times (mean, variance, values).
template <bool F32>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs p) {
    __shared__ float sh[4];
    const uint64_t row = blockIdx.x, at = row * p.x_stride;
    float s = 0.0f;
    for (uint32_t c = threadIdx.x; c < p.cols; c += 256) s += load<F32>(p.x, at + c);
    const float mean = block_sum(s, sh) / p.cols;
    s = 0.0f;
    for (uint32_t c = threadIdx.x; c < p.cols; c += 256) {
        const float d = load<F32>(p.x, at + c) - mean;
        s += d * d;
    }
    const float rstd = 1.0f / sqrtf(block_sum(s, sh) / p.cols + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    const float scale = p.out_scale ? *p.out_scale : 1.0f;
    for (uint32_t c = threadIdx.x; c < p.cols; c += 256) {
        const float v = (load<F32>(p.x, at + c) - mean) * rstd * load_w(p.weight, p.w_dtype, c, 1.0f) +
                        load_w(p.bias, p.w_dtype, c, 0.0f);
        const uint64_t o = row * p.y_stride + c;
        if (p.out_dtype == EC_FP32)
            ((float *)p.y)[o] = v;
        else if (p.out_dtype == EC_BF16)
            ((uint16_t *)p.y)[o] = f32_to_bf16(v);
        else
            ((uint8_t *)p.y)[o] = (uint8_t)f32_to_e4m3x4(v * scale, 0.0f, 0.0f, 0.0f);
    }
}

template <bool F32>
__global__ __launch_bounds__(256) void norm_grad_kernel(NormGradArgs p) {
    __shared__ float sh[4];
    const uint64_t row = blockIdx.x;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s = 0.0f, sh_ = 0.0f;
    for (uint32_t c = threadIdx.x; c < p.cols; c += 256) {
        const float h = (load<F32>(p.x, row * p.x_stride + c) - mean) * rstd;
        const float t = load<F32>(p.dy, row * p.dy_stride + c) * load_w(p.weight, p.w_dtype, c, 1.0f);
        s += t;
        sh_ += t * h;
    }
    const float mt = block_sum(s, sh) / p.cols, mth = block_sum(sh_, sh) / p.cols;
    for (uint32_t c = threadIdx.x; c < p.cols; c += 256) {
        const float h = (load<F32>(p.x, row * p.x_stride + c) - mean) * rstd;
        const float t = load<F32>(p.dy, row * p.dy_stride + c) * load_w(p.weight, p.w_dtype, c, 1.0f);
        float v = rstd * (t - mt - h * mth);
        if (p.dres) v += load<F32>(p.dres, row * p.dres_stride + c);
        const uint64_t o = row * p.dx_stride + c;
        if constexpr (F32)
            ((float *)p.dx)[o] = v;
        else
            ((uint16_t *)p.dx)[o] = f32_to_bf16(v);
    }
}

// Partial sums of dweight and dbias over a range of rows: one thread a column.
template <bool F32>
__global__ __launch_bounds__(256) void norm_grad_weight_kernel(NormGradArgs p) {
    const uint32_t c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    const uint64_t per = (p.rows + p.parts - 1) / p.parts, lo = blockIdx.y * per, hi = min(p.rows, lo + per);
    float dw = 0.0f, db = 0.0f;
    for (uint64_t r = lo; r < hi; ++r) {
        const float dy = load<F32>(p.dy, r * p.dy_stride + c);
        dw += dy * (load<F32>(p.x, r * p.x_stride + c) - p.mean[r]) * p.rstd[r];
        db += dy;
    }
    p.partial[((uint64_t)blockIdx.y * 2) * p.cols + c] = dw;
    p.partial[((uint64_t)blockIdx.y * 2 + 1) * p.cols + c] = db;
}

__global__ __launch_bounds__(256) void norm_grad_sum_kernel(NormGradArgs p) {
    const uint32_t c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float dw = 0.0f, db = 0.0f;
    for (uint32_t q = 0; q < p.parts; ++q) {
        dw += p.partial[((uint64_t)q * 2) * p.cols + c];
        db += p.partial[((uint64_t)q * 2 + 1) * p.cols + c];
    }
    if (p.dweight) p.dweight[c] = dw;
    if (p.dbias) p.dbias[c] = db;
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, hipStream_t s) {
    if (!a.rows) return hipSuccess;
    if (a.dtype == EC_FP32)
        norm_kernel<true><<<(uint32_t)a.rows, 256, 0, s>>>(a);
    else
        norm_kernel<false><<<(uint32_t)a.rows, 256, 0, s>>>(a);
    return hipGetLastError();
}

uint32_t norm_grad_parts(uint64_t rows, uint64_t) { return rows ? (uint32_t)((rows + 127) / 128 < 256 ? (rows + 127) / 128 : 256) : 1; }

hipError_t launch_norm_grad(const NormGradArgs &a, hipStream_t s) {
    const dim3 cols((a.cols + 255) / 256);
    if (a.rows && a.dx) {
        if (a.dtype == EC_FP32)
            norm_grad_kernel<true><<<(uint32_t)a.rows, 256, 0, s>>>(a);
        else
            norm_grad_kernel<false><<<(uint32_t)a.rows, 256, 0, s>>>(a);
    }
    if (a.dweight || a.dbias) {
        if (a.dtype == EC_FP32)
            norm_grad_weight_kernel<true><<<dim3(cols.x, a.parts), 256, 0, s>>>(a);
        else
            norm_grad_weight_kernel<false><<<dim3(cols.x, a.parts), 256, 0, s>>>(a);
        norm_grad_sum_kernel<<<cols, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace ec
