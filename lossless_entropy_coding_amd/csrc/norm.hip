// Layer norm, forward and backward.
#include "ffn_common.h"

namespace ec {
namespace {

// A row is held in the registers of THREADS threads, V chunks of eight
// neighbouring values each (chunk v of thread t starts at column
// 8 (v THREADS + t)), so x is read once and the variance is that of the
// centred values.  Both passes are bound by the bytes they move: at 8192 x
// 2048 in bf16 the forward pass takes 19.0 us (3.5 TB/s), the backward pass
// 36.3 us (3.7 TB/s) and 4.5 us for the sums of its partial rows; a copy
// reaches 4.8 TB/s.  One row of 2048 takes 2.7 us, a launch.
//
// WHOLE: the columns are a multiple of eight, so a chunk is whole or empty.
template <bool WHOLE>
__device__ __forceinline__ uint32_t left_of(uint32_t cols, uint32_t c) {
    if constexpr (WHOLE)
        return cols > c ? 8 : 0;
    else
        return cols > c ? cols - c : 0;
}

// Zeros where nothing is left.
template <bool WHOLE>
__device__ __forceinline__ void load_chunk(const void *p, uint32_t dtype, uint64_t at, uint32_t left, float *v) {
    if constexpr (WHOLE) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = 0.0f;
        if (left) load8(p, dtype, at, 8, v);
    } else {
        load8(p, dtype, at, left, v);
    }
}

// A chunk on its way: as it lies in memory where it is whole, so that a row
// loaded ahead takes half the registers in bf16.
template <bool F32, bool WHOLE>
struct Chunk {
    static constexpr bool kRaw = WHOLE && !F32;
    float v[kRaw ? 1 : 8];
    u32x4 raw;

    __device__ __forceinline__ void load(const void *p, uint64_t at, uint32_t left) {
        if constexpr (kRaw) {
            raw = u32x4{0, 0, 0, 0};
            if (left) raw = ((const AnyU32x4 *)((const uint16_t *)p + at))->v;
        } else {
            load_chunk<WHOLE>(p, F32 ? EC_FP32 : EC_BF16, at, left, v);
        }
    }

    __device__ __forceinline__ void get(float *o) const {
        if constexpr (kRaw) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                o[2 * q] = __uint_as_float(raw[q] << 16);
                o[2 * q + 1] = __uint_as_float(raw[q] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = v[q];
        }
    }
};

// weight or bias; `none` where there is none
template <bool WHOLE>
__device__ __forceinline__ void load_param(const void *p, uint32_t dtype, uint32_t c, uint32_t left, float none,
                                           float *v) {
    if (p) {
        load_chunk<WHOLE>(p, dtype, c, left, v);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = none;
    }
}

// Sums over a row's threads, the same value in every one of them.  Every
// thread of the workgroup calls it where a row has more than one wave.
template <int THREADS, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *sh) {
#pragma unroll
    for (int d = 32; d; d >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor(v[n], d);
    if constexpr (THREADS > 64) {
        constexpr int kWaves = THREADS / 64;
        const uint32_t wave = threadIdx.x >> 6, first = wave / kWaves * kWaves;
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) sh[n * 16 + wave] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) s += sh[n * 16 + first + w];
            v[n] = s;
        }
    }
}

template <bool F32, bool WHOLE, int BLOCK, int THREADS, int V>
__global__ __launch_bounds__(BLOCK) void norm_kernel(NormArgs p) {
    constexpr int kRows = BLOCK / THREADS;                          // a workgroup's rows at a time
    __shared__ float sh[32];
    const uint32_t t = threadIdx.x % THREADS;
    const float scale = p.out_scale ? *p.out_scale : 1.0f, cols = (float)p.cols;
    // weight and bias stay in registers over the rows, and the next row is
    // loaded while this one is worked on
    constexpr bool kKeep = V <= 4;
    float w[kKeep ? V : 1][8], b[kKeep ? V : 1][8];
    if constexpr (kKeep) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t c = 8 * (v * THREADS + t), left = left_of<WHOLE>(p.cols, c);
            load_param<WHOLE>(p.weight, p.w_dtype, c, left, 1.0f, w[v]);
            load_param<WHOLE>(p.bias, p.w_dtype, c, left, 0.0f, b[v]);
        }
    }
    Chunk<F32, WHOLE> ahead[V];
    const auto load = [&](uint64_t row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t c = 8 * (v * THREADS + t);
            ahead[v].load(p.x, row * p.x_stride + c, row < p.rows ? left_of<WHOLE>(p.cols, c) : 0);
        }
    };
    const uint64_t step = (uint64_t)gridDim.x * kRows;
    load((uint64_t)blockIdx.x * kRows + threadIdx.x / THREADS);
    for (uint64_t first = (uint64_t)blockIdx.x * kRows; first < p.rows; first += step) {
        const uint64_t row = first + threadIdx.x / THREADS;
        const bool in = row < p.rows;
        float x[V][8], s[1] = {0.0f}, m[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) ahead[v].get(x[v]);
        if (first + step < p.rows) load(row + step);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int q = 0; q < 8; ++q) s[0] += x[v][q];
        row_sum<THREADS>(s, sh);
        // The sum's rounding leaves `near` off by a part of itself, which a row
        // far from zero would take for its spread: the mean of what is left is
        // summed beside the squares and taken out of both.  A constant row's
        // mean becomes its value, and its variance zero.
        const float near = s[0] / cols;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t left = left_of<WHOLE>(p.cols, 8 * (v * THREADS + t));
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                x[v][q] -= near;
                m[0] += q < (int)left ? x[v][q] : 0.0f;
                m[1] += q < (int)left ? x[v][q] * x[v][q] : 0.0f;
            }
        }
        row_sum<THREADS>(m, sh);
        const float off = m[0] / cols, mean = near + off;
        const float var = __builtin_fmaf(-off, off, m[1] / cols);
        const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + p.eps);
        if (!in) continue;
        if (t == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t c = 8 * (v * THREADS + t), left = left_of<WHOLE>(p.cols, c);
            if (!left) break;
            const int k = kKeep ? v : 0;
            if constexpr (!kKeep) {
                load_param<WHOLE>(p.weight, p.w_dtype, c, left, 1.0f, w[0]);
                load_param<WHOLE>(p.bias, p.w_dtype, c, left, 0.0f, b[0]);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) x[v][q] = ((x[v][q] - off) * rstd * w[k][q] + b[k][q]) * scale;
            store8(p.y, p.out_dtype, row * p.y_stride + c, left, x[v]);
        }
    }
}

// Backward.  A workgroup walks over rows and keeps the sums of dweight and
// dbias for its columns in registers; they are joined over its rows in LDS
// and written once.  Rows wider than THREADS * V * 8 are cut into slices
// (blockIdx.y): each slice's workgroup sums over the whole row, but writes dx
// and the sums of its own columns only, so dx may not lie over x or dy there.
template <bool F32, bool WHOLE, int THREADS, int V>
__global__ __launch_bounds__(512) void norm_grad_kernel(NormGradArgs p) {
    constexpr int kRows = 512 / THREADS, kSlice = THREADS * V * 8;
    constexpr uint32_t kType = F32 ? EC_FP32 : EC_BF16;
    __shared__ float sh[32];
    __shared__ float join[kRows > 1 ? 2 * kSlice : 1];
    const uint32_t t = threadIdx.x % THREADS, r0 = threadIdx.x / THREADS, first = blockIdx.y * kSlice;
    const float cols = (float)p.cols;
    float dw[V][8] = {}, db[V][8] = {}, w[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint32_t c = first + 8 * (v * THREADS + t);
        load_param<WHOLE>(p.weight, p.w_dtype, c, left_of<WHOLE>(p.cols, c), 1.0f, w[v]);
    }
    // the next row is loaded while this one is worked on
    Chunk<F32, WHOLE> nx[V], nd[V], nr[V];
    float nmean, nrstd;
    const auto load = [&](uint64_t row) {
        const bool in = row < p.rows;
        nmean = in ? p.mean[row] : 0.0f;
        nrstd = in ? p.rstd[row] : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t c = first + 8 * (v * THREADS + t), left = in ? left_of<WHOLE>(p.cols, c) : 0;
            nx[v].load(p.x, row * p.x_stride + c, left);
            nd[v].load(p.dy, row * p.dy_stride + c, left);
            nr[v].load(p.dres, row * p.dres_stride + c, p.dres && p.dx ? left : 0);
        }
    };
    const uint64_t step = (uint64_t)gridDim.x * kRows;
    load((uint64_t)blockIdx.x * kRows + r0);
    for (uint64_t base = (uint64_t)blockIdx.x * kRows; base < p.rows; base += step) {
        const uint64_t row = base + r0;
        const bool in = row < p.rows;
        const float mean = nmean, rstd = nrstd;
        float h[V][8], dy[V][8], s[2] = {0.0f, 0.0f};
        Chunk<F32, WHOLE> dres[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nx[v].get(h[v]);
            nd[v].get(dy[v]);
            dres[v] = nr[v];
        }
        if (base + step < p.rows) load(row + step);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t left = left_of<WHOLE>(p.cols, first + 8 * (v * THREADS + t));
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                h[v][q] = q < (int)left ? (h[v][q] - mean) * rstd : 0.0f;
                const float g = dy[v][q] * w[v][q];
                s[0] += g;
                s[1] += g * h[v][q];
                dw[v][q] += dy[v][q] * h[v][q];
                db[v][q] += dy[v][q];
            }
        }
        if (!p.dx) continue;
        for (uint32_t other = 0; other < gridDim.y; ++other) {      // the row's other slices
            if (other == blockIdx.y) continue;
            for (int v = 0; v < V; ++v) {
                const uint32_t c = other * kSlice + 8 * (v * THREADS + t), left = in ? left_of<WHOLE>(p.cols, c) : 0;
                float ox[8], od[8], ow[8];
                load_chunk<WHOLE>(p.x, kType, row * p.x_stride + c, left, ox);
                load_chunk<WHOLE>(p.dy, kType, row * p.dy_stride + c, left, od);
                load_param<WHOLE>(p.weight, p.w_dtype, c, left, 1.0f, ow);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float g = q < (int)left ? od[q] * ow[q] : 0.0f;
                    s[0] += g;
                    s[1] += q < (int)left ? g * ((ox[q] - mean) * rstd) : 0.0f;
                }
            }
        }
        row_sum<THREADS>(s, sh);
        const float mt = s[0] / cols, mth = s[1] / cols;
        if (!in) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t c = first + 8 * (v * THREADS + t), left = left_of<WHOLE>(p.cols, c);
            if (!left) break;
            float o[8], res[8];
            dres[v].get(res);
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = rstd * (dy[v][q] * w[v][q] - mt - h[v][q] * mth) + res[q];
            store8(p.dx, kType, row * p.dx_stride + c, left, o);
        }
    }
    if (!p.partial) return;
    if constexpr (kRows > 1) {
        // the rows' threads add their sums in turn: the first's, plus the second's, ...
        for (uint32_t r = 0; r < (uint32_t)kRows; ++r) {
            if (r0 == r) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const uint32_t at = (v * 8 + q) * THREADS + t;
                        if (r) {
                            dw[v][q] += join[at];
                            db[v][q] += join[kSlice + at];
                        }
                        if (r + 1 < (uint32_t)kRows) {
                            join[at] = dw[v][q];
                            join[kSlice + at] = db[v][q];
                        }
                    }
            }
            __syncthreads();
        }
        if (r0 != kRows - 1) return;
    }
    float *o = p.partial + (uint64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint32_t c = first + 8 * (v * THREADS + t), left = left_of<WHOLE>(p.cols, c);
        if (!left) break;
        store8(o, EC_FP32, c, left, dw[v]);
        store8(o + p.cols, EC_FP32, c, left, db[v]);
    }
}

// Adds the parts in a fixed order: 16 columns by 16 threads that take every
// 16th part each.
__global__ __launch_bounds__(256) void norm_grad_sum_kernel(NormGradArgs p) {
    __shared__ float sh[16][17];
    const uint32_t x = threadIdx.x & 15, y = threadIdx.x >> 4;
    const uint64_t c = (uint64_t)blockIdx.x * 16 + x, n = 2 * (uint64_t)p.cols;
    float s = 0.0f;
    if (c < n)
#pragma unroll 8                            // loads of eight parts on the way
        for (uint32_t q = y; q < p.parts; q += 16) s += p.partial[q * n + c];
    sh[y][x] = s;
    __syncthreads();
    if (y || c >= n) return;
    for (int k = 1; k < 16; ++k) s += sh[k][x];
    if (c < p.cols) {
        if (p.dweight) p.dweight[c] = s;
    } else if (p.dbias) {
        p.dbias[c - p.cols] = s;
    }
}

template <bool F32, int BLOCK, int THREADS, int V>
void run_norm(const NormArgs &a, hipStream_t s) {
    constexpr int kRows = BLOCK / THREADS;
    const uint64_t need = (a.rows + kRows - 1) / kRows;
    // as many workgroups as run at a time, 16 waves a CU, each with several rows
    const uint64_t most = 256 * 1024 / BLOCK;
    const uint32_t blocks = (uint32_t)(need < most ? need : most);
    if (a.cols % 8 == 0)
        norm_kernel<F32, true, BLOCK, THREADS, V><<<blocks, BLOCK, 0, s>>>(a);
    else
        norm_kernel<F32, false, BLOCK, THREADS, V><<<blocks, BLOCK, 0, s>>>(a);
}

// Threads a row: one wave while a row fits its registers in four chunks a
// lane and there are rows enough for every CU (no barrier in the sums), more
// for longer rows, and for few rows, where the time is that of one row.
template <bool F32>
void pick_norm(const NormArgs &a, hipStream_t s) {
    const uint32_t c = a.cols;
    if (c <= 512)
        run_norm<F32, 256, 64, 1>(a, s);
    else if (c <= 2048 && a.rows >= 1024)
        c <= 1024 ? run_norm<F32, 256, 64, 2>(a, s) : run_norm<F32, 256, 64, 4>(a, s);
    else if (c <= 8192)
        c <= 2048 ? run_norm<F32, 256, 256, 1>(a, s)
                  : c <= 4096 ? run_norm<F32, 256, 256, 2>(a, s) : run_norm<F32, 256, 256, 4>(a, s);
    else if (c <= 16384)
        run_norm<F32, 1024, 1024, 2>(a, s);
    else
        c <= 32768 ? run_norm<F32, 1024, 1024, 4>(a, s) : run_norm<F32, 1024, 1024, 8>(a, s);
}

template <bool F32, int THREADS, int V>
void run_norm_grad(const NormGradArgs &a, hipStream_t s) {
    const dim3 grid(a.parts, (a.cols + THREADS * V * 8 - 1) / (THREADS * V * 8));
    if (a.cols % 8 == 0)
        norm_grad_kernel<F32, true, THREADS, V><<<grid, 512, 0, s>>>(a);
    else
        norm_grad_kernel<F32, false, THREADS, V><<<grid, 512, 0, s>>>(a);
}

// Threads a row in the backward pass: two chunks a thread, whose sums and
// values leave room for four waves a SIMD.
uint32_t grad_threads(uint64_t cols) { return cols <= 512 ? 64 : cols <= 2048 ? 128 : cols <= 4096 ? 256 : 512; }

template <bool F32>
void pick_norm_grad(const NormGradArgs &a, hipStream_t s) {
    switch (grad_threads(a.cols)) {
        case 64: run_norm_grad<F32, 64, 1>(a, s); break;
        case 128: a.cols <= 1024 ? run_norm_grad<F32, 128, 1>(a, s) : run_norm_grad<F32, 128, 2>(a, s); break;
        case 256: run_norm_grad<F32, 256, 2>(a, s); break;
        default: run_norm_grad<F32, 512, 2>(a, s);
    }
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, hipStream_t s) {
    if (!a.rows) return hipSuccess;
    a.dtype == EC_FP32 ? pick_norm<true>(a, s) : pick_norm<false>(a, s);
    return hipGetLastError();
}

// Workgroups of the backward pass, each with a row of sums to add: two a CU.
uint32_t norm_grad_parts(uint64_t rows, uint64_t cols) {
    const uint64_t at_once = 512 / grad_threads(cols), need = (rows + at_once - 1) / at_once;
    return (uint32_t)(need < 1 ? 1 : need < 512 ? need : 512);
}

// Only the widest kernel, of two chunks in 512 threads, cuts rows.
uint32_t norm_grad_slices(uint64_t cols) { return (uint32_t)((cols + 8191) / 8192); }

hipError_t launch_norm_grad(const NormGradArgs &a, hipStream_t s) {
    if (a.dx || a.partial) a.dtype == EC_FP32 ? pick_norm_grad<true>(a, s) : pick_norm_grad<false>(a, s);
    if (a.partial) norm_grad_sum_kernel<<<(2 * a.cols + 15) / 16, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace ec
