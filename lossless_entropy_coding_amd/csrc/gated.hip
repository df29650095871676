// The gated feed-forward block: act(x gate^T) * (x rest^T) in one product,
// dense and by expert, and the backward pass up to the products.
#include "product_kernel.h"

namespace ec {
namespace {

// ------------------------------------------------------------------ few rows
//
// As few_rows_kernel, with the 16 columns' rows of the gate and of the factor
// beside it: twice the loads of B on each of A.
template <int RT, int ACT>
__device__ __forceinline__ void few_gated_finish(const ProductArgs &p, const Place &q, const float *sums, uint32_t waves) {
    const uint32_t t = threadIdx.x, i = q.i0 + (t >> 1), j = q.j0 + (t & 1) * 8;
    if (t >= RT * 32 || i >= q.i1) return;
    const GatedColumns c = load_gated_columns(p, q.group, j);
    const float xs = p.x_scale ? p.x_scale[p.x_scales > 1 ? i : 0] : 1.0f, os = p.out_scale ? *p.out_scale : 1.0f;
    float gate[8] = {}, rest[8] = {};
    few_sums<RT>(sums, waves, gate);
    few_sums<RT>(sums + waves * RT * 16 * 20, waves, rest);
    finish8_gated<ACT>(p, i, j, gate, rest, c, xs, os, q.zero);
}

template <int RT>
struct FewGated {
    static constexpr int TI = RT * 16, TJ = 32;         // TJ: rows of B, for 16 columns
};

template <int RT, int W, bool E4M3>
__global__ __launch_bounds__(W * 64) void few_gated_kernel(ProductArgs p) {
    constexpr int ES = E4M3 ? 1 : 2, U = 4;             // steps whose loads are on the way in a lane
    using T = FewGated<RT>;
    __shared__ __attribute__((aligned(16))) float sums[2 * W * RT * 16 * 20];   // [half][wave][row][16 columns and a gap]
    if (p.groups && blockIdx.x == 0 && threadIdx.x < 64) check_offsets(p.offsets, p.groups, p.I, p.status);
    const Place q = find_place<T, kOpGated>(p, blockIdx.x);
    if (q.none) return;
    const uint32_t lane = threadIdx.x & 63, row = lane & 15, part = (lane >> 4) * 16;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    // rows and columns that do not exist repeat the last one: their sums are not stored
    const uint64_t column = min(q.j0 + row, p.J - 1);
    const char *b[2], *a[RT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        b[h] = (const char *)p.b + (q.group * p.b_group + (column + (h ? p.J : 0)) * p.b_j) * ES + part;
#pragma unroll
    for (int t = 0; t < RT; ++t) a[t] = (const char *)p.a + min(q.i0 + t * 16 + row, q.i1 - 1) * p.a_i * ES + part;
    const uint64_t bytes = (uint64_t)(q.c1 - q.c0) * ES;
    const uint32_t steps = (uint32_t)((bytes + 63) / 64), whole = (uint32_t)(bytes / 64);
    uint32_t s = (uint32_t)((uint64_t)steps * wave / W);
    const uint32_t s1 = (uint32_t)((uint64_t)steps * (wave + 1) / W);
    f32x4 acc[2][RT] = {};
    for (; s + U <= min(s1, whole); s += U) {
        u32x4 vb[U][2], va[U][RT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) vb[u][h] = ((const AnyByteU32x4 *)(b[h] + (uint64_t)(s + u) * 64))->v;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < RT; ++t) va[u][t] = ((const AnyByteU32x4 *)(a[t] + (uint64_t)(s + u) * 64))->v;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) few_multiply<RT, E4M3>(acc[h], vb[u][h], va[u]);
    }
    for (; s < s1; ++s) {
        u32x4 vb[2] = {}, va[RT] = {};
        const uint64_t at = (uint64_t)s * 64 + part;
        if (at < bytes) {
            const uint32_t n = (uint32_t)min(bytes - at, (uint64_t)16) / ES;    // 16 / ES, or the row's last values
            const auto value = [&](const char *from) {
                return n == 16 / ES ? ((const AnyByteU32x4 *)from)->v : few_values<ES>(from, n);
            };
#pragma unroll
            for (int h = 0; h < 2; ++h) vb[h] = value(b[h] + (uint64_t)s * 64);
#pragma unroll
            for (int t = 0; t < RT; ++t) va[t] = value(a[t] + (uint64_t)s * 64);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) few_multiply<RT, E4M3>(acc[h], vb[h], va);
    }
    // the accumulators hold row lane % 16, columns 4 (lane / 16) + r
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t)
            *(f32x4 *)(sums + ((h * W + wave) * (RT * 16) + t * 16 + row) * 20 + (lane >> 4) * 4) = acc[h][t];
    __syncthreads();
    switch (p.act) {
        case EC_ACT_GELU: few_gated_finish<RT, EC_ACT_GELU>(p, q, sums, W); break;
        case EC_ACT_SILU: few_gated_finish<RT, EC_ACT_SILU>(p, q, sums, W); break;
        case EC_ACT_RELU: few_gated_finish<RT, EC_ACT_RELU>(p, q, sums, W); break;
        default: few_gated_finish<RT, EC_ACT_NONE>(p, q, sums, W);
    }
}

template <int RT, bool E4M3>
void launch_few(const ProductArgs &a, const Plan &q, hipStream_t s) {
    if (q.waves == 4)
        few_gated_kernel<RT, 4, E4M3><<<(uint32_t)q.blocks, 256, 0, s>>>(a);
    else
        few_gated_kernel<RT, 8, E4M3><<<(uint32_t)q.blocks, 512, 0, s>>>(a);
}

template <class T>
void launch_tiles(const ProductArgs &a, const Plan &q, hipStream_t s) {
    if (a.dtype == EC_E4M3)
        product_kernel<T, kOpGated, true, false><<<(uint32_t)q.blocks, T::THREADS, 0, s>>>(a);
    else
        product_kernel<T, kOpGated, false, false><<<(uint32_t)q.blocks, T::THREADS, 0, s>>>(a);
    if (q.splits > 1) join_gated_kernel<T><<<q.tiles_i * q.tiles_j * T::NI, T::THREADS, 0, s>>>(a);
}

// ------------------------------------------------------------- backward pass
//
// dz = [dy rest act'(gate), dy act(gate)], rounded to bf16 for the matrix units
// of the products that follow, and the sums of its rows before the rounding.
// A workgroup takes 128 columns of both halves in one part of a group's rows,
// 16 threads of eight columns by 16 rows.  Bound by HBM: 10 bytes a value of
// dy, one pass over each.
constexpr uint32_t kGradCols = 128;

template <int ACT, bool SUM>
__global__ __launch_bounds__(256) void gated_grad_kernel(GatedGradArgs p, float *out, uint32_t parts) {
    __shared__ float sh[SUM ? 16 : 1][2][kGradCols + 4];
    const uint32_t g = blockIdx.y, part = blockIdx.z;
    uint32_t lo = 0, hi = p.m;
    if (p.groups) {
        if (blockIdx.x == 0 && g == 0 && part == 0 && threadIdx.x < 64) check_offsets(p.offsets, p.groups, p.m, p.status);
        group_range(p.offsets, p.m, g, &lo, &hi);
    }
    const uint64_t len = hi - lo;
    hi = lo + (uint32_t)(len * (part + 1) / parts);
    lo += (uint32_t)(len * part / parts);
    const uint32_t x = (threadIdx.x & 15) * 8, y = threadIdx.x >> 4, n = blockIdx.x * kGradCols + x;
    const uint32_t left = p.n > n ? p.n - n : 0;
    float s[2][8] = {};
    if (left) {
        const auto row = [&](uint32_t i, const float *dy, float *gate, float *rest) {
            float a[8], b[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                a[q] = dy[q] * rest[q] * act_slope<ACT>(gate[q]);
                b[q] = dy[q] * act_value<ACT>(gate[q]);
                if constexpr (SUM) {
                    s[0][q] += a[q];
                    s[1][q] += b[q];
                }
            }
            store8(p.dz, EC_BF16, i * p.pitch + n, left, a);
            store8(p.dz, EC_BF16, i * p.pitch + p.n + n, left, b);
            // the row's zeros, at most seven
            if (left <= 8)
                for (uint64_t c = 2 * (uint64_t)p.n; c < p.pitch; ++c) p.dz[i * p.pitch + c] = 0;
        };
        uint32_t i = lo + y;
        for (; i + 16 < hi; i += 32) {      // two rows on the way at a time
            float dy[2][8], gate[2][8], rest[2][8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint64_t r = i + 16 * k;
                load8_bf16(p.dy, r * p.dy_stride + n, left, dy[k]);
                load8_bf16(p.preact, r * p.preact_stride + n, left, gate[k]);
                load8_bf16(p.preact, r * p.preact_stride + p.n + n, left, rest[k]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) row(i + 16 * k, dy[k], gate[k], rest[k]);
        }
        if (i < hi) {
            float dy[8], gate[8], rest[8];
            load8_bf16(p.dy, (uint64_t)i * p.dy_stride + n, left, dy);
            load8_bf16(p.preact, (uint64_t)i * p.preact_stride + n, left, gate);
            load8_bf16(p.preact, (uint64_t)i * p.preact_stride + p.n + n, left, rest);
            row(i, dy, gate, rest);
        }
    }
    if constexpr (SUM) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 8; ++q) sh[y][h][x + q] = s[h][q];
        __syncthreads();
        const uint32_t h = threadIdx.x / kGradCols, c = threadIdx.x % kGradCols, col = blockIdx.x * kGradCols + c;
        if (col >= p.n) return;
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) t += sh[k][h][c];
        out[((uint64_t)part * gridDim.y + g) * 2 * p.n + (uint64_t)h * p.n + col] = t;
    }
}

template <int ACT>
void launch_grad(const GatedGradArgs &a, uint32_t parts, hipStream_t s) {
    const dim3 grid((uint32_t)ceil_div(a.n, kGradCols), a.groups ? a.groups : 1, parts);
    if (a.db)
        gated_grad_kernel<ACT, true><<<grid, 256, 0, s>>>(a, parts > 1 ? a.partial : a.db, parts);
    else
        gated_grad_kernel<ACT, false><<<grid, 256, 0, s>>>(a, nullptr, parts);
}

}  // namespace

hipError_t launch_gated(ProductArgs a, void *workspace, hipStream_t s) {
    if (!a.I || !a.J) return launch_check_offsets(a.offsets, a.groups, a.I, a.status, s);
    const Plan q = make_plan(a);
    if (q.none) return hipErrorInvalidValue;
    const hipError_t e = place_product(a, q, workspace, s);
    if (e != hipSuccess) return e;
    switch (q.shape) {
        case kHuge: launch_tiles<Huge>(a, q, s); break;
        case kEven: launch_tiles<Even>(a, q, s); break;
        case kSmall: launch_tiles<Small>(a, q, s); break;
        default:
            if (a.dtype == EC_E4M3)
                q.row_tiles == 1 ? launch_few<1, true>(a, q, s) : launch_few<2, true>(a, q, s);
            else
                q.row_tiles == 1 ? launch_few<1, false>(a, q, s) : launch_few<2, false>(a, q, s);
    }
    return hipGetLastError();
}

// Parts of the rows: enough workgroups for the card, each with 32 rows or more (of a group, on average).
uint32_t gated_grad_parts(const GatedGradArgs &a) {
    const uint64_t groups = a.groups ? a.groups : 1, blocks = ceil_div(a.n, kGradCols) * groups;
    uint64_t parts = ceil_div(2048, blocks ? blocks : 1);
    const uint64_t most = ceil_div(a.m, groups * 32);
    if (parts > most) parts = most;
    return (uint32_t)(parts < 1 ? 1 : parts);
}

hipError_t launch_gated_grad(const GatedGradArgs &a, hipStream_t s) {
    if (!a.n) return launch_check_offsets(a.offsets, a.groups, a.m, a.status, s);
    const uint32_t parts = gated_grad_parts(a);
    if (!launchable(ceil_div(a.n, kGradCols), 256)) return hipErrorInvalidValue;
    switch (a.act) {
        case EC_ACT_GELU: launch_grad<EC_ACT_GELU>(a, parts, s); break;
        case EC_ACT_SILU: launch_grad<EC_ACT_SILU>(a, parts, s); break;
        case EC_ACT_RELU: launch_grad<EC_ACT_RELU>(a, parts, s); break;
        default: launch_grad<EC_ACT_NONE>(a, parts, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.db || parts == 1) return e;
    return launch_column_join(a.partial, a.db, (uint64_t)(a.groups ? a.groups : 1) * 2 * a.n, parts, s);
}

}  // namespace ec
