// The gated feed-forward block: act(x gate^T) * (x rest^T) in one product,
// dense and by expert, and the backward pass up to the products.
#include "product_kernel.h"

namespace ec {
namespace {

// ------------------------------------------------------------------ few rows
//
// As few_rows_kernel, with the 16 columns' rows of the gate and of the factor
// beside it.  A wave takes both, or (SPLIT) half of the waves one and half the
// other: then a lane has eight loads of one stretch of memory on the way and
// not four of each of two.  By 2 x 16384 x 2048 bf16 weights, split over eight
// waves and not (us): one row 31.3 and 33.9, four 32.7 and 35.0; one by 2 x 8192
// x 8192 70 and 78.  The rule's borders, split and not:
// rows: eight by 2 x 16384 x 2048 34.4 and 35.4, x 1024 16.6 and 15.2; 16 rows
// x 2048 39.6 and 37.6, 17 46 and 42, where the loads of A weigh more; 64 rows over
// 32 experts of 2 x 1024 x 2048 in e4m3 34 and 28.8;
// workgroups: one row by 2 x 4096 x 8192 (256 of them) 38.5 and 32.9, 2 x 6144 x
// 8192 (384) 56.6 and 53.9, 2 x 8192 x 2048 (512) 14.9 and 15.7;
// bytes of a row, of which a wave has a quarter: one row by 2 x 16384 e4m3 rows
// of 2048 18.0 and 15.7, 4096 32.6 and 32.4, 8192 63 and 66; by 2 x 28672, 1024
// 17.4 and 14.9, 2048 29.5 and 28.8, 4096 51.0 and 52.7.  bf16 rows of 2048 bytes
// gain (2 x 28672: 28.5 and 29.5): they have half the conversions.
constexpr uint32_t kSplitBlocks = 512, kSplitRows = 4, kSplitLength = 4096;     // kSplitLength: of e4m3 rows

template <int RT>
struct FewGated {
    static constexpr int TI = RT * 16, TJ = 32;         // TJ: rows of B, for 16 columns
};

template <int RT, int ACT>
__device__ __forceinline__ void few_gated_finish(const ProductArgs &p, const Place &q, const float *sums, uint32_t parts) {
    const uint32_t t = threadIdx.x, i = q.i0 + (t >> 1), j = q.j0 + (t & 1) * 8;
    if (t >= RT * 32 || i >= q.i1) return;
    const GatedColumns c = load_gated_columns(p, q.group, j);
    const float xs = p.x_scale ? p.x_scale[p.x_scales > 1 ? i : 0] : 1.0f, os = p.out_scale ? *p.out_scale : 1.0f;
    float gate[8] = {}, rest[8] = {};
    few_sums<RT>(sums, parts, gate);
    few_sums<RT>(sums + parts * RT * 16 * 20, parts, rest);
    finish8_gated<ACT>(p, i, j, gate, rest, c, xs, os, q.zero);
}

template <int RT, int W, bool E4M3, bool SPLIT>
__global__ __launch_bounds__(W * 64) void few_gated_kernel(ProductArgs p) {
    // halves a wave takes, parts of the contraction, steps whose loads are on the way
    constexpr int ES = E4M3 ? 1 : 2, H = SPLIT ? 1 : 2, P = SPLIT ? W / 2 : W, U = 8 / H;
    using T = FewGated<RT>;
    __shared__ __attribute__((aligned(16))) float sums[2 * P * RT * 16 * 20];   // [half][part][row][16 columns and a gap]
    if (p.groups && blockIdx.x == 0 && threadIdx.x < 64) check_offsets(p.offsets, p.groups, p.I, p.status);
    const Place q = find_place<T, kOpGated>(p, blockIdx.x);
    if (q.none) return;
    const uint32_t lane = threadIdx.x & 63, row = lane & 15, chunk = (lane >> 4) * 16;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t half = wave / P, part = wave % P;
    // rows and columns that do not exist repeat the last one: their sums are not stored
    const uint64_t column = min(q.j0 + row, p.J - 1) + (uint64_t)half * p.J;
    const char *b[H], *a[RT];
#pragma unroll
    for (int h = 0; h < H; ++h)
        b[h] = (const char *)p.b + (q.group * p.b_group + (column + (uint64_t)h * p.J) * p.b_j) * ES + chunk;
#pragma unroll
    for (int t = 0; t < RT; ++t) a[t] = (const char *)p.a + min(q.i0 + t * 16 + row, q.i1 - 1) * p.a_i * ES + chunk;
    const uint64_t bytes = (uint64_t)(q.c1 - q.c0) * ES;
    const uint32_t steps = (uint32_t)((bytes + 63) / 64), whole = (uint32_t)(bytes / 64);
    uint32_t s = (uint32_t)((uint64_t)steps * part / P);
    const uint32_t s1 = (uint32_t)((uint64_t)steps * (part + 1) / P);
    f32x4 acc[H][RT] = {};
    for (; s + U <= min(s1, whole); s += U) {
        u32x4 vb[U][H], va[U][RT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < H; ++h) vb[u][h] = ((const AnyByteU32x4 *)(b[h] + (uint64_t)(s + u) * 64))->v;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < RT; ++t) va[u][t] = ((const AnyByteU32x4 *)(a[t] + (uint64_t)(s + u) * 64))->v;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < H; ++h) few_multiply<RT, E4M3>(acc[h], vb[u][h], va[u]);
    }
    for (; s < s1; ++s) {
        u32x4 vb[H] = {}, va[RT] = {};
        const uint64_t at = (uint64_t)s * 64 + chunk;
        if (at < bytes) {
            const uint32_t n = (uint32_t)min(bytes - at, (uint64_t)16) / ES;    // 16 / ES, or the row's last values
            const auto value = [&](const char *from) {
                return n == 16 / ES ? ((const AnyByteU32x4 *)from)->v : few_values<ES>(from, n);
            };
#pragma unroll
            for (int h = 0; h < H; ++h) vb[h] = value(b[h] + (uint64_t)s * 64);
#pragma unroll
            for (int t = 0; t < RT; ++t) va[t] = value(a[t] + (uint64_t)s * 64);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) few_multiply<RT, E4M3>(acc[h], vb[h], va);
    }
    // the accumulators hold row lane % 16, columns 4 (lane / 16) + r
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t)
            *(f32x4 *)(sums + (((half + h) * P + part) * (RT * 16) + t * 16 + row) * 20 + (lane >> 4) * 4) = acc[h][t];
    __syncthreads();
    switch (p.act) {
        case EC_ACT_GELU: few_gated_finish<RT, EC_ACT_GELU>(p, q, sums, P); break;
        case EC_ACT_SILU: few_gated_finish<RT, EC_ACT_SILU>(p, q, sums, P); break;
        case EC_ACT_RELU: few_gated_finish<RT, EC_ACT_RELU>(p, q, sums, P); break;
        default: few_gated_finish<RT, EC_ACT_NONE>(p, q, sums, P);
    }
}

template <bool E4M3>
void launch_few(const ProductArgs &a, const Plan &q, hipStream_t s) {
    const uint32_t n = (uint32_t)q.blocks;
    if (q.row_tiles == 2)
        q.waves == 4 ? few_gated_kernel<2, 4, E4M3, false><<<n, 256, 0, s>>>(a)
                     : few_gated_kernel<2, 8, E4M3, false><<<n, 512, 0, s>>>(a);
    else if (!a.groups && a.I <= kSplitRows && n >= kSplitBlocks && (!E4M3 || a.C >= kSplitLength) &&
             launchable(n, 512))            // the plan counted 256
        few_gated_kernel<1, 8, E4M3, true><<<n, 512, 0, s>>>(a);
    else
        q.waves == 4 ? few_gated_kernel<1, 4, E4M3, false><<<n, 256, 0, s>>>(a)
                     : few_gated_kernel<1, 8, E4M3, false><<<n, 512, 0, s>>>(a);
}

// A kernel for each activation: all of them in one are more than its registers bear.
void launch_wide_act(const ProductArgs &a, const Plan &q, hipStream_t s) {
    switch (a.act) {
        case EC_ACT_GELU: launch_wide<kOpGated, EC_ACT_GELU>(a, q, s); break;
        case EC_ACT_SILU: launch_wide<kOpGated, EC_ACT_SILU>(a, q, s); break;
        case EC_ACT_RELU: launch_wide<kOpGated, EC_ACT_RELU>(a, q, s); break;
        default: launch_wide<kOpGated, EC_ACT_NONE>(a, q, s);
    }
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
// A workgroup takes 128 columns of both halves in a slab of rows, 16 threads of
// eight columns by 16 rows; by group it takes the runs of groups in its slab
// one after the other.  The sums of slab s's run of group g are part s + g,
// which no other run has, and a group's parts are consecutive.  (Slabs and not
// parts of each group, since groups are uneven: 8192 rows by 1024 columns in 16
// groups 21 us, 35 with equal parts of every group.)  Bound by HBM: 10 bytes a
// value of dy, one pass over each; 2048 x 8192 with GELU 36 us (4.6 TB/s).
constexpr uint32_t kGradCols = 128;

struct Sums {
    float s[2][8];
};

template <int ACT, bool SUM>
__device__ __forceinline__ void grad_row(const GatedGradArgs &p, uint64_t i, uint32_t n, uint32_t left, const float *dy,
                                         const float *gate, const float *rest, Sums &sums) {
    float a[8], b[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        a[q] = dy[q] * rest[q] * act_slope<ACT>(gate[q]);
        b[q] = dy[q] * act_value<ACT>(gate[q]);
        if constexpr (SUM) {
            sums.s[0][q] += a[q];
            sums.s[1][q] += b[q];
        }
    }
    store8(p.dz, EC_BF16, i * p.pitch + n, left, a);
    store8(p.dz, EC_BF16, i * p.pitch + p.n + n, left, b);
    if (left <= 8)                          // the row's zeros, at most seven
        for (uint64_t c = 2 * (uint64_t)p.n; c < p.pitch; ++c) p.dz[i * p.pitch + c] = 0;
}

// Rows [lo, hi) of one group, their sums to out.
template <int ACT, bool SUM>
__device__ __forceinline__ void grad_run(const GatedGradArgs &p, uint32_t column, uint32_t lo, uint32_t hi, float *out) {
    __shared__ float sh[SUM ? 16 : 1][2][kGradCols + 4];
    const uint32_t x = (threadIdx.x & 15) * 8, y = threadIdx.x >> 4, n = column + x;
    const uint32_t left = p.n > n ? p.n - n : 0;
    Sums sums = {};
    if (left) {
        uint32_t i = lo + y;
        for (; (uint64_t)i + 16 < hi; i += 32) {        // two rows on the way at a time
            float dy[2][8], gate[2][8], rest[2][8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint64_t r = i + 16 * k;
                load8_bf16(p.dy, r * p.dy_stride + n, left, dy[k]);
                load8_bf16(p.preact, r * p.preact_stride + n, left, gate[k]);
                load8_bf16(p.preact, r * p.preact_stride + p.n + n, left, rest[k]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) grad_row<ACT, SUM>(p, i + 16 * k, n, left, dy[k], gate[k], rest[k], sums);
        }
        if (i < hi) {
            float dy[8], gate[8], rest[8];
            load8_bf16(p.dy, (uint64_t)i * p.dy_stride + n, left, dy);
            load8_bf16(p.preact, (uint64_t)i * p.preact_stride + n, left, gate);
            load8_bf16(p.preact, (uint64_t)i * p.preact_stride + p.n + n, left, rest);
            grad_row<ACT, SUM>(p, i, n, left, dy, gate, rest, sums);
        }
    }
    if constexpr (SUM) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 8; ++q) sh[y][h][x + q] = sums.s[h][q];
        __syncthreads();
        const uint32_t h = threadIdx.x / kGradCols, c = threadIdx.x % kGradCols;
        if (column + c < p.n) {
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < 16; ++k) t += sh[k][h][c];
            out[(uint64_t)h * p.n + column + c] = t;
        }
        __syncthreads();                    // before the next run's
    }
}

template <int ACT, bool SUM>
__global__ __launch_bounds__(256) void gated_grad_kernel(GatedGradArgs p, uint32_t column_blocks) {
    const uint32_t slab = blockIdx.x / column_blocks, column = (blockIdx.x - slab * column_blocks) * kGradCols;
    const uint32_t lo = slab * p.slab, hi = (uint32_t)min((uint64_t)lo + p.slab, (uint64_t)p.m);
    if (!p.groups) {
        grad_run<ACT, SUM>(p, column, lo, hi, SUM ? p.partial + (uint64_t)slab * 2 * p.n : nullptr);
        return;
    }
    if (blockIdx.x == 0 && threadIdx.x < 64) check_offsets(p.offsets, p.groups, p.m, p.status);
    // range r holds the rows of group r - 1 (the first and the last those of none)
    uint32_t edge = 0, start, end, n, sum;
    for (uint32_t base = 0; base < p.groups + 2 && edge < hi; base += 64) {
        scan_ranges(p.offsets, p.groups, p.m, p.m, base, edge, 0, &start, &end, &n, &sum);
        const uint32_t r = base + (threadIdx.x & 63);
        uint64_t mask = __ballot(r >= 1 && r <= p.groups && start < hi && end > lo && end > start);
        while (mask) {
            const int l = __ffsll((unsigned long long)mask) - 1;
            mask &= mask - 1;
            const uint32_t a = max(lo, (uint32_t)__builtin_amdgcn_readlane((int)start, l));
            const uint32_t b = min(hi, (uint32_t)__builtin_amdgcn_readlane((int)end, l)), g = base + l - 1;
            grad_run<ACT, SUM>(p, column, a, b, SUM ? p.partial + ((uint64_t)slab + g) * 2 * p.n : nullptr);
        }
        edge = (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
    }
}

// Adds a group's parts in a fixed order: 16 columns by 16 threads that take
// every 16th part each.
__global__ __launch_bounds__(256) void gated_sum_kernel(GatedGradArgs p) {
    __shared__ float sh[16][17];
    const uint32_t x = threadIdx.x & 15, y = threadIdx.x >> 4, g = blockIdx.y;
    const uint64_t c = (uint64_t)blockIdx.x * 16 + x, n = 2 * (uint64_t)p.n;
    uint32_t lo = 0, hi = p.m;
    if (p.groups) group_range(p.offsets, p.m, g, &lo, &hi);
    float s = 0.0f;
    if (c < n && lo < hi) {
        const uint64_t last = (hi - 1) / p.slab + (uint64_t)g;
#pragma unroll 4                            // loads of four parts on the way
        for (uint64_t q = lo / p.slab + (uint64_t)g + y; q <= last; q += 16) s += p.partial[q * n + c];
    }
    sh[y][x] = s;
    __syncthreads();
    if (y || c >= n) return;
    for (int k = 1; k < 16; ++k) s += sh[k][x];
    p.db[g * n + c] = s;
}

template <int ACT>
void launch_grad(const GatedGradArgs &a, uint32_t column_blocks, uint32_t blocks, hipStream_t s) {
    if (a.db)
        gated_grad_kernel<ACT, true><<<blocks, 256, 0, s>>>(a, column_blocks);
    else
        gated_grad_kernel<ACT, false><<<blocks, 256, 0, s>>>(a, column_blocks);
}

}  // namespace

hipError_t launch_gated(ProductArgs a, void *workspace, hipStream_t s) {
    if (!a.I || !a.J) return launch_check_offsets(a.offsets, a.groups, a.I, a.status, s);
    const Plan q = make_plan(a);
    if (q.none) return hipErrorInvalidValue;
    const hipError_t e = place_product(a, q, workspace, s);
    if (e != hipSuccess) return e;
    switch (q.shape) {
        case kHuge: runs_wide(a, q) ? launch_wide_act(a, q, s) : launch_tiles<Huge>(a, q, s); break;
        case kEven: launch_tiles<Even>(a, q, s); break;
        case kSmall: launch_tiles<Small>(a, q, s); break;
        case kTall: launch_tiles<Tall>(a, q, s); break;
        default:
            a.dtype == EC_E4M3 ? launch_few<true>(a, q, s) : launch_few<false>(a, q, s);
    }
    return hipGetLastError();
}

// Rows of a slab: 64, fewer where workgroups would not fill the card, more
// where parts would be over 1024 or workgroups too many for a launch.
uint32_t gated_grad_slab(uint32_t m, uint32_t n) {
    const uint64_t columns = ceil_div(n, kGradCols);
    uint32_t slab = 64;
    while (slab > 16 && columns * ceil_div(m, slab) < 1024) slab /= 2;
    while (ceil_div(m, slab) > 1024 || (slab < m && !launchable(columns * ceil_div(m, slab), 256))) slab *= 2;
    return slab;
}

bool gated_grad_fits(const GatedGradArgs &a) {
    return launchable(ceil_div(a.n, kGradCols) * ceil_div(a.m, a.slab), 256) &&
           (!a.db || launchable(ceil_div(2 * (uint64_t)a.n, 16), 256));
}

uint64_t gated_grad_workspace(const GatedGradArgs &a) {
    return a.db ? (ceil_div(a.m, a.slab) + a.groups) * 2 * a.n * 4 : 0;
}

hipError_t launch_gated_grad(const GatedGradArgs &a, hipStream_t s) {
    if (!a.n) return launch_check_offsets(a.offsets, a.groups, a.m, a.status, s);
    const uint64_t columns = ceil_div(a.n, kGradCols), blocks = columns * ceil_div(a.m, a.slab);
    const dim3 sums((uint32_t)ceil_div(2 * (uint64_t)a.n, 16), a.groups ? a.groups : 1);
    if (!gated_grad_fits(a)) return hipErrorInvalidValue;
    if (blocks) {
        switch (a.act) {
            case EC_ACT_GELU: launch_grad<EC_ACT_GELU>(a, (uint32_t)columns, (uint32_t)blocks, s); break;
            case EC_ACT_SILU: launch_grad<EC_ACT_SILU>(a, (uint32_t)columns, (uint32_t)blocks, s); break;
            case EC_ACT_RELU: launch_grad<EC_ACT_RELU>(a, (uint32_t)columns, (uint32_t)blocks, s); break;
            default: launch_grad<EC_ACT_NONE>(a, (uint32_t)columns, (uint32_t)blocks, s);
        }
    } else {
        const hipError_t e = launch_check_offsets(a.offsets, a.groups, a.m, a.status, s);
        if (e != hipSuccess) return e;
    }
    if (a.db) gated_sum_kernel<<<sums, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace ec
