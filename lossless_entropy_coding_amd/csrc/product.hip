// Matrix products with a fused epilogue, dense and grouped by expert.
#include <string.h>

#include "product_kernel.h"

namespace ec {
namespace {

// ------------------------------------------------------- rows made readable
//
// The products' loads take rows at 16-byte addresses whose contraction is a whole
// number of 16-byte chunks.  Any other factor is copied first: rows padded
// with zeros to 16 bytes, one after the other.
struct RowCopy {
    const void *p;
    uint64_t stride, group_stride, total;  // elements; total: 16-byte chunks of all groups
    uint32_t rows, cols, pitch;            // pitch of the copy's rows, elements
    void *out;
    uint32_t blocks;                       // 0: none
};

// Both factors in one launch: the first a.blocks workgroups copy a's.
template <typename E>
__global__ __launch_bounds__(256) void copy_rows_kernel(RowCopy a, RowCopy b) {
    constexpr uint32_t V = 16 / sizeof(E);
    const bool first = blockIdx.x < a.blocks;
    const RowCopy &k = first ? a : b;
    const uint32_t chunks = k.pitch / V;
    const uint64_t q = (uint64_t)(blockIdx.x - (first ? 0 : a.blocks)) * 256 + threadIdx.x;
    if (q >= k.total) return;
    uint64_t row, g;
    if (k.total >> 32) {
        row = q / chunks;
        g = row / k.rows;
    } else {                                // the same in short divisions
        row = (uint32_t)q / chunks;
        g = (uint32_t)row / k.rows;
    }
    const uint32_t c = (uint32_t)(q - row * chunks) * V;
    const E *in = (const E *)k.p + g * k.group_stride + (row - g * k.rows) * k.stride + c;
    union {
        E e[V];
        u32x4 w;
    } u;
    if (c + V <= k.cols) {
        u.w = ((const AnyByteU32x4 *)in)->v;
    } else {
        u.w = u32x4{0, 0, 0, 0};
#pragma unroll
        for (uint32_t n = 0; n < V; ++n)
            if (c + n < k.cols) u.e[n] = in[n];
    }
    ((u32x4 *)k.out)[q] = u.w;
}

// ---------------------------------------------------------------- column sums
//
// db[n] = sum of dy's rows.  A workgroup takes 128 columns of one part of a
// group's rows, 16 threads of eight columns by 16 rows; where that alone does
// not fill the card the rows are cut into parts, added in their order after.
constexpr uint32_t kSumCols = 128;

__global__ __launch_bounds__(256) void column_sum_kernel(ColumnSumArgs p, float *out, uint32_t parts) {
    __shared__ float sh[16][kSumCols + 4];
    const uint32_t g = blockIdx.y, part = blockIdx.z;
    uint32_t lo = 0, hi = p.m;
    if (p.groups) {
        if (blockIdx.x == 0 && g == 0 && part == 0 && threadIdx.x < 64) check_offsets(p.offsets, p.groups, p.m, p.status);
        group_range(p.offsets, p.m, g, &lo, &hi);
    }
    const uint64_t len = hi - lo;
    hi = lo + (uint32_t)(len * (part + 1) / parts);
    lo += (uint32_t)(len * part / parts);
    const uint32_t x = (threadIdx.x & 15) * 8, y = threadIdx.x >> 4, n = blockIdx.x * kSumCols + x;
    const uint32_t left = p.n > n ? p.n - n : 0;
    float s[8] = {};
    if (left) {
        uint32_t i = lo + y;
        for (; i + 48 < hi; i += 64) {      // four rows on the way at a time
            float v[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k) load8_bf16(p.dy, (uint64_t)(i + 16 * k) * p.dy_stride + n, left, v[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int q = 0; q < 8; ++q) s[q] += v[k][q];
        }
        for (; i < hi; i += 16) {
            float v[8];
            load8_bf16(p.dy, (uint64_t)i * p.dy_stride + n, left, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) s[q] += v[q];
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) sh[y][x + q] = s[q];
    __syncthreads();
    const uint32_t c = blockIdx.x * kSumCols + threadIdx.x;
    if (threadIdx.x >= kSumCols || c >= p.n) return;
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += sh[k][threadIdx.x];
    out[((uint64_t)part * gridDim.y + g) * p.n + c] = t;
}

__global__ __launch_bounds__(256) void column_join_kernel(const float *in, float *db, uint64_t n, uint32_t parts) {
    const uint64_t c = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= n) return;
    float s = 0.0f;
#pragma unroll 8                            // loads of eight parts on the way
    for (uint32_t q = 0; q < parts; ++q) s += in[q * n + c];
    db[c] = s;
}

// For a grouped product that has nothing to compute.
__global__ __launch_bounds__(64) void check_offsets_kernel(const int32_t *offsets, uint32_t groups, uint32_t m,
                                                           uint32_t *status) {
    check_offsets(offsets, groups, m, status);
}

// ---------------------------------------------------------------------- plan

// What a plan's time is made of, measured on whole runs (us): a stage of one
// workgroup alone on its CU, a stage per workgroup where every CU is full, and
// what a workgroup costs besides its stages; bf16 and e4m3.  The full rates
// are 1.25, 0.87, 0.51 and 1.17 PFLOP/s in bf16.  The last is for 129 to 256
// rows in a row of as many workgroups as CUs; whole calls with it and without
// (us): the loss of M rows x 32768 x 2048, M = 129 50.9 and 53.7, 160 52.4 and
// 55.4, 256 57.6 and 59.7, 320 67.1 and 66.7; gated M x 2 x 16384 x 2048 48.8 and
// 58.5, 50.0 and 59.8, 57.5 and 64.7, 70.5 and 70.2.  ec_linear_op's products do
// not have it: what they ran in before keeps its times.
struct ShapeCost {
    uint32_t TI, TJ, threads, per_cu;
    float alone[2], full[2], fixed;
};
constexpr ShapeCost kCost[] = {{256, 256, Huge::THREADS, 1, {0.55f, 1.1f}, {0.86f, 1.5f}, 10.0f},
                               {128, 128, Even::THREADS, 2, {0.25f, 0.43f}, {0.31f, 0.45f}, 5.0f},
                               {64, 64, Small::THREADS, 3, {0.17f, 0.28f}, {0.133f, 0.18f}, 6.0f},
                               {256, 128, Tall::THREADS, 1, {0.33f, 0.7f}, {0.46f, 0.85f}, 8.0f}};
constexpr uint64_t kCUs = 256;

bool aligned(const void *p, uint64_t stride, uint64_t group, uint64_t cols, uint32_t es, bool outer) {
    return !((((uintptr_t)p | (stride * es) | (group * es)) & 15) || (!outer && (cols * es & 15)));
}

// Whether the offsets of a stage's rows fit 31 bits: T rows of a tile where
// they are contiguous along the contraction, or the stage's rows of it.
bool reachable(uint64_t T, uint64_t stride, uint32_t es, bool outer) {
    return (outer ? kStageBytes / es : T) * stride * es + 65536 < (1ull << 31);
}

}  // namespace

Plan make_plan(const ProductArgs &a) {
    Plan q;
    memset(&q, 0, sizeof(q));
    const uint32_t es = a.dtype == EC_E4M3 ? 1 : 2;
    const bool outer_a = contracts_a_rows(a.op), outer_b = contracts_b_rows(a.op);
    const bool ragged = a.groups && !outer_a;
    const uint64_t groups = a.groups ? a.groups : 1;
    const uint64_t J = a.op == kOpGated ? 2 * (uint64_t)a.J : a.J;     // columns that tiles hold
    const bool joins = !a.groups && a.op != kOpRowStats && a.op != kOpLogitGrad;
    q.splits = 1;
    // Row tiles of a ragged product: at most one begun a group besides the whole ones.
    const auto most_tiles = [&](uint64_t tile) {
        return ragged ? a.I / tile + (a.I < groups + 2 ? a.I : groups + 2) : ceil_div(a.I, tile);
    };
    const auto few = [&](uint32_t row_tiles) {          // reads rows at any address, of any length
        q.shape = kFew;
        q.tiles_j = (uint32_t)ceil_div(a.J, 16);
        q.row_tiles = row_tiles;
        q.tiles_i = (uint32_t)most_tiles(16 * q.row_tiles);
        // Waves that share a contraction: with 1024 tiles four are enough
        // (16.4 us; 16.2 with eight), with 128 eight are better (13.4, 16.1).
        q.waves = (ragged ? groups : q.tiles_i) * q.tiles_j >= 2 * kCUs ? 4 : 8;
        q.blocks = (uint64_t)q.tiles_i * q.tiles_j;
        return launchable(q.blocks, q.waves * 64);
    };
    // Few rows a group, forward: one row by 16384 x 2048 weights takes 13.5 us
    // so, 20 us in tiles with a split contraction and its join.  17 to 32 rows:
    // one tile of 32 reads the weights once, but two of 16 use twice as many
    // CUs, so that the tiles of 16 columns must be enough for them all (17 rows:
    // 16384 columns 24 against 32 us, 2048 columns of 16384 e4m3 values 22
    // against 18), twice over by group, where rows are uneven (20 rows by 1024 x
    // 2048 a group, 32 groups: 50 us against 64, e4m3 22 against 38; uneven 61
    // against 58, e4m3 30 against 34; four uneven groups 13.7 against 12.3).
    // The average decides, since the host does not know the offsets: 1024 rows
    // of which 962 are in one of 32 groups take 90 us so and 45 in tiles.
    const uint64_t rows = ragged ? ceil_div(a.I, groups) : a.I;
    // The loss reads its rows again for every 16 entries of the vocabulary, and
    // with many of those, more than eight rows weigh more than the tiles' unused
    // ones.  Maxima and sums so and in tiles (us): 8 rows by 32768 x 2048 40.3 and
    // 42.2, 12 43.3 and 41.8, 16 47.0 and 42.4, 32 61.4 and 45.4; 32 by 131072 x 2048
    // 217 and 140; 16 by 16384 x 4096 45.8 and 41.7, by 8192 x 4096 23.7 and 34.3.
    // With gradients 32 by 32768 x 2048 184 and 152, by 8192 x 2048 64.7 and 72.9.
    const bool logits = a.op == kOpRowStats || a.op == kOpLogitGrad;
    const bool again = logits && rows > 8 && ceil_div(a.J, 16) >= 4 * kCUs;
    if (!outer_b && rows <= 32 && !again) {
        const bool fill = ceil_div(a.J, 16) * groups >= (ragged ? 2 : 1) * kCUs;
        if (few(rows > 16 && fill ? 2 : 1)) return q;
    }
    // The tiles and the number of splits with the least time, of the shapes
    // whose tiles reach their rows: where these lie, or else in a copy.
    const uint64_t a_rows = outer_a ? a.C : a.I, a_cols = outer_a ? a.I : a.C, a_stride = outer_a ? a.a_c : a.a_i;
    const uint64_t b_rows = outer_b ? a.C : J, b_cols = outer_b ? J : a.C, b_stride = outer_b ? a.b_c : a.b_j;
    const uint64_t a_pitch = round_up(a_cols, 16 / es), b_pitch = round_up(b_cols, 16 / es);
    const bool a_aligned = aligned(a.a, a_stride, 0, a.a_padded ? a_pitch : a_cols, es, outer_a);
    const bool b_aligned = aligned(a.b, b_stride, outer_a ? 0 : a.b_group, a.b_padded ? b_pitch : b_cols, es, outer_b);
    const uint64_t a_bytes = round_up(a_rows * a_pitch * es, 256);
    const uint64_t b_bytes = round_up((outer_a ? 1 : groups) * b_rows * b_pitch * es, 256);
    const uint64_t stages = ceil_div((outer_a ? ceil_div(a.C, groups) : (uint64_t)a.C) * es, kStageBytes);
    float best = 0.0f;
    for (uint32_t id = kHuge; id <= (a.op >= kOpGated ? kTall : kSmall); ++id) {
        const ShapeCost &c = kCost[id];
        float copies = 0.0f;                            // what this shape has copied and another need not, at 4 TB/s
        bool copy_a = false, copy_b = false;
        if (a.C) {
            copy_a = !a_aligned || !reachable(c.TI, a_stride, es, outer_a);
            copy_b = !b_aligned || !reachable(c.TJ, b_stride, es, outer_b);
            if ((copy_a && !reachable(c.TI, a_pitch, es, outer_a)) || (copy_b && !reachable(c.TJ, b_pitch, es, outer_b)))
                continue;
            if (!launchable(((copy_a ? a_bytes : 0) + (copy_b ? b_bytes : 0)) / 16 + 512, 1)) continue;
            copies = ((copy_a && a_aligned ? a_bytes : 0) + (copy_b && b_aligned ? b_bytes : 0)) * 0.5e-6f;
        }
        const uint64_t ti = ragged ? a.I / c.TI + (groups + 1) / 2 : ceil_div(a.I, c.TI);
        const uint64_t tiles = ti * ceil_div(J, c.TJ) * (outer_a ? groups : 1);
        if (!launchable(most_tiles(c.TI) * ceil_div(J, c.TJ) * (outer_a ? groups : 1), c.threads)) continue;
        for (uint32_t n = 1; n == 1 || (joins && n <= 32 && stages / n >= 8 && launchable(tiles * n, c.threads));
             n *= 2) {
            const uint64_t rounds = ceil_div(tiles * n, kCUs * c.per_cu), each = ceil_div(stages, n);
            const float alone = rounds * c.alone[es == 1], full = ceil_div(tiles * n, kCUs) * c.full[es == 1];
            float t = (alone > full ? alone : full) * each + c.fixed * rounds + copies;
            if (n > 1) t += 4.0f + (float)n * a.I * J * 1e-6f;      // the partial sums' bytes at 4 TB/s
            if (!best || t < best) {
                best = t;
                q.shape = id;
                q.splits = n;
                q.a_pitch = copy_a ? (uint32_t)a_pitch : 0;
                q.b_pitch = copy_b ? (uint32_t)b_pitch : 0;
            }
        }
    }
    if (!best) {                                        // rows of more than 32 MiB
        q.none = outer_b || !few(2);
        return q;
    }
    uint64_t at = q.a_pitch ? a_bytes : 0;
    q.b_at = at;
    if (q.b_pitch) at += b_bytes;
    const uint32_t TI = kCost[q.shape].TI, TJ = kCost[q.shape].TJ;
    const uint64_t ti = most_tiles(TI);
    q.tiles_i = (uint32_t)ti;
    q.tiles_j = (uint32_t)ceil_div(J, TJ);
    q.blocks = ti * q.tiles_j * (outer_a ? groups : 1);
    q.partial_at = at;
    if (q.splits > 1) {
        at += q.splits * q.blocks * TI * TJ * 4;
        q.blocks *= q.splits;
    }
    q.bytes = at;
    return q;
}

namespace {

template <class T, int OP, bool E4M3, bool SUM = false>
void launch_shape(const ProductArgs &a, const Plan &q, hipStream_t s) {
    product_kernel<T, OP, E4M3, SUM><<<(uint32_t)q.blocks, T::THREADS, 0, s>>>(a);
    if (q.splits > 1) join_kernel<T, OP><<<q.tiles_i * q.tiles_j * T::NI * T::NJ, T::THREADS, 0, s>>>(a);
}

template <class T>
void launch_op(const ProductArgs &a, const Plan &q, hipStream_t s) {
    const bool wide = T::TI == Wide::TI && a.act == EC_ACT_NONE && !a.db && runs_wide(a, q);
    if (a.op == EC_LINEAR_GRAD_INPUT)
        wide ? launch_wide<EC_LINEAR_GRAD_INPUT, EC_ACT_NONE>(a, q, s) : launch_shape<T, EC_LINEAR_GRAD_INPUT, false>(a, q, s);
    else if (a.op == EC_LINEAR_GRAD_WEIGHT && a.db)
        launch_shape<T, EC_LINEAR_GRAD_WEIGHT, false, true>(a, q, s);
    else if (a.op == EC_LINEAR_GRAD_WEIGHT)
        wide ? launch_wide<EC_LINEAR_GRAD_WEIGHT, EC_ACT_NONE>(a, q, s) : launch_shape<T, EC_LINEAR_GRAD_WEIGHT, false>(a, q, s);
    else if (a.dtype == EC_E4M3)
        launch_shape<T, EC_LINEAR_FORWARD, true>(a, q, s);
    else
        launch_shape<T, EC_LINEAR_FORWARD, false>(a, q, s);
}

template <int RT, bool E4M3>
void launch_few(const ProductArgs &a, const Plan &q, hipStream_t s) {
    const uint32_t n = (uint32_t)q.blocks;
    if (q.waves == 4)
        few_rows_kernel<RT, 4, E4M3><<<n, 256, 0, s>>>(a);
    else
        few_rows_kernel<RT, 8, E4M3><<<n, 512, 0, s>>>(a);
}

RowCopy row_copy(const void *p, uint64_t stride, uint64_t group_stride, uint64_t groups, uint64_t rows, uint64_t cols,
                 uint32_t es, void *out, uint32_t pitch) {
    RowCopy c = {p, stride, group_stride, groups * rows * (pitch * es / 16), (uint32_t)rows, (uint32_t)cols, pitch, out, 0};
    const uint64_t blocks = ceil_div(c.total, 256);
    c.blocks = blocks > 0x7FFFFFFF ? 0xFFFFFFFFu : (uint32_t)blocks;
    return c;
}

}  // namespace

hipError_t place_product(ProductArgs &a, const Plan &q, void *workspace, hipStream_t s) {
    const uint32_t es = a.dtype == EC_E4M3 ? 1 : 2;
    const bool outer_a = contracts_a_rows(a.op), outer_b = contracts_b_rows(a.op);
    const uint64_t J = a.op == kOpGated ? 2 * (uint64_t)a.J : a.J;
    char *ws = (char *)workspace;
    RowCopy ca = {}, cb = {};
    if (q.a_pitch) {
        const uint64_t rows = outer_a ? a.C : a.I, cols = outer_a ? a.I : a.C;
        ca = row_copy(a.a, outer_a ? a.a_c : a.a_i, 0, 1, rows, cols, es, ws + q.a_at, q.a_pitch);
        a.a = ws + q.a_at;
        (outer_a ? a.a_c : a.a_i) = q.a_pitch;
    }
    if (q.b_pitch) {
        const uint64_t rows = outer_b ? a.C : J, cols = outer_b ? J : a.C, groups = !outer_a && a.groups ? a.groups : 1;
        cb = row_copy(a.b, outer_b ? a.b_c : a.b_j, a.b_group, groups, rows, cols, es, ws + q.b_at, q.b_pitch);
        a.b = ws + q.b_at;
        (outer_b ? a.b_c : a.b_j) = q.b_pitch;
        a.b_group = rows * q.b_pitch;
    }
    const uint64_t copies = (uint64_t)ca.blocks + cb.blocks;
    if (!launchable(copies, 256)) return hipErrorInvalidValue;
    if (copies && es == 1)
        copy_rows_kernel<uint8_t><<<(uint32_t)copies, 256, 0, s>>>(ca, cb);
    else if (copies)
        copy_rows_kernel<uint16_t><<<(uint32_t)copies, 256, 0, s>>>(ca, cb);
    a.tiles_i = q.tiles_i;
    a.tiles_j = q.tiles_j;
    a.splits = q.splits;
    a.blocks = (uint32_t)q.blocks;
    a.partial = (float *)(ws + q.partial_at);
    return hipSuccess;
}

hipError_t launch_check_offsets(const int32_t *offsets, uint32_t groups, uint32_t m, uint32_t *status, hipStream_t s) {
    if (!groups || !status) return hipSuccess;
    check_offsets_kernel<<<1, 64, 0, s>>>(offsets, groups, m, status);
    return hipGetLastError();
}

bool product_sums_columns(const ProductArgs &a) {
    // The second launch and its join cost 8 - 10 us, the sums a tenth of the
    // product: up to 1024 rows that is less (see product_kernel).
    return a.op == EC_LINEAR_GRAD_WEIGHT && a.I && a.J && (a.groups || (a.C <= 1024 && make_plan(a).splits == 1));
}

bool product_fits(const ProductArgs &a) { return !a.I || !a.J || !make_plan(a).none; }

bool product_need(const ProductArgs &a, uint64_t *bytes) {
    *bytes = 0;
    if (!a.I || !a.J) return true;
    const Plan q = make_plan(a);
    *bytes = q.bytes;
    return !q.none;
}

uint64_t product_workspace(const ProductArgs &a) {
    if (!a.I || !a.J) return 0;
    return make_plan(a).bytes;
}

hipError_t launch_product(ProductArgs a, void *workspace, hipStream_t s) {
    if (!a.I || !a.J)
        return launch_check_offsets(a.offsets, a.groups, a.op == EC_LINEAR_GRAD_WEIGHT ? a.C : a.I, a.status, s);
    const Plan q = make_plan(a);
    if (q.none) return hipErrorInvalidValue;
    const hipError_t e = place_product(a, q, workspace, s);
    if (e != hipSuccess) return e;
    switch (q.shape) {
        case kHuge: launch_op<Huge>(a, q, s); break;
        case kEven: launch_op<Even>(a, q, s); break;
        case kSmall: launch_op<Small>(a, q, s); break;
        default:
            if (a.dtype == EC_E4M3)
                q.row_tiles == 1 ? launch_few<1, true>(a, q, s) : launch_few<2, true>(a, q, s);
            else
                q.row_tiles == 1 ? launch_few<1, false>(a, q, s) : launch_few<2, false>(a, q, s);
    }
    return hipGetLastError();
}

hipError_t launch_copy_rows(const void *in, uint64_t stride, uint64_t rows, uint64_t cols, uint32_t dtype, void *out,
                            uint64_t pitch, hipStream_t s) {
    const uint32_t es = dtype == EC_E4M3 ? 1 : 2;
    const RowCopy c = row_copy(in, stride, 0, 1, rows, cols, es, out, (uint32_t)pitch), none = {};
    if (!c.total) return hipSuccess;
    if (!launchable(c.blocks, 256)) return hipErrorInvalidValue;
    if (es == 1)
        copy_rows_kernel<uint8_t><<<c.blocks, 256, 0, s>>>(c, none);
    else
        copy_rows_kernel<uint16_t><<<c.blocks, 256, 0, s>>>(c, none);
    return hipGetLastError();
}

static uint32_t column_parts(const ColumnSumArgs &a) {
    const uint64_t groups = a.groups ? a.groups : 1, blocks = ceil_div(a.n, kSumCols) * groups;
    uint64_t parts = ceil_div(1024, blocks), most = ceil_div(a.m, groups * 64);
    if (parts > most) parts = most;
    return (uint32_t)(parts < 1 ? 1 : parts > 32 ? 32 : parts);
}

uint64_t column_sum_workspace(const ColumnSumArgs &a) {
    const uint32_t parts = a.n ? column_parts(a) : 1;
    return parts > 1 ? (uint64_t)parts * (a.groups ? a.groups : 1) * a.n * 4 : 0;
}

hipError_t launch_column_sum(const ColumnSumArgs &a, float *workspace, hipStream_t s) {
    if (!a.n) return launch_check_offsets(a.offsets, a.groups, a.m, a.status, s);
    const uint32_t parts = column_parts(a), groups = a.groups ? a.groups : 1;
    const uint64_t n = (uint64_t)groups * a.n;
    if (!launchable(ceil_div(a.n, kSumCols), 256) || (parts > 1 && !launchable(ceil_div(n, 256), 256)))
        return hipErrorInvalidValue;
    column_sum_kernel<<<dim3((uint32_t)ceil_div(a.n, kSumCols), groups, parts), 256, 0, s>>>(a, parts > 1 ? workspace : a.db,
                                                                                           parts);
    if (parts > 1) column_join_kernel<<<(uint32_t)ceil_div(n, 256), 256, 0, s>>>(workspace, a.db, n, parts);
    return hipGetLastError();
}

}  // namespace ec
