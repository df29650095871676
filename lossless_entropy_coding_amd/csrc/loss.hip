// Softmax cross entropy over a large vocabulary, from the products of the rows
// with the vocabulary's weights; the logits are never kept.
//
//   l = x w^T,  lse = log sum_v exp(l_v),  loss = lse - l_target
//   G = (exp(l - lse) - [target]) dloss,  dx = G w,  dw = G^T x
//
// Forward: one product whose epilogue leaves of each tile of logits every
// row's maximum and sum of exponentials (8 bytes for 256 logits), which a
// second launch joins.  Backward: by pieces of the vocabulary the logits are
// computed again, turned into G (bf16) in the epilogue, and multiplied with
// the piece's weights (added up in fp32 over the pieces) and with the rows.
// Rows without a target are left out of the backward pass before it begins; the
// last piece writes dx at the rows' own places (a launch of its own for that took
// 4.8 us at 1023 x 1000 and 10.9 at 4096 x 2048, and one piece needs no fp32 sums).
#include <string.h>

#include "product_kernel.h"

namespace ec {
namespace {

// -------------------------------------------------------------------- forward

__device__ __forceinline__ int64_t target_at(const LossArgs &p, uint32_t i) {
    return p.target_bytes == 8 ? ((const int64_t *)p.target)[i] : (int64_t)((const int32_t *)p.target)[i];
}

// Joins a row's parts: THREADS threads a row (a wave, or all 256 where rows
// are few), whose sums are joined in a fixed order.
template <int THREADS>
__global__ __launch_bounds__(256) void join_stats_kernel(LossArgs p, const float2 *stats, const float *hit, uint32_t tiles) {
    __shared__ float2 sh[4];
    const uint32_t i = blockIdx.x * (256 / THREADS) + threadIdx.x / THREADS, t = threadIdx.x % THREADS;
    if (i >= p.m) return;                   // the whole wave, or the workgroup
    float2 s = {-__builtin_inff(), 0.0f};
    const float2 *row = stats + (uint64_t)i * tiles;
#pragma unroll 4                            // loads of four parts on the way
    for (uint32_t k = t; k < tiles; k += THREADS) s = join_stats(s, row[k]);
#pragma unroll
    for (int d = 32; d; d >>= 1) s = join_stats(s, float2{__shfl_xor(s.x, d), __shfl_xor(s.y, d)});
    if constexpr (THREADS > 64) {
        if ((t & 63) == 0) sh[t >> 6] = s;
        __syncthreads();
        s = join_stats(join_stats(sh[0], sh[1]), join_stats(sh[2], sh[3]));
    }
    if (t) return;
    const float rest = logf(s.y), lse = s.x + rest;     // -inf where every logit is
    if (p.lse) p.lse[i] = lse;
    const int64_t target = target_at(p, i);
    const bool out = target != p.ignore && (target < 0 || target >= (int64_t)p.n);
    // From the maximum and not from lse, whose rounding may be more than a sure
    // row's whole loss (2^-24 of lse, that is 5e-4 at logits of 8192).  Neither
    // part is negative.
    p.loss[i] = target == p.ignore || out ? 0.0f : rest + (s.x - hit[i]);
    if (out && p.status) __hip_atomic_fetch_or(p.status, EC_S_BAD_TARGET, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ------------------------------------------------------------------- backward

// The rows with a target, in order: place[i] is row i's place among them, or
// -1; kept[] the rows themselves, *used their number.  One workgroup.
__global__ __launch_bounds__(1024) void keep_rows_kernel(LossArgs p, int32_t *place, uint32_t *kept, uint32_t *used) {
    __shared__ uint32_t waves[16];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t before = 0;
    bool bad = false;
    for (uint64_t base = 0; base < p.m; base += 1024) {
        const uint64_t i = base + threadIdx.x;
        bool keep = false;
        if (i < p.m) {
            const int64_t t = target_at(p, (uint32_t)i);
            keep = t != p.ignore && t >= 0 && t < (int64_t)p.n;
            bad |= t != p.ignore && !keep;
        }
        const uint64_t mask = __ballot(keep);
        if (lane == 0) waves[wave] = (uint32_t)__popcll(mask);
        __syncthreads();
        uint32_t at = before + (uint32_t)__popcll(mask & ((1ull << lane) - 1)), all = 0;
#pragma unroll
        for (uint32_t w = 0; w < 16; ++w) {
            if (w < wave) at += waves[w];
            all += waves[w];
        }
        if (i < p.m) place[i] = keep ? (int32_t)at : -1;
        if (keep) kept[at] = (uint32_t)i;
        before += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) *used = before;
    if (bad && p.status) __hip_atomic_fetch_or(p.status, EC_S_BAD_TARGET, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// x's rows with a target one after the other, padded with zeros to 16 bytes,
// with what the epilogues need of each; zeros in dx's other rows.  A wave takes
// a row.  COUNT: a workgroup counts the rows with a target before its own (4096
// rows: 16 KB from L2 on average) and keep_rows_kernel is not needed: 12.3 us at
// 4096 x 2048, where the two launches took 5.6 + 8.4.
template <bool COUNT>
__global__ __launch_bounds__(256) void gather_rows_kernel(LossArgs p, const int32_t *place, uint32_t *kept, uint32_t *used,
                                                          uint16_t *x, uint32_t pitch, float2 *row, int32_t *row_target) {
    __shared__ uint32_t sh[4];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, first = blockIdx.x * 4, i = first + wave;
    const auto keeps = [&](uint32_t r) {
        const int64_t t = target_at(p, r);
        return t != p.ignore && t >= 0 && t < (int64_t)p.n;
    };
    bool keep = false;
    int64_t target = 0;
    if (i < p.m) {
        target = target_at(p, i);
        keep = target != p.ignore && target >= 0 && target < (int64_t)p.n;
    }
    uint32_t at = 0;
    if constexpr (COUNT) {
        uint32_t n = 0;
        for (uint32_t r = threadIdx.x; r < first; r += 256) n += keeps(r) ? 1 : 0;
#pragma unroll
        for (int d = 32; d; d >>= 1) n += (uint32_t)__shfl_xor((int)n, d);
        if (lane == 0) sh[wave] = n;
        __syncthreads();
        at = sh[0] + sh[1] + sh[2] + sh[3];
        for (uint32_t r = first; r < i && r < p.m; ++r) at += keeps(r) ? 1 : 0;
        if (lane == 0 && (i + 1 == p.m || (p.m == 0 && i == 0))) *used = at + (keep ? 1 : 0);
        if (lane == 0 && i < p.m && !keep && target != p.ignore && p.status)
            __hip_atomic_fetch_or(p.status, EC_S_BAD_TARGET, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    } else if (i < p.m && keep) {
        at = (uint32_t)place[i];
    }
    if (i >= p.m) return;
    if (keep) {
        if (lane == 0) {
            if constexpr (COUNT) kept[at] = i;
            row[at] = float2{p.lse[i], p.dloss[p.dlosses > 1 ? i : 0]};
            row_target[at] = (int32_t)target;
        }
        for (uint64_t c = lane * 8; c < p.k; c += 512) {
            float v[8];
            load8_bf16(p.x, i * p.x_stride + c, (uint32_t)(p.k - c), v);
            store8(x, EC_BF16, (uint64_t)at * pitch + c, 8, v);
        }
    } else if (p.dx) {
        const float v[8] = {};
        for (uint64_t c = lane * 8; c < p.k; c += 512)
            store8(p.dx, EC_BF16, i * p.dx_stride + c, (uint32_t)(p.k - c), v);
    }
}

// ----------------------------------------------------------------- launches

template <class T, int OP>
void launch_tiles(const ProductArgs &a, const Plan &q, hipStream_t s) {
    product_kernel<T, OP, false, false><<<(uint32_t)q.blocks, T::THREADS, 0, s>>>(a);
    if constexpr (kJoins<OP>) {
        if (q.splits > 1) join_kernel<T, OP><<<q.tiles_i * q.tiles_j * T::NI * T::NJ, T::THREADS, 0, s>>>(a);
    }
}

template <int OP>
hipError_t launch_planned(ProductArgs a, const Plan &q, void *workspace, hipStream_t s) {
    if (q.none) return hipErrorInvalidValue;
    const hipError_t e = place_product(a, q, workspace, s);
    if (e != hipSuccess) return e;
    switch (q.shape) {
        case kHuge:
            if constexpr (OP == kOpRowStats)                // always Wide's
                launch_wide<OP, EC_ACT_NONE>(a, q, s);
            else
                runs_wide(a, q) ? launch_wide<OP, EC_ACT_NONE>(a, q, s) : launch_tiles<Huge, OP>(a, q, s);
            break;
        case kEven: launch_tiles<Even, OP>(a, q, s); break;
        case kSmall: launch_tiles<Small, OP>(a, q, s); break;
        case kTall: launch_tiles<Tall, OP>(a, q, s); break;
        default:
            if constexpr (!contracts_b_rows(OP)) {
                const uint32_t n = (uint32_t)q.blocks;
                if (q.row_tiles == 1)
                    q.waves == 4 ? few_rows_kernel<1, 4, false, OP><<<n, 256, 0, s>>>(a)
                                 : few_rows_kernel<1, 8, false, OP><<<n, 512, 0, s>>>(a);
                else
                    q.waves == 4 ? few_rows_kernel<2, 4, false, OP><<<n, 256, 0, s>>>(a)
                                 : few_rows_kernel<2, 8, false, OP><<<n, 512, 0, s>>>(a);
            }
    }
    return hipGetLastError();
}

template <int OP>
hipError_t launch_any(const ProductArgs &a, void *workspace, hipStream_t s) {
    return launch_planned<OP>(a, make_plan(a), workspace, s);
}

ProductArgs forward_product(const LossArgs &p) {
    ProductArgs a;
    memset(&a, 0, sizeof(a));
    a.op = kOpRowStats;
    a.dtype = EC_BF16;
    a.I = p.m;
    a.J = p.n;
    a.C = p.k;
    a.a = p.x;
    a.a_i = p.x_stride;
    a.a_c = 1;
    a.b = p.w;
    a.b_j = p.w_stride;
    a.b_c = 1;
    a.out_dtype = EC_FP32;
    a.target = p.target;
    a.target_bytes = p.target_bytes;
    return a;
}

// The pieces of the vocabulary and where the backward pass keeps what.
constexpr uint64_t kPieceBytes = 512ull << 20;  // of G
constexpr uint64_t kLeastPiece = 4096;
// Rows whose place every workgroup of the gathering launch counts by itself.
constexpr uint32_t kCountRows = 8192;

struct Pieces {
    uint32_t columns, pitch, x_pitch, w_pitch;  // w_pitch: 0 where w is read in place
    uint64_t place, kept, used, row, row_target, x, w, sum, g, product, bytes;     // place, sum: where needed
};

uint64_t take(uint64_t *at, uint64_t bytes) {
    const uint64_t here = *at;
    *at += round_up(bytes, 256);
    return here;
}

ProductArgs piece_product(const LossArgs &p, const Pieces &q, uint32_t op, uint32_t first, char *ws) {
    ProductArgs a;
    memset(&a, 0, sizeof(a));
    const uint32_t columns = p.n - first < q.columns ? p.n - first : q.columns;
    const void *w = q.w_pitch ? ws + q.w : (const char *)p.w + (uint64_t)first * p.w_stride * 2;
    const uint64_t w_stride = q.w_pitch ? q.w_pitch : p.w_stride;
    a.op = op;
    a.dtype = EC_BF16;
    a.used = (const uint32_t *)(ws + q.used);
    a.first = first;
    if (op == kOpLogitGrad) {
        a.I = p.m;
        a.J = columns;
        a.C = p.k;
        a.a = ws + q.x;
        a.a_i = q.x_pitch;
        a.a_c = 1;
        a.a_padded = true;
        a.b = w;
        a.b_j = w_stride;
        a.b_c = 1;
        a.b_padded = q.w_pitch != 0;
        a.row = (const float2 *)(ws + q.row);
        a.row_target = (const int32_t *)(ws + q.row_target);
        a.out = ws + q.g;
        a.out_stride = q.pitch;
        a.out_dtype = EC_BF16;
    } else if (op == kOpPieceInput) {
        a.I = p.m;
        a.J = p.k;
        a.C = columns;
        a.a = ws + q.g;
        a.a_i = q.pitch;
        a.a_c = 1;
        a.a_padded = true;
        a.b = w;
        a.b_j = 1;
        a.b_c = w_stride;
        a.sum_in = first ? (const float *)(ws + q.sum) : nullptr;
        if (p.n - first <= q.columns) {     // the last piece
            a.out = p.dx;
            a.out_stride = p.dx_stride;
            a.out_dtype = EC_BF16;
            a.kept = (const uint32_t *)(ws + q.kept);
        } else {
            a.out = ws + q.sum;
            a.out_stride = p.k;
            a.out_dtype = EC_FP32;
        }
    } else {
        a.I = columns;
        a.J = p.k;
        a.C = p.m;
        a.a = ws + q.g;
        a.a_i = 1;
        a.a_c = q.pitch;
        a.b = ws + q.x;
        a.b_j = 1;
        a.b_c = q.x_pitch;
        a.out = (char *)p.dw + (uint64_t)first * p.dw_stride * (p.dw_dtype == EC_FP32 ? 4 : 2);
        a.out_stride = p.dw_stride;
        a.out_dtype = p.dw_dtype;
    }
    return a;
}

// Whether a piece's products run: where first is 0, those of a whole piece,
// else those of the last.  *bytes: their workspace.
bool products_fit(const LossArgs &p, const Pieces &q, uint32_t first, uint64_t *bytes) {
    *bytes = 0;
    for (uint32_t op : {(uint32_t)kOpLogitGrad, (uint32_t)kOpPieceInput, (uint32_t)kOpPieceWeight}) {
        if ((op == kOpPieceInput && !p.dx) || (op == kOpPieceWeight && !p.dw)) continue;
        const ProductArgs a = piece_product(p, q, op, first, nullptr);
        if (!a.I || !a.J) continue;
        const Plan plan = make_plan(a);
        if (plan.none) return false;
        if (plan.bytes > *bytes) *bytes = plan.bytes;
    }
    return true;
}

bool lay_out(const LossArgs &p, Pieces *q) {
    memset(q, 0, sizeof(*q));
    uint64_t columns = kPieceBytes / (2 * (uint64_t)(p.m ? p.m : 1)) / 256 * 256;
    if (columns < kLeastPiece) columns = kLeastPiece;
    q->columns = (uint32_t)(columns < p.n ? columns : p.n);
    q->pitch = (uint32_t)round_up(q->columns, 8);
    const uint64_t pitch = round_up(p.k, 8);
    q->x_pitch = (uint32_t)pitch;
    const bool in_place = !((((uintptr_t)p.w | p.w_stride * 2) & 15) || (p.k & 7));
    q->w_pitch = in_place ? 0 : (uint32_t)pitch;
    uint64_t at = 0;
    q->place = take(&at, p.m > kCountRows ? (uint64_t)p.m * 4 : 0);
    q->kept = take(&at, (uint64_t)p.m * 4);
    q->used = take(&at, 4);
    q->row = take(&at, (uint64_t)p.m * 8);
    q->row_target = take(&at, (uint64_t)p.m * 4);
    q->x = take(&at, p.m * pitch * 2);
    q->w = take(&at, q->w_pitch ? q->columns * pitch * 2 : 0);
    q->sum = take(&at, p.dx && q->columns < p.n ? (uint64_t)p.m * p.k * 4 : 0);
    q->g = take(&at, (uint64_t)p.m * q->pitch * 2);
    q->product = at;
    const uint32_t last = (p.n - 1) / q->columns * q->columns;
    uint64_t whole, rest = 0;
    if (!products_fit(p, *q, 0, &whole) || (last && !products_fit(p, *q, last, &rest))) return false;
    q->bytes = at + (whole > rest ? whole : rest);
    // the launches that gather rows and copy w
    return launchable(ceil_div(p.m, 4), 256) && launchable(ceil_div(q->columns * (pitch / 8), 256), 256);
}

}  // namespace

static bool forward_need(const LossArgs &p, const Plan &q, uint64_t *bytes) {
    *bytes = round_up(q.bytes, 256) + round_up((uint64_t)p.m * q.tiles_j * 8, 256) + (uint64_t)p.m * 4;
    return !q.none && launchable(p.m, 256);
}

bool loss_need(const LossArgs &p, uint64_t *bytes) {
    *bytes = 0;
    return !p.m || forward_need(p, make_plan(forward_product(p)), bytes);
}

bool loss_grad_need(const LossArgs &p, uint64_t *bytes) {
    Pieces q;
    *bytes = 0;
    if (!lay_out(p, &q)) return false;
    *bytes = q.bytes;
    return true;
}

int run_loss(const LossArgs &p, void *workspace, uint64_t bytes, hipStream_t s) {
    if (!p.m) return EC_OK;
    ProductArgs a = forward_product(p);
    const Plan q = make_plan(a);
    uint64_t need;
    if (!forward_need(p, q, &need)) return EC_E_UNSUPPORTED;
    if (!workspace || bytes < need) return EC_E_INVAL;
    char *ws = (char *)workspace;
    a.stats = (float2 *)(ws + round_up(q.bytes, 256));
    a.hit = (float *)((char *)a.stats + round_up((uint64_t)p.m * q.tiles_j * 8, 256));
    const hipError_t e = launch_planned<kOpRowStats>(a, q, workspace, s);
    if (e != hipSuccess) return EC_E_HIP;
    if (p.m > 1024)
        join_stats_kernel<64><<<(p.m + 3) / 4, 256, 0, s>>>(p, a.stats, a.hit, q.tiles_j);
    else
        join_stats_kernel<256><<<p.m, 256, 0, s>>>(p, a.stats, a.hit, q.tiles_j);
    return hipGetLastError() == hipSuccess ? EC_OK : EC_E_HIP;
}

int run_loss_grad(const LossArgs &p, void *workspace, uint64_t bytes, hipStream_t s) {
    Pieces q;
    if (!lay_out(p, &q)) return EC_E_UNSUPPORTED;
    if (!workspace || bytes < q.bytes) return EC_E_INVAL;
    char *ws = (char *)workspace;
    int32_t *place = (int32_t *)(ws + q.place);
    uint32_t *kept = (uint32_t *)(ws + q.kept), *used = (uint32_t *)(ws + q.used);
    const auto gather = [&](auto kernel) {
        kernel<<<p.m > 4 ? (p.m + 3) / 4 : 1, 256, 0, s>>>(p, place, kept, used, (uint16_t *)(ws + q.x), q.x_pitch,
                                                          (float2 *)(ws + q.row), (int32_t *)(ws + q.row_target));
    };
    if (p.m > kCountRows) {
        keep_rows_kernel<<<1, 1024, 0, s>>>(p, place, kept, used);
        gather(gather_rows_kernel<false>);
    } else {
        gather(gather_rows_kernel<true>);
    }
    hipError_t e = hipGetLastError();
    for (uint32_t first = 0; e == hipSuccess && p.k && (p.dx || p.dw); first += q.columns) {
        const uint32_t columns = p.n - first < q.columns ? p.n - first : q.columns;
        if (q.w_pitch)
            e = launch_copy_rows((const char *)p.w + (uint64_t)first * p.w_stride * 2, p.w_stride, columns, p.k, EC_BF16,
                                 ws + q.w, q.w_pitch, s);
        if (e == hipSuccess && p.m) e = launch_any<kOpLogitGrad>(piece_product(p, q, kOpLogitGrad, first, ws), ws + q.product, s);
        if (e == hipSuccess && p.m && p.dx)
            e = launch_any<kOpPieceInput>(piece_product(p, q, kOpPieceInput, first, ws), ws + q.product, s);
        if (e == hipSuccess && p.dw)
            e = launch_any<kOpPieceWeight>(piece_product(p, q, kOpPieceWeight, first, ws), ws + q.product, s);
        if (p.n - first <= q.columns) break;
    }
    return e == hipSuccess ? EC_OK : EC_E_HIP;
}

}  // namespace ec
