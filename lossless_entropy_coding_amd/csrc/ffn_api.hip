// C ABI of the feed-forward operators, the loss and the weight update: argument checks and launches.
#include <math.h>
#include <string.h>

#include "ffn_common.h"
#include "train_common.h"

namespace ec {
namespace {

constexpr uint64_t kMaxSize = (1ull << 31) - 1;

uint64_t size_of(uint32_t dtype) { return dtype == EC_FP32 ? 4 : dtype == EC_BF16 ? 2 : dtype == EC_E4M3 ? 1 : 0; }

// A [rows, cols] tensor that may be absent: aligned to its element, with room
// for a row in its stride.
bool tensor_ok(const void *p, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t stride) {
    const uint64_t s = size_of(dtype);
    return s && ((uintptr_t)p & (s - 1)) == 0 && (rows <= 1 || stride >= cols) && stride < (1ull << 40);
}

// As tensor_ok, and present unless it has no elements.
bool factor_ok(const void *p, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t stride) {
    return (p || !rows || !cols) && tensor_ok(p, dtype, rows, cols, stride);
}

bool common_ok(const ec_linear_args *a) {
    if (!a || a->m > kMaxSize || a->n > kMaxSize || a->k > kMaxSize || a->act > EC_ACT_RELU) return false;
    if (a->groups > EC_MAX_GROUPS || (a->groups && (!a->d_offsets || ((uintptr_t)a->d_offsets & 3)))) return false;
    return ((uintptr_t)a->d_status & 3) == 0 && ((uintptr_t)a->d_workspace & 15) == 0;
}

bool group_stride_ok(const ec_linear_args *a, uint64_t rows, uint64_t cols, uint64_t stride, uint64_t group) {
    if (a->groups <= 1 || !rows || !cols) return true;
    return group >= (rows - 1) * stride + cols && group < (1ull << 48);
}

int check_forward(const ec_linear_args *a) {
    if (!common_ok(a)) return EC_E_INVAL;
    if (a->dtype != EC_BF16 && a->dtype != EC_E4M3) return EC_E_INVAL;
    if (!size_of(a->out_dtype)) return EC_E_INVAL;
    if (!factor_ok(a->d_x, a->dtype, a->m, a->k, a->x_stride)) return EC_E_INVAL;
    if (!factor_ok(a->d_w, a->dtype, a->n, a->k, a->w_stride)) return EC_E_INVAL;
    if (!group_stride_ok(a, a->n, a->k, a->w_stride, a->w_group_stride)) return EC_E_INVAL;
    if (!factor_ok(a->d_y, a->out_dtype, a->m, a->n, a->y_stride)) return EC_E_INVAL;
    if (a->d_bias && ((a->bias_dtype != EC_BF16 && a->bias_dtype != EC_FP32) ||
                      !tensor_ok(a->d_bias, a->bias_dtype, 1, a->n, a->n)))
        return EC_E_INVAL;
    if (!tensor_ok(a->d_residual, EC_BF16, a->m, a->n, a->d_residual ? a->residual_stride : a->n)) return EC_E_INVAL;
    if (!tensor_ok(a->d_preact, EC_BF16, a->m, a->n, a->d_preact ? a->preact_stride : a->n)) return EC_E_INVAL;
    if (a->d_x_scale && a->x_scales != 1 && a->x_scales != a->m) return EC_E_INVAL;
    if (a->d_w_scale && a->w_scales != 1 && a->w_scales != a->n) return EC_E_INVAL;
    if (((uintptr_t)a->d_x_scale | (uintptr_t)a->d_w_scale | (uintptr_t)a->d_out_scale) & 3) return EC_E_INVAL;
    if (a->d_out_scale && a->out_dtype != EC_E4M3) return EC_E_INVAL;
    return EC_OK;
}

int check_grad_input(const ec_linear_args *a) {
    if (!common_ok(a) || a->dtype != EC_BF16) return EC_E_INVAL;
    if (!factor_ok(a->d_dy, EC_BF16, a->m, a->n, a->dy_stride)) return EC_E_INVAL;
    if (!factor_ok(a->d_w, EC_BF16, a->n, a->k, a->w_stride)) return EC_E_INVAL;
    if (!group_stride_ok(a, a->n, a->k, a->w_stride, a->w_group_stride)) return EC_E_INVAL;
    if (!factor_ok(a->d_dx, EC_BF16, a->m, a->k, a->dx_stride)) return EC_E_INVAL;
    if (a->act != EC_ACT_NONE && !factor_ok(a->d_preact, EC_BF16, a->m, a->k, a->preact_stride)) return EC_E_INVAL;
    return EC_OK;
}

int check_grad_weight(const ec_linear_args *a) {
    if (!common_ok(a) || a->dtype != EC_BF16) return EC_E_INVAL;
    if (!factor_ok(a->d_dy, EC_BF16, a->m, a->n, a->dy_stride)) return EC_E_INVAL;
    if (a->d_dw) {
        if (a->out_dtype != EC_BF16 && a->out_dtype != EC_FP32) return EC_E_INVAL;
        if (!factor_ok(a->d_x, EC_BF16, a->m, a->k, a->x_stride)) return EC_E_INVAL;
        if (!factor_ok(a->d_dw, a->out_dtype, a->n, a->k, a->dw_stride)) return EC_E_INVAL;
        if (!group_stride_ok(a, a->n, a->k, a->dw_stride, a->dw_group_stride)) return EC_E_INVAL;
    }
    return ((uintptr_t)a->d_db & 3) == 0 ? EC_OK : EC_E_INVAL;
}

// Whether two [rows, cols] tensors share memory; of different strides, whether
// what they span does.
bool overlap(const void *p, uint64_t p_stride, const void *q, uint64_t q_stride, uint64_t rows, uint64_t cols,
             uint64_t size) {
    if (!rows || !cols) return false;
    const uint64_t a = (uint64_t)(uintptr_t)p, b = (uint64_t)(uintptr_t)q, row = cols * size;
    if (a + (rows - 1) * p_stride * size + row <= b || b + (rows - 1) * q_stride * size + row <= a) return false;
    if (rows == 1 || p_stride != q_stride) return true;
    const uint64_t step = p_stride * size, apart = (a < b ? b - a : a - b) % step;
    return apart < row || apart + row > step;       // not side by side
}

int hip_code(hipError_t e) { return e == hipSuccess ? EC_OK : EC_E_HIP; }

// A factor's row stride.  That of a single row may hold anything: the row's
// length (whole 16-byte chunks) instead, past which a tile finds its end.
uint64_t row_stride(uint64_t rows, uint64_t cols, uint64_t stride, uint32_t dtype) {
    const uint64_t chunk = 16 / size_of(dtype);
    return rows > 1 ? stride : (cols + chunk - 1) / chunk * chunk;
}

ProductArgs product(const ec_linear_args *a, uint32_t op) {
    ProductArgs p;
    memset(&p, 0, sizeof(p));
    p.op = op;
    p.dtype = a->dtype;
    p.groups = a->groups;
    p.offsets = a->d_offsets;
    p.status = a->d_status;
    p.preact = (uint16_t *)a->d_preact;
    p.preact_stride = a->preact_stride;
    if (op == EC_LINEAR_FORWARD) {
        p.I = (uint32_t)a->m;
        p.J = (uint32_t)a->n;
        p.C = (uint32_t)a->k;
        p.a = a->d_x;
        p.a_i = row_stride(a->m, a->k, a->x_stride, a->dtype);
        p.a_c = 1;
        p.b = a->d_w;
        p.b_j = row_stride(a->n, a->k, a->w_stride, a->dtype);
        p.b_c = 1;
        p.b_group = a->w_group_stride;
        p.act = a->act;
        p.out_dtype = a->out_dtype;
        p.bias_dtype = a->bias_dtype;
        p.x_scales = a->x_scales;
        p.w_scales = a->w_scales;
        p.bias = a->d_bias;
        p.residual = (const uint16_t *)a->d_residual;
        p.residual_stride = a->residual_stride;
        p.x_scale = a->d_x_scale;
        p.w_scale = a->d_w_scale;
        p.out_scale = a->d_out_scale;
        p.out = a->d_y;
        p.out_stride = a->y_stride;
    } else if (op == EC_LINEAR_GRAD_INPUT) {
        p.I = (uint32_t)a->m;
        p.J = (uint32_t)a->k;
        p.C = (uint32_t)a->n;
        p.a = a->d_dy;
        p.a_i = row_stride(a->m, a->n, a->dy_stride, a->dtype);
        p.a_c = 1;
        p.b = a->d_w;
        p.b_j = 1;
        p.b_c = row_stride(a->n, a->k, a->w_stride, a->dtype);
        p.b_group = a->w_group_stride;
        p.act = a->act;
        p.out_dtype = EC_BF16;
        p.out = a->d_dx;
        p.out_stride = a->dx_stride;
    } else {
        p.I = (uint32_t)a->n;
        p.J = (uint32_t)a->k;
        p.C = (uint32_t)a->m;
        p.a = a->d_dy;
        p.a_i = 1;
        p.a_c = row_stride(a->m, a->n, a->dy_stride, a->dtype);
        p.b = a->d_x;
        p.b_j = 1;
        p.b_c = row_stride(a->m, a->k, a->x_stride, a->dtype);
        p.out_dtype = a->out_dtype;
        p.out = a->d_dw;
        p.out_stride = a->dw_stride;
        p.out_group = a->dw_group_stride;
    }
    return p;
}

}  // namespace
}  // namespace ec

using namespace ec;

namespace {

int check(const ec_linear_args *a, uint32_t op) {
    switch (op) {
        case EC_LINEAR_FORWARD: return check_forward(a);
        case EC_LINEAR_GRAD_INPUT: return check_grad_input(a);
        case EC_LINEAR_GRAD_WEIGHT: return check_grad_weight(a);
    }
    return EC_E_INVAL;
}

bool has_product(const ec_linear_args *a, uint32_t op) { return op != EC_LINEAR_GRAD_WEIGHT || a->d_dw; }

ColumnSumArgs column_sum(const ec_linear_args *a) {
    ColumnSumArgs c;
    memset(&c, 0, sizeof(c));
    c.dy = (const uint16_t *)a->d_dy;
    c.dy_stride = a->dy_stride;
    c.m = (uint32_t)a->m;
    c.n = (uint32_t)a->n;
    c.groups = a->groups;
    c.offsets = a->d_offsets;
    c.db = a->d_db;
    c.status = a->d_dw ? nullptr : a->d_status;     // the product reports bad offsets
    return c;
}

int run_product(const ec_linear_args *a, const ProductArgs &p, hipStream_t stream) {
    if (!product_fits(p)) return EC_E_UNSUPPORTED;
    const uint64_t need = product_workspace(p);
    if (need && (!a->d_workspace || a->workspace_bytes < need)) return EC_E_INVAL;
    return hip_code(launch_product(p, a->d_workspace, stream));
}

}  // namespace

uint64_t linear_workspace_bytes(const ec_linear_args *a, uint32_t op) {
    if (check(a, op)) return 0;
    uint64_t need = has_product(a, op) ? product_workspace(product(a, op)) : 0;
    if (op == EC_LINEAR_GRAD_WEIGHT && a->d_db && !(a->d_dw && product_sums_columns(product(a, op)))) {
        // one after the other, in the same memory
        const uint64_t sums = column_sum_workspace(column_sum(a));
        need = sums > need ? sums : need;
    }
    return need;
}

int linear_forward(const ec_linear_args *a, hipStream_t stream) {
    const int rc = check_forward(a);
    return rc ? rc : run_product(a, product(a, EC_LINEAR_FORWARD), stream);
}

int linear_grad_input(const ec_linear_args *a, hipStream_t stream) {
    const int rc = check_grad_input(a);
    return rc ? rc : run_product(a, product(a, EC_LINEAR_GRAD_INPUT), stream);
}

int linear_grad_weight(const ec_linear_args *a, hipStream_t stream) {
    int rc = check_grad_weight(a);
    if (rc) return rc;
    if (a->d_dw) {
        ProductArgs p = product(a, EC_LINEAR_GRAD_WEIGHT);
        const bool both = a->d_db && product_sums_columns(p);
        if (both) p.db = a->d_db;
        if ((rc = run_product(a, p, stream)) || both) return rc;
    }
    if (!a->d_db)       // neither, as where n is 0
        return a->d_dw ? EC_OK : hip_code(launch_check_offsets(a->d_offsets, a->groups, (uint32_t)a->m, a->d_status, stream));
    const ColumnSumArgs c = column_sum(a);
    const uint64_t need = column_sum_workspace(c);
    if (need && (!a->d_workspace || a->workspace_bytes < need)) return EC_E_INVAL;
    return hip_code(launch_column_sum(c, (float *)a->d_workspace, stream));
}

int layer_norm_forward(const void *d_x, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t x_stride,
                       const void *d_weight, const void *d_bias, uint32_t w_dtype, float eps, void *d_y,
                       uint32_t out_dtype, uint64_t y_stride, const float *d_out_scale, float *d_mean,
                       float *d_rstd, hipStream_t stream) {
    if ((dtype != EC_BF16 && dtype != EC_FP32) || !cols || cols > 65536 || rows > kMaxSize || !size_of(out_dtype))
        return EC_E_INVAL;
    if ((d_weight || d_bias) && w_dtype != EC_BF16 && w_dtype != EC_FP32) return EC_E_INVAL;
    if (!factor_ok(d_x, dtype, rows, cols, x_stride) || !factor_ok(d_y, out_dtype, rows, cols, y_stride))
        return EC_E_INVAL;
    if ((d_weight && !tensor_ok(d_weight, w_dtype, 1, cols, cols)) || (d_bias && !tensor_ok(d_bias, w_dtype, 1, cols, cols)))
        return EC_E_INVAL;
    if (((uintptr_t)d_out_scale | (uintptr_t)d_mean | (uintptr_t)d_rstd) & 3) return EC_E_INVAL;
    if ((d_out_scale && out_dtype != EC_E4M3) || !(eps >= 0.0f)) return EC_E_INVAL;
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.x = d_x;
    a.rows = rows;
    a.x_stride = x_stride;
    a.cols = (uint32_t)cols;
    a.dtype = dtype;
    a.w_dtype = w_dtype;
    a.out_dtype = out_dtype;
    a.weight = d_weight;
    a.bias = d_bias;
    a.eps = eps;
    a.y = d_y;
    a.y_stride = y_stride;
    a.out_scale = d_out_scale;
    a.mean = d_mean;
    a.rstd = d_rstd;
    return hip_code(launch_norm(a, stream));
}

uint64_t layer_norm_grad_workspace_bytes(uint64_t rows, uint64_t cols) {
    if (!cols || cols > 65536 || rows > kMaxSize) return 0;
    return (uint64_t)norm_grad_parts(rows, cols) * 2 * cols * sizeof(float);
}

int layer_norm_grad(const void *d_dy, uint64_t dy_stride, const void *d_x, uint64_t x_stride, uint32_t dtype,
                    uint64_t rows, uint64_t cols, const float *d_mean, const float *d_rstd,
                    const void *d_weight, uint32_t w_dtype, const void *d_dres, uint64_t dres_stride, void *d_dx,
                    uint64_t dx_stride, float *d_dweight, float *d_dbias, void *d_workspace,
                    uint64_t workspace_bytes, hipStream_t stream) {
    if ((dtype != EC_BF16 && dtype != EC_FP32) || !cols || cols > 65536 || rows > kMaxSize) return EC_E_INVAL;
    if (d_weight && ((w_dtype != EC_BF16 && w_dtype != EC_FP32) || !tensor_ok(d_weight, w_dtype, 1, cols, cols)))
        return EC_E_INVAL;
    if (!factor_ok(d_dy, dtype, rows, cols, dy_stride) || !factor_ok(d_x, dtype, rows, cols, x_stride))
        return EC_E_INVAL;
    if (rows && (!d_mean || !d_rstd)) return EC_E_INVAL;
    if (d_dres && !tensor_ok(d_dres, dtype, rows, cols, dres_stride)) return EC_E_INVAL;
    if (d_dx && !tensor_ok(d_dx, dtype, rows, cols, dx_stride)) return EC_E_INVAL;
    // workgroups that share a row read all of it, in no order with its dx
    const uint64_t size = size_of(dtype);
    if (d_dx && norm_grad_slices(cols) > 1 &&
        (overlap(d_dx, dx_stride, d_x, x_stride, rows, cols, size) || overlap(d_dx, dx_stride, d_dy, dy_stride, rows, cols, size)))
        return EC_E_INVAL;
    if (((uintptr_t)d_mean | (uintptr_t)d_rstd | (uintptr_t)d_dweight | (uintptr_t)d_dbias) & 3) return EC_E_INVAL;
    if ((d_dweight || d_dbias) && (!d_workspace || ((uintptr_t)d_workspace & 15) ||
                                   workspace_bytes < layer_norm_grad_workspace_bytes(rows, cols)))
        return EC_E_INVAL;
    NormGradArgs a;
    memset(&a, 0, sizeof(a));
    a.dy = d_dy;
    a.x = d_x;
    a.weight = d_weight;
    a.dres = d_dres;
    a.rows = rows;
    a.dy_stride = dy_stride;
    a.x_stride = x_stride;
    a.dres_stride = dres_stride;
    a.dx_stride = dx_stride;
    a.cols = (uint32_t)cols;
    a.dtype = dtype;
    a.w_dtype = w_dtype;
    a.mean = d_mean;
    a.rstd = d_rstd;
    a.dx = d_dx;
    a.dweight = d_dweight;
    a.dbias = d_dbias;
    a.partial = d_dweight || d_dbias ? (float *)d_workspace : nullptr;
    a.parts = norm_grad_parts(rows, cols);
    return hip_code(launch_norm_grad(a, stream));
}

// ------------------------------------------------------------------ gated block

namespace {

// w and bias have 2 n rows; so does preact 2 n columns.
int check_gated(const ec_linear_args *a) {
    if (!common_ok(a) || a->n > kMaxSize / 2) return EC_E_INVAL;
    const uint64_t n = a->n, rows = 2 * n;
    if (a->dtype != EC_BF16 && a->dtype != EC_E4M3) return EC_E_INVAL;
    if (!size_of(a->out_dtype) || a->d_residual) return EC_E_INVAL;
    if (!factor_ok(a->d_x, a->dtype, a->m, a->k, a->x_stride)) return EC_E_INVAL;
    if (!factor_ok(a->d_w, a->dtype, rows, a->k, a->w_stride)) return EC_E_INVAL;
    if (!group_stride_ok(a, rows, a->k, a->w_stride, a->w_group_stride)) return EC_E_INVAL;
    if (!factor_ok(a->d_y, a->out_dtype, a->m, n, a->y_stride)) return EC_E_INVAL;
    if (a->d_bias && ((a->bias_dtype != EC_BF16 && a->bias_dtype != EC_FP32) ||
                      !tensor_ok(a->d_bias, a->bias_dtype, 1, rows, rows)))
        return EC_E_INVAL;
    if (!tensor_ok(a->d_preact, EC_BF16, a->m, rows, a->d_preact ? a->preact_stride : rows)) return EC_E_INVAL;
    if (a->d_x_scale && a->x_scales != 1 && a->x_scales != a->m) return EC_E_INVAL;
    if (a->d_w_scale && a->w_scales != 1 && a->w_scales != rows) return EC_E_INVAL;
    if (((uintptr_t)a->d_x_scale | (uintptr_t)a->d_w_scale | (uintptr_t)a->d_out_scale) & 3) return EC_E_INVAL;
    if (a->d_out_scale && a->out_dtype != EC_E4M3) return EC_E_INVAL;
    return EC_OK;
}

int check_gated_grad(const ec_linear_args *a) {
    if (!common_ok(a) || a->n > kMaxSize / 2 || a->dtype != EC_BF16) return EC_E_INVAL;
    const uint64_t n = a->n, rows = 2 * n;
    if (!factor_ok(a->d_dy, EC_BF16, a->m, n, a->dy_stride)) return EC_E_INVAL;
    if (!factor_ok(a->d_preact, EC_BF16, a->m, rows, a->preact_stride)) return EC_E_INVAL;
    if (a->d_dx) {
        if (!factor_ok(a->d_w, EC_BF16, rows, a->k, a->w_stride)) return EC_E_INVAL;
        if (!group_stride_ok(a, rows, a->k, a->w_stride, a->w_group_stride)) return EC_E_INVAL;
        if (!tensor_ok(a->d_dx, EC_BF16, a->m, a->k, a->dx_stride)) return EC_E_INVAL;
    }
    if (a->d_dw) {
        if (a->out_dtype != EC_BF16 && a->out_dtype != EC_FP32) return EC_E_INVAL;
        if (!factor_ok(a->d_x, EC_BF16, a->m, a->k, a->x_stride)) return EC_E_INVAL;
        if (!tensor_ok(a->d_dw, a->out_dtype, rows, a->k, a->dw_stride)) return EC_E_INVAL;
        if (!group_stride_ok(a, rows, a->k, a->dw_stride, a->dw_group_stride)) return EC_E_INVAL;
    }
    return ((uintptr_t)a->d_db & 3) == 0 ? EC_OK : EC_E_INVAL;
}

ProductArgs gated_product(const ec_linear_args *a) {
    ProductArgs p = product(a, EC_LINEAR_FORWARD);
    p.op = kOpGated;
    p.b_j = row_stride(2 * a->n, a->k, a->w_stride, a->dtype);
    return p;
}

// The backward pass: where dz and the sums' parts lie, and its two products.
struct GatedGrad {
    GatedGradArgs grad;
    ProductArgs dx, dw;
    uint64_t partial, product, bytes;       // workspace
    bool fits;
};

GatedGrad gated_grad(const ec_linear_args *a, void *workspace) {
    GatedGrad q;
    memset(&q, 0, sizeof(q));
    char *ws = (char *)workspace;
    GatedGradArgs &g = q.grad;
    g.dy = (const uint16_t *)a->d_dy;
    g.dy_stride = a->dy_stride;
    g.preact = (const uint16_t *)a->d_preact;
    g.preact_stride = a->preact_stride;
    g.m = (uint32_t)a->m;
    g.n = (uint32_t)a->n;
    g.groups = a->groups;
    g.act = a->act;
    g.offsets = a->d_offsets;
    g.status = a->d_status;
    g.dz = (uint16_t *)ws;
    g.pitch = (2 * a->n + 7) / 8 * 8;
    g.db = a->d_db;
    g.slab = gated_grad_slab(g.m, g.n);
    q.partial = (a->m * g.pitch * 2 + 255) / 256 * 256;
    q.product = q.partial + (gated_grad_workspace(g) + 255) / 256 * 256;
    g.partial = (float *)(ws + q.partial);
    q.bytes = q.product;
    q.fits = gated_grad_fits(g);
    uint64_t need;
    // the products of dz, as of the gradient of a product with 2 n columns
    ec_linear_args l = *a;
    l.n = 2 * a->n;
    l.act = EC_ACT_NONE;
    l.d_dy = g.dz;
    l.dy_stride = g.pitch;
    l.d_preact = nullptr;
    l.d_db = nullptr;
    l.d_status = nullptr;
    if (a->d_dx) {
        q.dx = product(&l, EC_LINEAR_GRAD_INPUT);
        q.dx.a_i = g.pitch;
        q.dx.a_padded = true;
        q.fits = product_need(q.dx, &need) && q.fits;
        q.bytes = q.product + need > q.bytes ? q.product + need : q.bytes;
    }
    if (a->d_dw) {
        q.dw = product(&l, EC_LINEAR_GRAD_WEIGHT);
        q.dw.a_c = g.pitch;
        q.fits = product_need(q.dw, &need) && q.fits;
        q.bytes = q.product + need > q.bytes ? q.product + need : q.bytes;
    }
    return q;
}

}  // namespace

uint64_t gated_linear_workspace_bytes(const ec_linear_args *a) {
    if (check_gated(a)) return 0;
    return product_workspace(gated_product(a));
}

int gated_linear_forward(const ec_linear_args *a, hipStream_t stream) {
    const int rc = check_gated(a);
    if (rc) return rc;
    const ProductArgs p = gated_product(a);
    uint64_t need;
    if (!product_need(p, &need)) return EC_E_UNSUPPORTED;
    if (need && (!a->d_workspace || a->workspace_bytes < need)) return EC_E_INVAL;
    return hip_code(launch_gated(p, a->d_workspace, stream));
}

uint64_t gated_linear_grad_workspace_bytes(const ec_linear_args *a) {
    if (check_gated_grad(a)) return 0;
    const GatedGrad q = gated_grad(a, nullptr);
    return q.fits ? q.bytes : 0;
}

int gated_linear_grad(const ec_linear_args *a, hipStream_t stream) {
    const int rc = check_gated_grad(a);
    if (rc) return rc;
    const GatedGrad q = gated_grad(a, a->d_workspace);
    if (!q.fits) return EC_E_UNSUPPORTED;
    if (q.bytes && (!a->d_workspace || a->workspace_bytes < q.bytes)) return EC_E_INVAL;
    hipError_t e = launch_gated_grad(q.grad, stream);
    char *const ws = (char *)a->d_workspace + q.product;
    if (e == hipSuccess && a->d_dx) e = launch_product(q.dx, ws, stream);
    if (e == hipSuccess && a->d_dw) e = launch_product(q.dw, ws, stream);
    return hip_code(e);
}

// --------------------------------------------------------------- cross entropy

namespace {

bool loss_ok(const ec_loss_args *a) {
    if (!a || a->m > kMaxSize || !a->n || a->n > kMaxSize || a->k > kMaxSize) return false;
    if (a->target_bytes != 4 && a->target_bytes != 8) return false;
    if (!factor_ok(a->d_x, EC_BF16, a->m, a->k, a->x_stride) || !factor_ok(a->d_w, EC_BF16, a->n, a->k, a->w_stride))
        return false;
    if (a->m && (!a->d_target || ((uintptr_t)a->d_target & (a->target_bytes - 1)))) return false;
    return !(((uintptr_t)a->d_lse | (uintptr_t)a->d_status) & 3) && !((uintptr_t)a->d_workspace & 15);
}

LossArgs loss_args(const ec_loss_args *a) {
    LossArgs p;
    memset(&p, 0, sizeof(p));
    p.x = a->d_x;
    p.x_stride = row_stride(a->m, a->k, a->x_stride, EC_BF16);
    p.w = a->d_w;
    p.w_stride = row_stride(a->n, a->k, a->w_stride, EC_BF16);
    p.m = (uint32_t)a->m;
    p.n = (uint32_t)a->n;
    p.k = (uint32_t)a->k;
    p.target = a->d_target;
    p.target_bytes = a->target_bytes;
    p.ignore = a->ignore_index;
    p.loss = a->d_loss;
    p.lse = a->d_lse;
    p.dloss = a->d_dloss;
    p.dlosses = a->dlosses;
    p.dx = a->d_dx;
    p.dx_stride = a->dx_stride;
    p.dw = a->d_dw;
    p.dw_stride = a->dw_stride;
    p.dw_dtype = a->dw_dtype;
    p.status = a->d_status;
    return p;
}

int check_loss(const ec_loss_args *a) {
    if (!loss_ok(a) || (a->m && !a->d_loss) || ((uintptr_t)a->d_loss & 3)) return EC_E_INVAL;
    return EC_OK;
}

int check_loss_grad(const ec_loss_args *a) {
    if (!loss_ok(a) || (a->m && (!a->d_lse || !a->d_dloss)) || ((uintptr_t)a->d_dloss & 3)) return EC_E_INVAL;
    if (a->dlosses != 1 && a->dlosses != a->m) return EC_E_INVAL;
    if (a->d_dx && !tensor_ok(a->d_dx, EC_BF16, a->m, a->k, a->dx_stride)) return EC_E_INVAL;
    if (a->d_dw && ((a->dw_dtype != EC_BF16 && a->dw_dtype != EC_FP32) ||
                    !tensor_ok(a->d_dw, a->dw_dtype, a->n, a->k, a->dw_stride)))
        return EC_E_INVAL;
    return EC_OK;
}

}  // namespace

uint64_t linear_cross_entropy_workspace_bytes(const ec_loss_args *a) {
    uint64_t need;
    return !check_loss(a) && loss_need(loss_args(a), &need) ? need : 0;
}

int linear_cross_entropy(const ec_loss_args *a, hipStream_t stream) {
    const int rc = check_loss(a);
    return rc ? rc : run_loss(loss_args(a), a->d_workspace, a->workspace_bytes, stream);
}

uint64_t linear_cross_entropy_grad_workspace_bytes(const ec_loss_args *a) {
    uint64_t need;
    return !check_loss_grad(a) && loss_grad_need(loss_args(a), &need) ? need : 0;
}

int linear_cross_entropy_grad(const ec_loss_args *a, hipStream_t stream) {
    const int rc = check_loss_grad(a);
    return rc ? rc : run_loss_grad(loss_args(a), a->d_workspace, a->workspace_bytes, stream);
}

// ----------------------------------------------------------------------- AdamW

uint64_t adamw_state_blocks(uint64_t n) { return adamw_blocks(n); }

int adamw_step(const ec_adamw_tensor *tensors, uint32_t count, const ec_adamw_args *a, hipStream_t stream) {
    if (!a || (count && !tensors)) return EC_E_INVAL;
    if (a->state_dtype != EC_FP32 && a->state_dtype != EC_E4M3) return EC_E_INVAL;
    const bool coded = a->state_dtype == EC_E4M3;
    if (!a->d_steps || ((uintptr_t)a->d_steps & 3) || (((uintptr_t)a->d_lr | (uintptr_t)a->d_grad_scale) & 3))
        return EC_E_INVAL;
    if (!(a->beta1 >= 0.0 && a->beta1 < 1.0 && a->beta2 >= 0.0 && a->beta2 < 1.0 && a->eps >= 0.0)) return EC_E_INVAL;
    uint64_t blocks = 0;
    for (uint32_t i = 0; i < count; ++i) {
        const ec_adamw_tensor &t = tensors[i];
        if (t.n > (1ull << 40) || (t.grad_dtype != EC_BF16 && t.grad_dtype != EC_FP32)) return EC_E_INVAL;
        if (t.n && (!t.d_param || !t.d_grad)) return EC_E_INVAL;
        if (((uintptr_t)t.d_param & 3) || ((uintptr_t)t.d_grad & (t.grad_dtype == EC_BF16 ? 1 : 3)) || ((uintptr_t)t.d_copy & 1))
            return EC_E_INVAL;
        blocks += adamw_blocks(t.n);
        if (blocks > kAdamBlocks) return EC_E_UNSUPPORTED;
    }
    if (blocks > a->state_blocks) return EC_E_INVAL;
    if (blocks && (!a->d_m || !a->d_v || (((uintptr_t)a->d_m | (uintptr_t)a->d_v) & 15))) return EC_E_INVAL;
    if (coded && blocks && (!a->d_m_scale || !a->d_v_scale || (((uintptr_t)a->d_m_scale | (uintptr_t)a->d_v_scale) & 3)))
        return EC_E_INVAL;
    AdamArgs p;
    memset(&p, 0, sizeof(p));
    p.m = a->d_m;
    p.v = a->d_v;
    p.m_scale = a->d_m_scale;
    p.v_scale = a->d_v_scale;
    p.steps = a->d_steps;
    p.lr_at = a->d_lr;
    p.grad_scale = a->d_grad_scale;
    p.lr = (float)a->lr;
    p.b1 = (float)a->beta1;
    p.b2 = (float)a->beta2;
    p.rest1 = (float)(1.0 - a->beta1);
    p.rest2 = (float)(1.0 - a->beta2);
    p.log_b1 = (float)log(a->beta1);
    p.log_b2 = (float)log(a->beta2);
    p.eps = (float)a->eps;
    p.seed = a->seed;
    p.e4m3 = coded;
    AdamBatch batch(p, stream);
    uint64_t block = 0;
    hipError_t e = hipSuccess;
    for (uint32_t i = 0; i < count && e == hipSuccess; ++i) {
        const ec_adamw_tensor &t = tensors[i];
        e = batch.add(AdamTensor{t.d_param, t.d_grad, t.d_copy, t.n, block, t.weight_decay, t.grad_dtype == EC_BF16});
        block += adamw_blocks(t.n);
    }
    return hip_code(e == hipSuccess ? batch.finish() : e);
}
