// C ABI of the dense operators beside the routed layer (declared in
// include/moe_routed.h): argument checks on the host, then kernel launches on
// the caller's stream, as in abi.cpp.
#include "checks.hpp"
#include "launch.hpp"

#include <initializer_list>

namespace {

constexpr int64_t kMaxCols = (int64_t)1 << 20;  // row lengths and strides, elements

// a row-major [*][cols] operand with row stride ld
bool rows_ok(int64_t cols, int64_t ld) { return ld >= cols && ld <= kMaxCols; }

// an array that may be left out
bool aligned_or_null(const void *p, size_t a) { return !p || aligned(p, a); }

bool result_ok(int dtype, int operand) { return dtype == MOE_F32 || dtype == operand; }

bool act_ok(int act, int first) { return act >= first && act <= MOE_ACT_GELU; }

// an output that may be one of the inputs: element by element, so with the same stride
bool in_place_ok(const void *out, int64_t ldo, const void *in, int64_t ldi, int T)
{
    return !in || out != in || ldo == ldi || T == 1;
}

// outputs that are asked for lie apart
bool apart(const void *a, const void *b) { return !a || a != b; }

// an output that is asked for is none of a call's other arguments
bool apart_from(const void *out, std::initializer_list<const void *> others)
{
    for (const void *p : others)
        if (!apart(out, p)) return false;
    return true;
}

int linear_sizes(int T, int d, int n, int64_t ldx, int64_t ldw, int dtype)
{
    if (T < 1 || d < 1 || n < 1 || T > kI32Max - 1024 || !dtype_ok(dtype)) return MOE_EINVAL;
    if (!rows_ok(d, ldx) || !rows_ok(n, ldw)) return MOE_EINVAL;
    return MOE_OK;
}

int balance_sizes(int T, int E, int K)
{
    if (T < 1 || E < 1 || K < 1 || K > E) return MOE_EINVAL;
    if (E > MOE_MAX_EXPERTS || K > MOE_ROUTE_MAX_K) return MOE_EUNSUPPORTED;
    if ((int64_t)T * E > kI32Max * 4 || (int64_t)T * K > kI32Max) return MOE_EINVAL;
    return MOE_OK;
}

bool workspace_ok(const void *p, size_t have, size_t need)
{
    return need == 0 || (aligned(p, 256) && have >= need);
}

}  // namespace

extern "C" {

int moe_linear_workspace(int T, int d, int n, int64_t ldx, int64_t ldw, int dtype, size_t *bytes)
{
    if (!bytes) return MOE_EINVAL;
    const int rc = linear_sizes(T, d, n, ldx, ldw, dtype);
    if (rc == MOE_OK && !moe::linear_fits(T, n, d, dtype)) return MOE_EINVAL;
    if (rc == MOE_OK) *bytes = (size_t)moe::linear_space(T, d, n, ldx, ldw, dtype).total;
    return rc;
}

int moe_linear_shape(int M, int N, int K, int dtype, int *tile, int *split)
{
    if (!tile || !split || M < 1 || N < 1 || K < 1 || M > kI32Max - 1024 || N > kI32Max - 1024 ||
        K > kI32Max - 1024 || !dtype_ok(dtype))
        return MOE_EINVAL;
    moe::linear_shape(M, N, K, dtype, tile, split);
    return MOE_OK;
}

int moe_linear(const void *x, int64_t ldx, const void *w, int64_t ldw, const void *bias,
               const void *residual, int64_t ldr, int residual_dtype, int dtype, int act, int T,
               int d, int n, void *workspace, size_t ws_bytes, void *out, int64_t ldo,
               int out_dtype, moe_stream_t stream)
{
    size_t need = 0;
    const int rc = moe_linear_workspace(T, d, n, ldx, ldw, dtype, &need);
    if (rc != MOE_OK) return rc;
    if (!act_ok(act, MOE_ACT_NONE) || !result_ok(out_dtype, dtype) || !rows_ok(n, ldo))
        return MOE_EINVAL;
    if (residual && (!result_ok(residual_dtype, dtype) || !rows_ok(n, ldr))) return MOE_EINVAL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned_or_null(bias, 16) ||
        !aligned_or_null(residual, 16) || !workspace_ok(workspace, ws_bytes, need))
        return MOE_EINVAL;
    if (out == x || out == w || out == bias || (need && out == workspace)) return MOE_EINVAL;
    if (out == residual && (residual_dtype != out_dtype || (ldr != ldo && T > 1))) return MOE_EINVAL;
    moe::LinearCall c;
    c.x = x;
    c.w = w;
    c.bias = bias;
    c.residual = residual;
    c.out = out;
    c.ldx = ldx;
    c.ldw = ldw;
    c.ldr = residual ? ldr : n;
    c.ldo = ldo;
    c.dtype = dtype;
    c.res_dtype = residual ? residual_dtype : dtype;
    c.out_dtype = out_dtype;
    c.act = act;
    c.T = T;
    c.d = d;
    c.n = n;
    return moe::launch_linear(c, workspace, as_stream(stream)) == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_linear_backward_workspace(int T, int d, int n, int64_t ldx, int64_t ldw, int64_t lddz,
                                  int dtype, int grads, size_t *bytes)
{
    if (!bytes || grads < 1 || grads > (MOE_GRAD_X | MOE_GRAD_W | MOE_GRAD_BIAS)) return MOE_EINVAL;
    // the stride of an operand that the gradients do not read is not looked at
    const int rc = linear_sizes(T, d, n, grads & MOE_GRAD_W ? ldx : d, grads & MOE_GRAD_X ? ldw : n,
                                dtype);
    if (rc != MOE_OK) return rc;
    if (!rows_ok(n, lddz)) return MOE_EINVAL;
    if ((grads & MOE_GRAD_X && !moe::linear_fits(T, d, n, dtype)) ||
        (grads & MOE_GRAD_W && !moe::linear_fits(d, n, T, dtype)))
        return MOE_EINVAL;
    *bytes = (size_t)moe::linear_backward_space(T, d, n, ldx, ldw, lddz, dtype,
                                                grads & MOE_GRAD_X, grads & MOE_GRAD_W,
                                                grads & MOE_GRAD_BIAS)
                 .total;
    return MOE_OK;
}

int moe_linear_backward(const void *x, int64_t ldx, const void *w, int64_t ldw, const void *dz,
                        int64_t lddz, int dtype, int T, int d, int n, void *workspace,
                        size_t ws_bytes, void *dx, int64_t lddx, void *dw, int64_t lddw, void *db,
                        int grad_dtype, moe_stream_t stream)
{
    const int grads = (dx ? MOE_GRAD_X : 0) | (dw ? MOE_GRAD_W : 0) | (db ? MOE_GRAD_BIAS : 0);
    size_t need = 0;
    const int rc = moe_linear_backward_workspace(T, d, n, ldx, ldw, lddz, dtype, grads, &need);
    if (rc != MOE_OK) return rc;
    if (!aligned(dz, 16) || !workspace_ok(workspace, ws_bytes, need)) return MOE_EINVAL;
    if (dx && (!aligned(dx, 16) || !aligned(w, 16) || !rows_ok(d, lddx))) return MOE_EINVAL;
    if (dw && (!aligned(dw, 16) || !aligned(x, 16) || !rows_ok(n, lddw))) return MOE_EINVAL;
    if (db && !aligned(db, 16)) return MOE_EINVAL;
    if ((dw || db) && !result_ok(grad_dtype, dtype)) return MOE_EINVAL;
    for (const void *p : {(const void *)dx, (const void *)dw, (const void *)db})
        if (p && (p == dz || (dw && p == x) || (dx && p == w) || (need && p == workspace)))
            return MOE_EINVAL;
    if (!apart(dx, dw) || !apart(dx, db) || !apart(dw, db)) return MOE_EINVAL;
    moe::LinearBackwardCall c;
    c.x = x;
    c.w = w;
    c.dz = dz;
    c.dx = dx;
    c.dw = dw;
    c.db = db;
    c.ldx = ldx;
    c.ldw = ldw;
    c.lddz = lddz;
    c.lddx = lddx;
    c.lddw = lddw;
    c.dtype = dtype;
    c.grad_dtype = grad_dtype;
    c.T = T;
    c.d = d;
    c.n = n;
    return moe::launch_linear_backward(c, workspace, as_stream(stream)) == hipSuccess ? MOE_OK
                                                                                      : MOE_EHIP;
}

int moe_balance_workspace(int T, int E, int K, size_t *bytes)
{
    if (!bytes) return MOE_EINVAL;
    const int rc = balance_sizes(T, E, K);
    if (rc == MOE_OK) *bytes = (size_t)moe::balance_workspace(T, E);
    return rc;
}

int moe_balance_loss(const float *logits, const int32_t *ids, int T, int E, int K, void *workspace,
                     size_t ws_bytes, int32_t *cnt, float *prob, float *loss, moe_stream_t stream)
{
    size_t need = 0;
    const int rc = moe_balance_workspace(T, E, K, &need);
    if (rc != MOE_OK) return rc;
    if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(cnt, 4) || !aligned(prob, 4) ||
        !aligned(loss, 4) || !workspace_ok(workspace, ws_bytes, need))
        return MOE_EINVAL;
    // (with one address for both inputs there are no results to keep apart)
    if (static_cast<const void *>(logits) != ids &&
        (!apart_from(cnt, {logits, ids, workspace, prob, loss}) ||
         !apart_from(prob, {logits, ids, workspace, loss}) ||
         !apart_from(loss, {logits, ids, workspace})))
        return MOE_EINVAL;
    return moe::launch_balance_loss(logits, ids, T, E, K, cnt, prob, loss, workspace,
                                    as_stream(stream)) == hipSuccess
               ? MOE_OK
               : MOE_EHIP;
}

int moe_route_backward(const float *logits, const int32_t *ids, const float *w, const float *dw,
                       const int32_t *cnt, const float *dloss, int T, int E, int K, void *dlogits,
                       int dtype, moe_stream_t stream)
{
    const int rc = balance_sizes(T, E, K);
    if (rc != MOE_OK) return rc;
    if (!dtype_ok(dtype) || (!dw && !dloss)) return MOE_EINVAL;
    if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(cnt, 4) ||
        !aligned(dlogits, (size_t)elem_bytes(dtype)) || !aligned_or_null(dw, 4) ||
        !aligned_or_null(dloss, 4) || (dw && !aligned(w, 4)))
        return MOE_EINVAL;
    if (!apart_from(dlogits, {logits, ids, dw, cnt, dloss}) || (dw && dlogits == w))
        return MOE_EINVAL;
    return moe::launch_route_backward(logits, ids, w, dw, cnt, dloss, T, E, K, dlogits, dtype,
                                      as_stream(stream)) == hipSuccess
               ? MOE_OK
               : MOE_EHIP;
}

int moe_act_forward(const void *g, int64_t ldg, const void *u, int64_t ldu, int dtype, int act,
                    int T, int f, void *h, int64_t ldh, uint8_t *g8, uint8_t *gs, uint8_t *u8,
                    uint8_t *us, moe_stream_t stream)
{
    if (T < 1 || f < 1 || !dtype_ok(dtype) || !act_ok(act, MOE_ACT_RELU)) return MOE_EINVAL;
    if (!rows_ok(f, ldg) || !rows_ok(f, ldh) || (u && !rows_ok(f, ldu))) return MOE_EINVAL;
    if (!aligned(g, 16) || !aligned_or_null(u, 16) || !aligned(h, 16)) return MOE_EINVAL;
    // a checkpoint is whole (codes and scales of g, and of u if there is one) or absent
    const bool keep = g8 != nullptr;
    if ((gs != nullptr) != keep || (u8 != nullptr) != (keep && u) || (us != nullptr) != (keep && u))
        return MOE_EINVAL;
    if (!aligned_or_null(g8, 16) || !aligned_or_null(u8, 16)) return MOE_EINVAL;
    if (!in_place_ok(h, ldh, g, ldg, T) || !in_place_ok(h, ldh, u, ldu, T) ||
        !apart_from(g8, {g, u, h, gs, u8, us}) || !apart_from(gs, {g, u, h, u8, us}) ||
        !apart_from(u8, {g, u, h, us}) || !apart_from(us, {g, u, h}))
        return MOE_EINVAL;
    return moe::launch_act_forward(g, ldg, u, ldu, dtype, act, T, f, h, ldh, g8, gs, u8, us,
                                   as_stream(stream)) == hipSuccess
               ? MOE_OK
               : MOE_EHIP;
}

int moe_act_backward(const uint8_t *g8, const uint8_t *gs, const uint8_t *u8, const uint8_t *us,
                     const void *dh, int64_t lddh, int dtype, int act, int T, int f, void *dg,
                     int64_t lddg, void *du, int64_t lddu, void *h, int64_t ldh,
                     moe_stream_t stream)
{
    if (T < 1 || f < 1 || !dtype_ok(dtype) || !act_ok(act, MOE_ACT_RELU)) return MOE_EINVAL;
    if (!rows_ok(f, lddh) || !rows_ok(f, lddg) || (h && !rows_ok(f, ldh))) return MOE_EINVAL;
    if (!aligned(g8, 16) || !gs || !aligned(dh, 16) || !aligned(dg, 16) || !aligned_or_null(h, 16))
        return MOE_EINVAL;
    // u's codes, scales and gradient go together
    if ((u8 != nullptr) != (us != nullptr) || (u8 != nullptr) != (du != nullptr)) return MOE_EINVAL;
    if (u8 && (!aligned(u8, 16) || !aligned(du, 16) || !rows_ok(f, lddu))) return MOE_EINVAL;
    if (!in_place_ok(dg, lddg, dh, lddh, T) || !in_place_ok(dh, lddh, du, lddu, T) ||
        !in_place_ok(dh, lddh, h, ldh, T) || !apart(dg, du) || !apart(dg, h) || !apart(du, h))
        return MOE_EINVAL;
    // (in place of dh, an output lies where dh lies)
    for (const void *out : {(const void *)dg, (const void *)du, (const void *)h})
        if (out != dh && !apart_from(out, {g8, gs, u8, us})) return MOE_EINVAL;
    return moe::launch_act_backward(g8, gs, u8, us, dh, lddh, dtype, act, T, f, dg, lddg, du, lddu,
                                    h, ldh, as_stream(stream)) == hipSuccess
               ? MOE_OK
               : MOE_EHIP;
}

}  // extern "C"
