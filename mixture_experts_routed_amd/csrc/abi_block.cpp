// C ABI of the operators around the routed layer's block (declared in
// include/moe_routed.h): routing by scores, norms with gate and residual. Argument
// checks on the host, then kernel launches on the caller's stream.
#include "checks.hpp"
#include "dense_checks.hpp"
#include "launch.hpp"

#include <math.h>

namespace {

// -> MOE_OK or an error: sizes as for moe_route_topk
int score_sizes(int score, int T, int E, int K, float scale)
{
    if (T < 1 || E < 1 || K < 1 || K > E) return MOE_EINVAL;
    if (E > MOE_MAX_EXPERTS || K > MOE_ROUTE_MAX_K) return MOE_EUNSUPPORTED;
    if ((int64_t)T * E > kI32Max * 4 || (int64_t)T * K > kI32Max) return MOE_EINVAL;
    if ((score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || !isfinite(scale))
        return MOE_EINVAL;
    return MOE_OK;
}

int norm_sizes(int T, int d)
{
    if (T < 1 || d < 1 || T > kI32Max - 1024) return MOE_EINVAL;
    return d > MOE_NORM_MAX_D ? MOE_EUNSUPPORTED : MOE_OK;
}

// an operand of a row-major [T][d] matrix, and one that may be left out
bool matrix_ok(const void *p, int d, int64_t ld) { return aligned(p, 16) && rows_ok(d, ld); }
bool matrix_or_null(const void *p, int d, int64_t ld) { return !p || matrix_ok(p, d, ld); }

// the gate's pointer, kind and stride; it goes with y
bool gate_ok(const void *gate, int64_t ld, int kind, const void *y, int d)
{
    if (kind < MOE_GATE_NONE || kind > MOE_GATE_FULL || (gate != nullptr) != (kind != MOE_GATE_NONE))
        return false;
    return !gate || (y && aligned(gate, 16) && (kind != MOE_GATE_FULL || rows_ok(d, ld)));
}

}  // namespace

extern "C" {

int moe_route_scored(const float *logits, const float *bias, int score, int T, int E, int K,
                     int groups, int keep, int group_top, int renorm, float scale, int32_t *ids,
                     float *w, moe_stream_t stream)
{
    const int rc = score_sizes(score, T, E, K, scale);
    if (rc != MOE_OK) return rc;
    if (groups < 1 || E % groups || keep < 1 || keep > groups || group_top < 1 ||
        group_top > E / groups || K > keep * (E / groups))
        return MOE_EINVAL;
    if (groups > MOE_SCORE_MAX_GROUPS || group_top > 2) return MOE_EUNSUPPORTED;
    if (!aligned(logits, 4) || !aligned_or_null(bias, 4) || !aligned(ids, 4) || !aligned(w, 4))
        return MOE_EINVAL;
    if (!apart_from(ids, {logits, bias, w}) || !apart_from(w, {logits, bias})) return MOE_EINVAL;
    moe::ScoreCall c;
    c.logits = logits;
    c.bias = bias;
    c.T = T;
    c.E = E;
    c.K = K;
    c.groups = groups;
    c.keep = keep;
    c.group_top = group_top;
    c.sigmoid = score == MOE_SCORE_SIGMOID;
    c.renorm = renorm != 0;
    c.scale = scale;
    c.ids = ids;
    c.w = w;
    return moe::launch_route_scored(c, as_stream(stream)) == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_route_scored_backward(const float *logits, const int32_t *ids, const float *dw,
                              const void *add, int score, int T, int E, int K, int renorm,
                              float scale, void *dlogits, int dtype, moe_stream_t stream)
{
    const int rc = score_sizes(score, T, E, K, scale);
    if (rc != MOE_OK) return rc;
    if (!dtype_ok(dtype)) return MOE_EINVAL;
    const size_t es = (size_t)elem_bytes(dtype);
    if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(dw, 4) || !aligned(dlogits, es) ||
        !aligned_or_null(add, es))
        return MOE_EINVAL;
    if (!apart_from(dlogits, {logits, ids, dw})) return MOE_EINVAL;
    moe::ScoreBackwardCall c;
    c.logits = logits;
    c.dw = dw;
    c.ids = ids;
    c.add = add;
    c.dlogits = dlogits;
    c.T = T;
    c.E = E;
    c.K = K;
    c.dtype = dtype;
    c.sigmoid = score == MOE_SCORE_SIGMOID;
    c.renorm = renorm != 0;
    c.scale = scale;
    return moe::launch_route_scored_backward(c, as_stream(stream)) == hipSuccess ? MOE_OK
                                                                                 : MOE_EHIP;
}

int moe_norm(const void *r, int64_t ldr, int r_dtype, const void *y, int64_t ldy, int y_dtype,
             const void *w_post, const void *gate, int64_t ldgate, int gate_kind,
             const void *w_pre, int dtype, int T, int d, float alpha, float eps, void *z,
             int64_t ldz, void *h, int64_t ldh, float *stats, moe_stream_t stream)
{
    const int rc = norm_sizes(T, d);
    if (rc != MOE_OK) return rc;
    if (!dtype_ok(dtype) || !result_ok(r_dtype, dtype) || (y && !result_ok(y_dtype, dtype)) ||
        !isfinite(alpha) || !(eps >= 7.888609052210118e-31f) || !isfinite(eps))  // 2^-100
        return MOE_EINVAL;
    if (!matrix_ok(r, d, ldr) || !matrix_or_null(y, d, ldy) || !matrix_or_null(z, d, ldz) ||
        !matrix_or_null(h, d, ldh) || !aligned_or_null(w_post, 16) || !aligned_or_null(w_pre, 16) ||
        !aligned_or_null(stats, 4) || !gate_ok(gate, ldgate, gate_kind, y, d))
        return MOE_EINVAL;
    // what goes together
    if ((!y && !w_pre) || (w_post && !y) || (z != nullptr) != (y != nullptr) ||
        (h != nullptr) != (w_pre != nullptr))
        return MOE_EINVAL;
    if (!apart_from(z, {y, w_post, gate, w_pre, h, stats}) ||
        !apart_from(h, {r, w_post, gate, w_pre, stats}) ||
        !apart_from(stats, {r, y, w_post, gate, w_pre}))
        return MOE_EINVAL;
    if (!in_place_ok(z, ldz, r, ldr, T) || !in_place_ok(h, ldh, y, ldy, T) ||
        (h && h == y && y_dtype != dtype))
        return MOE_EINVAL;
    moe::NormCall c;
    c.r = r;
    c.y = y;
    c.w_post = w_post;
    c.gate = gate;
    c.w_pre = w_pre;
    c.z = z;
    c.h = h;
    c.stats = stats;
    c.ldr = ldr;
    c.ldy = ldy;
    c.ldgate = ldgate;
    c.ldz = ldz;
    c.ldh = ldh;
    c.dtype = dtype;
    c.T = T;
    c.d = d;
    c.gate_kind = gate_kind;
    c.r32 = r_dtype == MOE_F32;
    c.y32 = y && y_dtype == MOE_F32;
    c.alpha = alpha;
    c.eps = eps;
    return moe::launch_norm(c, as_stream(stream)) == hipSuccess ? MOE_OK : MOE_EHIP;
}

int moe_norm_backward_workspace(int T, int d, size_t *bytes)
{
    if (!bytes) return MOE_EINVAL;
    const int rc = norm_sizes(T, d);
    if (rc == MOE_OK) *bytes = moe::norm_backward_workspace(T, d);
    return rc;
}

int moe_norm_backward(const void *dz, int64_t lddz, const void *dh, int64_t lddh, const void *z,
                      int64_t ldz, int r_dtype, const void *y, int64_t ldy, int y_dtype,
                      const void *w_post, const void *gate, int64_t ldgate, int gate_kind,
                      const void *w_pre, const float *stats, int dtype, int T, int d, float alpha,
                      void *workspace, size_t ws_bytes, void *dr, int64_t lddr, void *dy,
                      int64_t lddy, void *dgate, int64_t lddgate, void *dw_post, void *dw_pre,
                      int grad_dtype, moe_stream_t stream)
{
    size_t need = 0;
    const int rc = moe_norm_backward_workspace(T, d, &need);
    if (rc != MOE_OK) return rc;
    if (!dtype_ok(dtype) || !result_ok(r_dtype, dtype) || (y && !result_ok(y_dtype, dtype)) ||
        !result_ok(grad_dtype, dtype) || !isfinite(alpha))
        return MOE_EINVAL;
    if (!matrix_or_null(dz, d, lddz) || !matrix_or_null(dh, d, lddh) || !matrix_or_null(y, d, ldy) ||
        !matrix_ok(z, d, ldz) || !matrix_ok(dr, d, lddr) || !matrix_or_null(dy, d, lddy) ||
        !aligned_or_null(w_post, 16) || !aligned_or_null(w_pre, 16) || !aligned(stats, 4) ||
        !aligned_or_null(dgate, 16) || !aligned_or_null(dw_post, 16) ||
        !aligned_or_null(dw_pre, 16) || !workspace_ok(workspace, ws_bytes, need) ||
        !gate_ok(gate, ldgate, gate_kind, y, d))
        return MOE_EINVAL;
    if (gate_kind == MOE_GATE_FULL && dgate && !rows_ok(d, lddgate)) return MOE_EINVAL;
    // what goes together
    if ((!y && !w_pre) || (w_post && !y) || (dh != nullptr) != (w_pre != nullptr) || (!dz && !dh) ||
        (dy && !y) || (dgate && !gate) || (dw_post && !w_post) || (dw_pre && !w_pre))
        return MOE_EINVAL;
    if (!apart_from(dr, {dh, z, y, w_post, gate, w_pre, stats, workspace, dy, dgate, dw_post, dw_pre}) ||
        !apart_from(dy, {dz, dh, z, y, w_post, gate, w_pre, stats, workspace, dgate, dw_post, dw_pre}) ||
        !apart_from(dgate, {dz, dh, z, y, w_post, gate, w_pre, stats, workspace, dw_post, dw_pre}) ||
        !apart_from(dw_post, {dz, dh, z, y, w_post, gate, w_pre, stats, workspace, dw_pre}) ||
        !apart_from(dw_pre, {dz, dh, z, y, w_post, gate, w_pre, stats, workspace}))
        return MOE_EINVAL;
    if (!in_place_ok(dr, lddr, dz, lddz, T)) return MOE_EINVAL;
    moe::NormBackwardCall c;
    c.dz = dz;
    c.dh = dh;
    c.z = z;
    c.y = y;
    c.w_post = w_post;
    c.gate = gate;
    c.w_pre = w_pre;
    c.stats = stats;
    c.dr = dr;
    c.dy = dy;
    c.dgate = dgate;
    c.dw_post = dw_post;
    c.dw_pre = dw_pre;
    c.lddz = lddz;
    c.lddh = lddh;
    c.ldz = ldz;
    c.ldy = ldy;
    c.ldgate = ldgate;
    c.lddr = lddr;
    c.lddy = lddy;
    c.lddgate = lddgate;
    c.dtype = dtype;
    c.T = T;
    c.d = d;
    c.gate_kind = gate_kind;
    c.r32 = r_dtype == MOE_F32;
    c.y32 = y && y_dtype == MOE_F32;
    c.grad32 = grad_dtype == MOE_F32;
    c.alpha = alpha;
    return moe::launch_norm_backward(c, workspace, as_stream(stream)) == hipSuccess ? MOE_OK
                                                                                    : MOE_EHIP;
}

}  // extern "C"
