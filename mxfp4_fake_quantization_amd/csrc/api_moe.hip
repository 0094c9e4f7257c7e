// api_moe.hip -- the extern "C" entry points of the mixture-of-experts
// operators (include/mxfp4.h).  As in api.hip: arguments are validated on the
// host before anything is enqueued, the kernels run on the caller's stream,
// nothing is allocated or synchronized.
#include "api_common.h"
#include "moe_kernels.h"
#include "mxfp4_kernels.h"
#include "mxgemm_act.h"

using namespace mxfp4_api;

namespace {

mxfp4_status_t check_act(int32_t act) {
  if ((act < MXACT_NONE || act > MXACT_GELU) && act != MXACT_SWIGLU && act != MXACT_GEGLU)
    return fail(MXFP4_EUNSUPPORTED, "act %d is not one of the MXACT_ activations", act);
  return MXFP4_OK;
}

mxfp4_status_t check_route(const mxfp4_moe_route_t *d) {
  if (!d) return fail(MXFP4_EINVAL, "desc is NULL");
  MXFP4_TRY(check_dtype(d->dtype));
  if (d->score != MXMOE_SOFTMAX && d->score != MXMOE_SIGMOID)
    return fail(MXFP4_EINVAL, "score %d is not MXMOE_SOFTMAX or MXMOE_SIGMOID", d->score);
  if (d->renormalize != 0 && d->renormalize != 1)
    return fail(MXFP4_EINVAL, "renormalize must be 0 or 1 (got %d)", d->renormalize);
  if (d->tokens < 0) return fail(MXFP4_EINVAL, "negative tokens %lld", (long long)d->tokens);
  if (d->experts < 1 || d->experts > mxfp4::kRouteMaxExperts)
    return fail(MXFP4_EUNSUPPORTED, "experts %d is not in [1, %d]", d->experts, mxfp4::kRouteMaxExperts);
  if (d->k < 1 || d->k > mxfp4::kRouteMaxK || d->k > d->experts)
    return fail(MXFP4_EUNSUPPORTED, "k %d is not in [1, %d] or above the %d experts", d->k, mxfp4::kRouteMaxK,
                d->experts);
  if (d->num_groups < 1 || d->num_groups > mxfp4::kRouteMaxGroups || d->experts % d->num_groups != 0)
    return fail(MXFP4_EINVAL, "num_groups %d is not in [1, %d] or does not divide the %d experts", d->num_groups,
                mxfp4::kRouteMaxGroups, d->experts);
  if (d->topk_groups < 1 || d->topk_groups > d->num_groups)
    return fail(MXFP4_EINVAL, "topk_groups %d is not in [1, %d]", d->topk_groups, d->num_groups);
  if ((int64_t)d->topk_groups * (d->experts / d->num_groups) < d->k)
    return fail(MXFP4_EINVAL, "%d groups of %d experts hold fewer than k = %d", d->topk_groups,
                d->experts / d->num_groups, d->k);
  if (d->tokens > INT64_MAX / 8 / d->experts) return fail(MXFP4_EINVAL, "tokens * experts overflows");
  if (d->reserved != 0) return fail(MXFP4_EINVAL, "reserved fields must be 0");
  return MXFP4_OK;
}

mxfp4_status_t check_slots(int64_t tokens, int32_t k, int64_t cols, int64_t n_rows, const char *what) {
  if (tokens < 0 || cols < 0 || n_rows < 0)
    return fail(MXFP4_EINVAL, "negative shape: tokens %lld, cols %lld, %s %lld", (long long)tokens, (long long)cols,
                what, (long long)n_rows);
  if (k < 1 || k > mxfp4::kRouteMaxK)
    return fail(MXFP4_EUNSUPPORTED, "k %d is not in [1, %d]", k, mxfp4::kRouteMaxK);
  const int64_t most = tokens > n_rows ? tokens : n_rows;
  if (cols > 0 && most > INT64_MAX / 8 / cols) return fail(MXFP4_EINVAL, "rows * cols overflows");
  if (n_rows > INT32_MAX) return fail(MXFP4_EUNSUPPORTED, "%s %lld is above 2^31 - 1", what, (long long)n_rows);
  return MXFP4_OK;
}

}  // namespace

extern "C" {

mxfp4_status_t mxfp4_moe_route(const mxfp4_moe_route_t *desc, const void *logits, const float *bias, float *weights,
                               int32_t *ids, void *stream) {
  MXFP4_TRY(check_route(desc));
  if (desc->tokens == 0) return ok();
  MXFP4_TRY(check_elems(logits, desc->dtype, "logits"));
  MXFP4_TRY(check_opt(bias, 4, "bias"));
  MXFP4_TRY(check_ptr(weights, 4, "weights"));
  MXFP4_TRY(check_ptr(ids, 4, "ids"));
  if (!apart({weights, ids}, {logits, bias})) return fail(MXFP4_EINVAL, "outputs alias each other or an input");
  mxfp4::RouteLaunch L{desc->dtype, desc->score, desc->renormalize, desc->tokens, desc->experts, desc->k,
                       desc->num_groups, desc->topk_groups, desc->scale, logits, bias, weights, ids};
  return hip_status(mxfp4::launch_route(L, static_cast<hipStream_t>(stream)), "routing launch");
}

mxfp4_status_t mxfp4_moe_route_bwd(const mxfp4_moe_route_t *desc, const float *grad_weights, const void *logits,
                                   const int32_t *ids, void *grad_logits, void *stream) {
  MXFP4_TRY(check_route(desc));
  if (desc->tokens == 0) return ok();
  MXFP4_TRY(check_ptr(grad_weights, 4, "grad_weights"));
  MXFP4_TRY(check_elems(logits, desc->dtype, "logits"));
  MXFP4_TRY(check_ptr(ids, 4, "ids"));
  MXFP4_TRY(check_elems(grad_logits, desc->dtype, "grad_logits"));
  if (!apart({grad_logits}, {grad_weights, logits, ids})) return fail(MXFP4_EINVAL, "grad_logits aliases an input");
  mxfp4::RouteBwdLaunch L{desc->dtype, desc->score, desc->renormalize, desc->tokens, desc->experts, desc->k,
                          desc->scale, grad_weights, logits, ids, grad_logits};
  return hip_status(mxfp4::launch_route_bwd(L, static_cast<hipStream_t>(stream)), "routing backward launch");
}

int64_t mxfp4_moe_plan_workspace(int64_t slots, int32_t experts) {
  if (slots < 0 || slots > INT32_MAX || experts < 1 || experts > mxfp4::kRouteMaxExperts) return -1;
  return 4 * mxfp4::plan_workspace(slots, experts);
}

mxfp4_status_t mxfp4_moe_plan(int64_t slots, int32_t experts, const int32_t *ids, int64_t *group_list, int32_t *rows,
                              void *workspace, int64_t workspace_bytes, void *stream) {
  if (slots < 0) return fail(MXFP4_EINVAL, "negative slots %lld", (long long)slots);
  if (slots > INT32_MAX) return fail(MXFP4_EUNSUPPORTED, "slots %lld is above 2^31 - 1", (long long)slots);
  if (experts < 1 || experts > mxfp4::kRouteMaxExperts)
    return fail(MXFP4_EUNSUPPORTED, "experts %d is not in [1, %d]", experts, mxfp4::kRouteMaxExperts);
  MXFP4_TRY(check_ptr(group_list, 8, "group_list"));
  if (slots > 0) {
    MXFP4_TRY(check_ptr(ids, 4, "ids"));
    MXFP4_TRY(check_ptr(rows, 4, "rows"));
  }
  const int64_t need = 4 * mxfp4::plan_workspace(slots, experts);
  if (need > 0) {
    MXFP4_TRY(check_ptr(workspace, 4, "workspace"));
    if (workspace_bytes < need)
      return fail(MXFP4_EINVAL, "workspace holds %lld bytes; the call needs %lld", (long long)workspace_bytes,
                  (long long)need);
  }
  if (!apart({group_list, rows, need > 0 ? workspace : nullptr}, {ids}))
    return fail(MXFP4_EINVAL, "outputs alias each other or ids");
  mxfp4::PlanLaunch L{slots, experts, ids, group_list, rows, static_cast<int32_t *>(workspace)};
  return hip_status(mxfp4::launch_plan(L, static_cast<hipStream_t>(stream)), "plan launch");
}

mxfp4_status_t mxfp4_moe_dispatch(const mxfp4_desc_t *desc, int32_t fmt, const void *x, const int32_t *rows, int32_t k,
                                  int64_t out_rows, void *y, uint8_t *q, uint8_t *scales, void *stream) {
  int64_t n;
  MXFP4_TRY(check_desc(desc, false, &n));
  MXFP4_TRY(check_slots(desc->rows, k, desc->cols, out_rows, "out_rows"));
  if (q && fmt != MXFP8_E4M3 && fmt != MXFP8_E5M2)
    return fail(MXFP4_EINVAL, "fmt %d is not MXFP8_E4M3 or MXFP8_E5M2", fmt);
  if (n == 0 || out_rows == 0) return ok();  // an array without elements may be NULL
  if (!y && !q) return fail(MXFP4_EINVAL, "no output given");
  if (!q != !scales) return fail(MXFP4_EINVAL, "q and scales come together");
  MXFP4_TRY(check_elems(x, desc->dtype, "x"));
  MXFP4_TRY(check_ptr(rows, 4, "rows"));
  if (y) MXFP4_TRY(check_elems(y, desc->dtype, "y"));
  if (!apart({y, q, scales}, {x, rows})) return fail(MXFP4_EINVAL, "outputs alias each other or an input");
  mxfp4::DispatchLaunch L{desc->dtype, fmt, desc->block, desc->rows, desc->cols, out_rows, k, x, rows, y, q, scales};
  return hip_status(mxfp4::launch_dispatch(L, static_cast<hipStream_t>(stream)), "dispatch launch");
}

mxfp4_status_t mxfp4_moe_combine(int32_t dtype, int64_t tokens, int64_t cols, int32_t k, int64_t in_rows, const void *h,
                                 const int32_t *rows, const float *weights, const void *residual, void *y,
                                 void *stream) {
  MXFP4_TRY(check_dtype(dtype));
  MXFP4_TRY(check_slots(tokens, k, cols, in_rows, "in_rows"));
  if (tokens == 0 || cols == 0) return ok();
  if (in_rows > 0) MXFP4_TRY(check_elems(h, dtype, "h"));
  MXFP4_TRY(check_ptr(rows, 4, "rows"));
  MXFP4_TRY(check_opt(weights, 4, "weights"));
  if (residual) MXFP4_TRY(check_elems(residual, dtype, "residual"));
  MXFP4_TRY(check_elems(y, dtype, "y"));
  // y may be the residual (the token's row is read before it is written)
  if (!apart({y}, {h, rows, weights, residual == y ? nullptr : residual}))
    return fail(MXFP4_EINVAL, "y aliases an input");
  mxfp4::CombineLaunch L{dtype, tokens, cols, in_rows, k, h, rows, weights, residual, y};
  return hip_status(mxfp4::launch_combine(L, static_cast<hipStream_t>(stream)), "combine launch");
}

mxfp4_status_t mxfp4_moe_combine_bwd(int32_t dtype, int64_t tokens, int64_t cols, int32_t k, int64_t in_rows,
                                     const void *grad_y, const void *h, const int32_t *rows, const float *weights,
                                     void *grad_h, float *grad_weights, void *stream) {
  MXFP4_TRY(check_dtype(dtype));
  MXFP4_TRY(check_slots(tokens, k, cols, in_rows, "in_rows"));
  const bool empty = cols == 0;  // every dot product is 0 then
  // no output elements: grad_h may be NULL because it is empty
  if (tokens == 0 || ((empty || in_rows == 0) && !grad_weights)) return ok();
  if (!grad_h && !grad_weights) return fail(MXFP4_EINVAL, "no output given");
  if (!empty) MXFP4_TRY(check_elems(grad_y, dtype, "grad_y"));
  MXFP4_TRY(check_ptr(rows, 4, "rows"));
  if (grad_weights && in_rows > 0 && !empty) MXFP4_TRY(check_elems(h, dtype, "h"));
  MXFP4_TRY(check_opt(weights, 4, "weights"));
  if (grad_h && in_rows > 0 && !empty) MXFP4_TRY(check_elems(grad_h, dtype, "grad_h"));
  MXFP4_TRY(check_opt(grad_weights, 4, "grad_weights"));
  if (!apart({grad_h, grad_weights}, {grad_y, grad_weights ? h : nullptr, rows, weights}))
    return fail(MXFP4_EINVAL, "outputs alias each other or an input");
  mxfp4::CombineBwdLaunch L{dtype, tokens, cols, in_rows, k, grad_y, h, rows, weights, grad_h, grad_weights};
  return hip_status(mxfp4::launch_combine_bwd(L, static_cast<hipStream_t>(stream)), "combine backward launch");
}

mxfp4_status_t mxfp4_grouped_matmul_act(int64_t M, int64_t N, int64_t K, const mxfp4_mx_operand_t *a,
                                        const mxfp4_mx_operand_t *b, const int64_t *group_list, int32_t num_groups,
                                        int32_t group_list_type, const mxfp4_epilogue_t *ep, int32_t out_dtype, void *c,
                                        int64_t ldc, void *stream) {
  if (M < 0 || N < 0 || K < 0) return fail(MXFP4_EINVAL, "negative shape");
  if (K % 32 != 0) return fail(MXFP4_EINVAL, "K %lld is not a multiple of 32", (long long)K);
  if (group_list && (num_groups < 1 || (group_list_type != 0 && group_list_type != 1)))
    return fail(MXFP4_EINVAL, "num_groups must be >= 1 and group_list_type 0 or 1");
  if (!ep) return fail(MXFP4_EINVAL, "epilogue is NULL");
  MXFP4_TRY(check_act(ep->act));
  if (ep->reserved != 0) return fail(MXFP4_EINVAL, "reserved fields must be 0");
  if (out_dtype != MXGEMM_OUT_BF16 && out_dtype != MXGEMM_OUT_F32)
    return fail(MXFP4_EUNSUPPORTED, "out_dtype %d is not MXGEMM_OUT_BF16 or MXGEMM_OUT_F32", out_dtype);
  const bool gated = ep->act & 4;
  const int32_t dtype = out_dtype == MXGEMM_OUT_F32 ? MXFP4_F32 : MXFP4_BF16;
  if (M == 0 || N == 0) return ok();
  if (K == 0) return fail(MXFP4_EUNSUPPORTED, "K must be > 0");
  MXFP4_TRY(check_opt(group_list, 8, "group_list"));
  MXFP4_TRY(check_operand(a, "a", true, K, 0, true));
  MXFP4_TRY(check_operand(b, "b", true, K, 0, false));
  if (b->fmt == MXGEMM_E5M2) return fail(MXFP4_EUNSUPPORTED, "b->fmt must be MXGEMM_E2M1 or MXGEMM_E4M3");
  // gated: the up rows are reached by 32-bit offsets from the gate rows
  if (gated && (N > (1 << 24) || (N + 256) * (b->ld > b->ld_scales ? b->ld : b->ld_scales) >= (int64_t)1 << 32))
    return fail(MXFP4_EUNSUPPORTED, "the gate half of b (N * ld) must stay below 2^32 bytes");
  MXFP4_TRY(check_elems(c, dtype, "c"));
  if (ldc < N) return fail(MXFP4_EINVAL, "ldc %lld < N %lld", (long long)ldc, (long long)N);
  MXFP4_TRY(check_opt(ep->bias, 4, "bias"));
  if (ep->bias_stride < 0) return fail(MXFP4_EINVAL, "bias_stride must be >= 0");
  if (ep->residual) {
    MXFP4_TRY(check_elems(ep->residual, dtype, "residual"));
    if (ep->ld_residual < N) return fail(MXFP4_EINVAL, "ld_residual %lld < N %lld", (long long)ep->ld_residual, (long long)N);
    if (ep->residual == c && ep->ld_residual != ldc) return fail(MXFP4_EINVAL, "c over the residual needs the same ld");
  }
  if (ep->z) {
    MXFP4_TRY(check_elems(ep->z, dtype, "z"));
    if (ep->ld_z < (gated ? 2 : 1) * N)
      return fail(MXFP4_EINVAL, "ld_z %lld is below the %lld columns of z", (long long)ep->ld_z, (long long)((gated ? 2 : 1) * N));
  }
  if (!apart({c, ep->z}, {a->data, a->scales, b->data, b->scales, group_list, ep->bias,
                          ep->residual == c ? nullptr : ep->residual}))
    return fail(MXFP4_EINVAL, "an output aliases an input or another output");
  mxfp4::GemmLaunch L{};
  L.a_fmt = a->fmt;
  L.b_fmt = b->fmt;
  L.a_block = a->block;
  L.b_block = b->block;
  L.out_f32 = out_dtype == MXGEMM_OUT_F32;
  L.M = M;
  L.N = N;
  L.K = K;
  L.a = static_cast<const uint8_t *>(a->data);
  L.as = a->scales;
  L.b = static_cast<const uint8_t *>(b->data);
  L.bs = b->scales;
  L.lda = a->ld;
  L.ldas = a->ld_scales;
  L.ldb = b->ld;
  L.ldbs = b->ld_scales;
  L.b_gs = b->group_stride;
  L.b_gss = b->group_stride_scales;
  L.ldc = ldc;
  L.c = c;
  L.group_list = group_list;
  L.num_groups = group_list ? num_groups : 1;
  L.list_type = group_list_type;
  const mxfp4::ActArgs e{ep->bias, ep->bias_stride, ep->residual, ep->ld_residual, ep->z, ep->ld_z, ep->act & 3};
  return hip_status(mxfp4::launch_gemm_act(L, e, gated, static_cast<hipStream_t>(stream)), "grouped matmul launch");
}

int64_t mxfp4_act_bwd_workspace(int32_t act, int64_t rows, int64_t cols, int32_t num_groups) {
  if (check_act(act) != MXFP4_OK || rows < 0 || cols < 0 || num_groups < 0) return -1;
  const int64_t zc = cols * (act & 4 ? 2 : 1);
  if (zc > 0 && rows / 32 + num_groups + 2 > INT64_MAX / 8 / zc) return -1;
  return 4 * mxfp4::act_bwd_workspace(rows, zc, num_groups);
}

mxfp4_status_t mxfp4_act_bwd(int32_t dtype, int32_t act, int64_t rows, int64_t cols, const void *grad_c, const void *z,
                             void *grad_z, float *grad_bias, const int64_t *group_list, int32_t num_groups,
                             int32_t group_list_type, void *workspace, int64_t workspace_bytes, void *stream) {
  MXFP4_TRY(check_dtype(dtype));
  MXFP4_TRY(check_act(act));
  if (rows < 0 || cols < 0) return fail(MXFP4_EINVAL, "negative shape %lld x %lld", (long long)rows, (long long)cols);
  if (cols > 0 && rows > INT64_MAX / 16 / cols) return fail(MXFP4_EINVAL, "rows * cols overflows");
  if (group_list && (num_groups < 1 || (group_list_type != 0 && group_list_type != 1)))
    return fail(MXFP4_EINVAL, "num_groups must be >= 1 and group_list_type 0 or 1");
  MXFP4_TRY(check_opt(group_list, 8, "group_list"));
  if (cols == 0 || (rows == 0 && !grad_bias)) return ok();
  if (rows > 0) {
    MXFP4_TRY(check_elems(grad_c, dtype, "grad_c"));
    MXFP4_TRY(check_elems(z, dtype, "z"));
    MXFP4_TRY(check_elems(grad_z, dtype, "grad_z"));
  }
  const int32_t groups = group_list ? num_groups : 0;
  if (grad_bias) {
    MXFP4_TRY(check_ptr(grad_bias, 4, "grad_bias"));
    const int64_t need = mxfp4_act_bwd_workspace(act, rows, cols, groups);
    if (need > 0) MXFP4_TRY(check_ptr(workspace, 4, "workspace"));
    if (workspace_bytes < need)
      return fail(MXFP4_EINVAL, "workspace holds %lld bytes; the call needs %lld", (long long)workspace_bytes,
                  (long long)need);
  }
  // plain activations: grad_z may be grad_c or z (an element is read before it is written)
  const bool in_place = !(act & 4);
  if (!apart({grad_z, grad_bias, grad_bias ? workspace : nullptr},
             {in_place && grad_z == grad_c ? nullptr : grad_c, in_place && grad_z == z ? nullptr : z, group_list}))
    return fail(MXFP4_EINVAL, "an output aliases an input or another output");
  mxfp4::ActBwdLaunch L{dtype, act, rows, cols, grad_c, z, grad_z, grad_bias, group_list, groups, group_list_type,
                        static_cast<float *>(workspace)};
  return hip_status(mxfp4::launch_act_bwd(L, static_cast<hipStream_t>(stream)), "activation backward launch");
}

}  // extern "C"
