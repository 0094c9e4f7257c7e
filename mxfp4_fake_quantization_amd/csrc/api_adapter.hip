// api_adapter.hip -- the extern "C" entry points of the low-rank adapters and of
// the gradient norm (include/mxfp4.h).  As in api.hip: arguments are validated on
// the host before anything is enqueued, the kernels run on the caller's stream,
// nothing is allocated or synchronized.
#include "adapter_kernels.h"
#include "api_common.h"
#include "grad_norm_kernels.h"
#include "mxfp4_kernels.h"

#include <algorithm>
#include <new>
#include <vector>

using namespace mxfp4_api;

namespace {

constexpr int64_t kMostFeatures = (int64_t)1 << 24, kMostTokens = (int64_t)1 << 26;

mxfp4_status_t check_adapter(const mxfp4_adapter_t *d) {
  if (!d) return fail(MXFP4_EINVAL, "desc is NULL");
  MXFP4_TRY(check_dtype(d->dtype));
  if (d->reserved != 0) return fail(MXFP4_EINVAL, "reserved fields must be 0");
  if (d->rank < 1 || d->rank > mxfp4::kAdapterMaxRank)
    return fail(MXFP4_EUNSUPPORTED, "rank %d is not in [1, %d]", d->rank, mxfp4::kAdapterMaxRank);
  if (d->adapters < 1) return fail(MXFP4_EINVAL, "adapters %d is below 1", d->adapters);
  if (d->tokens < 0 || d->tokens > kMostTokens)
    return fail(d->tokens < 0 ? MXFP4_EINVAL : MXFP4_EUNSUPPORTED, "tokens %lld is not in [0, 2^26]",
                (long long)d->tokens);
  if (d->in_features < 1 || d->out_features < 1)
    return fail(MXFP4_EINVAL, "in_features %lld and out_features %lld must be >= 1", (long long)d->in_features,
                (long long)d->out_features);
  if (d->in_features > kMostFeatures || d->out_features > kMostFeatures)
    return fail(MXFP4_EUNSUPPORTED, "in_features and out_features above 2^24 are not supported");
  // A launch has below 2^32 threads: 256 for each of the second product's tiles.  (The first
  // product has a workgroup for each 64 rows, or some 2048 where that is more.)
  const int64_t most = d->in_features > d->out_features ? d->in_features : d->out_features;
  const int64_t rows = mxfp4::kAdapterLeastRows, cols = mxfp4::kAdapterLeastCols;
  if ((d->tokens + rows - 1) / rows * ((most + cols - 1) / cols) >= (int64_t)1 << 24)
    return fail(MXFP4_EUNSUPPORTED, "%lld tokens of %lld features are more than one call takes", (long long)d->tokens,
                (long long)most);
  return MXFP4_OK;
}

mxfp4_status_t check_rows(const void *p, int64_t ld, int64_t cols, int32_t dtype, const char *what) {
  MXFP4_TRY(check_elems(p, dtype, what));
  if (ld < cols || ld > (int64_t)1 << 26)
    return fail(MXFP4_EINVAL, "%s: %lld elements between rows of %lld", what, (long long)ld, (long long)cols);
  return MXFP4_OK;
}

mxfp4_status_t check_space(const void *workspace, int64_t have, int64_t need) {
  if (need == 0) return MXFP4_OK;
  MXFP4_TRY(check_ptr(workspace, 16, "workspace"));
  if (have < need)
    return fail(MXFP4_EINVAL, "workspace holds %lld bytes; the call needs %lld", (long long)have, (long long)need);
  return MXFP4_OK;
}

// Workgroups of the weight gradients' launches, 256 threads each: pieces by columns, and 256 elements of
// the summed gradients; a launch has below 2^32 threads.
mxfp4_status_t check_trained(const mxfp4_adapter_t *d) {
  if (d->adapters > mxfp4::kAdapterMaxTrained)
    return fail(MXFP4_EUNSUPPORTED, "the backward pass takes up to %d adapters, got %d", mxfp4::kAdapterMaxTrained,
                d->adapters);
  const int64_t sum = d->in_features + d->out_features;
  const int64_t pieces = d->tokens / 128 + (d->adapters < d->tokens ? d->adapters : d->tokens);
  if (pieces * (sum / 64 + 2) >= (int64_t)1 << 24 || d->adapters * (d->rank * sum / 256 + 2) >= (int64_t)1 << 24)
    return fail(MXFP4_EUNSUPPORTED, "%d adapters of %lld features and %lld tokens are more than one call takes",
                d->adapters, (long long)sum, (long long)d->tokens);
  return MXFP4_OK;
}

// What clipping writes must not meet: a tensor given twice would be scaled twice, in an order that
// hangs on the workgroups.  (The sort of 448 tensors in no order takes 14 us of the host's time.)
struct Span {
  uintptr_t lo, hi;
  bool read;  // a gradient with its output elsewhere: may meet another one
};
bool meets(const std::vector<Span> &spans) {
  uintptr_t any = 0, written = 0;
  for (const Span &s : spans) {
    if (s.lo < (s.read ? written : any)) return true;
    any = std::max(any, s.hi);
    if (!s.read) written = std::max(written, s.hi);
  }
  return false;
}
mxfp4_status_t check_clip_spans(int32_t n, const mxfp4_grad_item_t *items, const float *norm, const void *workspace,
                                int64_t workspace_bytes) {
  try {
    std::vector<Span> spans;
    spans.reserve(2 * (size_t)n);
    const uintptr_t nlo = reinterpret_cast<uintptr_t>(norm), nhi = nlo + 4;
    const uintptr_t wlo = reinterpret_cast<uintptr_t>(workspace), whi = wlo + (uintptr_t)workspace_bytes;
    bool good = true;
    auto add = [&](const void *p, int64_t bytes, bool read) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      if (bytes == 0) return;
      const Span s{at, at + (uintptr_t)bytes, read};
      good = good && (s.hi <= nlo || s.lo >= nhi) && (s.hi <= wlo || s.lo >= whi);
      spans.push_back(s);
    };
    for (int32_t i = 0; i < n; ++i) {
      const int64_t bytes = items[i].count * (items[i].dtype == MXFP4_F32 ? 4 : 2);
      add(items[i].out, bytes, false);
      if (items[i].grad != items[i].out) add(items[i].grad, bytes, true);
    }
    auto before = [](const Span &a, const Span &b) { return a.lo < b.lo; };
    if (!std::is_sorted(spans.begin(), spans.end(), before)) std::sort(spans.begin(), spans.end(), before);
    if (!good || meets(spans)) return fail(MXFP4_EINVAL, "a clipped tensor overlaps another tensor, the norm or the workspace");
  } catch (const std::bad_alloc &) {
    return fail(MXFP4_EUNSUPPORTED, "no host memory to check %d tensors", n);
  }
  return MXFP4_OK;
}

mxfp4_status_t check_norm(int32_t norm_type, int32_t n, const mxfp4_grad_item_t *items, bool outs, int64_t *elements) {
  if (norm_type != MXNORM_INF && norm_type != MXNORM_L1 && norm_type != MXNORM_L2)
    return fail(MXFP4_EUNSUPPORTED, "norm_type %d is not MXNORM_INF, MXNORM_L1 or MXNORM_L2", norm_type);
  if (n < 0) return fail(MXFP4_EINVAL, "negative number of tensors %d", n);
  if (n > 0 && !items) return fail(MXFP4_EINVAL, "items is NULL");
  *elements = 0;
  for (int32_t i = 0; i < n; ++i) {
    const mxfp4_grad_item_t &t = items[i];
    MXFP4_TRY(check_dtype(t.dtype));
    if (t.reserved != 0) return fail(MXFP4_EINVAL, "reserved fields must be 0");
    if (t.count < 0 || t.count > INT64_MAX / 16 || *elements > INT64_MAX / 16 - t.count)
      return fail(MXFP4_EINVAL, "tensor %d holds %lld elements", i, (long long)t.count);
    if (t.count == 0) continue;
    *elements += t.count;
    MXFP4_TRY(check_elems(t.grad, t.dtype, "grad"));
    if (outs) MXFP4_TRY(check_elems(t.out, t.dtype, "out"));
  }
  return MXFP4_OK;
}

}  // namespace

extern "C" {

int64_t mxfp4_adapter_workspace(const mxfp4_adapter_t *desc) {
  if (check_adapter(desc) != MXFP4_OK) return -1;
  mxfp4::AdapterLaunch L{};
  L.dtype = desc->dtype;
  L.rank = desc->rank;
  L.adapters = desc->adapters;
  L.tokens = desc->tokens;
  L.in = desc->in_features;
  L.out = desc->out_features;
  return 4 * mxfp4::adapter_workspace(L);
}

mxfp4_status_t mxfp4_adapter_fwd(const mxfp4_adapter_t *desc, const void *x, int64_t ldx, const void *a, const void *b,
                                 const float *scale, const int32_t *ids, const void *base, int64_t ld_base, void *y,
                                 int64_t ldy, float *u, void *workspace, int64_t workspace_bytes, void *stream) {
  MXFP4_TRY(check_adapter(desc));
  const int32_t dt = desc->dtype;
  if (desc->tokens == 0) return ok();
  MXFP4_TRY(check_rows(x, ldx, desc->in_features, dt, "x"));
  MXFP4_TRY(check_elems(a, dt, "a"));
  MXFP4_TRY(check_elems(b, dt, "b"));
  MXFP4_TRY(check_opt(scale, 4, "scale"));
  MXFP4_TRY(check_opt(ids, 4, "ids"));
  if (base) MXFP4_TRY(check_rows(base, ld_base, desc->out_features, dt, "base"));
  MXFP4_TRY(check_rows(y, ldy, desc->out_features, dt, "y"));
  if (base == y && ld_base != ldy) return fail(MXFP4_EINVAL, "y over base needs the same row length");
  MXFP4_TRY(check_opt(u, 4, "u"));
  const int64_t need = mxfp4_adapter_workspace(desc);
  MXFP4_TRY(check_space(workspace, workspace_bytes, need));
  if (!apart({y, u, workspace}, {x, a, b, scale, ids, base == y ? nullptr : base}))
    return fail(MXFP4_EINVAL, "an output aliases an input or another output");
  mxfp4::AdapterLaunch L{dt,  desc->rank, desc->adapters, desc->tokens, desc->in_features, desc->out_features,
                         x,   ldx,        a,              b,            scale,             ids,
                         base, ld_base,   y,              ldy,          u,                 static_cast<float *>(workspace)};
  return hip_status(mxfp4::launch_adapter(L, static_cast<hipStream_t>(stream)), "adapter launch");
}

int64_t mxfp4_adapter_bwd_workspace(const mxfp4_adapter_t *desc, int32_t grad_a, int32_t grad_b) {
  if (check_adapter(desc) != MXFP4_OK || check_trained(desc) != MXFP4_OK) return -1;
  return mxfp4::adapter_bwd_workspace(desc->tokens, desc->in_features, desc->out_features, desc->rank, desc->adapters,
                                      grad_a != 0, grad_b != 0);
}

mxfp4_status_t mxfp4_adapter_bwd(const mxfp4_adapter_t *desc, const void *grad_y, int64_t ld_grad_y, const void *x,
                                 int64_t ldx, const void *a, const void *b, const float *scale, const int32_t *ids,
                                 const float *u, const void *base, int64_t ld_base, void *grad_x, int64_t ld_grad_x,
                                 void *grad_a, void *grad_b, void *workspace, int64_t workspace_bytes, void *stream) {
  MXFP4_TRY(check_adapter(desc));
  MXFP4_TRY(check_trained(desc));
  const int32_t dt = desc->dtype;
  if (!grad_a && !grad_b) {
    if (desc->tokens == 0) return ok();  // grad_x may be NULL because it is empty
    if (!grad_x) return fail(MXFP4_EINVAL, "no output given");
  }
  if (grad_a) MXFP4_TRY(check_elems(grad_a, dt, "grad_a"));
  if (grad_b) MXFP4_TRY(check_elems(grad_b, dt, "grad_b"));
  if (desc->tokens > 0) {
    MXFP4_TRY(check_rows(grad_y, ld_grad_y, desc->out_features, dt, "grad_y"));
    if (grad_a) MXFP4_TRY(check_rows(x, ldx, desc->in_features, dt, "x"));
    if (grad_x) MXFP4_TRY(check_elems(a, dt, "a"));
    MXFP4_TRY(check_elems(b, dt, "b"));
    MXFP4_TRY(check_opt(scale, 4, "scale"));
    MXFP4_TRY(check_opt(ids, 4, "ids"));
    if (grad_b) MXFP4_TRY(check_ptr(u, 4, "u"));
    if (grad_x) {
      MXFP4_TRY(check_rows(grad_x, ld_grad_x, desc->in_features, dt, "grad_x"));
      if (base) MXFP4_TRY(check_rows(base, ld_base, desc->in_features, dt, "base"));
      if (base == grad_x && ld_base != ld_grad_x)
        return fail(MXFP4_EINVAL, "grad_x over base needs the same row length");
    }
  }
  const int64_t need = mxfp4_adapter_bwd_workspace(desc, grad_a != nullptr, grad_b != nullptr);
  MXFP4_TRY(check_space(workspace, workspace_bytes, need));
  if (!apart({grad_x, grad_a, grad_b, workspace}, {grad_y, grad_a ? x : nullptr, a, b, scale, ids, grad_b ? u : nullptr,
                                                   base == grad_x ? nullptr : base}))
    return fail(MXFP4_EINVAL, "an output aliases an input or another output");
  mxfp4::AdapterBwdLaunch L{dt, desc->rank, desc->adapters, desc->tokens, desc->in_features, desc->out_features,
                            grad_y, ld_grad_y, x, ldx, a, b, scale, ids, u, base, ld_base, grad_x, ld_grad_x,
                            grad_a, grad_b, static_cast<uint8_t *>(workspace)};
  return hip_status(mxfp4::launch_adapter_bwd(L, static_cast<hipStream_t>(stream)), "adapter backward launch");
}

int64_t mxfp4_grad_norm_workspace(int32_t n, int64_t elements) {
  if (n < 0 || elements < 0 || elements > INT64_MAX / 16) return -1;
  return 8 * mxfp4::grad_norm_workspace(n, elements);
}

mxfp4_status_t mxfp4_grad_norm(int32_t norm_type, int32_t n, const mxfp4_grad_item_t *items, float *norm, void *workspace,
                               int64_t workspace_bytes, void *stream) {
  int64_t elements;
  MXFP4_TRY(check_norm(norm_type, n, items, false, &elements));
  MXFP4_TRY(check_ptr(norm, 4, "norm"));
  MXFP4_TRY(check_space(workspace, workspace_bytes, mxfp4_grad_norm_workspace(n, elements)));
  mxfp4::GradNormLaunch L{items, n, norm_type, static_cast<double *>(workspace), norm, false, false, 0.0f};
  return hip_status(mxfp4::launch_grad_norm(L, static_cast<hipStream_t>(stream)), "gradient norm launch");
}

mxfp4_status_t mxfp4_grad_clip(int32_t norm_type, int32_t n, const mxfp4_grad_item_t *items, float max_norm,
                               int32_t compute_norm, float *norm, void *workspace, int64_t workspace_bytes,
                               void *stream) {
  int64_t elements;
  MXFP4_TRY(check_norm(norm_type, n, items, true, &elements));
  if (compute_norm != 0 && compute_norm != 1) return fail(MXFP4_EINVAL, "compute_norm must be 0 or 1 (got %d)", compute_norm);
  if (!(max_norm >= 0.0f)) return fail(MXFP4_EINVAL, "max_norm must be >= 0 (got %g)", (double)max_norm);
  MXFP4_TRY(check_ptr(norm, 4, "norm"));
  const int64_t need = compute_norm ? mxfp4_grad_norm_workspace(n, elements) : 0;
  MXFP4_TRY(check_space(workspace, workspace_bytes, need));
  MXFP4_TRY(check_clip_spans(n, items, norm, workspace, need));
  mxfp4::GradNormLaunch L{items, n, norm_type, static_cast<double *>(workspace), norm, true, !compute_norm, max_norm};
  return hip_status(mxfp4::launch_grad_norm(L, static_cast<hipStream_t>(stream)), "gradient clipping launch");
}

}  // extern "C"
