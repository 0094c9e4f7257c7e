// api_common.h -- what the C-ABI sources share: the thread's error message, the
// pointer and shape checks, and the HIP status mapping.
#pragma once

#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>
#include <string>

#include <hip/hip_runtime.h>

#include "../../include/mxfp4.h"

namespace mxfp4_api {

inline std::string &last_error() {
  static thread_local std::string message;
  return message;
}

inline mxfp4_status_t fail(mxfp4_status_t st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  last_error() = buf;
  return st;
}

inline mxfp4_status_t ok() {
  last_error().clear();
  return MXFP4_OK;
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Common descriptor checks; sets *n to rows * cols.
inline mxfp4_status_t check_desc(const mxfp4_desc_t *d, bool need_rule, int64_t *n) {
  if (!d) return fail(MXFP4_EINVAL, "desc is NULL");
  if (d->dtype != MXFP4_BF16 && d->dtype != MXFP4_F32)
    return fail(MXFP4_EUNSUPPORTED, "dtype %d is not MXFP4_BF16 or MXFP4_F32", d->dtype);
  if (d->block != 32 && d->block != 128)
    return fail(MXFP4_EUNSUPPORTED, "block %d is not 32 or 128", d->block);
  if (d->reserved0 != 0 || d->reserved1 != 0) return fail(MXFP4_EINVAL, "reserved fields must be 0");
  if (d->rows < 0 || d->cols < 0) return fail(MXFP4_EINVAL, "negative shape %lld x %lld",
                                              (long long)d->rows, (long long)d->cols);
  if (d->cols > 0 && d->rows > INT64_MAX / 4 / d->cols)
    return fail(MXFP4_EINVAL, "rows * cols overflows");
  if (need_rule) {
    if (d->rule != MXFP4_RULE_FLOOR && d->rule != MXFP4_RULE_AMCT)
      return fail(MXFP4_EINVAL, "unknown rule %d", d->rule);
    if (d->rule == MXFP4_RULE_AMCT && !(d->scale_factor > 0.0f))
      return fail(MXFP4_EINVAL, "scale_factor must be > 0 (got %g)", (double)d->scale_factor);
  }
  *n = d->rows * d->cols;
  return MXFP4_OK;
}

inline mxfp4_status_t check_ptr(const void *p, uintptr_t align, const char *what) {
  if (!p) return fail(MXFP4_EINVAL, "%s is NULL", what);
  if (!aligned(p, align)) return fail(MXFP4_EINVAL, "%s is not %u-byte aligned", what, (unsigned)align);
  return MXFP4_OK;
}

inline mxfp4_status_t check_opt(const void *p, uintptr_t align, const char *what) {
  return p ? check_ptr(p, align, what) : MXFP4_OK;
}

inline mxfp4_status_t hip_status(hipError_t e, const char *what) {
  if (e != hipSuccess) return fail(MXFP4_EHIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

#define MXFP4_TRY(expr)                      \
  do {                                       \
    mxfp4_status_t st_ = (expr);             \
    if (st_ != MXFP4_OK) return st_;         \
  } while (0)

// Distinct non-NULL pointers (NULL entries are skipped).
inline bool distinct(std::initializer_list<const void *> ps) {
  const void *seen[16];
  int n = 0;
  for (const void *p : ps) {
    if (!p) continue;
    for (int i = 0; i < n; ++i)
      if (seen[i] == p) return false;
    seen[n++] = p;
  }
  return true;
}

inline mxfp4_status_t check_dtype(int32_t dtype) {
  if (dtype != MXFP4_BF16 && dtype != MXFP4_F32)
    return fail(MXFP4_EUNSUPPORTED, "dtype %d is not MXFP4_BF16 or MXFP4_F32", dtype);
  return MXFP4_OK;
}

// Outputs apart from each other and from every input (NULL entries are
// skipped); inputs may share memory.
inline bool apart(std::initializer_list<const void *> outs, std::initializer_list<const void *> ins) {
  if (!distinct(outs)) return false;
  for (const void *o : outs)
    for (const void *i : ins)
      if (o && o == i) return false;
  return true;
}

// Pointers of elements: aligned to one element.
inline mxfp4_status_t check_elems(const void *p, int32_t dtype, const char *what) {
  return check_ptr(p, dtype == MXFP4_F32 ? 4 : 2, what);
}

// One operand of the grouped products.
inline mxfp4_status_t check_operand(const mxfp4_mx_operand_t *o, const char *what, bool rows_split, int64_t K,
                             int64_t k_blocks, bool is_a) {
  if (!o) return fail(MXFP4_EINVAL, "%s is NULL", what);
  if (is_a ? (o->fmt != MXGEMM_E4M3 && o->fmt != MXGEMM_E5M2)
           : (o->fmt != MXGEMM_E4M3 && o->fmt != MXGEMM_E5M2 && o->fmt != MXGEMM_E2M1))
    return fail(MXFP4_EUNSUPPORTED, "%s->fmt %d is not supported", what, o->fmt);
  if (o->block != 32 && o->block != 128)
    return fail(MXFP4_EUNSUPPORTED, "%s->block %d is not 32 or 128", what, o->block);
  if (!rows_split && o->block != 32)
    return fail(MXFP4_EUNSUPPORTED, "%s->block must be 32 when groups split K", what);
  const int64_t kel = rows_split ? K : k_blocks * 32;  // K extent of a row
  if (kel > 0) {  // rows without elements are not read, and their arrays may be NULL
    MXFP4_TRY(check_ptr(o->data, 16, what));
    if (!o->scales) return fail(MXFP4_EINVAL, "%s->scales is NULL", what);
  }
  const int64_t row_bytes = o->fmt == MXGEMM_E2M1 ? kel / 2 : kel;
  const int64_t nblk = (kel + o->block - 1) / o->block;
  if (o->ld % 16 != 0 || o->ld < row_bytes)
    return fail(MXFP4_EINVAL, "%s->ld %lld must be a multiple of 16 and >= %lld", what, (long long)o->ld,
                (long long)row_bytes);
  if (o->ld > (int64_t)1 << 24) return fail(MXFP4_EUNSUPPORTED, "%s->ld is above 2^24 bytes", what);
  if (o->ld_scales < nblk || o->ld_scales > (int64_t)1 << 24)
    return fail(MXFP4_EINVAL, "%s->ld_scales %lld must be >= %lld (and below 2^24)", what,
                (long long)o->ld_scales, (long long)nblk);
  if (o->group_stride < 0 || o->group_stride_scales < 0 || o->group_stride % 16 != 0)
    return fail(MXFP4_EINVAL, "%s group strides must be >= 0 (data: a multiple of 16)", what);
  return MXFP4_OK;
}

}  // namespace mxfp4_api
