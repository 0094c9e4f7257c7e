// adapter_kernels.h -- host-side launch descriptors of the low-rank adapters'
// kernels and of the gradient norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxfp4 {

constexpr int kAdapterMaxRank = 128;
constexpr int kAdapterMaxTrained = 1024;  // adapters of a backward pass
// The second product's smallest tile, of 256 threads: what bounds a call's size (the kernel asserts it).
constexpr int kAdapterLeastRows = 32, kAdapterLeastCols = 256;

// y = base + s u B^T, u = x A^T, with the adapter of each row.
struct AdapterLaunch {
  int dtype, rank, adapters;
  int64_t tokens, in, out;
  const void *x;          // [tokens, ldx]
  int64_t ldx;
  const void *a;          // [adapters, rank, in]
  const void *b;          // [adapters, out, rank]
  const float *scale;     // [adapters] or NULL (1)
  const int32_t *ids;     // [tokens] or NULL (adapter 0)
  const void *base;       // [tokens, ld_base] or NULL
  int64_t ld_base;
  void *y;                // [tokens, ldy]
  int64_t ldy;
  float *u;               // [tokens, rank] or NULL
  float *workspace;       // adapter_workspace floats
};
int64_t adapter_workspace(const AdapterLaunch &L);  // by its sizes alone
hipError_t launch_adapter(const AdapterLaunch &L, hipStream_t stream);

struct AdapterBwdLaunch {
  int dtype, rank, adapters;
  int64_t tokens, in, out;
  const void *grad_y;     // [tokens, ld_gy]
  int64_t ld_gy;
  const void *x;          // [tokens, ldx]; NULL without grad_a
  int64_t ldx;
  const void *a, *b;
  const float *scale;
  const int32_t *ids;
  const float *u;         // [tokens, rank]; NULL without grad_b
  const void *base;       // added to grad_x, [tokens, ld_base], or NULL
  int64_t ld_base;
  void *grad_x;           // [tokens, ld_gx] or NULL
  int64_t ld_gx;
  void *grad_a, *grad_b;  // of a's and b's shape, or NULL
  uint8_t *workspace;     // adapter_bwd_workspace bytes
};
int64_t adapter_bwd_workspace(int64_t tokens, int64_t in, int64_t out, int rank, int adapters, bool grad_a, bool grad_b);
hipError_t launch_adapter_bwd(const AdapterBwdLaunch &L, hipStream_t stream);

}  // namespace mxfp4
