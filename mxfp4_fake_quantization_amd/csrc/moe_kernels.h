// moe_kernels.h -- host-side launch descriptors of the mixture-of-experts
// kernels (routing, token permutation, the epilogue's backward).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxfp4 {

// Expert choice per token.  score: 0 softmax, 1 sigmoid.
constexpr int kRouteMaxExperts = 1024, kRouteMaxK = 64, kRouteMaxGroups = 64;
struct RouteLaunch {
  int dtype, score, renorm;
  int64_t tokens;
  int experts, k, groups, topk_groups;
  float scale;
  const void *logits;  // [tokens, experts]
  const float *bias;   // [experts] or NULL
  float *weights;      // [tokens, k]
  int32_t *ids;        // [tokens, k]
};
hipError_t launch_route(const RouteLaunch &L, hipStream_t stream);

struct RouteBwdLaunch {
  int dtype, score, renorm;
  int64_t tokens;
  int experts, k;
  float scale;
  const float *grad_weights;  // [tokens, k]
  const void *logits;
  const int32_t *ids;
  void *grad_logits;          // [tokens, experts]
};
hipError_t launch_route_bwd(const RouteBwdLaunch &L, hipStream_t stream);

// Slots (token, choice) -> rows in expert order, and rows per expert.
struct PlanLaunch {
  int64_t slots;
  int experts;
  const int32_t *ids;   // [slots]
  int64_t *group_list;  // [experts] counts
  int32_t *rows;        // [slots]
  int32_t *workspace;   // plan_workspace(slots, experts) int32
};
int64_t plan_workspace(int64_t slots, int experts);
hipError_t launch_plan(const PlanLaunch &L, hipStream_t stream);

// Token rows copied (y) and / or quantized to MXFP8 (q, scales) at their slots' rows.
struct DispatchLaunch {
  int dtype, fmt, block;  // fmt: 0 E4M3, 1 E5M2
  int64_t tokens, cols, out_rows;
  int k;
  const void *x;
  const int32_t *rows;  // [tokens, k]
  void *y;              // [out_rows, cols] or NULL
  uint8_t *q;           // [out_rows, cols] or NULL
  uint8_t *scales;      // [out_rows, ceil(cols / block)]
};
hipError_t launch_dispatch(const DispatchLaunch &L, hipStream_t stream);

struct CombineLaunch {
  int dtype;
  int64_t tokens, cols, in_rows;
  int k;
  const void *h;          // [in_rows, cols]
  const int32_t *rows;    // [tokens, k]
  const float *weights;   // [tokens, k] or NULL (1)
  const void *residual;   // [tokens, cols] or NULL
  void *y;                // [tokens, cols]
};
hipError_t launch_combine(const CombineLaunch &L, hipStream_t stream);

struct CombineBwdLaunch {
  int dtype;
  int64_t tokens, cols, in_rows;
  int k;
  const void *grad_y;
  const void *h;         // NULL when grad_weights is
  const int32_t *rows;
  const float *weights;  // NULL (1)
  void *grad_h;          // NULL: not wanted
  float *grad_weights;   // NULL: not wanted
};
hipError_t launch_combine_bwd(const CombineBwdLaunch &L, hipStream_t stream);

// The grouped MX product (rows-split groups) with its epilogue; act: kind
// (0 none, 1 relu, 2 silu, 3 gelu) + 4 for the gated form, in which B has 2 N rows.
struct GemmLaunch;
struct ActArgs;
hipError_t launch_act_tiles(const GemmLaunch &L, const ActArgs &e, hipStream_t stream);
hipError_t launch_gated_tiles(const GemmLaunch &L, const ActArgs &e, hipStream_t stream);
hipError_t launch_gemm_act(const GemmLaunch &L, const ActArgs &e, bool gated, hipStream_t stream);

// Backward of the epilogue: grad_z = grad_c * act'(z), and its column sums per group.
struct ActBwdLaunch {
  int dtype, act;
  int64_t rows, cols;     // cols: of grad_c; z and grad_z have twice as many when gated
  const void *grad_c, *z;
  void *grad_z;
  float *grad_bias;       // [groups, columns of z] or NULL
  const int64_t *group_list;
  int num_groups, list_type;
  float *workspace;       // act_bwd_workspace floats when grad_bias is given
};
int64_t act_bwd_workspace(int64_t rows, int64_t zcols, int num_groups);
hipError_t launch_act_bwd(const ActBwdLaunch &L, hipStream_t stream);

}  // namespace mxfp4
