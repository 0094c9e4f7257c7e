// adapter_fwd_kernels.hip -- low-rank adapters of many requests beside a shared
// projection on gfx950: y[t] = base[t] + s_i B_i (A_i x[t]), i = ids[t].
#include "adapter_launch.h"

namespace mxfp4 {
int64_t adapter_workspace(int64_t tokens, int64_t in, int64_t out, int rank, int adapters, int dtype) {
  return tokens * rank * shrink_splits(tokens, in);
}

hipError_t launch_adapter(const AdapterLaunch &L, hipStream_t stream) {
  const int splits = shrink_splits(L.tokens, L.in);
  const bool keep = L.u != nullptr;
  float *u = splits == 1 && keep ? L.u : L.workspace;
  const int64_t part = L.tokens * L.rank;
  ShrinkArgs S{static_cast<const uint8_t *>(L.x), static_cast<const uint8_t *>(L.a), L.ids, nullptr, u, L.tokens, L.ldx,
               L.in, part, L.adapters, L.rank, splits, shrink_slots(L.tokens, L.adapters, splits),
               window_count(L.tokens)};
  hipError_t e = launch_shrink<false>(L.dtype, S, PlanArgs{}, stream);
  if (e != hipSuccess) return e;
  ExpandArgs E{u, static_cast<const uint8_t *>(L.b), L.ids, L.scale, static_cast<const uint8_t *>(L.base),
               static_cast<uint8_t *>(L.y), u == L.u ? nullptr : L.u, L.tokens, L.out, L.ld_base, L.ldy, part,
               L.adapters, L.rank, splits};
  return launch_expand<false>(L.dtype, E, stream);
}

}  // namespace mxfp4
