// mxgemm_gated_kernels.hip -- the grouped MX product with a gated activation:
// the gate and the up columns of an output in one tile.
#include "moe_kernels.h"
#include "mxgemm_act_launch.h"

namespace mxfp4 {

hipError_t launch_gated_tiles(const GemmLaunch &L, const ActArgs &e, hipStream_t st) { return act_tiles_any<2>(L, e, st); }

}  // namespace mxfp4
