// mxgemm_act_kernels.hip -- the grouped MX product with bias, activation and
// residual on every column (256 x 256 tiles and their 128 x 128 tail).
#include "moe_kernels.h"
#include "mxgemm_act_launch.h"

namespace mxfp4 {

hipError_t launch_act_tiles(const GemmLaunch &L, const ActArgs &e, hipStream_t st) { return act_tiles_any<1>(L, e, st); }

}  // namespace mxfp4
