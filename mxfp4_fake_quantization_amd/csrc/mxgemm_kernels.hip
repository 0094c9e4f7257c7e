// mxgemm_kernels.hip -- the plain grouped MX matrix product: the kernels of
// mxgemm_tile.h without an epilogue, and their launches.
#include "mxgemm_tile.h"

namespace mxfp4 {
namespace {

template <int AF, int BF, bool S4, bool SMALL>
__global__ __launch_bounds__((GemmShape<BF, SMALL>::threads), (GemmShape<BF, SMALL>::per_cu)) void mxgemm_kernel(GemmArgs P) {
  mxgemm_tile<AF, BF, S4, SMALL, 0>(P, ActArgs{});
}

template <int AF, int BF, bool SMALL>
hipError_t gemm_launch_one(const GemmArgs &a, int64_t grid, hipStream_t st) {
  const dim3 block(GemmShape<BF, SMALL>::threads);
  if (a.s4)
    hipLaunchKernelGGL((mxgemm_kernel<AF, BF, true, SMALL>), dim3((unsigned)grid), block, 0, st, a);
  else
    hipLaunchKernelGGL((mxgemm_kernel<AF, BF, false, SMALL>), dim3((unsigned)grid), block, 0, st, a);
  return hipGetLastError();
}

template <int AF, int BF>
hipError_t gemm_launch(const GemmArgs &a0, hipStream_t st) {
  GemmArgs a = a0;
  constexpr int64_t BM = GemmShape<BF>::BM, BN = GemmShape<BF>::BN;
  static_assert(BM == 256 && BN == 256, "row-split tiles are 256 x 256 units");
  a.tiles_n = (a.N + BN - 1) / BN;
  if (a.group_type == 0) {
    // upper bound of the M tiles: every group adds at most one partial tile
    a.tiles_m = (a.M + BM - 1) / BM + (a.gl ? a.G : 0);
    a.total = a.tiles_m * a.tiles_n;
    if (a.total <= 0) return hipSuccess;
    if (a.total > 0x7FFFFFFF) return hipErrorInvalidValue;
    a.ncu = device_cus();
    const int64_t half = a.ncu / 2;
    // the big tiles (none when even the upper bound is a tail of at most
    // half a round), then, for rows of at most 8 N-tiles, the tail's small
    // tiles: 4 per big tile, at most half a round of big tiles (workgroups
    // without a tile return at once)
    a.row_order = a.tiles_n <= 8;
    if (a.total > half || !a.row_order) {
      const hipError_t e = gemm_launch_one<AF, BF, false>(a, a.total, st);
      if (e != hipSuccess) return e;
    }
    const int64_t small = 4 * (a.total < half ? a.total : half);
    return small > 0 && a.row_order ? gemm_launch_one<AF, BF, true>(a, small, st) : hipSuccess;
  }
  a.tiles_m = (a.M + BM - 1) / BM;
  a.total = a.tiles_m * a.tiles_n * a.G;
  if (a.total <= 0) return hipSuccess;
  if (a.total > 0x7FFFFFFF) return hipErrorInvalidValue;
  return gemm_launch_one<AF, BF, false>(a, a.total, st);
}

template <int AF>
hipError_t gemm_launch_b(int bf, const GemmArgs &a, hipStream_t st) {
  switch (bf) {
    case kFmtE4M3: return gemm_launch<AF, kFmtE4M3>(a, st);
    case kFmtE5M2: return gemm_launch<AF, kFmtE5M2>(a, st);
    default: return gemm_launch<AF, kFmtE2M1>(a, st);
  }
}

}  // namespace

hipError_t launch_mx_gemm(const GemmLaunch &L, hipStream_t st) {
  const GemmArgs a = gemm_args(L);
  return L.a_fmt == kFmtE4M3 ? gemm_launch_b<kFmtE4M3>(L.b_fmt, a, st) : gemm_launch_b<kFmtE5M2>(L.b_fmt, a, st);
}

}  // namespace mxfp4
