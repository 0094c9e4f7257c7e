// mxgemm_act_launch.h -- launches of the tiled product with an epilogue; each
// epilogue form (EPI of mxgemm_tile.h) is instantiated in a source of its own.
#pragma once

#include "mxgemm_tile.h"

namespace mxfp4 {
namespace {

template <int AF, int BF, bool S4, bool SMALL, int EPI>
__global__ __launch_bounds__((GemmShape<BF, SMALL>::threads), (GemmShape<BF, SMALL>::per_cu)) void mxgemm_act_kernel(
    GemmArgs P, ActArgs E) {
  mxgemm_tile<AF, BF, S4, SMALL, EPI>(P, E);
}

template <int AF, int BF, bool SMALL, int EPI>
hipError_t act_tiles_one(const GemmArgs &a, const ActArgs &e, int64_t grid, hipStream_t st) {
  const dim3 block(GemmShape<BF, SMALL>::threads);
  if (a.s4)
    hipLaunchKernelGGL((mxgemm_act_kernel<AF, BF, true, SMALL, EPI>), dim3((unsigned)grid), block, 0, st, a, e);
  else
    hipLaunchKernelGGL((mxgemm_act_kernel<AF, BF, false, SMALL, EPI>), dim3((unsigned)grid), block, 0, st, a, e);
  return hipGetLastError();
}

// The tiles as in the plain product (row split): see gemm_launch.
template <int AF, int BF, int EPI>
hipError_t act_tiles(const GemmArgs &a0, const ActArgs &e, hipStream_t st) {
  GemmArgs a = a0;
  constexpr int64_t BM = GemmShape<BF>::BM, BNO = GemmShape<BF>::BN / (EPI == 2 ? 2 : 1);
  a.tiles_n = (a.N + BNO - 1) / BNO;
  a.tiles_m = (a.M + BM - 1) / BM + (a.gl ? a.G : 0);
  a.total = a.tiles_m * a.tiles_n;
  if (a.total > 0x7FFFFFFF) return hipErrorInvalidValue;
  a.ncu = device_cus();
  const int64_t half = a.ncu / 2;
  // Row order with its tail launch up to 32 tiles a row, wider ones in bands for
  // the weights' re-reads.  Measured, row order / bands: the tail's small tiles
  // save up to 40 % where the rounds are few (5000 rows in 8 groups, 2048 -> 2560,
  // 10 tiles a row, 50 / 82 us, -> 4864, 19 tiles, 94 / 125; 4099 rows, 4096 ->
  // 4095 98 / 157; 16384 rows, 7168 -> 2 x 2304, 18 tiles, 562 / 607), bands 1 - 5 %
  // where there are many (16384 rows, 2048 -> 4096, 16 tiles, 230 / 225, -> 8192,
  // 32 tiles, 421 / 408; 32768 rows, 2048 -> 7168, 28 tiles, 695 / 663).
  a.row_order = a.tiles_n <= 32;
  if (a.total > half || !a.row_order) {
    const hipError_t r = act_tiles_one<AF, BF, false, EPI>(a, e, a.total, st);
    if (r != hipSuccess) return r;
  }
  const int64_t small = 4 * (a.total < half ? a.total : half);
  return a.row_order ? act_tiles_one<AF, BF, true, EPI>(a, e, small, st) : hipSuccess;
}

template <int EPI>
hipError_t act_tiles_any(const GemmLaunch &L, const ActArgs &e, hipStream_t st) {
  const GemmArgs a = gemm_args(L);
  if (L.a_fmt == kFmtE4M3)
    return L.b_fmt == kFmtE2M1 ? act_tiles<kFmtE4M3, kFmtE2M1, EPI>(a, e, st) : act_tiles<kFmtE4M3, kFmtE4M3, EPI>(a, e, st);
  return L.b_fmt == kFmtE2M1 ? act_tiles<kFmtE5M2, kFmtE2M1, EPI>(a, e, st) : act_tiles<kFmtE5M2, kFmtE4M3, EPI>(a, e, st);
}

}  // namespace
}  // namespace mxfp4
