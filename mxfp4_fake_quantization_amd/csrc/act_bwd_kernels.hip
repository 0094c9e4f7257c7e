// act_bwd_kernels.hip -- backward of the product's epilogue on gfx950: the
// gradient through the activation, and the bias gradient per group.
//
//   dz = dc act'(z);   gated, z = (gate, up): dgate = dc up act'(gate),
//   dup = dc act(gate);   dbias_g = the sum of group g's rows of dz in fp32.
//   silu' = s (1 + x (1 - s)), s = 1 / (1 + exp(-x));  gelu' = Phi(x) + x phi(x)
//
// A workgroup takes a run of consecutive rows (of one group: the runs restart
// at every group start, as the grouped quantizers' blocks do) and 256 columns,
// 8 a lane, its rows eight at a time.  Each lane keeps its columns' sums, the
// lanes of a column meet in LDS, and a second launch adds the runs' sums in
// order: no atomics, the same bits every time.  Bound by the bytes of z, dc and
// dz.
#include "moe_kernels.h"
#include "mxfp4_groups.h"
#include "mxgemm_act.h"

namespace mxfp4 {
namespace {

constexpr int kActBwdThreads = 256;
// Rows of a run and lanes side by side (8 columns each), logarithms.  Small
// pieces spread evenly over the CUs: swiglu with bias on 32768 x 2 x 2048 takes
// 128 us (5.2 TB/s).  Measured when it took 138: 64-row runs 146, 64 lanes 151,
// 256 lanes of 64-row runs (two workgroups a CU and a few more) 176.
constexpr int kRunLog = 5, kColsLog = 5;

struct ActBwdArgs {
  const uint8_t *dc, *z;
  uint8_t *dz;
  float *part;  // [runs, zcols] or NULL
  const int64_t *gl;
  int64_t rows, cols, zcols;
  int G, list_type, act;
  int tx_log;       // lanes side by side in a row
  int64_t ctiles;   // column tiles
};

template <int ACT>
__device__ __forceinline__ float act_slope(float x, float *value) {
  if (ACT == kActRelu) {
    *value = x < 0.0f ? 0.0f : x;
    return x > 0.0f ? 1.0f : 0.0f;
  }
  if (ACT == kActSilu) {
    const float s = sigmoid_f(x);
    *value = x * s;
    return s * (1.0f + x * (1.0f - s));
  }
  if (ACT == kActGelu) {
    float gauss;
    const float cdf = normal_cdf(x, &gauss);
    *value = x * cdf;
    return fmaf(x * 0.398942280f, gauss, cdf);
  }
  *value = x;
  return 1.0f;
}

template <int DT, bool GATED, int ACT>
__global__ __launch_bounds__(kActBwdThreads) void act_bwd_kernel(ActBwdArgs A) {
  constexpr int ES = Row8<DT>::ES, NS = GATED ? 16 : 8;
  const int tx = threadIdx.x & ((1 << A.tx_log) - 1), ty = threadIdx.x >> A.tx_log;
  const int64_t ct = blockIdx.x % A.ctiles, run = blockIdx.x / A.ctiles;
  int64_t r0, len;
  if (A.gl) {
    block_row_uniform(A.gl, A.G, A.list_type, A.rows, kRunLog, run, &r0, &len);
  } else {
    r0 = run << kRunLog;
    len = A.rows - r0 < (1 << kRunLog) ? A.rows - r0 : 1 << kRunLog;
  }
  const int64_t c0 = ((ct << A.tx_log) + tx) * 8;
  const int n = A.cols - c0 >= 8 ? 8 : (A.cols > c0 ? (int)(A.cols - c0) : 0);
  float sum[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) sum[j] = 0.0f;
  const int step = kActBwdThreads >> A.tx_log;
#pragma unroll 2
  for (int64_t r = n ? r0 + ty : r0 + len; r < r0 + len; r += step) {
    uint32_t wd[Row8<DT>::NW], wz[Row8<DT>::NW], wu[Row8<DT>::NW];
    const int64_t zat = (r * A.zcols + c0) * ES;
    load8<DT>(wd, A.dc + (r * A.cols + c0) * ES, n);
    load8<DT>(wz, A.z + zat, n);
    if (GATED) load8<DT>(wu, A.z + zat + A.cols * ES, n);
    float f[8], fu[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float value;
      const float slope = act_slope<ACT>(elem<DT>(wz, j), &value);
      const float d = elem<DT>(wd, j);
      f[j] = GATED ? d * elem<DT>(wu, j) * slope : d * slope;
      fu[j] = d * value;
      sum[j] += f[j];
      if (GATED) sum[NS - 8 + j] += fu[j];
    }
    uint32_t o[Row8<DT>::NW];
    pack8<DT>(o, f);
    store8<DT>(A.dz + zat, o, n);
    if (GATED) {
      pack8<DT>(o, fu);
      store8<DT>(A.dz + zat + A.cols * ES, o, n);
    }
  }
  if (!A.part || len <= 0) return;  // the same for the workgroup
  __shared__ float meet[NS][kActBwdThreads];
#pragma unroll
  for (int j = 0; j < NS; ++j) meet[j][threadIdx.x] = sum[j];
  __syncthreads();
  // thread t adds the lanes of column t's partials, in row order
  const int width = 8 << A.tx_log;  // columns of the tile
  for (int t = threadIdx.x; t < (GATED ? 2 : 1) * width; t += kActBwdThreads) {
    const int up = t >= width ? 1 : 0, col = t - up * width;
    const int64_t c = (ct << A.tx_log) * 8 + col;
    if (c >= A.cols) continue;
    float s = 0.0f;
    for (int y = 0; y < step; ++y) s += meet[(8 * up + (col & 7)) % NS][(y << A.tx_log) + (col >> 3)];
    A.part[run * A.zcols + c + up * A.cols] = s;
  }
}

// dbias[g, c]: the sums of the group's runs.  64 columns a workgroup, a quarter
// of the runs each wave, in order, then the quarters in order (one thread a
// column for all runs took 20 us for 129 runs of 4096 columns, ahead of its
// loads' latency only).
__global__ __launch_bounds__(kActBwdThreads) void bias_sum_kernel(const float *part, const int64_t *gl, int G,
                                                                  int list_type, int64_t rows, int64_t zcols,
                                                                  int64_t ctiles, float *out) {
  __shared__ float quarter[kActBwdThreads / 64][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = (int)(blockIdx.x / ctiles);
  const int64_t c = (blockIdx.x % ctiles) * 64 + lane;
  int64_t first = 0, n = (rows + (1 << kRunLog) - 1) >> kRunLog;
  if (gl) group_block_span(gl, G, list_type, rows, kRunLog, g, &first, &n);
  const int64_t per = (n + 3) >> 2, lo = wave * per, hi = lo + per < n ? lo + per : n;
  float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (c < zcols) {
    const float *p = part + first * zcols + c;
    int64_t i = lo;
    for (; i + 8 <= hi; i += 8)
#pragma unroll
      for (int u = 0; u < 8; ++u) s[u] += p[(i + u) * zcols];
    for (; i < hi; ++i) s[0] += p[i * zcols];
  }
  quarter[wave][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  if (wave == 0 && c < zcols)
    out[(int64_t)g * zcols + c] = (quarter[0][lane] + quarter[1][lane]) + (quarter[2][lane] + quarter[3][lane]);
}

int64_t runs_of(int64_t rows, int groups) {  // at most: every group adds one partial run
  return ((rows + (1 << kRunLog) - 1) >> kRunLog) + groups;
}

template <int DT, bool GATED>
hipError_t act_bwd_launch(const ActBwdArgs &a, int64_t grid, hipStream_t st) {
  hipError_t r = hipErrorInvalidValue;
  switch (a.act) {
    case kActNone:
      if (!GATED) hipLaunchKernelGGL((act_bwd_kernel<DT, false, kActNone>), dim3((unsigned)grid), dim3(kActBwdThreads), 0, st, a);
      break;
    case kActRelu:
      if (!GATED) hipLaunchKernelGGL((act_bwd_kernel<DT, false, kActRelu>), dim3((unsigned)grid), dim3(kActBwdThreads), 0, st, a);
      break;
    case kActSilu:
      hipLaunchKernelGGL((act_bwd_kernel<DT, GATED, kActSilu>), dim3((unsigned)grid), dim3(kActBwdThreads), 0, st, a);
      break;
    default:
      hipLaunchKernelGGL((act_bwd_kernel<DT, GATED, kActGelu>), dim3((unsigned)grid), dim3(kActBwdThreads), 0, st, a);
  }
  r = hipGetLastError();
  return r;
}

}  // namespace

int64_t act_bwd_workspace(int64_t rows, int64_t zcols, int num_groups) { return runs_of(rows, num_groups) * zcols; }

hipError_t launch_act_bwd(const ActBwdLaunch &L, hipStream_t st) {
  ActBwdArgs a{};
  const bool gated = L.act & 4;
  a.dc = static_cast<const uint8_t *>(L.grad_c);
  a.z = static_cast<const uint8_t *>(L.z);
  a.dz = static_cast<uint8_t *>(L.grad_z);
  a.part = L.grad_bias ? L.workspace : nullptr;
  a.gl = L.group_list;
  a.rows = L.rows;
  a.cols = L.cols;
  a.zcols = L.cols * (gated ? 2 : 1);
  a.G = L.num_groups;
  a.list_type = L.list_type;
  a.act = L.act & 3;
  while (a.tx_log < kColsLog && (int64_t)(8 << a.tx_log) < L.cols) ++a.tx_log;
  a.ctiles = (L.cols + (8 << a.tx_log) - 1) / (8 << a.tx_log);
  const int64_t runs = a.gl ? runs_of(L.rows, L.num_groups) : (L.rows + (1 << kRunLog) - 1) >> kRunLog;
  const int64_t grid = runs * a.ctiles;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (grid > 0) {
    const hipError_t r = L.dtype == kBF16 ? (gated ? act_bwd_launch<kBF16, true>(a, grid, st) : act_bwd_launch<kBF16, false>(a, grid, st))
                                          : (gated ? act_bwd_launch<kF32, true>(a, grid, st) : act_bwd_launch<kF32, false>(a, grid, st));
    if (r != hipSuccess) return r;
  }
  if (!L.grad_bias) return hipSuccess;
  const int64_t bt = (a.zcols + 63) / 64;
  const int64_t groups = L.group_list ? L.num_groups : 1;
  if (bt * groups > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL(bias_sum_kernel, dim3((unsigned)(bt * groups)), dim3(kActBwdThreads), 0, st, a.part, L.group_list,
                     L.num_groups, L.list_type, L.rows, a.zcols, bt, L.grad_bias);
  return hipGetLastError();
}

}  // namespace mxfp4
