// moe_rows_kernels.hip -- tokens into expert order and back on gfx950.
//
// The experts' product takes the rows of expert 0, then of expert 1, ... (its
// group_list holds the counts).  The plan ranks the slots (token t, choice j)
// in that order, equal experts by slot: rows[t, j] is the slot's row, -1 for a
// slot without an expert.  Dispatch writes a token's row to its k rows (as it
// is, or as MXFP8, quantized once); combine sums a token's k rows with its
// weights.  Everything is addressed by token, so no kernel needs the inverse
// order and no sum uses atomics: results do not depend on timing.
#include "moe_kernels.h"
#include "mxfp4_device.h"
#include "mxfp4_kernels.h"
#include "mxfp4_rows8.h"

namespace mxfp4 {
namespace {

// ---- plan --------------------------------------------------------------------
//
// A stable counting sort by expert.  A workgroup of 16 waves takes a chunk of
// consecutive slots, each wave a consecutive part of it, 64 at a time: the
// lanes of a step that hold the same expert are found by one ballot per bit
// of the expert number, which gives a slot's rank among them, and the wave's
// running counts (one row of LDS counters per wave) the rank before the step.
// One chunk (up to kPlanOne slots): one launch.  More: a first launch counts
// every chunk, the second adds up the counts of the chunks before its own (one
// thread an expert, chunk after chunk, took 10 us of latency for 32 chunks).

constexpr int kPlanWaves = 16, kPlanThreads = 64 * kPlanWaves;
constexpr int64_t kPlanOne = 8192;
constexpr int kPlanMaxChunks = 256;

int64_t plan_chunk(int64_t slots) {
  if (slots <= kPlanOne) {  // as few steps a wave as there are
    const int64_t c = (slots + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
    return c < kPlanThreads ? kPlanThreads : c;
  }
  const int64_t per = (slots + kPlanMaxChunks - 1) / kPlanMaxChunks;
  const int64_t c = (per + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
  return c < 2048 ? 2048 : c;
}

struct PlanArgs {
  const int32_t *ids;
  int64_t *group_list;
  int32_t *rows, *hist;  // hist [chunks, experts]
  int64_t slots, chunk;
  int experts, bits, chunks;
};

__device__ __forceinline__ int plan_id(const PlanArgs &A, int64_t i, int64_t end) {
  if (i >= end) return A.experts;
  const int e = A.ids[i];
  return e >= 0 && e < A.experts ? e : A.experts;  // the last number: slots without an expert
}

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(PlanArgs A) {
  __shared__ int32_t cnt[kRouteMaxExperts];
  for (int e = threadIdx.x; e < A.experts; e += kPlanThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * A.chunk;
  const int64_t end = lo + A.chunk < A.slots ? lo + A.chunk : A.slots;
  for (int64_t i = lo + threadIdx.x; i < end; i += kPlanThreads) {
    const int e = plan_id(A, i, end);
    if (e < A.experts) atomicAdd(&cnt[e], 1);  // a count: the order of the additions does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < A.experts; e += kPlanThreads) A.hist[(int64_t)blockIdx.x * A.experts + e] = cnt[e];
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs A) {
  __shared__ int32_t cnt[kPlanWaves][kRouteMaxExperts];
  __shared__ int32_t sum[2][kRouteMaxExperts];
  __shared__ int32_t wsum[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid & 63; e < A.experts; e += 64) cnt[wave][e] = 0;
  if (tid < A.experts) sum[0][tid] = sum[1][tid] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * A.chunk;
  const int64_t end = lo + A.chunk < A.slots ? lo + A.chunk : A.slots;
  const int64_t part = A.chunk / kPlanWaves;  // a multiple of 64
  const int64_t wlo = lo + wave * part;
  const int64_t wend = wlo + part < end ? wlo + part : end;
  for (int64_t i = wlo + lane; i < wend; i += 64) {
    const int e = plan_id(A, i, wend);
    if (e < A.experts) atomicAdd(&cnt[wave][e], 1);
  }
  __syncthreads();
  // the chunks' counts, all threads over (chunk, expert): an expert's slots
  // before this chunk, and all of them (integer sums: any order)
  if (A.chunks > 1) {
    const int n = A.chunks * A.experts;
#pragma unroll 4
    for (int i = tid; i < n; i += kPlanThreads) {
      const int b = i / A.experts, e = i - b * A.experts;
      const int32_t c = A.hist[i];
      if (c) {
        atomicAdd(&sum[0][e], c);
        if (b < (int)blockIdx.x) atomicAdd(&sum[1][e], c);
      }
    }
    __syncthreads();
  }
  // expert e, one a thread
  int32_t before = 0, total = 0;
  if (tid < A.experts) {
    if (A.chunks > 1) {
      total = sum[0][tid];
      before = sum[1][tid];
    } else {
      for (int w = 0; w < kPlanWaves; ++w) total += cnt[w][tid];
    }
    if (blockIdx.x == 0) A.group_list[tid] = total;
  }
  // exclusive scan of the totals over the experts
  int32_t incl = total;
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int32_t at = incl - total + before;
  for (int w = 0; w < wave; ++w) at += wsum[w];
  if (tid < A.experts) {
    for (int w = 0; w < kPlanWaves; ++w) {
      const int32_t c = cnt[w][tid];
      cnt[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();
  // Every lane of a wave takes part in the ballots: the loop count is the wave's.
  for (int64_t base = wlo; base < wend; base += 64) {
    const int64_t i = base + lane;
    const int e = plan_id(A, i, wend);
    uint64_t same = ~0ull;
    for (int b = 0; b < A.bits; ++b) {
      const uint64_t on = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? on : ~on;
    }
    const uint64_t below = (1ull << lane) - 1;
    if (e < A.experts) {
      const int32_t first = cnt[wave][e];
      A.rows[i] = first + (int32_t)__popcll(same & below);
      // the group's last lane moves the count on (a wave's LDS operations keep
      // their order: the reads above come first)
      if ((same >> lane) == 1ull) cnt[wave][e] = first + (int32_t)__popcll(same);
    } else if (i < wend) {
      A.rows[i] = -1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- dispatch ------------------------------------------------------------------
//
// A workgroup takes 1024 elements of one token, 8 a lane, quantizes them once
// (the OCP MX rule of the row-wise MXFP8 kernel: E8M0 scale from the exponent
// of the block's largest magnitude, exact scaling, hardware conversion) and
// stores them to the token's k rows, 512 contiguous bytes a wave.  Bound by
// the bytes written.

struct DispatchArgs {
  const uint8_t *x;
  const int32_t *rows;
  uint8_t *y, *q, *scales;
  int64_t tokens, cols, nb, out_rows;
  int k, chunks;  // workgroups a row of tokens
  int tx_log;
};

constexpr int kDispatchThreads = 128, kDispatchLog = 7;

// Lanes of a workgroup: 2^tx_log side by side in a token's row, the tokens
// below each other.  WIDE: one token a workgroup, so slots are the same for all
// lanes and their rows and weights come by scalar loads, which the branches
// around them, taken lane by lane at the end of a row, do not touch.
typedef const int32_t __attribute__((address_space(4))) *scalar_i32;
typedef const float __attribute__((address_space(4))) *scalar_f32;

// Row of slot i, -1 outside [0, n), and its weight.
template <bool WIDE>
__device__ __forceinline__ int slot_row(const int32_t *rows, int64_t i, int64_t n) {
  const int r = WIDE ? ((scalar_i32)(uint64_t)rows)[i] : rows[i];
  return r >= 0 && r < n ? r : -1;
}
template <bool WIDE>
__device__ __forceinline__ float slot_weight(const float *weights, int64_t i) {
  if (!weights) return 1.0f;
  return WIDE ? ((scalar_f32)(uint64_t)weights)[i] : weights[i];
}

// log2 of the lanes side by side: as many as the row has 8-element pieces, at
// least 4 (a 32-element block), at most `most`.
int lanes_log(int64_t cols, int least, int most) {
  int l = least;
  while (l < most && ((int64_t)8 << l) < cols) ++l;
  return l;
}

template <int DT, int FMT, int G, bool WIDE>
__global__ __launch_bounds__(kDispatchThreads) void dispatch_kernel(DispatchArgs A) {
  constexpr int ES = Row8<DT>::ES;
  constexpr float MAXN = FMT == kE4M3 ? 448.0f : 57344.0f;
  constexpr int EMAX = FMT == kE4M3 ? 8 : 15;
  const int tx_log = WIDE ? kDispatchLog : A.tx_log;
  int64_t t = blockIdx.x / A.chunks;
  if (!WIDE) t = (t << (kDispatchLog - tx_log)) + (threadIdx.x >> tx_log);
  const int64_t c0 = ((int64_t)(blockIdx.x % A.chunks << tx_log) + (threadIdx.x & ((1 << tx_log) - 1))) * 8;
  const int64_t left = WIDE || t < A.tokens ? A.cols - c0 : 0;
  const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
  uint32_t w[Row8<DT>::NW];
  load8<DT>(w, A.x + (t * A.cols + c0) * ES, n);
  uint32_t lo = 0, hi = 0, e8 = 0;
  if (A.q) {
    uint32_t am = 0;
    if (DT == kBF16) {
      const uint32_t m = pk_max(pk_max(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                pk_max(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
      am = max32(m & 0xFFFFu, m >> 16) << 16;
    } else {
#pragma unroll
      for (int j = 0; j < Row8<DT>::NW; ++j) am = max32(am, w[j] & 0x7FFFFFFFu);
    }
    am = group_max<G>(am);
    const int eb = (int)(am >> 23);
    e8 = eb > EMAX ? (uint32_t)(eb - EMAX) : 0u;
    const float s = bits_f32((254u - e8) << 23);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_fmed3f(elem<DT>(w, j) * s, -MAXN, MAXN);
    auto two = [](float a, float b, uint32_t old, auto high) {
      constexpr bool HI = decltype(high)::value;
      return FMT == kE4M3 ? (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HI)
                          : (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(a, b, (int)old, HI);
    };
    lo = two(v[2], v[3], two(v[0], v[1], 0, std::false_type{}), std::true_type{});
    hi = two(v[6], v[7], two(v[4], v[5], 0, std::false_type{}), std::true_type{});
  }
  if (n == 0) return;
  const bool head = (threadIdx.x & (G - 1)) == 0;
  for (int j = 0; j < A.k; ++j) {
    const int64_t r = slot_row<WIDE>(A.rows, t * A.k + j, A.out_rows);
    if (r < 0) continue;
    if (A.y) store8<DT>(A.y + (r * A.cols + c0) * ES, w, n);
    if (A.q) {
      uint8_t *dst = A.q + r * A.cols + c0;
      if (n == 8) {
        const u32x2 pk = {lo, hi};
        __builtin_nontemporal_store(pk, reinterpret_cast<u32x2_a1 *>(dst));
      } else {
        const uint64_t pk = (uint64_t)lo | ((uint64_t)hi << 32);
        for (int b = 0; b < n; ++b) dst[b] = (uint8_t)(pk >> (8 * b));
      }
      if (head) A.scales[r * A.nb + c0 / (8 * G)] = (uint8_t)e8;
    }
  }
}

// ---- combine -------------------------------------------------------------------
//
// A lane sums 8 elements of a token over its k rows in 32 bits, in the order
// of the choices; the rows' loads are independent, eight in flight at a time.
// Bound by the bytes read.

struct CombineArgs {
  const uint8_t *h;
  const int32_t *rows;
  const float *weights;
  const uint8_t *residual;
  uint8_t *y;
  int64_t tokens, cols, in_rows;
  int k, chunks, tx_log;
};

constexpr int kCombineThreads = 128, kCombineLog = 7;
constexpr int kAhead = 8;

template <int DT, bool WIDE>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(CombineArgs A) {
  constexpr int ES = Row8<DT>::ES;
  const int tx_log = WIDE ? kCombineLog : A.tx_log;
  int64_t t = blockIdx.x / A.chunks;
  if (!WIDE) t = (t << (kCombineLog - tx_log)) + (threadIdx.x >> tx_log);
  if (!WIDE && t >= A.tokens) return;
  const int64_t c0 = ((int64_t)(blockIdx.x % A.chunks << tx_log) + (threadIdx.x & ((1 << tx_log) - 1))) * 8;
  const int64_t left = A.cols - c0;
  const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  for (int j0 = 0; j0 < A.k; j0 += kAhead) {
    uint32_t w[kAhead][Row8<DT>::NW];
    int r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      r[u] = j0 + u < A.k ? slot_row<WIDE>(A.rows, t * A.k + j0 + u, A.in_rows) : -1;
      if (r[u] >= 0) load8<DT>(w[u], A.h + ((int64_t)r[u] * A.cols + c0) * ES, n);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (r[u] < 0) continue;
      const float wt = slot_weight<WIDE>(A.weights, t * A.k + j0 + u);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += wt * elem<DT>(w[u], j);
    }
  }
  if (n == 0) return;
  if (A.residual) {
    uint32_t w[Row8<DT>::NW];
    load8<DT>(w, A.residual + (t * A.cols + c0) * ES, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += elem<DT>(w, j);
  }
  uint32_t o[Row8<DT>::NW];
  pack8<DT>(o, acc);
  store8<DT>(A.y + (t * A.cols + c0) * ES, o, n);
}

// ---- combine backward ------------------------------------------------------------
//
// grad_h = w * dy leaves as it is formed; the dot products of dy with up to 8
// rows at a time stay in registers until the end of the row.  Rows of up to
// 512 elements: one piece a lane, tokens below each other in a wave, the sums
// by lane exchanges.  Longer ones: a workgroup a token, 2048 elements a pass,
// where the waves' sums meet in LDS.  Both add in an order fixed by the shape.
// Bound by the bytes.

struct CombineBwdArgs {
  const uint8_t *gy, *h;
  const int32_t *rows;
  const float *weights;
  uint8_t *gh;
  float *gw;
  int64_t tokens, cols, in_rows;
  int k, tx_log;
};

constexpr int kCombineBwdThreads = 256, kDots = 8;

// One piece of dy against slots j0 .. j0 + 7 of token t: rows out, dots on.
template <int DT, bool WIDE>
__device__ __forceinline__ void combine_bwd_piece(const CombineBwdArgs &A, int64_t t, int j0, int64_t c0, int n,
                                                  float (&dot)[kDots]) {
  constexpr int ES = Row8<DT>::ES;
  uint32_t wy[Row8<DT>::NW], wh[kDots][Row8<DT>::NW];
  int r[kDots];
  // every load before the first store, which may not move over them
  load8<DT>(wy, A.gy + (t * A.cols + c0) * ES, n);
#pragma unroll
  for (int u = 0; u < kDots; ++u) {
    r[u] = j0 + u < A.k ? slot_row<WIDE>(A.rows, t * A.k + j0 + u, A.in_rows) : -1;
    if (A.gw && r[u] >= 0) load8<DT>(wh[u], A.h + ((int64_t)r[u] * A.cols + c0) * ES, n);
  }
#pragma unroll
  for (int u = 0; u < kDots; ++u) {
    if (r[u] < 0) continue;
    if (A.gw) {
#pragma unroll
      for (int j = 0; j < 8; ++j) dot[u] += elem<DT>(wy, j) * elem<DT>(wh[u], j);
    }
    if (A.gh) {
      const float wt = slot_weight<WIDE>(A.weights, t * A.k + j0 + u);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = wt * elem<DT>(wy, j);
      uint32_t o[Row8<DT>::NW];
      pack8<DT>(o, f);
      store8<DT>(A.gh + ((int64_t)r[u] * A.cols + c0) * ES, o, n);
    }
  }
}

template <int DT>
__global__ __launch_bounds__(kCombineBwdThreads) void combine_bwd_kernel(CombineBwdArgs A) {
  __shared__ float part[kCombineBwdThreads / 64][kDots];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j0 = 0; j0 < A.k; j0 += kDots) {
    float dot[kDots];
#pragma unroll
    for (int u = 0; u < kDots; ++u) dot[u] = 0.0f;
    for (int64_t c0 = (int64_t)threadIdx.x * 8; c0 < A.cols; c0 += kCombineBwdThreads * 8)
      combine_bwd_piece<DT, true>(A, t, j0, c0, A.cols - c0 >= 8 ? 8 : (int)(A.cols - c0), dot);
    if (!A.gw) continue;  // the same for the whole launch
#pragma unroll
    for (int u = 0; u < kDots; ++u) {
      float s = dot[u];
      for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
      if (lane == 0) part[wave][u] = s;
    }
    __syncthreads();
    if (threadIdx.x < kDots && j0 + (int)threadIdx.x < A.k) {
      float s = 0.0f;
      for (int w = 0; w < kCombineBwdThreads / 64; ++w) s += part[w][threadIdx.x];
      A.gw[t * A.k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

template <int DT>
__global__ __launch_bounds__(kCombineBwdThreads) void combine_bwd_narrow_kernel(CombineBwdArgs A) {
  const int tx = threadIdx.x & ((1 << A.tx_log) - 1);
  const int64_t t = ((int64_t)blockIdx.x * kCombineBwdThreads + threadIdx.x) >> A.tx_log;
  const int64_t c0 = (int64_t)tx * 8;
  const int64_t left = t < A.tokens ? A.cols - c0 : 0;
  const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
  for (int j0 = 0; j0 < A.k; j0 += kDots) {
    float dot[kDots];
#pragma unroll
    for (int u = 0; u < kDots; ++u) dot[u] = 0.0f;
    if (n > 0) combine_bwd_piece<DT, false>(A, t, j0, c0, n, dot);
    if (!A.gw) continue;
#pragma unroll
    for (int u = 0; u < kDots; ++u) {
      float s = dot[u];
      for (int d = 1; d < (1 << A.tx_log); d <<= 1) s += __shfl_xor(s, d);
      if (tx == 0 && t < A.tokens && j0 + u < A.k) A.gw[t * A.k + j0 + u] = s;
    }
  }
}

template <int DT, int FMT, int G>
hipError_t dispatch_one(const DispatchArgs &a, int64_t grid, hipStream_t st) {
  if (a.tx_log == kDispatchLog)
    hipLaunchKernelGGL((dispatch_kernel<DT, FMT, G, true>), dim3((unsigned)grid), dim3(kDispatchThreads), 0, st, a);
  else
    hipLaunchKernelGGL((dispatch_kernel<DT, FMT, G, false>), dim3((unsigned)grid), dim3(kDispatchThreads), 0, st, a);
  return hipGetLastError();
}
template <int DT, int FMT>
hipError_t dispatch_g(const DispatchArgs &a, int block, int64_t grid, hipStream_t st) {
  return block == 128 ? dispatch_one<DT, FMT, 16>(a, grid, st) : dispatch_one<DT, FMT, 4>(a, grid, st);
}

template <int DT>
hipError_t combine_one(const CombineArgs &a, int64_t grid, hipStream_t st) {
  if (a.tx_log == kCombineLog)
    hipLaunchKernelGGL((combine_kernel<DT, true>), dim3((unsigned)grid), dim3(kCombineThreads), 0, st, a);
  else
    hipLaunchKernelGGL((combine_kernel<DT, false>), dim3((unsigned)grid), dim3(kCombineThreads), 0, st, a);
  return hipGetLastError();
}

template <int DT>
hipError_t combine_bwd_one(CombineBwdArgs &a, hipStream_t st) {
  constexpr int64_t kNarrow = 512;
  if (a.cols <= kNarrow) {
    a.tx_log = lanes_log(a.cols, 0, 6);
    const int64_t per = kCombineBwdThreads >> a.tx_log, grid = (a.tokens + per - 1) / per;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((combine_bwd_narrow_kernel<DT>), dim3((unsigned)grid), dim3(kCombineBwdThreads), 0, st, a);
  } else {
    if (a.tokens > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((combine_bwd_kernel<DT>), dim3((unsigned)a.tokens), dim3(kCombineBwdThreads), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace

int64_t plan_workspace(int64_t slots, int experts) {
  const int64_t c = plan_chunk(slots), n = (slots + c - 1) / c;
  return n > 1 ? n * experts : 0;
}

hipError_t launch_plan(const PlanLaunch &L, hipStream_t st) {
  PlanArgs a{};
  a.ids = L.ids;
  a.group_list = L.group_list;
  a.rows = L.rows;
  a.hist = L.workspace;
  a.slots = L.slots;
  a.chunk = plan_chunk(L.slots);
  a.experts = L.experts;
  while ((1 << a.bits) <= L.experts) ++a.bits;  // numbers 0 .. experts
  a.chunks = L.slots > 0 ? (int)((L.slots + a.chunk - 1) / a.chunk) : 1;
  if (a.chunks > 1) {
    hipLaunchKernelGGL(plan_count_kernel, dim3(a.chunks), dim3(kPlanThreads), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(plan_kernel, dim3(a.chunks), dim3(kPlanThreads), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_dispatch(const DispatchLaunch &L, hipStream_t st) {
  DispatchArgs a{};
  a.x = static_cast<const uint8_t *>(L.x);
  a.rows = L.rows;
  a.y = static_cast<uint8_t *>(L.y);
  a.q = L.q;
  a.scales = L.scales;
  a.cols = L.cols;
  a.nb = (L.cols + L.block - 1) / L.block;
  a.out_rows = L.out_rows;
  a.k = L.k;
  a.tokens = L.tokens;
  a.tx_log = lanes_log(L.cols, L.block == 128 ? 4 : 2, kDispatchLog);
  const int64_t chunks = (L.cols + (8 << a.tx_log) - 1) / (8 << a.tx_log);
  const int64_t per = kDispatchThreads >> a.tx_log, grid = chunks * ((L.tokens + per - 1) / per);
  if (chunks > 0x7FFFFFFF || grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  a.chunks = (int)chunks;
  if (L.dtype == kBF16)
    return L.fmt == kE4M3 ? dispatch_g<kBF16, kE4M3>(a, L.block, grid, st) : dispatch_g<kBF16, kE5M2>(a, L.block, grid, st);
  return L.fmt == kE4M3 ? dispatch_g<kF32, kE4M3>(a, L.block, grid, st) : dispatch_g<kF32, kE5M2>(a, L.block, grid, st);
}

hipError_t launch_combine(const CombineLaunch &L, hipStream_t st) {
  CombineArgs a{};
  a.h = static_cast<const uint8_t *>(L.h);
  a.rows = L.rows;
  a.weights = L.weights;
  a.residual = static_cast<const uint8_t *>(L.residual);
  a.y = static_cast<uint8_t *>(L.y);
  a.cols = L.cols;
  a.in_rows = L.in_rows;
  a.k = L.k;
  a.tokens = L.tokens;
  a.tx_log = lanes_log(L.cols, 0, kCombineLog);
  const int64_t chunks = (L.cols + (8 << a.tx_log) - 1) / (8 << a.tx_log);
  const int64_t per = kCombineThreads >> a.tx_log, grid = chunks * ((L.tokens + per - 1) / per);
  if (chunks > 0x7FFFFFFF || grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  a.chunks = (int)chunks;
  return L.dtype == kBF16 ? combine_one<kBF16>(a, grid, st) : combine_one<kF32>(a, grid, st);
}

hipError_t launch_combine_bwd(const CombineBwdLaunch &L, hipStream_t st) {
  CombineBwdArgs a{};
  a.gy = static_cast<const uint8_t *>(L.grad_y);
  a.h = static_cast<const uint8_t *>(L.h);
  a.rows = L.rows;
  a.weights = L.weights;
  a.gh = static_cast<uint8_t *>(L.grad_h);
  a.gw = L.grad_weights;
  a.cols = L.cols;
  a.in_rows = L.in_rows;
  a.k = L.k;
  a.tokens = L.tokens;
  return L.dtype == kBF16 ? combine_bwd_one<kBF16>(a, st) : combine_bwd_one<kF32>(a, st);
}

}  // namespace mxfp4
