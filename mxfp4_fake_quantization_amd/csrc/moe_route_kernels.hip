// moe_route_kernels.hip -- the choice of experts for each token, and its
// gradient, on gfx950.
//
// Forward, per token with logits l[E]: scores s = softmax(l) or
// 1 / (1 + exp(-l)); selection values v = s + bias (with a bias or groups), or
// v = l, which orders the experts as s does without its rounding.  Experts
// whose logit or value is -inf or NaN cannot be chosen.  With groups, a
// group's value is the sum of its two largest v and the best topk_groups
// groups stay.  The k largest v are chosen, equal values by lowest index.
// w = scale * s of the chosen, divided by their sum when renormalised.
//
// Work split: L = 16 lanes hold a token (4 tokens a wave; 64 lanes for more
// than 32 values a lane or k > 16), every lane V consecutive experts of ONE
// group (lanes are dealt to the groups first), so the loads are 16-byte
// pieces, group sums are reductions over a lane range, and the maximum of a
// token is one chain of DPP row operations.  Up to k = 8 (16 lanes a token) the
// lanes sort their values and merge them (top_by_sorting); where that does not
// settle the choice, and for larger k, each of k steps takes the token's largest
// v and its lowest index by two such chains and clears it.  Bound by VALU work,
// not by the logits' bytes: 32768 tokens of 256 experts in 8 groups, k = 8, take
// 17 us; the VALU issues for 87 % of the busy cycles (1005 instructions a wave).
#include "moe_kernels.h"
#include "mxfp4_device.h"
#include "mxfp4_rows8.h"

namespace mxfp4 {
namespace {

constexpr int kRouteThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ uint32_t fbits(float f) { return __builtin_bit_cast(uint32_t, f); }

// Reductions over the aligned L lanes of a token.  Every step pairs two groups
// of lanes that already agree (mirrors of half a row and of a row swap quads
// and halves), so both sides add the same two numbers and all lanes end with
// the same bits: a sum that differed between lanes would order equal experts
// by the lane that holds them.
constexpr int kDppRowHalfMirror = 0x141, kDppRowMirror = 0x140;
template <int L, typename OP>
__device__ __forceinline__ float reduce_f(float v, OP op) {
  v = op(v, bits_f32(dpp<kDppQuadXor1>(fbits(v))));
  v = op(v, bits_f32(dpp<kDppQuadXor2>(fbits(v))));
  v = op(v, bits_f32(dpp<kDppRowHalfMirror>(fbits(v))));
  v = op(v, bits_f32(dpp<kDppRowMirror>(fbits(v))));
  if (L == 64) {
    v = op(v, bits_f32(lane_xor16(fbits(v))));
    v = op(v, bits_f32(lane_xor32(fbits(v))));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float max_lanes(float v) {
  return reduce_f<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
  return reduce_f<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ uint32_t min_lanes(uint32_t v) {
  auto op = [](uint32_t a, uint32_t b) { return a < b ? a : b; };
  v = op(v, dpp<kDppQuadXor1>(v));
  v = op(v, dpp<kDppQuadXor2>(v));
  v = op(v, dpp<kDppRowHalfMirror>(v));
  v = op(v, dpp<kDppRowMirror>(v));
  if (L == 64) {
    v = op(v, lane_xor16(v));
    v = op(v, lane_xor32(v));
  }
  return v;
}

// exp(x) and 1 / (1 + exp(-x)) on the hardware 2^x and reciprocal, 1 ulp each:
// the product with log2 e rounds the exponent, a relative error of |x| 2^-24.
// (expf and an IEEE division took route_prefill's 256 scores a token 6 us.)
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(1.44269504f * x); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x)); }

template <int DT>
__device__ __forceinline__ float load_one(const uint8_t *p, int64_t i) {
  if (DT == kBF16) return bits_f32((uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << 16);
  return reinterpret_cast<const float *>(p)[i];
}

// V consecutive elements from element `at`; those past cnt read as -inf (from
// the row's first element, without a branch a value: 16 of them around the
// bias took route_prefill 14 us).  vec: whole pieces of PE elements, aligned.
template <int DT, int V>
struct Pieces {
  static constexpr int ES = DT == kBF16 ? 2 : 4;
  static constexpr int PE = V * ES < 16 ? V : 16 / ES;  // elements of a piece
  static constexpr int PW = PE * ES / 4;                // words of a piece
};
template <int DT, int V>
__device__ __forceinline__ void load_values(const uint8_t *p, int64_t row, int e0, int cnt, bool vec, float (&l)[V]) {
  using P = Pieces<DT, V>;
  typedef uint32_t words __attribute__((ext_vector_type(P::PW)));
  if (vec) {
    words w[V / P::PE];
#pragma unroll
    for (int q = 0; q < V / P::PE; ++q)
      w[q] = *reinterpret_cast<const words *>(p + (row + (q * P::PE < cnt ? e0 + q * P::PE : 0)) * P::ES);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int q = j / P::PE, i = j % P::PE;
      const float x = DT == kBF16 ? bits_f32(i & 1 ? w[q][(i >> 1) % P::PW] & 0xFFFF0000u : w[q][(i >> 1) % P::PW] << 16)
                                  : bits_f32(w[q][i % P::PW]);
      l[j] = j < cnt ? x : kNegInf;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float x = load_one<DT>(p, row + (j < cnt ? e0 + j : 0));
      l[j] = j < cnt ? x : kNegInf;
    }
  }
}

// ---- the k <= 8 largest by sorting (16 lanes a token) ----------------------
//
// Each lane sorts its values, the lanes' first 8 merge pairwise in four steps
// (the larger of a_i and b_7-i are the 8 largest of both, and need three
// compare steps to be in order), after which every lane holds the token's 8
// largest values.  The k-th of them is a threshold that picks the experts, and
// the number of larger ones is an expert's rank.  This needs the k values
// different from each other and from all others; where they are not, or fewer
// than k experts are live, the caller's step-by-step choice runs instead (for
// all tokens of the wave).  Measured on 32768 tokens of 256 experts,
// bf16 or fp32 logits, k = 8, no bias: 12.3 us against 15.6 step by step.
constexpr int kTop = 8;

__device__ __forceinline__ void order(float &a, float &b) {  // a >= b
  const float hi = fmaxf(a, b), lo = fminf(a, b);
  a = hi;
  b = lo;
}

// Descending; Batcher's odd-even merge sort.
template <int N>
__device__ __forceinline__ void sort_desc(float (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j < N - k; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(v[i + j], v[i + j + k]);
}

template <int CTRL>
__device__ __forceinline__ void merge_top(float (&t)[kTop]) {
  float c[kTop];
#pragma unroll
  for (int i = 0; i < kTop; ++i) c[i] = fmaxf(t[i], bits_f32(dpp<CTRL>(fbits(t[kTop - 1 - i]))));
#pragma unroll
  for (int d = kTop / 2; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < kTop; ++i)
      if (!(i & d)) order(c[i], c[i + d]);
#pragma unroll
  for (int i = 0; i < kTop; ++i) t[i] = c[i];
}

// bf16 values leave 16 bits of the fp32 free: the expert's number goes there so
// that equal logits are ordered by lowest index and no two values are equal.
// -0 counts as +0; infinities stay as they are.
template <int V>
__device__ __forceinline__ void tag_bf16(float (&v)[V], int e0) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t b = fbits(v[j] + 0.0f), e = (uint32_t)(e0 + j);
    const uint32_t t = b | ((b >> 31) ? e : 0xFFFFu - e);
    v[j] = (b & 0x7F800000u) == 0x7F800000u ? v[j] : bits_f32(t);
  }
}

// False (for the whole wave) where the values do not settle the choice.
template <int V>
__device__ __forceinline__ bool top_by_sorting(const float (&v)[V], int e0, int k, int slot, int li, int *mine) {
  __shared__ int ids[kRouteThreads / 16][kTop];
  float s[V], t[kTop];
#pragma unroll
  for (int j = 0; j < V; ++j) s[j] = v[j];
  sort_desc<V>(s);
#pragma unroll
  for (int i = 0; i < kTop; ++i) t[i] = i < V ? s[i % V] : kNegInf;
  merge_top<kDppQuadXor1>(t);
  merge_top<kDppQuadXor2>(t);
  merge_top<kDppRowHalfMirror>(t);
  merge_top<kDppRowMirror>(t);
  float last = t[0];
  bool equal = false;
#pragma unroll
  for (int i = 1; i < kTop; ++i) {
    if (i < k) {  // the same for the launch
      equal |= t[i] == t[i - 1];
      last = t[i];
    }
  }
  uint32_t picked = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) picked |= v[j] >= last ? 1u << j : 0u;
  int n = __popc(picked);
  n += (int)dpp<kDppQuadXor1>((uint32_t)n);
  n += (int)dpp<kDppQuadXor2>((uint32_t)n);
  n += (int)dpp<kDppRowHalfMirror>((uint32_t)n);
  n += (int)dpp<kDppRowMirror>((uint32_t)n);
  if (__ballot(equal || n != k || !(last > kNegInf))) return false;
  while (__ballot(picked != 0)) {
    const int j = __ffs((int)picked) - 1;  // -1: nothing left in this lane
    picked &= picked - 1;
    float x = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) x = i == j ? v[i] : x;
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kTop; ++i) rank += t[i] > x ? 1 : 0;
    if (j >= 0) ids[slot][rank & (kTop - 1)] = e0 + j;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  *mine = li < k ? ids[slot][li & (kTop - 1)] : -1;
  return true;
}

struct RouteArgs {
  const uint8_t *logits;
  const float *bias;
  float *weights;
  int32_t *ids;
  int64_t tokens;
  int experts, k, groups, topk_groups;
  int size, lpg_log, vr;  // experts a group, log2 lanes a group, experts a lane
  int score, renorm, vec, bias_vec;
  float scale;
};

template <int DT, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs A) {
  const int lane = threadIdx.x & 63, li = lane & (L - 1);
  const int64_t tok = (int64_t)blockIdx.x * (kRouteThreads / L) + threadIdx.x / L;
  const int64_t t = tok < A.tokens ? tok : A.tokens - 1;  // spare lanes repeat the last token, and store nothing
  const int g = li >> A.lpg_log, sub = li & ((1 << A.lpg_log) - 1);
  const int e0 = g * A.size + sub * A.vr;
  int cnt = g < A.groups ? A.size - sub * A.vr : 0;
  cnt = cnt < 0 ? 0 : (cnt < A.vr ? cnt : A.vr);
  const int64_t row = t * A.experts;

  float v[V];
  load_values<DT, V>(A.logits, row, e0, cnt, A.vec, v);

  // softmax needs the row's maximum and sum, unless only the chosen logits matter
  const bool by_score = A.bias || A.groups > 1;
  float top = 0.0f, inv = 1.0f;
  if (A.score == 0) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, v[j]);
    top = max_lanes<L>(m);
    top = top > kNegInf ? top : 0.0f;
    if (by_score || !A.renorm) {
      float ex[V], sum = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ex[j] = exp_fast(v[j] - top);
        sum += ex[j];
      }
      sum = sum_lanes<L>(sum);
      inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      if (by_score) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = v[j] > kNegInf ? ex[j] * inv : kNegInf;
      }
    }
  } else if (by_score) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = v[j] > kNegInf ? sigmoid(v[j]) : kNegInf;
  }
  if (A.bias) {
    float b[V];
    load_values<kF32, V>(reinterpret_cast<const uint8_t *>(A.bias), 0, e0, cnt, A.bias_vec, b);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += b[j];
  }
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = v[j] > kNegInf ? v[j] : kNegInf;  // NaN is never chosen

  if (A.groups > 1) {
    float t1 = kNegInf, t2 = kNegInf;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      t2 = fmaxf(t2, fminf(t1, v[j]));
      t1 = fmaxf(t1, v[j]);
    }
    for (int d = 1; d < (1 << A.lpg_log); d <<= 1) {
      const float o1 = __shfl_xor(t1, d), o2 = __shfl_xor(t2, d);
      t2 = fmaxf(fmaxf(t2, o2), fminf(t1, o1));
      t1 = fmaxf(t1, o1);
    }
    const float gv = t1 > kNegInf ? t1 + (t2 > kNegInf ? t2 : 0.0f) : kNegInf;
    int rank = 0;
    for (int o = 0; o < A.groups; ++o) {
      const float ov = __shfl(gv, (lane & ~(L - 1)) + (o << A.lpg_log));
      rank += (ov > gv || (ov == gv && o < g)) ? 1 : 0;
    }
    if (rank >= A.topk_groups) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = kNegInf;
    }
  }

  int mine = -1;  // lane i of the token keeps its i-th choice
  bool chosen = false;
  if constexpr (L == 16) {
    if (A.k <= kTop) {
      if (DT == kBF16 && !by_score) tag_bf16<V>(v, e0);
      chosen = top_by_sorting<V>(v, e0, A.k, threadIdx.x >> 4, li, &mine);
    }
  }
  if (!chosen) {
    for (int i = 0; i < A.k; ++i) {
      float m = v[0];
#pragma unroll
      for (int j = 1; j < V; ++j) m = fmaxf(m, v[j]);
      const float best = max_lanes<L>(m);
      int at = 0;
#pragma unroll
      for (int j = V - 1; j >= 0; --j) at = v[j] == best ? j : at;
      const bool live = best > kNegInf;
      const uint32_t win = min_lanes<L>(live && m == best ? (uint32_t)(e0 + at) : 0xFFFFFFFFu);
      const int jw = live ? (int)win - e0 : -1;
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = j == jw ? kNegInf : v[j];
      mine = li == i ? (int)win : mine;  // 0xFFFFFFFF is -1
    }
  }

  const bool has = li < A.k && mine >= 0;
  float s = 0.0f;
  if (has) {
    const float l = load_one<DT>(A.logits, row + mine);
    s = A.score == 0 ? exp_fast(l - top) * inv : sigmoid(l);
  }
  if (A.renorm) {
    const float total = sum_lanes<L>(s);
    s = total == 0.0f ? 0.0f : s / total;
  }
  if (li < A.k && tok < A.tokens) {
    A.weights[tok * A.k + li] = s * A.scale;
    A.ids[tok * A.k + li] = mine;
  }
}

// ---- backward --------------------------------------------------------------
//
// The choice is constant.  With d = scale * grad_weights of the chosen and p
// their scores (renormalised: p / sum p):
//   sigmoid            dl_j = d_j s_j (1 - s_j)
//   sigmoid, renorm.   dl_j = (d_j - sum_i d_i p_i) / sum s * s_j (1 - s_j)
//   softmax            dl_e = s_e (d_e - sum_j d_j s_j)       for every expert
//   softmax, renorm.   dl_j = p_j (d_j - sum_i d_i p_i)       for the chosen
// Only the third reads the whole row of logits; the others gather k of them.
// The row of d (or of dl) is put together in LDS, so the dense gradient
// leaves in whole pieces.  Bound by the gradient's bytes.

struct RouteBwdArgs {
  const float *gw;
  const uint8_t *logits;
  const int32_t *ids;
  uint8_t *gl;
  int64_t tokens;
  int experts, k, vr;
  int score, renorm, vec;
  float scale;
};

template <int DT, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void route_bwd_kernel(RouteBwdArgs A) {
  using P = Pieces<DT, V>;
  constexpr int TOK = kRouteThreads / L;
  __shared__ __align__(16) float srow[TOK][L * V];
  const int li = threadIdx.x & (L - 1), slot = threadIdx.x / L;
  const int64_t tok = (int64_t)blockIdx.x * TOK + slot;
  const bool in = tok < A.tokens;
  const int64_t t = in ? tok : A.tokens - 1;
  const int64_t row = t * A.experts;
  const int e0 = li * A.vr;
  int cnt = A.experts - e0;
  cnt = cnt < 0 ? 0 : (cnt < A.vr ? cnt : A.vr);

#pragma unroll
  for (int j = 0; j < V; ++j) srow[slot][j * L + li] = 0.0f;

  const bool dense = A.score == 0 && !A.renorm;
  float ex[V], top = 0.0f, inv = 1.0f;
  if (dense) {
    load_values<DT, V>(A.logits, row, e0, cnt, A.vec, ex);
    float m = ex[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, ex[j]);
    top = max_lanes<L>(m);
    top = top > kNegInf ? top : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      ex[j] = exp_fast(ex[j] - top);
      sum += ex[j];
    }
    sum = sum_lanes<L>(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  int id = -1;
  float d = 0.0f, l = kNegInf;
  if (li < A.k) {
    id = A.ids[t * A.k + li];
    if (id < 0 || id >= A.experts) {
      id = -1;
    } else {
      d = A.gw[t * A.k + li] * A.scale;
      l = load_one<DT>(A.logits, row + id);
    }
  }
  float out, dot = 0.0f;
  if (dense) {
    dot = sum_lanes<L>(id >= 0 ? d * (exp_fast(l - top) * inv) : 0.0f);
    out = d;
  } else {
    float s;
    if (A.score == 0) {
      top = max_lanes<L>(l);
      s = id >= 0 ? exp_fast(l - top) : 0.0f;
    } else {
      s = id >= 0 ? sigmoid(l) : 0.0f;
    }
    float p = s, r = 1.0f;
    if (A.renorm) {
      const float total = sum_lanes<L>(s);
      r = total == 0.0f ? 0.0f : 1.0f / total;
      p = s * r;
      d -= sum_lanes<L>(id >= 0 ? d * p : 0.0f);
    }
    out = A.score == 0 ? p * d : d * r * s * (1.0f - s);
  }
  __syncthreads();
  if (id >= 0) srow[slot][id] = out;
  __syncthreads();
  if (!in) return;
  float o[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float x = j < cnt ? srow[slot][e0 + j] : 0.0f;
    o[j] = dense ? ex[j] * inv * (x - dot) : x;
  }
  typedef uint32_t words __attribute__((ext_vector_type(P::PW)));
  if (A.vec) {
#pragma unroll
    for (int q = 0; q < V / P::PE; ++q) {
      if (q * P::PE >= cnt) break;
      words w;
#pragma unroll
      for (int j = 0; j < P::PW; ++j)
        w[j] = DT == kBF16 ? pack_bf16(o[(q * P::PE + 2 * j) % V], o[(q * P::PE + 2 * j + 1) % V])
                           : fbits(o[(q * P::PE + j) % V]);
      *reinterpret_cast<words *>(A.gl + (row + e0 + q * P::PE) * P::ES) = w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j >= cnt) break;
      if (DT == kBF16) reinterpret_cast<uint16_t *>(A.gl)[row + e0 + j] = (uint16_t)pack_bf16(o[j], 0.0f);
      else reinterpret_cast<float *>(A.gl)[row + e0 + j] = o[j];
    }
  }
}

bool pieces_fit(const void *p, int es, int v, int vr, int size, int experts) {
  const int pe = v * es < 16 ? v : 16 / es;
  return (uintptr_t)p % (pe * es) == 0 && vr % pe == 0 && size % vr == 0 && experts % pe == 0;
}

template <int DT, int L, int V>
hipError_t route_one(RouteArgs &a, hipStream_t st) {
  constexpr int TOK = kRouteThreads / L;
  a.vec = pieces_fit(a.logits, DT == kBF16 ? 2 : 4, V, a.vr, a.size, a.experts);
  a.bias_vec = a.bias && pieces_fit(a.bias, 4, V, a.vr, a.size, a.experts);
  const int64_t n = (a.tokens + TOK - 1) / TOK;
  if (n > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((route_kernel<DT, L, V>), dim3((unsigned)n), dim3(kRouteThreads), 0, st, a);
  return hipGetLastError();
}
template <int DT, int L, int V>
hipError_t route_bwd_one(RouteBwdArgs &a, hipStream_t st) {
  constexpr int TOK = kRouteThreads / L;
  a.vec = pieces_fit(a.logits, DT == kBF16 ? 2 : 4, V, a.vr, a.experts, a.experts) && (uintptr_t)a.gl % 16 == 0;
  const int64_t n = (a.tokens + TOK - 1) / TOK;
  if (n > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((route_bwd_kernel<DT, L, V>), dim3((unsigned)n), dim3(kRouteThreads), 0, st, a);
  return hipGetLastError();
}

// Lanes and experts a lane: groups get a power of two of the token's lanes.
// False where L lanes cannot hold the row with at most `most` values each.
bool lay_out(int L, int most, int experts, int groups, int k, int *size, int *lpg_log, int *vr) {
  int gl = 0;
  while ((1 << gl) < groups) ++gl;
  if ((1 << gl) > L || k > L) return false;
  int log_l = 0;
  while ((1 << log_l) < L) ++log_l;
  *size = experts / groups;
  *lpg_log = log_l - gl;
  const int lpg = 1 << *lpg_log;
  *vr = (*size + lpg - 1) / lpg;
  return *vr <= most;
}

template <int DT>
hipError_t route_launch(RouteArgs &a, hipStream_t st) {
  // 16 lanes a token as long as they hold it: 512 experts in 32 values a lane
  // take 30 us for 32768 tokens, as 8 values in 64 lanes 45
  if (lay_out(16, 32, a.experts, a.groups, a.k, &a.size, &a.lpg_log, &a.vr)) {
    if (a.vr <= 4) return route_one<DT, 16, 4>(a, st);
    if (a.vr <= 8) return route_one<DT, 16, 8>(a, st);
    if (a.vr <= 16) return route_one<DT, 16, 16>(a, st);
    return route_one<DT, 16, 32>(a, st);
  }
  if (!lay_out(64, 32, a.experts, a.groups, a.k, &a.size, &a.lpg_log, &a.vr)) return hipErrorInvalidValue;
  if (a.vr <= 8) return route_one<DT, 64, 8>(a, st);
  if (a.vr <= 16) return route_one<DT, 64, 16>(a, st);
  return route_one<DT, 64, 32>(a, st);
}

template <int DT>
hipError_t route_bwd_launch(RouteBwdArgs &a, hipStream_t st) {
  int size, lpg_log;
  if (lay_out(16, 16, a.experts, 1, a.k, &size, &lpg_log, &a.vr)) {
    if (a.vr <= 4) return route_bwd_one<DT, 16, 4>(a, st);
    if (a.vr <= 8) return route_bwd_one<DT, 16, 8>(a, st);
    return route_bwd_one<DT, 16, 16>(a, st);
  }
  if (!lay_out(64, 32, a.experts, 1, a.k, &size, &lpg_log, &a.vr)) return hipErrorInvalidValue;
  if (a.vr <= 8) return route_bwd_one<DT, 64, 8>(a, st);
  return route_bwd_one<DT, 64, 16>(a, st);
}

}  // namespace

hipError_t launch_route(const RouteLaunch &R, hipStream_t st) {
  RouteArgs a{};
  a.logits = static_cast<const uint8_t *>(R.logits);
  a.bias = R.bias;
  a.weights = R.weights;
  a.ids = R.ids;
  a.tokens = R.tokens;
  a.experts = R.experts;
  a.k = R.k;
  a.groups = R.groups;
  a.topk_groups = R.topk_groups;
  a.score = R.score;
  a.renorm = R.renorm;
  a.scale = R.scale;
  return R.dtype == kBF16 ? route_launch<kBF16>(a, st) : route_launch<kF32>(a, st);
}

hipError_t launch_route_bwd(const RouteBwdLaunch &R, hipStream_t st) {
  RouteBwdArgs a{};
  a.gw = R.grad_weights;
  a.logits = static_cast<const uint8_t *>(R.logits);
  a.ids = R.ids;
  a.gl = static_cast<uint8_t *>(R.grad_logits);
  a.tokens = R.tokens;
  a.experts = R.experts;
  a.k = R.k;
  a.score = R.score;
  a.renorm = R.renorm;
  a.scale = R.scale;
  return R.dtype == kBF16 ? route_bwd_launch<kBF16>(a, st) : route_bwd_launch<kF32>(a, st);
}

}  // namespace mxfp4
