// grad_norm_kernels.hip -- the norm over many gradient tensors, and clipping, on
// gfx950:
//     norm = (sum over all tensors of |g|^p)^(1/p), p = 1 or 2, or max |g|;
//     out  = g * min(1, max_norm / (norm + 1e-6)).
// Bound by the bytes: the gradients once for the norm, once more (from the 256 MB
// cache, where they fit) and written once for clipping (235 MB 38 us, 6.2 TB/s; 1.9 GB in
// and out 277 + 770 us, 6.8 and 4.9 TB/s).  448 tensors of odd sizes that lie apart, 115 MB in
// fp32: norm 31.5 us, clipping in place 85.7 (end to end, and so one tensor: 21.5 and 60).  Sums are held in 64 bits
// throughout: the squares of any fp32 values neither overflow nor vanish, and the
// matrix-free arithmetic of two double operations an element hides behind the
// loads.  A workgroup sums a contiguous run of chunks and writes one partial sum;
// the partial sums are added in a fixed order: no atomics, the same bits each time.
//
// Tensors come as kernel arguments, up to 4 KB of them a launch: nothing is copied to the
// device, and the call can be captured.
#include "grad_norm_kernels.h"
#include "mxfp4_device.h"
#include "mxfp4_kernels.h"
#include "mxfp4_rows8.h"

namespace mxfp4 {
namespace {

constexpr int kNormThreads = 256, kLoads = 8;          // 16-byte loads of a thread and chunk
constexpr int kChunkBytes = kNormThreads * 16 * kLoads;
constexpr int kMostGroups = 2048;                      // workgroups of a launch

// The tensors of a launch, as many as 4000 bytes of arguments hold.  OUT: with outputs apart from
// the gradients.
template <bool OUT>
struct Batch {
  static constexpr int N = OUT ? 180 : 284;
  const uint8_t *grad[N];
  uint8_t *out[OUT ? N : 1];
  uint32_t end[N];          // chunks up to and with the tensor's
  uint16_t tail[N];         // elements of its last chunk * 2, + 1 for fp32
  int n;
  uint32_t chunks;
};
static_assert(sizeof(Batch<true>) <= 4000 && sizeof(Batch<false>) <= 4000, "kernel arguments stay below 4 KB");

// Sum or maximum of |g|^p over a chunk, per thread.
template <int P>
__device__ __forceinline__ double joined(double a, double b) {
  if (P == 0) return b > a || b != b ? b : a;  // a NaN stays
  return a + b;
}
template <int P>
__device__ __forceinline__ double term(double acc, float g) {
  const double d = (double)__builtin_fabsf(g);
  if (P == 0) return joined<0>(acc, d);
  return P == 1 ? acc + d : __builtin_fma(d, d, acc);
}

template <int P>
__device__ __forceinline__ double wave_joined(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = joined<P>(v, __shfl_xor(v, d));
  return v;
}

// Of a whole workgroup, in every thread.
template <int P, int WAVES>
__device__ __forceinline__ double group_joined(double v, double *lds) {
  v = wave_joined<P>(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) v = joined<P>(v, lds[w]);
  return v;
}

template <int P>
__device__ __forceinline__ float norm_of(double v) {
  return (float)(P == 2 ? __builtin_sqrt(v) : v);
}

// A chunk's place: the thread's first element and how many the chunk has from there.
struct Place {
  const uint8_t *p;
  uint8_t *out;
  int left;
  bool f32;
};
template <bool OUT>
__device__ __forceinline__ Place place(const Batch<OUT> &B, uint32_t chunk, int item) {
  const int t = B.tail[item];
  const bool f32 = t & 1;
  const int64_t first = (int64_t)(chunk - (item ? B.end[item - 1] : 0)) * kChunkBytes + threadIdx.x * 16;
  const int count = chunk + 1 == B.end[item] ? t >> 1 : kChunkBytes / (f32 ? 4 : 2);
  const uint8_t *p = B.grad[item] + first;
  return {p, OUT ? B.out[item] + first : const_cast<uint8_t *>(p), count - (int)threadIdx.x * (f32 ? 4 : 8), f32};
}
// Elements between a thread's loads of a chunk.
__device__ __forceinline__ int step_of(bool f32) { return kNormThreads * (f32 ? 4 : 8); }

template <bool NT>
__device__ __forceinline__ void load_chunk(u32x4 (&w)[kLoads], const Place &at) {
  const int per = at.f32 ? 4 : 8, step = step_of(at.f32);
  if (at.left >= (kLoads - 1) * step + per) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const u32x4_a2 *p = reinterpret_cast<const u32x4_a2 *>(at.p + i * (kNormThreads * 16));
      w[i] = NT ? __builtin_nontemporal_load(p) : *p;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int n = at.left - i * step;
    const uint8_t *p = at.p + i * (kNormThreads * 16);
    w[i] = u32x4{0, 0, 0, 0};
    if (n >= per) {
      w[i] = *reinterpret_cast<const u32x4_a2 *>(p);
    } else if (at.f32) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) w[i][j] = reinterpret_cast<const uint32_t *>(p)[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) w[i][j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[j] << (16 * (j & 1));
    }
  }
}

template <bool OUT>
__device__ __forceinline__ int item_of(const Batch<OUT> &B, uint32_t chunk) {
  int lo = 0, hi = B.n - 1;  // the first item whose end is past the chunk
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (chunk < B.end[mid]) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// partial: one double a workgroup; or, NULL, the norm itself.  NT: the gradients are not read
// again, or too many for the 256 MB cache: they pass by it.  (A norm of 235 MB 38 us, else 43.
// Norm and clipping, through the cache / by it: in place 128 MB 69 / 74 us, 192 MB 118 / 118, 256 MB 160 /
// 161, 320 MB 203 / 198, 512 MB 318 / 299, 1.8 GB 1101 / 1056; out of place 128 MB 67 / 79, 256 MB 133 / 153,
// 320 MB 172 / 190, 512 MB 282 / 295, 1 GB 578 / 581, 1.8 GB 1061 / 1053.)
template <int P, bool NT>
__global__ __launch_bounds__(kNormThreads) void grad_norm_kernel(Batch<false> B, double *partial, float *norm) {
  __shared__ double lds[kNormThreads / 64];
  const uint32_t lo = (uint32_t)((uint64_t)B.chunks * blockIdx.x / gridDim.x);
  const uint32_t hi = (uint32_t)((uint64_t)B.chunks * (blockIdx.x + 1) / gridDim.x);
  double acc[2] = {0, 0};
  int item = item_of(B, lo);
  for (uint32_t c = lo; c < hi; ++c) {
    while (c >= B.end[item]) ++item;
    const Place at = place(B, c, item);
    u32x4 w[kLoads];
    load_chunk<NT>(w, at);
    if (at.f32) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j & 1] = term<P>(acc[j & 1], bits_f32(w[i][j]));
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[0] = term<P>(acc[0], bits_f32(w[i][j] << 16));
          acc[1] = term<P>(acc[1], bits_f32(w[i][j] & 0xFFFF0000u));
        }
    }
  }
  const double v = group_joined<P, kNormThreads / 64>(joined<P>(acc[0], acc[1]), lds);
  if (threadIdx.x == 0) {
    if (partial) partial[blockIdx.x] = v;
    else *norm = norm_of<P>(v);
  }
}

// The partial sums joined: thread t takes t, t + THREADS, ...
template <int P, int THREADS>
__device__ __forceinline__ double all_partials(const double *partial, int n, double *lds) {
  double v = 0;
  for (int i = threadIdx.x; i < n; i += THREADS) v = joined<P>(v, partial[i]);
  return group_joined<P, THREADS / 64>(v, lds);
}

constexpr int kFinalThreads = 256;
template <int P>
__global__ __launch_bounds__(kFinalThreads) void grad_norm_final_kernel(const double *partial, int n, float *norm) {
  __shared__ double lds[kFinalThreads / 64];
  const double v = all_partials<P, kFinalThreads>(partial, n, lds);
  if (threadIdx.x == 0) *norm = norm_of<P>(v);
}

// partial NULL: the norm is given.  Every workgroup joins the partial sums (they stay
// in the cache); the first one of a launch with `write` stores the norm.  The chunks
// are taken in the opposite order, the last read first: they are still in the cache, which
// the outputs pass by (117 MB in and out: both passes 62 us, 78 through it).
template <int P, bool OUT>
__global__ __launch_bounds__(kNormThreads) void grad_clip_kernel(Batch<OUT> B, const double *partial, int n, float *norm,
                                                                 float max_norm, bool write) {
  __shared__ double lds[kNormThreads / 64];
  float v;
  if (partial) {
    v = norm_of<P>(all_partials<P, kNormThreads>(partial, n, lds));
    if (write && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  } else {
    v = *norm;
  }
  // a NaN norm clips to NaN, an infinite one to 0
  const float ratio = max_norm / (v + 1e-6f);
  const float coef = ratio >= 1.0f ? 1.0f : ratio;
  const uint32_t g = gridDim.x - 1 - blockIdx.x;
  const uint32_t lo = (uint32_t)((uint64_t)B.chunks * g / gridDim.x);
  const uint32_t hi = (uint32_t)((uint64_t)B.chunks * (g + 1) / gridDim.x);
  if (lo >= hi) return;
  int item = item_of(B, hi - 1);
  for (uint32_t c = hi; c-- > lo;) {
    while (item > 0 && c < B.end[item - 1]) --item;
    const Place at = place(B, c, item);
    if (coef == 1.0f && at.p == at.out) continue;
    u32x4 w[kLoads];
    load_chunk<false>(w, at);
    const int per = at.f32 ? 4 : 8, step = step_of(at.f32);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (at.f32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i][j] = __builtin_bit_cast(uint32_t, bits_f32(w[i][j]) * coef);
      } else if (coef != 1.0f) {  // (a copy keeps a NaN's bits)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[i][j] = pack_bf16(bits_f32(w[i][j] << 16) * coef, bits_f32(w[i][j] & 0xFFFF0000u) * coef);
      }
      const int left = at.left - i * step;
      uint8_t *p = at.out + i * (kNormThreads * 16);
      if (left >= per) {
        __builtin_nontemporal_store(w[i], reinterpret_cast<u32x4_a2 *>(p));
      } else if (at.f32) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < left) reinterpret_cast<uint32_t *>(p)[j] = w[i][j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) reinterpret_cast<uint16_t *>(p)[j] = (uint16_t)(w[i][j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

// ---- host ------------------------------------------------------------------------------

uint32_t chunks_of(const GradTensor &t) {
  const int64_t bytes = t.count * (t.dtype == kF32 ? 4 : 2);
  return (uint32_t)((bytes + kChunkBytes - 1) / kChunkBytes);
}

// Tensors that follow one another in memory (and whose outputs do) are one to the
// kernels: the gradients of a flat bucket take one launch, however many they are.
bool follows(const GradTensor &a, const GradTensor &b, bool outs) {
  const int64_t bytes = a.count * (a.dtype == kF32 ? 4 : 2);
  return a.dtype == b.dtype && static_cast<const uint8_t *>(a.grad) + bytes == b.grad &&
         (!outs || static_cast<uint8_t *>(a.out) + bytes == b.out);
}

constexpr uint32_t kMostChunks = 1u << 30;  // of a launch

// Calls f(batch, first partial, workgroups) for each launch.
template <bool OUT, typename F>
hipError_t each_batch(const GradNormLaunch &L, F f) {
  Batch<OUT> B;
  B.n = 0;
  B.chunks = 0;
  int at = 0;
  auto send = [&]() {
    if (!B.n) return hipSuccess;
    // as many chunks for each workgroup, but for one
    const uint32_t each = (B.chunks + kMostGroups - 1) / kMostGroups;
    const int groups = (int)((B.chunks + each - 1) / each);
    const hipError_t e = f(B, at, groups);
    at += groups;
    B.n = 0;
    B.chunks = 0;
    return e;
  };
  for (int i = 0; i < L.n;) {
    GradTensor t = L.tensors[i++];
    if (!t.count) continue;
    while (i < L.n && follows(t, L.tensors[i], OUT)) t.count += L.tensors[i++].count;
    const int64_t es = t.dtype == kF32 ? 4 : 2, most = (int64_t)(kMostChunks / 2) * (kChunkBytes / es);
    while (t.count > 0) {  // (a tensor of more chunks than a launch takes goes in parts)
      GradTensor part = t;
      if (part.count > most) part.count = most;
      const uint32_t c = chunks_of(part);
      if (B.n == Batch<OUT>::N || B.chunks + c > kMostChunks) {
        const hipError_t e = send();
        if (e != hipSuccess) return e;
      }
      B.grad[B.n] = static_cast<const uint8_t *>(part.grad);
      if (OUT) B.out[B.n] = static_cast<uint8_t *>(part.out);
      B.tail[B.n] = (uint16_t)(2 * (part.count - (c - 1) * (kChunkBytes / es)) + (part.dtype == kF32));
      B.chunks += c;
      B.end[B.n++] = B.chunks;
      t.count -= part.count;
      t.grad = static_cast<const uint8_t *>(t.grad) + part.count * es;
      if (OUT) t.out = static_cast<uint8_t *>(t.out) + part.count * es;
    }
  }
  return send();
}

// One workgroup does it all: a handful of chunks cost less than a second launch (in a graph 1 / 4 / 6
// chunks 3.4 / 5.7 / 7.3 us, two launches 5.3; a launch of its own costs the host about 3 us more).
constexpr uint32_t kAlone = 4;

template <int P>
hipError_t norm_and_clip(const GradNormLaunch &L, hipStream_t stream) {
  int n = 0;
  const double *partial = L.given ? nullptr : L.workspace;
  if (!L.given) {
    uint64_t chunks = 0, bytes = 0;
    for (int i = 0; i < L.n; ++i) {
      chunks += chunks_of(L.tensors[i]);
      bytes += L.tensors[i].count * (L.tensors[i].dtype == kF32 ? 4 : 2);
    }
    const bool pass_by = !L.clip || bytes > (uint64_t)256 << 20;
    const bool alone = !L.clip && chunks <= kAlone && chunks > 0 && L.n <= Batch<false>::N;
    const hipError_t e = each_batch<false>(L, [&](const Batch<false> &B, int at, int groups) {
      double *to = alone ? nullptr : L.workspace + at;
      if (pass_by) grad_norm_kernel<P, true><<<alone ? 1 : groups, kNormThreads, 0, stream>>>(B, to, L.norm);
      else grad_norm_kernel<P, false><<<groups, kNormThreads, 0, stream>>>(B, to, L.norm);
      n = at + groups;
      return hipGetLastError();
    });
    if (e != hipSuccess || alone) return e;
    if (!L.clip || n == 0) {
      grad_norm_final_kernel<P><<<1, kFinalThreads, 0, stream>>>(L.workspace, n, L.norm);
      return hipGetLastError();
    }
  }
  if (!L.clip) return hipSuccess;
  bool in_place = true;
  for (int i = 0; i < L.n; ++i) in_place = in_place && (L.tensors[i].count == 0 || L.tensors[i].grad == L.tensors[i].out);
  auto launch = [&](const auto &B, int at, int groups) {
    constexpr bool OUT = sizeof(B.out) > sizeof(void *);
    grad_clip_kernel<P, OUT><<<groups, kNormThreads, 0, stream>>>(B, partial, n, L.norm, L.max_norm, at == 0);
    return hipGetLastError();
  };
  return in_place ? each_batch<false>(L, launch) : each_batch<true>(L, launch);
}

}  // namespace

int64_t grad_norm_workspace(int64_t n, int64_t elements) {
  // a launch takes Batch::N tensors, a part of one, or kMostChunks chunks
  const int64_t chunks = elements * 4 / kChunkBytes + n, launches = n / Batch<false>::N + 1 + 4 * (chunks / kMostChunks + 1);
  const int64_t most = launches * kMostGroups;
  return chunks < most ? chunks : most;
}

hipError_t launch_grad_norm(const GradNormLaunch &L, hipStream_t stream) {
  if (L.order == 0) return norm_and_clip<0>(L, stream);
  return L.order == 1 ? norm_and_clip<1>(L, stream) : norm_and_clip<2>(L, stream);
}

}  // namespace mxfp4
