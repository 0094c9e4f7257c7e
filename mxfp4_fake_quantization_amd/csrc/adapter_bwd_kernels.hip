// adapter_bwd_kernels.hip -- the backward pass of the low-rank adapters on gfx950:
//     du[t] = s_i grad_y[t] B_i              (shrink with B read across its rows)
//     grad_x[t] = base[t] + du[t] A_i        (expand with A read across its rows)
//     grad_A_i = sum over t of du[t]^T x[t],  grad_B_i = s_i sum over t of grad_y[t]^T u[t]
// i = ids[t].  grad_y is read twice, x once; the sums over rows are split into
// pieces whose parts are added in a fixed order: no atomics, the same bits each time.
#include "adapter_launch.h"

namespace mxfp4 {
namespace {

// ---- weight gradients ----------------------------------------------------------------
//
// out[r, c] = sum over an adapter's rows t of v[t, r] z[t, c], (v, z) = (du, x) or
// (u, grad_y).  A workgroup takes 16 PE columns of a piece of rows, its four waves
// every fourth step of KF rows.  The sum runs down the rows of both operands, so a
// lane loads PE rows of 16 bytes and turns them in registers (one v_perm per two
// bf16 elements, no LDS): its 16 bytes are then column PE l + j of fragment j.
// v, in fp32, is split into three bf16 operands as in the other products.  Bound by the
// bytes of x and grad_y: 16384 tokens, 4096 -> 4096, rank 16 50 us (5.4 TB/s); 8191
// tokens, 7168 -> 2048, rank 64 60 us (2.5 TB/s: v, split for four tiles of ranks, and three
// products of each take the rest of the time).

constexpr int kGradWaves = 4;

struct GradSide {
  const uint8_t *z;    // [tokens, ld]
  const float *v;      // [tokens, rank]
  float *part;         // [pieces][rank * cols]
  int64_t ld, cols;
  int groups;          // of columns; 0: not wanted
};

struct GradArgs {
  GradSide a, b;
  const int32_t *order, *first;
  const int4 *pieces;
  int adapters, rank;
};

template <int DT, int RT, int MODE>
__global__ __launch_bounds__(64 * kGradWaves) void adapter_grad_kernel(GradArgs A) {
  using T = Tile<DT>;
  __shared__ float sums[kGradWaves][T::PE][64][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
  const int groups = A.a.groups + A.b.groups;
  const int piece = blockIdx.x / groups, g = blockIdx.x % groups;
  if (piece >= A.first[A.adapters]) return;
  const bool is_b = g >= A.a.groups;
  const GradSide S = is_b ? A.b : A.a;
  const int64_t n0 = (int64_t)(is_b ? g - A.a.groups : g) * (16 * T::PE);
  const int4 pc = A.pieces[piece];
  const int count = pc.z;
  const int32_t *order = A.order + pc.y;
  const int64_t col = n0 + T::PE * i;
  const RowPiece<DT, MODE> piece_z(col, S.cols);
  int vr[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) vr[r] = 16 * r + i < A.rank ? 16 * r + i : A.rank - 1;
  f32x4 acc[RT][T::PE];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < T::PE; ++j) acc[r][j] = f32x4{0, 0, 0, 0};
  for (int st = wave; st * T::KF < count; st += kGradWaves) {
    const int at = st * T::KF + T::PE * q;
    int32_t row[T::PE];
#pragma unroll
    for (int e = 0; e < T::PE; ++e) row[e] = order[at + e < count ? at + e : count - 1];
    u32x4 z[T::PE];
    float v[RT][T::PE];
#pragma unroll
    for (int e = 0; e < T::PE; ++e) {
      z[e] = piece_z.raw(S.z + row[e] * S.ld * T::ES);
#pragma unroll
      for (int r = 0; r < RT; ++r) v[r][e] = S.v[(int64_t)row[e] * A.rank + vr[r]];
    }
    if constexpr (MODE == kCut) {
#pragma unroll
      for (int e = 0; e < T::PE; ++e) z[e] = piece_z.settled(z[e]);
    }
    if ((st + 1) * T::KF > count) {  // rows past the piece count as 0
#pragma unroll
      for (int e = 0; e < T::PE; ++e)
        if (at + e >= count) {
          z[e] = u32x4{0, 0, 0, 0};
#pragma unroll
          for (int r = 0; r < RT; ++r) v[r][e] = 0.0f;
        }
    }
    u32x4 vf[DT == kBF16 ? 3 : 1][RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      if constexpr (DT == kBF16) {
        const Parts p = parts_of(v[r]);
        vf[0][r] = p.hi;
        vf[1][r] = p.mid;
        vf[2][r] = p.lo;
      } else {
#pragma unroll
        for (int d = 0; d < 4; ++d) vf[0][r][d] = __builtin_bit_cast(uint32_t, v[r][d]);
      }
    }
#pragma unroll
    for (int j = 0; j < T::PE; ++j) {
      const u32x4 zf = turned<DT>(z, j);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (auto &part : vf) acc[r][j] = mma<DT>(part[r], zf, acc[r][j]);
    }
  }
  // the waves' sums, 16 ranks at a time
  float *out = S.part + (int64_t)piece * A.rank * S.cols;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < T::PE; ++j) *reinterpret_cast<f32x4 *>(sums[wave][j][lane]) = acc[r][j];
    __syncthreads();
    if (!is_b) {  // [rank, cols]: a wave takes rank 4 q + wave, a lane PE columns
      const int rank = 16 * r + 4 * q + wave;
      if (rank < A.rank) {
        float f[T::PE];
#pragma unroll
        for (int j = 0; j < T::PE; ++j) {
          f[j] = sums[0][j][lane][wave];
#pragma unroll
          for (int w = 1; w < kGradWaves; ++w) f[j] += sums[w][j][lane][wave];
        }
        float *p = out + rank * S.cols + col;
#pragma unroll
        for (int j = 0; j < T::PE; ++j)
          if (col + j < S.cols) p[j] = f[j];
      }
    } else {  // [cols, rank]: a wave takes every fourth column, a lane 4 ranks
      for (int j = wave; j < T::PE; j += kGradWaves) {
        f32x4 f = *reinterpret_cast<f32x4 *>(sums[0][j][lane]);
#pragma unroll
        for (int w = 1; w < kGradWaves; ++w) f += *reinterpret_cast<f32x4 *>(sums[w][j][lane]);
        const int r0 = 16 * r + 4 * q;
        float *p = out + (col + j) * A.rank + r0;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (col + j < S.cols && r0 + v < A.rank) p[v] = f[v];
      }
    }
  }
}

// Each adapter's pieces added up, in a fixed order, and rounded once; 0 for an adapter
// without rows.
struct GradSumArgs {
  const float *part_a, *part_b;
  uint8_t *grad_a, *grad_b;
  const int32_t *first;
  const float *scale;
  int64_t size_a, size_b;        // elements of an adapter's gradient
  int blocks_a, blocks_b;        // workgroups of each
};
// Four groups of 64 threads share out the pieces, four loads of each under way at a
// time (16 pieces one after the other took 7 us).
constexpr int kSumLanes = 64, kSumGroups = 4, kSumEach = 4, kSumThreads = kSumLanes * kSumGroups;

template <int DT>
__global__ __launch_bounds__(kSumThreads) void adapter_grad_sum_kernel(GradSumArgs A) {
  __shared__ f32x4 sums[kSumGroups][kSumLanes];
  const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
  const int blocks = A.blocks_a + A.blocks_b;
  const int a = blockIdx.x / blocks;
  int b = blockIdx.x % blocks;
  const bool is_b = b >= A.blocks_a;
  if (is_b) b -= A.blocks_a;
  const int64_t size = is_b ? A.size_b : A.size_a;
  const float *part = is_b ? A.part_b : A.part_a;
  uint8_t *out = is_b ? A.grad_b : A.grad_a;
  const int64_t e0 = ((int64_t)b * kSumLanes + lane) * kSumEach;
  const int lo = A.first[a], hi = A.first[a + 1];
  const float s = is_b && A.scale ? A.scale[a] : 1.0f;
  f32x4 f = {0, 0, 0, 0};
  auto piece = [&](int p) {
    const uint8_t *at = reinterpret_cast<const uint8_t *>(part + p * size);
    return size >= 4 ? RowPiece<kF32, kCut>(e0, size).load(at) : ld_single<kF32>(at, size - e0);
  };
  if (e0 < size) {
    int p = lo + group;
    for (; p + 3 * kSumGroups < hi; p += 4 * kSumGroups) {
      u32x4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = piece(p + k * kSumGroups);
#pragma unroll
      for (int k = 0; k < 4; ++k) f += __builtin_bit_cast(f32x4, v[k]);
    }
    for (; p < hi; p += kSumGroups) f += __builtin_bit_cast(f32x4, piece(p));
  }
  sums[group][lane] = f;
  __syncthreads();
  if (group > 0 || e0 >= size) return;
#pragma unroll
  for (int g = 1; g < kSumGroups; ++g) f += sums[g][lane];
#pragma unroll
  for (int j = 0; j < kSumEach; ++j)
    if (e0 + j < size) {
      const int64_t at = a * size + e0 + j;
      if (DT == kBF16) reinterpret_cast<uint16_t *>(out)[at] = (uint16_t)pack_bf16(s * f[j], 0.0f);
      else reinterpret_cast<float *>(out)[at] = s * f[j];
    }
}

// du from its parts, as the kernel of grad_x adds them where that is wanted too.
__global__ __launch_bounds__(256) void adapter_parts_kernel(const float *parts, float *du, int64_t part, int splits) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e < part) du[e] = parts_sum(parts + e, part, splits);
}

// ---- host ------------------------------------------------------------------------------

// Rows of a piece: about 512 workgroups over the columns of both gradients.  (Gradients of A and B, 4096 ->
// 4096, rank 16: 16384 tokens 79 us, with 1024 workgroups 82.3, 256 83.1; 2048 tokens 26.9, 29.8, 26.6;
// 8192 tokens, 7168 -> 2048, rank 64, 4 adapters: 82, 84.9, 83.9.)
int piece_rows(int64_t tokens, int64_t in, int64_t out) {
  const int64_t groups = (in + 127) / 128 + (out + 127) / 128;
  const int64_t per = (tokens * groups / 512 + 127) / 128 * 128;
  return (int)(per < 128 ? 128 : per > 4096 ? 4096 : per);
}

struct BwdSpace {  // offsets of the workspace's parts, 16-byte aligned
  int64_t du, parts, order, first, pieces, part_a, part_b, total;
  int64_t most;    // pieces
  int rows;
};
BwdSpace bwd_space(int64_t tokens, int64_t in, int64_t out, int rank, int adapters, bool grad_a, bool grad_b) {
  BwdSpace S;
  int64_t at = 0;
  auto take = [&at](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 15) / 16 * 16;
    return here;
  };
  S.rows = piece_rows(tokens, in, out);
  S.most = tokens / S.rows + (adapters < tokens ? adapters : tokens);
  S.du = take(4 * tokens * rank);
  const int splits = shrink_splits(tokens, out);
  S.parts = take(splits > 1 ? 4 * tokens * rank * splits : 0);
  const bool any = grad_a || grad_b;
  S.order = take(any ? 4 * tokens : 0);
  S.first = take(any ? 4 * (int64_t)(adapters + 1) : 0);
  S.pieces = take(any ? 16 * S.most : 0);
  S.part_a = take(grad_a ? 4 * S.most * rank * in : 0);
  S.part_b = take(grad_b ? 4 * S.most * rank * out : 0);
  S.total = at;
  return S;
}

template <int DT>
hipError_t launch_grads(const AdapterBwdLaunch &L, const BwdSpace &S, int mode, hipStream_t stream) {
  constexpr int cols = 16 * Tile<DT>::PE;
  uint8_t *ws = L.workspace;
  float *part_a = reinterpret_cast<float *>(ws + S.part_a), *part_b = reinterpret_cast<float *>(ws + S.part_b);
  const int32_t *first = reinterpret_cast<const int32_t *>(ws + S.first);
  GradArgs G{};
  if (L.grad_a) G.a = {static_cast<const uint8_t *>(L.x), reinterpret_cast<const float *>(ws + S.du), part_a, L.ldx, L.in,
                       (int)((L.in + cols - 1) / cols)};
  if (L.grad_b) G.b = {static_cast<const uint8_t *>(L.grad_y), L.u, part_b, L.ld_gy, L.out,
                       (int)((L.out + cols - 1) / cols)};
  G.order = reinterpret_cast<const int32_t *>(ws + S.order);
  G.first = first;
  G.pieces = reinterpret_cast<const int4 *>(ws + S.pieces);
  G.adapters = L.adapters;
  G.rank = L.rank;
  if (S.most > 0) {
    const unsigned grid = (unsigned)(S.most * (G.a.groups + G.b.groups));
    by_rank_and_mode(L.rank, mode, [&](auto rt, auto m) {
      adapter_grad_kernel<DT, decltype(rt)::value, decltype(m)::value><<<grid, 64 * kGradWaves, 0, stream>>>(G);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t sa = L.grad_a ? L.rank * L.in : 0, sb = L.grad_b ? L.rank * L.out : 0;
  constexpr int each = kSumLanes * kSumEach;
  GradSumArgs R{part_a, part_b, static_cast<uint8_t *>(L.grad_a), static_cast<uint8_t *>(L.grad_b), first, L.scale, sa, sb,
                (int)((sa + each - 1) / each), (int)((sb + each - 1) / each)};
  adapter_grad_sum_kernel<DT><<<(unsigned)((R.blocks_a + R.blocks_b) * L.adapters), kSumThreads, 0, stream>>>(R);
  return hipGetLastError();
}

template <int DT>
hipError_t backward(const AdapterBwdLaunch &L, hipStream_t stream) {
  const int mode = piece_mode(DT, L.tokens, L.in, L.out, L.rank);
  const BwdSpace S = bwd_space(L.tokens, L.in, L.out, L.rank, L.adapters, L.grad_a, L.grad_b);
  uint8_t *ws = L.workspace;
  float *du = reinterpret_cast<float *>(ws + S.du);
  PlanArgs P{};
  if (L.grad_a || L.grad_b) {
    P.order = reinterpret_cast<int32_t *>(ws + S.order);
    P.first = reinterpret_cast<int32_t *>(ws + S.first);
    P.pieces = reinterpret_cast<int4 *>(ws + S.pieces);
    P.rows = S.rows;
    P.blocks = plan_blocks(L.tokens);
    while ((1 << P.bits) < L.adapters) ++P.bits;
  }
  const int64_t part = L.tokens * L.rank;
  const int splits = shrink_splits(L.tokens, L.out);
  float *parts = splits > 1 ? reinterpret_cast<float *>(ws + S.parts) : du;
  ShrinkArgs D{static_cast<const uint8_t *>(L.grad_y), static_cast<const uint8_t *>(L.b), L.ids, L.scale, parts, L.tokens,
               L.ld_gy, L.out, part, L.adapters, L.rank, splits, shrink_slots(L.tokens, L.adapters, splits),
               L.grad_x || L.grad_a ? window_count(L.tokens) : 0};
  hipError_t e = launch_shrink<DT, true>(D, P, mode, stream);
  if (e != hipSuccess) return e;
  if (L.grad_x && L.tokens > 0) {
    ExpandArgs X{parts, static_cast<const uint8_t *>(L.a), L.ids, nullptr, static_cast<const uint8_t *>(L.base),
                 static_cast<uint8_t *>(L.grad_x), splits > 1 && L.grad_a ? du : nullptr, L.tokens, L.in, L.ld_base,
                 L.ld_gx, part, L.adapters, L.rank, splits};
    e = launch_expand<DT, true>(X, mode, stream);
    if (e != hipSuccess) return e;
  }
  if (L.grad_a && !L.grad_x && splits > 1 && part > 0) {
    adapter_parts_kernel<<<(unsigned)((part + 255) / 256), 256, 0, stream>>>(parts, du, part, splits);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!L.grad_a && !L.grad_b) return hipSuccess;
  return launch_grads<DT>(L, S, mode, stream);
}

}  // namespace

int64_t adapter_bwd_workspace(int64_t tokens, int64_t in, int64_t out, int rank, int adapters, bool grad_a, bool grad_b) {
  return bwd_space(tokens, in, out, rank, adapters, grad_a, grad_b).total;
}

hipError_t launch_adapter_bwd(const AdapterBwdLaunch &L, hipStream_t stream) {
  return L.dtype == kBF16 ? backward<kBF16>(L, stream) : backward<kF32>(L, stream);
}

}  // namespace mxfp4
