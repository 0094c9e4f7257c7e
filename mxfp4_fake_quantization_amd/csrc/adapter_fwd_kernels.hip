// adapter_fwd_kernels.hip -- low-rank adapters of many requests beside a shared
// projection on gfx950: y[t] = base[t] + s_i B_i (A_i x[t]), i = ids[t].
//
// Two launches, u = x A^T and y = base + s u B^T; many rows as in adapter_launch.h, few
// rows (decode) as below.
#include "adapter_launch.h"

namespace mxfp4 {
namespace {

// ---- few rows ----------------------------------------------------------------------
//
// Bound by reading each adapter's weights once, and by latency: many small workgroups,
// each with all its loads under way at once.  A workgroup takes the rows of one adapter
// in a window of 64 (it is the workgroup of the first of them; those of the others end
// at once) and a part of the long dimension (u) or of the columns (y).
// One launch that computed u again for every part of the columns read A once a part
// through each CU's L1 at 64 bytes a clock: 64 tokens of 48 adapters, 8192 -> 28672, rank
// 16 took 51 us (two launches 6.9 + 19.6, 46 MB of B at 2.3 TB/s), one token 4096 -> 4096
// 9.4 (3.7 + 5.1).

struct FewArgs {
  const uint8_t *x, *a, *b;
  const int32_t *ids;
  const float *scale;
  const uint8_t *base;
  uint8_t *y;
  float *u;             // [splits][tokens, rank]
  float *u_out;         // [tokens, rank] or NULL
  int64_t tokens, in, out, ldx, ld_base, ldy, part;
  int adapters, rank, splits, parts;
};

constexpr int kFewWaves = 4;

// The rows of one adapter in a window.
struct FewRows {
  int64_t row0;
  int own, n, line;     // line: lane t holds the t-th row
  bool mine;            // this workgroup's
  __device__ __forceinline__ FewRows(const FewArgs &A, int m, int lane) {
    row0 = m / kWindow * kWindow;
    const int id = row0 + lane < A.tokens ? row_adapter(A.ids, row0 + lane, A.adapters) : -2;
    own = __builtin_amdgcn_readlane(id, m % kWindow);
    const uint64_t match = __ballot(id == own);
    mine = __builtin_ctzll(match) == m % kWindow;
    n = __popcll(match);
    line = lined_up(match, lane);
  }
  // Row `at`, the last one from n on (every lane takes part).
  __device__ __forceinline__ int64_t row(int at) const {
    return row0 + __builtin_amdgcn_ds_bpermute((at < n ? at : n - 1) << 2, line);
  }
};

// The rows' tiles of 16 are taken together (NT: one, or up to four), so that the weights
// are loaded once for all of them.
template <int DT, int RT, int MODE, int NT>
__device__ __forceinline__ void few_u(const FewArgs &A, const FewRows &R, f32x4 (*part)[RT][64], int lane, int wave) {
  using T = Tile<DT>;
  // fragments of a turn, as the registers allow
  constexpr int U = NT == 1 ? (RT <= 1 ? 8 : RT <= 4 ? 4 : 2) : RT <= 1 ? 4 : RT <= 4 ? 2 : 1;
  const int i = lane & 15, q = lane >> 4;
  float *u = A.u + blockIdx.y * A.part;
  const uint8_t *wa = A.a + (int64_t)R.own * A.rank * A.in * T::ES;
  uint32_t at_w[RT];  // the lane's row of each 16 ranks, from the first (few_rows() bounds it)
#pragma unroll
  for (int r = 0; r < RT; ++r) at_w[r] = ((16 * r + i < A.rank ? 16 * r + i : A.rank - 1) * (uint32_t)A.in + T::PE * q) * T::ES;
  const int64_t turns = A.in / (U * T::KF);
  const int first = blockIdx.y * kFewWaves + wave, step = kFewWaves * A.splits;
  int64_t row[NT];
  const uint8_t *xp[NT];
  f32x4 acc[NT][RT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    row[t] = R.row(16 * t + i);
    xp[t] = A.x + row[t] * A.ldx * T::ES;
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[t][r] = f32x4{0, 0, 0, 0};
  }
  for (int64_t turn = first; turn < turns; turn += step) {
    u32x4 xf[NT][U], wf[U][RT];
#pragma unroll
    for (int c = 0; c < U; ++c)
#pragma unroll
      for (int r = 0; r < RT; ++r) wf[c][r] = ld_frag(wa + (turn * U + c) * T::KF * T::ES + at_w[r]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int c = 0; c < U; ++c) xf[t][c] = u32x4{0, 0, 0, 0};
      if (16 * t + i < R.n) {  // (lanes without a row would cost the L1 a cycle for each 64 bytes)
#pragma unroll
        for (int c = 0; c < U; ++c) xf[t][c] = ld_frag(xp[t] + ((turn * U + c) * T::KF + T::PE * q) * T::ES);
      }
    }
#pragma unroll
    for (int c = 0; c < U; ++c)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[t][r] = mma<DT>(wf[c][r], xf[t][c], acc[t][r]);
  }
  // the rest of the row, fragment by fragment
  for (int64_t k0 = (turns * U + first) * T::KF; k0 < A.in; k0 += step * T::KF) {
    const RowPiece<DT, MODE> piece(k0 + T::PE * q, A.in);
    u32x4 xf[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xf[t] = piece.load(xp[t]);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const u32x4 wf = piece.load(wa + at_w[r] - T::PE * q * T::ES);
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t][r] = mma<DT>(wf, xf[t], acc[t][r]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    __syncthreads();  // the tile before has been read
#pragma unroll
    for (int r = 0; r < RT; ++r) part[wave][r][lane] = acc[t][r];
    __syncthreads();
    for (int r = wave; r < RT; r += kFewWaves) {
      f32x4 sum = part[0][r][lane];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) sum += part[w][r][lane];
      const int r0 = 16 * r + 4 * q;
      if (16 * t + i < R.n) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (r0 + v < A.rank) u[row[t] * A.rank + r0 + v] = sum[v];
      }
    }
  }
}

template <int DT, int RT, int MODE>
__global__ __launch_bounds__(64 * kFewWaves) void adapter_few_u_kernel(FewArgs A) {
  __shared__ f32x4 part[kFewWaves][RT][64];
  const int m = blockIdx.x;
  if (m >= A.tokens) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const FewRows R(A, m, lane);
  if (!R.mine || R.own < 0) return;
  if (R.n <= 16) few_u<DT, RT, MODE, 1>(A, R, part, lane, wave);
  else few_u<DT, RT, MODE, kWindow / 16>(A, R, part, lane, wave);
}

// Columns are the rows of the first operand here: tile j of a run has columns 16 j to
// 16 j + 15, whose weights are one contiguous piece of B, and a lane's results are four
// consecutive columns of token l % 16.  (The other way round, as for many rows, a tile's
// weights come in 16 pieces; that way pays in stores, of which few rows have few.)
template <int DT>
struct Quad {  // four consecutive elements of a row
  uint32_t w[DT == kBF16 ? 2 : 4];
  __device__ __forceinline__ void load(const uint8_t *p, int64_t left, bool inside) {
    if (inside) {
      if constexpr (DT == kBF16) {
        typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
        const u32x2 v = *reinterpret_cast<const u32x2_a2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
      } else {
        const u32x4 v = ld_frag(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e % (DT == kBF16 ? 2 : 4)] = v[e];
      }
    } else {
      const u32x4 v = ld_single<DT>(p, left < 4 ? left : 4);
#pragma unroll
      for (int e = 0; e < (DT == kBF16 ? 2 : 4); ++e) w[e] = v[e];
    }
  }
  __device__ __forceinline__ void add(f32x4 f) {
    if constexpr (DT == kBF16) {
#pragma unroll
      for (int d = 0; d < 2; ++d)
        w[d] = pack_bf16(bits_f32(w[d] << 16) + f[2 * d], bits_f32(w[d] & 0xFFFF0000u) + f[2 * d + 1]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e % (DT == kBF16 ? 2 : 4)] = __builtin_bit_cast(uint32_t, bits_f32(w[e % (DT == kBF16 ? 2 : 4)]) + f[e]);
    }
  }
  __device__ __forceinline__ void store(uint8_t *p, int64_t left, bool inside) const {
    if (inside) {
      if constexpr (DT == kBF16) {
        typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
        *reinterpret_cast<u32x2_a2 *>(p) = u32x2{w[0], w[1]};
      } else {
        *reinterpret_cast<u32x4_a1 *>(p) = u32x4{w[0], w[1], w[2 % (DT == kBF16 ? 2 : 4)], w[3 % (DT == kBF16 ? 2 : 4)]};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) {
          if (DT == kBF16) reinterpret_cast<uint16_t *>(p)[e] = (uint16_t)(w[(e >> 1) % 2] >> (16 * (e & 1)));
          else reinterpret_cast<uint32_t *>(p)[e] = w[e % (DT == kBF16 ? 2 : 4)];
        }
    }
  }
};

// Tiles of a run.  (With 8, both kernels: one token of rank 16 9.3 us instead of 8.4, 32 / 128 / 256 rows of 48
// adapters, 4096 -> 4096, 10.4 / 12.5 / 14.4 instead of 9.5 / 12.0 / 13.4, 32 rows of 8 adapters of rank 64, 4096 ->
// 14336, 21.3 instead of 18.6.)
constexpr int kFewTiles = 4;

template <int DT, int RT, int MODE>
__device__ __forceinline__ void few_y(const FewArgs &A, const FewRows &R,
                                      u32x4 (*us)[Expand<DT, frag_count<DT>(RT), false, MODE>::UF][64], int lane, int wave) {
  using T = Tile<DT>;
  using X = Expand<DT, frag_count<DT>(RT), false, MODE>;
  constexpr int F = X::F, TILES = kFewTiles, COLS = 16 * TILES;
  const int i = lane & 15, q = lane >> 4, own = R.own, n = R.n;
  const int64_t runs = (A.out + COLS - 1) / COLS;
  const int64_t first = blockIdx.y * kFewWaves + wave, step = kFewWaves * A.parts;
  const uint8_t *wb = A.b + (int64_t)(own < 0 ? 0 : own) * A.out * A.rank * T::ES;
  const uint8_t *w_last = wb + A.out * A.rank * T::ES - 16;
  // The lane's pieces of a run's weights lie at one distance each from the run's first
  // row, which is the wave's: loads take no arithmetic (it was what bound this kernel).
  uint32_t at_w[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int r0 = X::rank0(f, q);
    at_w[f] = (i * A.rank + (r0 < A.rank ? r0 : 0)) * T::ES;
  }
  const uint32_t tile_bytes = 16 * A.rank * T::ES;
  const bool full = MODE == kExact && A.rank == 16 * RT;  // no fragment holds a rank past the last
  // (rows shorter than a piece end in the last 16 bytes: one run more is met with care)
  auto inside = [&](int64_t n0) { return MODE != kSingle && n0 + COLS + (MODE == kCut ? T::PE : 0) <= A.out; };
  u32x4 w[F][TILES];
  auto load = [&](int64_t n0) {
    if (inside(n0)) {
      const uint8_t *from = wb + n0 * A.rank * T::ES;
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int j = 0; j < TILES; ++j) w[f][j] = ld_frag(from + j * tile_bytes + at_w[f]);
    } else {
#pragma unroll 1
      for (int j = 0; j < TILES; ++j) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const int64_t col = n0 + 16 * j + i;
          const int r0 = X::rank0(f, q);
          const uint8_t *p = wb + ((col < A.out ? col : A.out - 1) * A.rank + (r0 < A.rank ? r0 : 0)) * T::ES;
          const u32x4 v = settle_inside<DT, MODE>(ld_inside<DT, MODE>(p, w_last, A.rank - r0), p, w_last, A.rank - r0);
#pragma unroll
          for (int k = 0; k < TILES; ++k)
            if (k == j) w[f][k] = v;
        }
      }
    }
  };
  // base of tile t of the rows; the first one's is under way with the weights and u
  Quad<DT> out[TILES];
  auto fetch = [&](int64_t n0, int t) {
    const int64_t left = A.out - n0 - 4 * q, row = R.row(16 * t + i);
    const bool in = n0 + COLS <= A.out;
#pragma unroll
    for (int j = 0; j < TILES; ++j) out[j] = Quad<DT>{};
    if (A.base && 16 * t + i < n) {
      const uint8_t *from = A.base + (row * A.ld_base + 4 * q + n0) * T::ES;
#pragma unroll
      for (int j = 0; j < TILES; ++j) out[j].load(from + 16 * j * T::ES, left - 16 * j, in);
    }
  };
  if (own >= 0 && first < runs) load(first * COLS);
  if (first < runs) fetch(first * COLS, 0);
  if (own >= 0) {
    if (16 * wave < n) {  // u's fragments, wave w those of tile w
      const float s = A.scale ? A.scale[own] : 1.0f;
      const float *up = A.u + R.row(16 * wave + i) * A.rank;
      const uint8_t *u_last = reinterpret_cast<const uint8_t *>(A.u + A.tokens * A.rank - 4);
      u32x4 uf[X::UF];
      X::u_frags(uf, A.rank, q, [&](float(&v)[T::PE], int r, int rest) {
#pragma unroll
        for (int e = 0; e < T::PE; ++e) v[e] = 0.0f;
#pragma unroll 2
        for (int k = 0; k < A.splits; ++k) {
#pragma unroll
          for (int h = 0; h < T::PE; h += 4) {
            const uint8_t *p = reinterpret_cast<const uint8_t *>(up + k * A.part + (rest > h ? r + h : 0));
            const uint8_t *end = u_last + k * A.part * 4;
            const u32x4 g = settle_inside<kF32, MODE>(ld_inside<kF32, MODE>(p, end, rest - h), p, end, rest - h);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h + e] += bits_f32(g[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < T::PE; ++e) v[e] *= s;
      });
#pragma unroll
      for (int f = 0; f < X::UF; ++f) us[wave][f][lane] = uf[f];
    }
  }
  static_assert(kFewWaves >= kWindow / 16, "a wave for every tile's fragments");
  __syncthreads();
  for (int64_t run = first; run < runs; run += step) {
    const int64_t n0 = run * COLS, left = A.out - n0 - 4 * q;
    const bool in = n0 + COLS <= A.out;
    if (run > first) {
      if (own >= 0) load(n0);
      fetch(n0, 0);
    }
    bool settled = full || !inside(n0);
#pragma unroll 1
    for (int t = 0; 16 * t < n; ++t) {  // (the weights stay for all tiles of rows)
      const int64_t row = R.row(16 * t + i);
      const bool wanted = 16 * t + i < n;
      if (t > 0) fetch(n0, t);
      if (own >= 0) {
        if (!settled) {
#pragma unroll
          for (int f = 0; f < F; ++f)
#pragma unroll
            for (int j = 0; j < TILES; ++j) w[f][j] = only<DT>(w[f][j], A.rank - X::rank0(f, q));
          settled = true;
        }
        u32x4 uf[X::UF];
#pragma unroll
        for (int f = 0; f < X::UF; ++f) uf[f] = us[t][f][lane];
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
          f32x4 acc = {0, 0, 0, 0};
#pragma unroll
          for (int f = 0; f < X::UF; ++f) acc = mma<DT>(w[f % F][j], uf[f], acc);
          out[j].add(acc);
        }
      }
      if (wanted && (own >= 0 || A.base != A.y)) {
        uint8_t *to = A.y + (row * A.ldy + 4 * q + n0) * T::ES;
#pragma unroll
        for (int j = 0; j < TILES; ++j) out[j].store(to + 16 * j * T::ES, left - 16 * j, in);
      }
    }
  }
  if (A.u_out && blockIdx.y == 0) {
    const int count = n * A.rank;
    for (int e0 = 0; e0 < count; e0 += 64 * kFewWaves) {
      const int e = e0 + threadIdx.x, t = e / A.rank;
      const int64_t at = R.row(t) * A.rank + (e - t * A.rank);  // (every lane takes part)
      if (e < count) A.u_out[at] = own >= 0 ? parts_sum(A.u + at, A.part, A.splits) : 0.0f;
    }
  }
}

template <int DT, int RT, int MODE>
__global__ __launch_bounds__(64 * kFewWaves) void adapter_few_y_kernel(FewArgs A) {
  __shared__ u32x4 us[kWindow / 16][Expand<DT, frag_count<DT>(RT), false, MODE>::UF][64];
  const int m = blockIdx.x;
  if (m >= A.tokens) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const FewRows R(A, m, lane);
  if (!R.mine) return;
  few_y<DT, RT, MODE>(A, R, us, lane, wave);
}

// Few rows, and few of an adapter: up to 16 on average, one tile; the weights' reading is all there is.
// (4096 -> 4096, rank 16, 48 adapters: 32 / 256 / 512 rows take 9.5 / 13.4 / 22.0 us, as many rows 42.9 /
// 29.1 / 23.7; one adapter: 16 / 32 / 256 rows 9.5 / 12.2 / 19.7, as many 13.1 / 13.6 / 13.7; 4096 -> 14336, rank
// 64, 8 adapters: 128 / 256 rows 22.7 / 37.3, as many 29.5 / 26.1.  A's rows are reached by 32-bit distances.)
bool few_rows(const AdapterLaunch &L) {
  return L.tokens <= 256 && L.tokens <= 16 * (int64_t)L.adapters && L.rank * L.in < (int64_t)1 << 29;
}

// Parts of the long dimension, for about 512 workgroups, each wave with 8 KB or more of an
// adapter's weights.
int few_splits(const AdapterLaunch &L) {
  const int64_t most = L.adapters < L.tokens ? L.adapters : L.tokens;
  const int64_t useful = (L.in * L.rank * (L.dtype == kBF16 ? 2 : 4) + 8192 * kFewWaves - 1) / (8192 * kFewWaves);
  int64_t s = most > 0 ? 512 / most : 1;
  if (s > useful) s = useful;
  // y's kernel adds the parts up (up to 1 / 2 / 4 / 8 / 12 parts, 4096 -> 4096: one token of rank 16 10.6 / 8.8 /
  // 8.3 / 8.3 / 8.3 us, rank 64 23.4 / 16.1 / 12.9 / 13.0 / 15.2, rank 128 40.6 / 26.7 / 20.2 / 18.8 / 21.7; 64 tokens
  // of 48 adapters, rank 16, 8192 -> 28672 28.8 / 25.6 / 25.0 / 27.1 / 27.1, rank 64, 4096 -> 4096
  // 30.2 / 22.6 / 19.9 / 21.7 / 23.1)
  constexpr int cap = 4;
  if (s > cap) s = cap;
  return s < 1 ? 1 : (int)s;
}

template <int DT>
hipError_t launch_few(const AdapterLaunch &L, hipStream_t stream) {
  const int cols = 16 * kFewTiles;
  const int64_t most = L.adapters < L.tokens ? L.adapters : L.tokens;
  const int64_t useful = ((L.out + cols - 1) / cols + kFewWaves - 1) / kFewWaves;
  int64_t parts = 2048 / most;  // (48 adapters, 8192 -> 28672, both kernels: 26.1 us; twice as many 27.7, two thirds 24.0; 4096 -> 14336 alike)
  if (parts > useful) parts = useful;
  if (parts < 1) parts = 1;
  const int splits = few_splits(L), mode = piece_mode(DT, L.tokens, L.in, L.out, L.rank);
  float *u = splits == 1 && L.u ? L.u : L.workspace;
  FewArgs A{static_cast<const uint8_t *>(L.x), static_cast<const uint8_t *>(L.a), static_cast<const uint8_t *>(L.b), L.ids,
            L.scale, static_cast<const uint8_t *>(L.base), static_cast<uint8_t *>(L.y), u, L.u, L.tokens, L.in, L.out, L.ldx,
            L.ld_base, L.ldy, L.tokens * L.rank, L.adapters, L.rank, splits, (int)parts};
  // (an odd number of rows: the parts of one go to all XCDs in turn)
  by_rank_and_mode(L.rank, mode, [&](auto rt, auto m) {
    adapter_few_u_kernel<DT, decltype(rt)::value, decltype(m)::value>
        <<<dim3((unsigned)L.tokens | 1, (unsigned)splits), 64 * kFewWaves, 0, stream>>>(A);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  by_rank_and_mode(L.rank, mode, [&](auto rt, auto m) {
    adapter_few_y_kernel<DT, decltype(rt)::value, decltype(m)::value>
        <<<dim3((unsigned)L.tokens | 1, (unsigned)parts), 64 * kFewWaves, 0, stream>>>(A);
  });
  return hipGetLastError();
}

template <int DT>
hipError_t launch_many(const AdapterLaunch &L, hipStream_t stream) {
  const int splits = shrink_splits(L.tokens, L.in), mode = piece_mode(DT, L.tokens, L.in, L.out, L.rank);
  float *u = splits == 1 && L.u ? L.u : L.workspace;
  const int64_t part = L.tokens * L.rank;
  ShrinkArgs S{static_cast<const uint8_t *>(L.x), static_cast<const uint8_t *>(L.a), L.ids, nullptr, u, L.tokens, L.ldx,
               L.in, part, L.adapters, L.rank, splits, shrink_slots(L.tokens, L.adapters, splits),
               window_count(L.tokens)};
  const hipError_t e = launch_shrink<DT, false>(S, PlanArgs{}, mode, stream);
  if (e != hipSuccess) return e;
  ExpandArgs E{u, static_cast<const uint8_t *>(L.b), L.ids, L.scale, static_cast<const uint8_t *>(L.base),
               static_cast<uint8_t *>(L.y), u == L.u ? nullptr : L.u, L.tokens, L.out, L.ld_base, L.ldy, part,
               L.adapters, L.rank, splits};
  return launch_expand<DT, false>(E, mode, stream);
}

}  // namespace

int64_t adapter_workspace(const AdapterLaunch &L) {
  return L.tokens * L.rank * (few_rows(L) ? few_splits(L) : shrink_splits(L.tokens, L.in));
}

hipError_t launch_adapter(const AdapterLaunch &L, hipStream_t stream) {
  if (few_rows(L)) return L.dtype == kBF16 ? launch_few<kBF16>(L, stream) : launch_few<kF32>(L, stream);
  return L.dtype == kBF16 ? launch_many<kBF16>(L, stream) : launch_many<kF32>(L, stream);
}

}  // namespace mxfp4
