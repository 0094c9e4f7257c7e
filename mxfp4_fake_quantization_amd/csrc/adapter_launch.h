// adapter_launch.h -- the shrink and expand kernels of the low-rank adapters
// (adapter_device.h) and their launches, for the forward pass (ACROSS false) and
// the backward pass (ACROSS true: the transposed weights).
#pragma once

#include "adapter_device.h"

namespace mxfp4 {
namespace {

struct ShrinkArgs {
  const uint8_t *x, *w;
  const int32_t *ids;
  const float *scale;  // of each adapter, or NULL
  float *u;            // [splits][tokens, rank]
  int64_t tokens, ldx, K, part;
  int adapters, rank, splits;
};

struct ExpandArgs {
  const float *u;
  const uint8_t *w;
  const int32_t *ids;
  const float *scale;
  const uint8_t *base;
  uint8_t *y;
  float *u_out;        // the sum of the splits, where it is wanted apart
  int64_t tokens, N, ld_base, ldy, part;
  int adapters, rank, splits;
};

// ---- rows in adapter order ---------------------------------------------------------
//
// The weight gradients sum over an adapter's rows, wherever they are: a stable
// counting sort of the tokens by adapter, cut into pieces of at most `rows` rows
// of one adapter.  One workgroup does it while the others of the same launch
// compute du.

struct PlanArgs {
  int32_t *order;   // [tokens] rows, sorted by adapter
  int32_t *first;   // [adapters + 1] each adapter's first piece, and their number
  int4 *pieces;     // adapter, first place in order, rows
  int rows, bits;   // bits of an adapter's number
};

template <int WAVES>
__device__ void plan_rows(const PlanArgs &P, const int32_t *ids, int64_t tokens, int adapters, int32_t *cnt) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < WAVES * adapters; e += 64 * WAVES) cnt[e] = 0;
  __syncthreads();
  const int64_t part = (tokens + 64 * WAVES - 1) / (64 * WAVES) * 64;
  const int64_t lo = wave * part, hi = lo + part < tokens ? lo + part : tokens;
  int32_t *mine = cnt + wave * adapters;
  for (int64_t i = lo + lane; i < hi; i += 64) {
    const int id = row_adapter(ids, i, adapters);
    if (id >= 0) atomicAdd(&mine[id], 1);  // a count: the order of the additions does not matter
  }
  __syncthreads();
  if (wave == 0) {  // first places and pieces, 64 adapters at a time
    int32_t at = 0, piece = 0;
    for (int e0 = 0; e0 < adapters; e0 += 64) {
      const int e = e0 + lane;
      int32_t total = 0;
      if (e < adapters)
        for (int w = 0; w < WAVES; ++w) total += cnt[w * adapters + e];
      const int32_t np = (total + P.rows - 1) / P.rows;
      int32_t st = total, sp = np;
      for (int d = 1; d < 64; d <<= 1) {
        const int32_t ot = __shfl_up(st, d), op = __shfl_up(sp, d);
        if (lane >= d) {
          st += ot;
          sp += op;
        }
      }
      int32_t start = at + st - total;
      const int32_t fp = piece + sp - np;
      at += __shfl(st, 63);
      piece += __shfl(sp, 63);
      if (e < adapters) {
        P.first[e] = fp;
        for (int p = 0; p < np; ++p) {
          const int32_t left = total - p * P.rows;
          P.pieces[fp + p] = make_int4(e, start + p * P.rows, left < P.rows ? left : P.rows, 0);
        }
        for (int w = 0; w < WAVES; ++w) {
          const int32_t c = cnt[w * adapters + e];
          cnt[w * adapters + e] = start;
          start += c;
        }
      }
    }
    if (lane == 0) P.first[adapters] = piece;
  }
  __syncthreads();
  // Every lane of a wave takes part in the ballots: the loop count is the wave's.
  for (int64_t base = lo; base < hi; base += 64) {
    const int64_t i = base + lane;
    const int id = i < hi ? row_adapter(ids, i, adapters) : -1;
    uint64_t same = __ballot(id >= 0);
    for (int b = 0; b < P.bits; ++b) {
      const uint64_t on = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? on : ~on;
    }
    if (id >= 0) {
      const int32_t at = mine[id];
      P.order[at + __popcll(same & ((1ull << lane) - 1))] = (int32_t)i;
      // the group's last lane moves the count on (a wave's LDS operations keep
      // their order: the reads above come first)
      if ((same >> lane) == 1ull) mine[id] = at + (int32_t)__popcll(same);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- shrink ----------------------------------------------------------------------
//
// A workgroup takes tiles of 16 MT rows of one adapter in a window; its eight
// waves share out the blocks of the long dimension and add their parts in LDS, in
// the order of the waves.

constexpr int kShrinkWaves = 8;

template <int DT, int RT, int MT, bool ACROSS>
__global__ __launch_bounds__(64 * kShrinkWaves) void adapter_shrink_kernel(ShrinkArgs A, PlanArgs P) {
  using T = Tile<DT>;
  __shared__ f32x4 part[kShrinkWaves][MT * RT][64];
  int block = blockIdx.x;
  if constexpr (ACROSS) {  // the backward pass
    if (P.order && --block < 0) {
      __shared__ int32_t cnt[kShrinkWaves * kAdapterMaxTrained];
      plan_rows<kShrinkWaves>(P, A.ids, A.tokens, A.adapters, cnt);
      return;
    }
  }
  constexpr int SLOTS = kWindow / (16 * MT);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
  const int64_t row0 = (int64_t)(block / SLOTS) * kWindow;
  const int slot = block % SLOTS;
  const bool live = row0 + lane < A.tokens;
  const int id = live ? row_adapter(A.ids, row0 + lane, A.adapters) : -1;
  float *u = A.u + (int64_t)blockIdx.y * A.part;
  const int64_t blocks = (A.K + 4 * T::KF - 1) / (4 * T::KF);
  const int64_t lo = blocks * blockIdx.y / A.splits, hi = blocks * (blockIdx.y + 1) / A.splits;
  // rows without an adapter: u = 0
  if (slot == 0 && wave == 0 && live && id < 0)
    for (int r = 0; r < A.rank; ++r) u[(row0 + lane) * A.rank + r] = 0.0f;
  int seen = 0;
  for (uint64_t rem = __ballot(id >= 0); rem;) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(rem));
    const uint64_t match = __ballot(id == a);
    rem &= ~match;
    const int n = __popcll(match), tiles = (n + 16 * MT - 1) / (16 * MT);
    const int line = lined_up(match, lane);
    const uint8_t *w = A.w + (int64_t)a * A.rank * A.K * T::ES;
    // this workgroup's tiles of the window's: slot, slot + SLOTS, ...
    for (int j = (slot - seen % SLOTS + SLOTS) % SLOTS; j < tiles; j += SLOTS) {
      const uint8_t *xrow[MT];
      int row[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int at = 16 * (j * MT + m) + i;
        const int to = __builtin_amdgcn_ds_bpermute(at << 2, line);  // (every lane takes part)
        row[m] = at < n ? to : -1;
      }
      const int first = __builtin_amdgcn_readfirstlane(row[0]);  // at 16 j MT < n
#pragma unroll
      for (int m = 0; m < MT; ++m) xrow[m] = A.x + (row0 + (row[m] < 0 ? first : row[m])) * A.ldx * T::ES;
      f32x4 acc[MT][RT];
      shrink_part<DT, RT, MT, ACROSS>(acc, xrow, w, A.K, A.rank, lo + wave, hi, kShrinkWaves, lane);
      __syncthreads();  // the tile before has been read
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r) part[wave][m * RT + r][lane] = acc[m][r];
      __syncthreads();
      const float s = A.scale ? A.scale[a] : 1.0f;
      for (int e = wave; e < MT * RT; e += kShrinkWaves) {
        f32x4 sum = part[0][e][lane];
#pragma unroll
        for (int v = 1; v < kShrinkWaves; ++v) sum += part[v][e][lane];
        const int at = 16 * (j * MT + e / RT) + i;
        const int to = __builtin_amdgcn_ds_bpermute(at << 2, line);
        const int r0 = 16 * (e % RT) + 4 * q;
        if (at < n) {
          float *p = u + (row0 + to) * A.rank + r0;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (r0 + v < A.rank) p[v] = s * sum[v];
        }
      }
    }
    seen += tiles;
  }
}

// ---- expand ----------------------------------------------------------------------

constexpr int kExpandWaves = 4;

template <int DT, int NF, bool ACROSS>
__global__ __launch_bounds__(64 * kExpandWaves) void adapter_expand_kernel(ExpandArgs A, int chunks) {
  using T = Tile<DT>;
  using X = Expand<DT, NF, ACROSS>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
  const int64_t row0 = (int64_t)(blockIdx.x / chunks) * kWindow;
  const int chunk = blockIdx.x % chunks;
  const int64_t n0 = ((int64_t)chunk * kExpandWaves + wave) * X::COLS;
  const bool live = row0 + lane < A.tokens;
  const int id = live ? row_adapter(A.ids, row0 + lane, A.adapters) : -1;
  if (A.u_out && chunk == 0) {
    const int64_t from = row0 * A.rank;
    const int64_t count = (A.tokens - row0 < kWindow ? A.tokens - row0 : kWindow) * A.rank;
    for (int64_t e = threadIdx.x; e < count; e += 64 * kExpandWaves) {
      float s = A.u[from + e];
      for (int k = 1; k < A.splits; ++k) s += A.u[k * A.part + from + e];
      A.u_out[from + e] = s;
    }
  }
  if (n0 >= A.N) return;
  const bool inside = n0 + X::COLS <= A.N, whole = A.rank % T::PE == 0;
  for (uint64_t rem = __ballot(live); rem;) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(rem));
    const uint64_t match = __ballot(id == a) & __ballot(live);
    rem &= ~match;
    const int n = __popcll(match);
    const int line = lined_up(match, lane);
    if (a < 0 && A.base == A.y) continue;  // already there
    X W;
    if (a >= 0) W.load(A.w + (int64_t)a * A.N * A.rank * T::ES, A.N, A.rank, n0, lane);
    const float s = a >= 0 && A.scale ? A.scale[a] : 1.0f;
    for (int j = 0; 16 * j < n; ++j) {
      const int at = 16 * j + i;
      const int to = __builtin_amdgcn_ds_bpermute((at < n ? at : 16 * j) << 2, line);
      const int64_t row = row0 + to;
      u32x4 base[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int64_t col = n0 + X::piece(p, q);
        const uint8_t *from = A.base + (row * A.ld_base + col) * T::ES;
        if (!A.base) base[p] = u32x4{0, 0, 0, 0};
        else if (inside) base[p] = ld_frag(from);
        else base[p] = ld_frag_n<DT>(from, A.N - col);
      }
      if (a >= 0) {
        u32x4 uf[X::UF];
        X::u_frags(uf, A.rank, q, [&](float(&v)[T::PE], int r, int left) {
          const float *up = A.u + row * A.rank + (whole && left <= 0 ? 0 : r);
#pragma unroll
          for (int e = 0; e < T::PE; ++e) v[e] = 0.0f;
          for (int k = 0; k < A.splits; ++k) {
#pragma unroll
            for (int h = 0; h < T::PE; h += 4) {
              const uint8_t *p = reinterpret_cast<const uint8_t *>(up + k * A.part + h);
              const u32x4 t = whole ? ld_frag(p) : ld_frag_n<kF32>(p, left - h);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[h + e] += bits_f32(t[e]);
            }
          }
#pragma unroll
          for (int e = 0; e < T::PE; ++e) v[e] = whole && left <= 0 ? 0.0f : v[e] * s;
        });
        f32x4 acc[T::PE];
        W.product(acc, uf);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          float f[T::PE];
#pragma unroll
          for (int e = 0; e < T::PE; ++e) f[e] = X::at(acc, p, e);
          base[p] = add_base<DT>(base[p], f);
        }
      }
      if (at < n) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int64_t col = n0 + X::piece(p, q);
          uint8_t *to_y = A.y + (row * A.ldy + col) * T::ES;
          if (inside) *reinterpret_cast<u32x4_a1 *>(to_y) = base[p];
          else st_frag_n<DT>(to_y, base[p], A.N - col);
        }
      }
    }
  }
}

// ---- launches ----------------------------------------------------------------------

// Parts of the long dimension: as many as fill the chip's 256 CUs twice, each with
// work for the eight waves.
inline int shrink_splits(int64_t tokens, int64_t K) {
  const int64_t groups = (tokens + 15) / 16;
  const int64_t most = (K + 1023) / 1024;
  int64_t s = 512 / (groups > 0 ? groups : 1);
  if (s > most) s = most;
  return s < 1 ? 1 : (int)s;
}

template <int DT, bool ACROSS>
hipError_t launch_shrink_dt(const ShrinkArgs &A, const PlanArgs &P, hipStream_t stream) {
  const int64_t windows = (A.tokens + kWindow - 1) / kWindow;
  const int rt = (A.rank + 15) / 16;
  const dim3 grid((unsigned)(windows * 4 + (P.order ? 1 : 0)), A.splits);
  const int th = 64 * kShrinkWaves;
  if (rt <= 1) adapter_shrink_kernel<DT, 1, 1, ACROSS><<<grid, th, 0, stream>>>(A, P);
  else if (rt <= 2) adapter_shrink_kernel<DT, 2, 1, ACROSS><<<grid, th, 0, stream>>>(A, P);
  else if (rt <= 4) adapter_shrink_kernel<DT, 4, 1, ACROSS><<<grid, th, 0, stream>>>(A, P);
  else adapter_shrink_kernel<DT, 8, 1, ACROSS><<<grid, th, 0, stream>>>(A, P);
  return hipGetLastError();
}

template <bool ACROSS>
hipError_t launch_shrink(int dtype, const ShrinkArgs &A, const PlanArgs &P, hipStream_t stream) {
  return dtype == kBF16 ? launch_shrink_dt<kBF16, ACROSS>(A, P, stream) : launch_shrink_dt<kF32, ACROSS>(A, P, stream);
}

template <int DT, bool ACROSS>
hipError_t launch_expand_dt(const ExpandArgs &A, hipStream_t stream) {
  const int64_t windows = (A.tokens + kWindow - 1) / kWindow;
  const int64_t cols = kExpandWaves * Expand<DT, 1, ACROSS>::COLS;
  const int chunks = (int)((A.N + cols - 1) / cols);
  const int rt = (A.rank + 15) / 16;
  const dim3 grid((unsigned)(windows * chunks));
  const int th = 64 * kExpandWaves;
  if (rt <= 1) adapter_expand_kernel<DT, frag_count<DT>(1), ACROSS><<<grid, th, 0, stream>>>(A, chunks);
  else if (rt <= 2) adapter_expand_kernel<DT, frag_count<DT>(2), ACROSS><<<grid, th, 0, stream>>>(A, chunks);
  else if (rt <= 4) adapter_expand_kernel<DT, frag_count<DT>(4), ACROSS><<<grid, th, 0, stream>>>(A, chunks);
  else adapter_expand_kernel<DT, frag_count<DT>(8), ACROSS><<<grid, th, 0, stream>>>(A, chunks);
  return hipGetLastError();
}

template <bool ACROSS>
hipError_t launch_expand(int dtype, const ExpandArgs &A, hipStream_t stream) {
  return dtype == kBF16 ? launch_expand_dt<kBF16, ACROSS>(A, stream) : launch_expand_dt<kF32, ACROSS>(A, stream);
}

}  // namespace
}  // namespace mxfp4
