// adapter_launch.h -- the shrink and expand kernels of the low-rank adapters
// (adapter_device.h) and their launches, for the forward pass (ACROSS false) and
// the backward pass (ACROSS true: the transposed weights).
#pragma once

#include "adapter_device.h"

#include <type_traits>

namespace mxfp4 {
namespace {

struct ShrinkArgs {
  const uint8_t *x, *w;
  const int32_t *ids;
  const float *scale;  // of each adapter, or NULL
  float *u;            // [splits][tokens, rank]
  int64_t tokens, ldx, K, part;
  int adapters, rank, splits, slots;
  int windows;         // 0: only the plan is wanted
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
// of one adapter.  It runs in workgroups of its own beside those that compute du, each
// of which counts all tokens and places a part of them (one workgroup for all took 34 us
// for 16384 tokens, longer than du).

struct PlanArgs {
  int32_t *order;   // [tokens] rows, sorted by adapter
  int32_t *first;   // [adapters + 1] each adapter's first piece, and their number
  int4 *pieces;     // adapter, first place in order, rows
  int rows, bits;   // bits of an adapter's number
  int blocks;       // workgroups
};

constexpr int kPlanStep = 256;  // tokens of a wave's step: four a lane

inline int plan_blocks(int64_t tokens) {
  const int64_t b = (tokens + 1023) / 1024;
  return b > 64 ? 64 : b < 1 ? 1 : (int)b;
}

// lds: (WAVES + 2) * adapters numbers.
template <int WAVES>
__device__ void plan_rows(const PlanArgs &P, const int32_t *ids, int64_t tokens, int adapters, int32_t *lds, int block) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int32_t *total = lds, *before = lds + adapters, *cnt = lds + 2 * adapters;
  for (int e = tid; e < (WAVES + 2) * adapters; e += 64 * WAVES) lds[e] = 0;
  __syncthreads();
  const int64_t chunk = (tokens + (int64_t)P.blocks * kPlanStep - 1) / ((int64_t)P.blocks * kPlanStep) * kPlanStep;
  const int64_t lo = block * chunk < tokens ? block * chunk : tokens, hi = lo + chunk < tokens ? lo + chunk : tokens;
  // All tokens, a step of 256 a wave, two steps' loads at a time; a step of one adapter, as
  // most are, is one addition.  (Integer sums: any order.)
  constexpr int AHEAD = 2;
  for (int64_t base = wave * kPlanStep; base < tokens; base += AHEAD * WAVES * kPlanStep) {
    int32_t id[AHEAD][4];
#pragma unroll
    for (int s = 0; s < AHEAD; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t i = base + s * WAVES * kPlanStep + 4 * lane + e;
        const int v = ids ? ids[i < tokens ? i : tokens - 1] : 0;
        id[s][e] = i < tokens && v >= 0 && v < adapters ? v : -1;
      }
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) {
      const bool early = base + s * WAVES * kPlanStep < lo;  // (lo is a multiple of the step)
      const int one = __builtin_amdgcn_readfirstlane(id[s][0]);
      const bool alike = id[s][0] == one && id[s][1] == one && id[s][2] == one && id[s][3] == one;
      if (__ballot(alike) == ~0ull) {
        if (lane == 0 && one >= 0) {
          atomicAdd(&total[one], kPlanStep);
          if (early) atomicAdd(&before[one], kPlanStep);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (id[s][e] >= 0) {
            atomicAdd(&total[id[s][e]], 1);
            if (early) atomicAdd(&before[id[s][e]], 1);
          }
      }
    }
  }
  // this workgroup's tokens by wave
  const int64_t part = chunk / WAVES, wlo = lo + wave * part < hi ? lo + wave * part : hi;
  const int64_t whi = wlo + part < hi ? wlo + part : hi;
  int32_t *mine = cnt + wave * adapters;
  for (int64_t i = wlo + lane; i < whi; i += 64) {
    const int id = row_adapter(ids, i, adapters);
    if (id >= 0) atomicAdd(&mine[id], 1);
  }
  __syncthreads();
  if (wave == 0) {  // first places and pieces, 64 adapters at a time
    int32_t at = 0, piece = 0;
    for (int e0 = 0; e0 < adapters; e0 += 64) {
      const int e = e0 + lane;
      const int32_t n = e < adapters ? total[e] : 0;
      const int32_t np = (n + P.rows - 1) / P.rows;
      int32_t st = n, sp = np;
      for (int d = 1; d < 64; d <<= 1) {
        const int32_t ot = __shfl_up(st, d), op = __shfl_up(sp, d);
        if (lane >= d) {
          st += ot;
          sp += op;
        }
      }
      const int32_t start = at + st - n, fp = piece + sp - np;
      at += __shfl(st, 63);
      piece += __shfl(sp, 63);
      if (e < adapters) {
        if (block == 0) {
          P.first[e] = fp;
          for (int p = 0; p < np; ++p) {
            const int32_t left = n - p * P.rows;
            P.pieces[fp + p] = make_int4(e, start + p * P.rows, left < P.rows ? left : P.rows, 0);
          }
        }
        int32_t here = start + before[e];
        for (int w = 0; w < WAVES; ++w) {
          const int32_t c = cnt[w * adapters + e];
          cnt[w * adapters + e] = here;
          here += c;
        }
      }
    }
    if (lane == 0 && block == 0) P.first[adapters] = piece;
  }
  __syncthreads();
  // Every lane of a wave takes part in the ballots: the loop count is the wave's.
  for (int64_t base = wlo; base < whi; base += 64) {
    const int64_t i = base + lane;
    const int id = i < whi ? row_adapter(ids, i, adapters) : -1;
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

// Workgroup id -> place in [0, total) such that each of the 8 XCDs (workgroups go to
// them in turn) has a run of consecutive places: neighbouring windows mostly hold one
// adapter, whose weights then stay in that XCD's L2.
__device__ __forceinline__ int64_t xcd_share(int64_t id, int64_t total) {
  const int64_t q = total >> 3, r = total & 7, x = id & 7;
  return x * q + (x < r ? x : r) + (id >> 3);
}

// ---- shrink ----------------------------------------------------------------------
//
// A workgroup takes the rows of one adapter in a window of 64, wave w the w-th 16 of
// them, over a part of the long dimension.  256 bytes of every row and of every
// rank's weights at a time go through LDS (two buffers, the next block's loads in
// flight during a block's products): global reads are 256 consecutive bytes of a
// row, and the weights are read once for all four waves.  Piece p of LDS row r lies
// at p ^ (r % 16), which spreads a fragment's 16 rows over all banks.  Bound by reading x
// (8192 x 7168 bf16, 16 adapters of rank 32: 35 us, 3.6 TB/s; 4096 x 4096 fp32, rank 8:
// 14.4 us, 4.7 TB/s).
//
// Windows of several adapters: workgroup `slot` of a window takes every slots-th of
// its adapters.

constexpr int kShrinkWaves = 4, kShrinkThreads = 64 * kShrinkWaves;
constexpr int kBlockBytes = 256, kPieces = kBlockBytes / 16;

__device__ __forceinline__ int piece_at(int row, int piece) { return row * kPieces + (piece ^ (row & 15)); }

template <int DT, int RT, bool ACROSS, int MODE>
__global__ __launch_bounds__(kShrinkThreads) void adapter_shrink_kernel(ShrinkArgs A, PlanArgs P) {
  using T = Tile<DT>;
  constexpr int BK = kBlockBytes / T::ES;        // elements of a block
  constexpr int XP = kWindow * kPieces / kShrinkThreads;  // pieces of x a thread stages
  // pieces of W: of its rows, or (ACROSS) squares of PE x PE elements, PE pieces each
  constexpr int WT = ACROSS ? kPieces * (16 * RT / T::PE) : 16 * RT * kPieces;
  constexpr int WP = (WT + kShrinkThreads - 1) / kShrinkThreads, WN = ACROSS ? T::PE : 1;
  __shared__ u32x4 xs[2][kWindow * kPieces];
  __shared__ u32x4 ws[2][16 * RT * kPieces];
  int64_t block = blockIdx.x;
  if constexpr (ACROSS) {  // the backward pass
    if (P.order) {
      static_assert(sizeof xs >= sizeof(int32_t) * (kShrinkWaves + 2) * kAdapterMaxTrained, "the plan's counts");
      if (block < P.blocks)
        plan_rows<kShrinkWaves>(P, A.ids, A.tokens, A.adapters, reinterpret_cast<int32_t *>(xs), (int)block);
      block -= (P.blocks + 7) / 8 * 8;  // (the others keep their XCDs)
      if (block < 0) return;
    }
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, q = lane >> 4;
  // (window, part) pairs, in the outer order of the slots: those of windows with one
  // adapter have nothing to do
  const int64_t pairs = (int64_t)A.windows * A.splits;
  const int slot = (int)(block / ((pairs + 7) / 8 * 8));
  block -= slot * ((pairs + 7) / 8 * 8);
  if (block >= pairs) return;
  const int64_t pair = xcd_share(block, pairs);
  const int split = (int)(pair % A.splits);
  const int64_t row0 = pair / A.splits * kWindow;
  const bool live = row0 + lane < A.tokens;
  const int id = live ? row_adapter(A.ids, row0 + lane, A.adapters) : -1;
  float *u = A.u + split * A.part;
  const int64_t blocks = (A.K + BK - 1) / BK;
  const int64_t lo = blocks * split / A.splits, hi = blocks * (split + 1) / A.splits;
  // rows without an adapter: u = 0
  if (slot == 0 && wave == 0 && live && id < 0)
    for (int r = 0; r < A.rank; ++r) u[(row0 + lane) * A.rank + r] = 0.0f;
  int seen = 0;
  for (uint64_t rem = __ballot(id >= 0); rem; ++seen) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(rem));
    const uint64_t match = __ballot(id == a);
    rem &= ~match;
    if (seen % A.slots != slot) continue;
    const int n = __popcll(match);
    const int line = lined_up(match, lane);
    const uint8_t *w = A.w + (int64_t)a * A.rank * A.K * T::ES;
    // the thread's rows of x: tid / 16 and every 16th from there (rows past the last repeat it)
    const uint8_t *xrow[XP];
#pragma unroll
    for (int j = 0; j < XP; ++j) {
      const int r = tid / kPieces + j * (kShrinkThreads / kPieces);
      const int to = __builtin_amdgcn_ds_bpermute((r < n ? r : n - 1) << 2, line);
      xrow[j] = A.x + (row0 + to) * A.ldx * T::ES;
    }
    const uint8_t *w_last = w + A.K * A.rank * T::ES - 16;
    struct Stage {
      u32x4 x[XP], w[WP][WN];
    };
    Stage s0, s1;  // blocks on their way
    // Block blk; WHOLE: it lies inside the rows.  No load hangs on a condition (but for
    // kSingle), so the compiler waits for the loads it needs, not for all under way.
    auto load = [&](Stage &S, int64_t blk, auto whole) {
      constexpr bool WHOLE = decltype(whole)::value;
      const int64_t k0 = blk * BK;
      const RowPiece<DT, MODE> xp(k0 + T::PE * (tid % kPieces), A.K);
#pragma unroll
      for (int j = 0; j < XP; ++j)
        S.x[j] = WHOLE ? ld_frag(xrow[j] + (k0 + T::PE * (tid % kPieces)) * T::ES) : xp.load(xrow[j]);
#pragma unroll
      for (int j = 0; j < WP; ++j) {
        const int e = tid + j * kShrinkThreads;
        if constexpr (ACROSS) {  // PE rows k of PE ranks (threads past the last square repeat it)
          const int t = WT % kShrinkThreads == 0 || e < WT ? e : WT - 1;
          const int64_t k = k0 + T::PE * (t % kPieces);
          const int r = T::PE * (t / kPieces);
#pragma unroll
          for (int v = 0; v < WN; ++v) {
            if constexpr (WHOLE) {  // (ranks past the last hold anything)
              S.w[j][v] = ld_frag(w + ((k + v) * A.rank + (r < A.rank ? r : 0)) * T::ES);
            } else {
              const uint8_t *p = w + ((k + v < A.K ? k + v : A.K - 1) * A.rank + (r < A.rank ? r : 0)) * T::ES;
              const u32x4 t = settle_inside<DT, MODE>(ld_inside<DT, MODE>(p, w_last, A.rank - r), p, w_last, A.rank - r);
              S.w[j][v] = k + v < A.K ? t : u32x4{0, 0, 0, 0};
            }
          }
        } else {
          const int r = e / kPieces;  // (WT is a multiple of the threads)
          const uint8_t *row = w + (r < A.rank ? r : A.rank - 1) * A.K * T::ES;
          const int64_t k = k0 + T::PE * (e % kPieces);
          S.w[j][0] = WHOLE ? ld_frag(row + k * T::ES) : RowPiece<DT, MODE>(k, A.K).load(row);
        }
      }
    };
    auto store = [&](const Stage &S, int buf) {
#pragma unroll
      for (int j = 0; j < XP; ++j)
        xs[buf][piece_at(tid / kPieces + j * (kShrinkThreads / kPieces), tid % kPieces)] = S.x[j];
#pragma unroll
      for (int j = 0; j < WP; ++j) {
        const int e = tid + j * kShrinkThreads;
        if constexpr (ACROSS) {
          if (WT % kShrinkThreads == 0 || e < WT)
#pragma unroll
            for (int v = 0; v < WN; ++v)
              ws[buf][piece_at(T::PE * (e / kPieces) + v, e % kPieces)] = turned<DT>(S.w[j], v);
        } else {
          ws[buf][piece_at(e / kPieces, e % kPieces)] = S.w[j][0];
        }
      }
    };
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0, 0, 0, 0};
    auto compute = [&](int buf) {
      if (16 * wave >= n) return;
#pragma unroll
      for (int c = 0; c < kPieces / 4; ++c) {
        const u32x4 xf = xs[buf][piece_at(16 * wave + i, 4 * c + q)];
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = mma<DT>(ws[buf][piece_at(16 * r + i, 4 * c + q)], xf, acc[r]);
      }
    };
    __syncthreads();  // the adapter before has been read
    // Two blocks' loads are under way while one is computed.  Workgroups start at
    // different blocks: rows a power of two apart would all ask the same few memory
    // channels at a time otherwise.
    using Yes = std::integral_constant<bool, true>;
    using No = std::integral_constant<bool, false>;
    // blocks inside the rows; (ACROSS) and whose pieces of short rows end inside W
    const int64_t inside = (A.K - (ACROSS && MODE != kExact ? T::PE : 0)) / BK;
    const int64_t full = hi <= inside ? hi : inside > lo ? inside : lo;
    const int64_t count = full - lo;
    if (count > 0) {
      int64_t next = lo + (pair / A.splits * 5) % count;
      auto following = [&]() {
        const int64_t here = next;
        if (++next == full) next = lo;
        return here;
      };
      load(s0, following(), Yes());
      load(s1, following(), Yes());
      store(s0, 0);
      __syncthreads();
      // (blocks past the last are loaded again and not used)
      for (int64_t b = 0; b < count; b += 2) {
        load(s0, following(), Yes());
        compute(0);
        store(s1, 1);
        __syncthreads();
        if (b + 1 < count) {
          load(s1, following(), Yes());
          compute(1);
          store(s0, 0);
          __syncthreads();
        }
      }
    }
    for (int64_t blk = full; blk < hi; ++blk) {
      load(s0, blk, No());
      __syncthreads();
      store(s0, 0);
      __syncthreads();
      compute(0);
    }
    const float s = A.scale ? A.scale[a] : 1.0f;
    const int at = 16 * wave + i;
    const int to = __builtin_amdgcn_ds_bpermute(at << 2, line);  // (every lane takes part)
    if (at < n) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int r0 = 16 * r + 4 * q;
        float *p = u + (row0 + to) * A.rank + r0;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (r0 + v < A.rank) p[v] = s * acc[r][v];
      }
    }
  }
}

// ---- expand ----------------------------------------------------------------------

constexpr int kExpandWaves = 4;

__device__ __forceinline__ float parts_sum(const float *u, int64_t part, int splits) {
  float s = u[0];
  for (int k = 1; k < splits; ++k) s += u[k * part];
  return s;
}

// A workgroup takes 64 rows by 4 waves of columns.  Everything that does not hang on
// the rows' adapters is under way before those are known: the base of all rows
// (the wave's 16 KB) and u, of which wave w makes the fragments of rows 16 w to 16 w +
// 15 for all.  Then the adapters of the window pass one after the other; a row takes
// the result of its own one, so that no other adapter's values (an infinity, say) reach it.
// Bound by the bytes of base and y: 8192 x 7168 bf16, rank 32 51.5 us (4.7 TB/s), 4096 x 4096
// fp32, rank 8 27.1 us (5.0 TB/s), both with their base.
// Rows of a workgroup: 64, with the 16-byte pieces of 128 columns a row; 32 in fp32, whose registers
// then leave room for a wave more.  (Both kernels of the forward, 4096 rows and columns, bf16 of rank 64 /
// 128: 36.9 / 69.1 us, with 32 rows 43.6 / 88.3.  fp32 of rank 8 41.7 us and, now that the tiles are
// kept apart below, 40.4 with 64 rows; rank 64 / 128 91.5 / 161.6, and 79.6 / 140.4.)
template <int DT>
constexpr int kExpandRows = DT == kBF16 ? 64 : 32;
static_assert(kExpandRows<kBF16> >= kAdapterLeastRows && kExpandRows<kF32> >= kAdapterLeastRows &&
                  kExpandWaves * 16 * Tile<kF32>::PE >= kAdapterLeastCols && 64 * kExpandWaves == 256,
              "the check of a call's size counts these tiles");
// Waves a SIMD; what lets the weights stay in registers.  (bf16 of rank 65 to 128, 1000 rows and columns:
// 41 us with one wave, 46 with two and registers spilled; 4096 rows and columns 69 and 62.  fp32 is
// faster with two and 12 to 19 spilled, 4096 rows and columns 162 us, else 193; 209 for the weights across
// ragged rows.)
template <int DT, int NF>
constexpr int kExpandOccupancy = NF <= 1 ? (DT == kBF16 ? 3 : 4) : DT == kBF16 && NF >= 4 ? 1 : 2;

template <int DT, int NF, bool ACROSS, int MODE>
__global__ __launch_bounds__(64 * kExpandWaves, (kExpandOccupancy<DT, NF>)) void adapter_expand_kernel(ExpandArgs A,
                                                                                                           int chunks) {
  using T = Tile<DT>;
  using X = Expand<DT, NF, ACROSS, MODE>;
  constexpr int ROWS = kExpandRows<DT>, TILES = ROWS / 16;
  __shared__ u32x4 us[TILES][X::UF][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, q = lane >> 4;
  const int64_t tile = xcd_share(blockIdx.x, gridDim.x);
  const int64_t row0 = tile / chunks * ROWS;
  const int chunk = (int)(tile % chunks);
  const int64_t n0 = ((int64_t)chunk * kExpandWaves + wave) * X::COLS;
  const int rows = A.tokens - row0 < ROWS ? (int)(A.tokens - row0) : ROWS;
  const int id = lane < rows ? row_adapter(A.ids, row0 + lane, A.adapters) : -2;
  const bool mine = n0 < A.N;  // (a wave past the columns still makes fragments)
  const bool inside = (int64_t)(chunk + 1) * kExpandWaves * X::COLS <= A.N && rows == ROWS;
  const int64_t col = n0 + T::PE * i;
  // out[j][v]: row 16 j + 4 q + v; base at first
  u32x4 out[TILES][4];
  if (inside && A.base) {
    const uint8_t *from = A.base + (row0 * A.ld_base + n0) * T::ES;
    const uint32_t mine_at = (4 * q * (uint32_t)A.ld_base + T::PE * i) * T::ES;  // (the rest is the wave's)
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {  // (unaligned rows share cache lines between their pieces)
        const uint8_t *p = from + (16 * j + v) * A.ld_base * T::ES + mine_at;
        out[j][v] = MODE == kExact ? ld_frag_nt(p) : ld_frag(p);
      }
  } else if (A.base && mine) {  // rows and columns past the last hold anything
    const RowPiece<DT, MODE> piece(col, A.N);
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * j + 4 * q + v;
        out[j][v] = piece.raw(A.base + (row0 + (r < rows ? r : rows - 1)) * A.ld_base * T::ES);
      }
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) out[j][v] = piece.settled(out[j][v]);
  } else {
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) out[j][v] = u32x4{0, 0, 0, 0};
  }
  const uint64_t live = ~0ull >> (64 - rows);
  uint64_t rem = __ballot(id >= 0);
  X W;
  auto weights = [&](int a) {
    if (mine) W.load({A.w + (int64_t)a * A.N * A.rank * T::ES, A.N, n0, A.rank, lane});
  };
  int a = 0;
  if (rem) {
    a = __builtin_amdgcn_readlane(id, __builtin_ctzll(rem));
    weights(a);
    if (wave < TILES) {
      // fragments of the rows' own u, the row's scale in it; 0 for a row without an adapter
      const int r_u = 16 * wave + i;
      const int own = __builtin_amdgcn_ds_bpermute(r_u << 2, id);
      const float s = own < 0 ? 0.0f : A.scale ? A.scale[own] : 1.0f;
      const float *up = A.u + (row0 + (r_u < rows ? r_u : rows - 1)) * A.rank;
      const uint8_t *u_last = reinterpret_cast<const uint8_t *>(A.u + A.tokens * A.rank - 4);
      u32x4 uf[X::UF];
      X::u_frags(uf, A.rank, q, [&](float(&v)[T::PE], int r, int left) {
#pragma unroll
        for (int e = 0; e < T::PE; ++e) v[e] = 0.0f;
        for (int k = 0; k < A.splits; ++k) {
#pragma unroll
          for (int h = 0; h < T::PE; h += 4) {
            const uint8_t *p = reinterpret_cast<const uint8_t *>(up + k * A.part + (left > h ? r + h : 0));
            const uint8_t *end = u_last + k * A.part * 4;
            const u32x4 t = settle_inside<kF32, MODE>(ld_inside<kF32, MODE>(p, end, left - h), p, end, left - h);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h + e] += bits_f32(t[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < T::PE; ++e) v[e] = own < 0 ? 0.0f : v[e] * s;
      });
#pragma unroll
      for (int f = 0; f < X::UF; ++f) us[wave][f][lane] = uf[f];
    }
    if (A.u_out && chunk == 0) {
      for (int e = threadIdx.x; e < rows * A.rank; e += 64 * kExpandWaves)
        A.u_out[row0 * A.rank + e] = parts_sum(A.u + row0 * A.rank + e, A.part, A.splits);
    }
  } else if (A.u_out && chunk == 0) {
    for (int e = threadIdx.x; e < rows * A.rank; e += 64 * kExpandWaves) A.u_out[row0 * A.rank + e] = 0.0f;
  }
  __syncthreads();
  if (!mine) return;
  while (rem) {
    const uint64_t match = __ballot(id == a);
    rem &= ~match;
    W.settle({A.w + (int64_t)a * A.N * A.rank * T::ES, A.N, n0, A.rank, lane});
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const uint32_t here = (uint32_t)(match >> (16 * j)) & 0xFFFFu;
      if (!here) continue;
#pragma unroll
      for (int h = 0; h < T::PE; h += 4) {  // four tiles at a time, for the registers
        __builtin_amdgcn_sched_barrier(0);  // (fragments of several tiles at once: up to five registers spilled)
        f32x4 acc[4];
        W.product(acc, h, [&](int f) { return us[j][f][lane]; });
        if (here == 0xFFFFu) {
#pragma unroll
          for (int v = 0; v < 4; ++v) add_products<DT>(out[j][v], acc, h, v);
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if ((here >> (4 * q + v)) & 1) add_products<DT>(out[j][v], acc, h, v);
        }
      }
    }
    if (rem) {
      a = __builtin_amdgcn_readlane(id, __builtin_ctzll(rem));
      weights(a);
    }
  }
  // rows without an adapter are in place already where y is base
  const uint64_t wanted = A.base == A.y ? __ballot(id >= 0) : live;
  if (inside && wanted == live) {
    uint8_t *to = A.y + (row0 * A.ldy + n0) * T::ES;
    const uint32_t mine_at = (4 * q * (uint32_t)A.ldy + T::PE * i) * T::ES;
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        __builtin_nontemporal_store(out[j][v], reinterpret_cast<u32x4_a1 *>(to + (16 * j + v) * A.ldy * T::ES + mine_at));
  } else {
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * j + 4 * q + v;
        if ((wanted >> r) & 1) st_frag_n<DT>(A.y + ((row0 + r) * A.ldy + col) * T::ES, out[j][v], A.N - col);
      }
  }
}

// ---- launches ----------------------------------------------------------------------

inline int window_count(int64_t tokens) { return (int)((tokens + kWindow - 1) / kWindow); }

// Parts of the long dimension: as many as put a workgroup on each of the 256 CUs. The second kernel
// adds the parts up once a tile of columns, so fewer are better there (both kernels, with one workgroup a CU,
// two, and half a one: 8192 tokens, 7168 -> 7168, rank 32 80.2 / 85.7 / 86.5 us; gradient of x, rank 64 73 / 80
// / 89; 4096 tokens of fp32, rank 8 41.7 / 44.8 / 47.9; all gradients of 8191 tokens, 7168 -> 2048, rank 64 149.5 /
// 161.6 / 143).
inline int shrink_splits(int64_t tokens, int64_t K) {
  const int64_t windows = window_count(tokens);
  const int64_t most = (K + 511) / 512;
  int64_t s = 256 / (windows > 0 ? windows : 1);
  if (s > most) s = most;
  if (s > 16) s = 16;
  return s < 1 ? 1 : (int)s;
}

// Workgroups that share a window's adapters: up to 2048 workgroups in all, of which those beyond a
// window's adapters end at once (1531 rows of 24 adapters 13.6 us, with 1024 13.2; 8192 rows of 16 alike).
inline int shrink_slots(int64_t tokens, int adapters, int splits) {
  const int64_t windows = window_count(tokens);
  int64_t s = 2048 / ((windows > 0 ? windows : 1) * splits);
  if (s > 64) s = 64;
  if (s > adapters) s = adapters;
  return s < 1 ? 1 : (int)s;
}

// How the rows' pieces are met (adapter_device.h).
inline int piece_mode(int dtype, int64_t tokens, int64_t in, int64_t out, int rank) {
  const int pe = dtype == kBF16 ? 8 : 4;
  if (in % pe == 0 && out % pe == 0 && rank % pe == 0) return kExact;
  return in < pe || out < pe || tokens * rank < 4 ? kSingle : kCut;
}

// Calls f(rank tiles, mode) with both as constants.  Problems of kSingle are tiny:
// one form of the kernels serves all ranks.
template <typename F>
void by_rank_and_mode(int rank, int mode, F f) {
  using std::integral_constant;
  const int rt = (rank + 15) / 16;
  auto ranks = [&](auto m) {
    if (rt <= 1) f(integral_constant<int, 1>(), m);
    else if (rt <= 2) f(integral_constant<int, 2>(), m);
    else if (rt <= 4) f(integral_constant<int, 4>(), m);
    else f(integral_constant<int, 8>(), m);
  };
  if (mode == kExact) ranks(integral_constant<int, kExact>());
  else if (mode == kCut) ranks(integral_constant<int, kCut>());
  else f(integral_constant<int, 8>(), integral_constant<int, kSingle>());
}

template <int DT, bool ACROSS>
hipError_t launch_shrink(const ShrinkArgs &A, const PlanArgs &P, int mode, hipStream_t stream) {
  const int64_t pairs = (int64_t)A.windows * A.splits;
  const dim3 grid((unsigned)((pairs + 7) / 8 * 8 * A.slots + (P.order ? (P.blocks + 7) / 8 * 8 : 0)));
  by_rank_and_mode(A.rank, mode, [&](auto rt, auto m) {
    adapter_shrink_kernel<DT, decltype(rt)::value, ACROSS, decltype(m)::value><<<grid, kShrinkThreads, 0, stream>>>(A, P);
  });
  return hipGetLastError();
}

template <int DT, bool ACROSS>
hipError_t launch_expand(const ExpandArgs &A, int mode, hipStream_t stream) {
  const int64_t windows = (A.tokens + kExpandRows<DT> - 1) / kExpandRows<DT>;
  const int64_t cols = kExpandWaves * 16 * Tile<DT>::PE;
  const int chunks = (int)((A.N + cols - 1) / cols);
  const dim3 grid((unsigned)(windows * chunks));
  by_rank_and_mode(A.rank, mode, [&](auto rt, auto m) {
    adapter_expand_kernel<DT, frag_count<DT>(decltype(rt)::value), ACROSS, decltype(m)::value>
        <<<grid, 64 * kExpandWaves, 0, stream>>>(A, chunks);
  });
  return hipGetLastError();
}

}  // namespace
}  // namespace mxfp4
