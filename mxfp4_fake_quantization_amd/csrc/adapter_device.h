// adapter_device.h -- what the low-rank adapters' kernels share: matrix-core
// tiles of 16-byte fragments, the rows of a window by adapter, and the two
// products
//     u[t, r] = sum_k x[t, k] W[r, k]     ("shrink": k long, r <= 128)
//     y[t, n] = base[t, n] + sum_r u[t, r] W[n, r]     ("expand")
// with the weights of each row's adapter.  The forward pass has W = A [r, in],
// then W = B [out, r]; the backward pass has the same products with the
// transposes of B and A, which are read across their rows.
//
// Fragments.  An operand of a 16 x 16 tile is 16 bytes a lane: lane l holds row
// l % 16 and, of the summed dimension, 8 bf16 (one v_mfma 16x16x32) or 4 fp32
// values (four v_mfma 16x16x4, one a component) of part q = l / 16.  A sum does
// not depend on the order of its terms as long as both operands agree, so every
// fragment is one contiguous 16-byte piece of a row.  The result's lane l holds
// row 4 q + v (v = 0..3) of the first operand and row l % 16 of the second.
//
// u is kept in fp32.  As an operand of a bf16 product it is split into three parts,
// u = hi + mid + lo: 8 bits toward 0 of u, of the rest, and what is left then, at most 8 of
// u's 24 bits, so nothing is lost (but below 2^-133) and y is rounded once, to its type.
// All three have u's sign and are 0 for 0 alone, so an infinite weight or row gives what u
// does.  (Two parts lose 2^-16 of u, more than y itself where the terms cancel.  The third
// costs 1 to 4 % of the products' time, 8 % of all gradients' of 4096 rows and columns of
// rank 128: 144 -> 157 us.)
#pragma once

#include "adapter_kernels.h"
#include "mxfp4_rows8.h"

namespace mxfp4 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef u32x4 u32x4_a1 __attribute__((aligned(2)));

template <int DT>
struct Tile {
  static constexpr int ES = DT == kBF16 ? 2 : 4;  // bytes of an element
  static constexpr int PE = 16 / ES;              // elements of a fragment's lane
  static constexpr int KF = 4 * PE;               // summed elements of a fragment
};

template <int DT>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == kBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(bits_f32(a[i]), bits_f32(b[i]), c, 0, 0, 0);
    return c;
  }
}

// ---- pieces of 16 bytes ----------------------------------------------------------
//
// A row's last piece may be cut short, and rows start at any element (the hardware
// takes unaligned accesses).  How a kernel meets that, chosen by its sizes:
//   kExact   every row has a whole number of pieces: a piece is there or not;
//   kCut     rows of any length: a piece that sticks out is loaded from the last 16
//            bytes of its row (or array) and shifted down, zeros following, so the load
//            itself hangs on no condition and the loads of a loop stay in flight
//            together (a branch around a load made the compiler wait for all of them);
//   kSingle  rows shorter than a piece: element by element.
enum { kExact = 0, kCut = 1, kSingle = 2 };

__device__ __forceinline__ u32x4 ld_frag(const uint8_t *p) { return *reinterpret_cast<const u32x4_a1 *>(p); }
__device__ __forceinline__ u32x4 ld_frag_nt(const uint8_t *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a1 *>(p));
}

// The first n elements of a piece, the others 0.
template <int DT>
__device__ __forceinline__ u32x4 ld_single(const uint8_t *p, int64_t n) {
  u32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < Tile<DT>::PE; ++j)
    if (j < n) {
      if (DT == kBF16) w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[j] << (16 * (j & 1));
      else w[j & 3] = reinterpret_cast<const uint32_t *>(p)[j];
    }
  return w;
}

// A piece without its first d elements, zeros following; none for d >= PE.
template <int DT>
__device__ __forceinline__ u32x4 shifted(u32x4 w, int d) {
  if (d <= 0) return w;
  if (d >= Tile<DT>::PE) return u32x4{0, 0, 0, 0};
  const int bits = d * 8 * Tile<DT>::ES;
  if (bits & 64) w = u32x4{w[2], w[3], 0, 0};
  if (bits & 32) w = u32x4{w[1], w[2], w[3], 0};
  if (DT == kBF16 && (bits & 16))
    w = u32x4{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16};
  return w;
}

// The first n elements, the others 0.
template <int DT>
__device__ __forceinline__ u32x4 only(u32x4 w, int n) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if (DT == kBF16) w[d] = n >= 2 * d + 2 ? w[d] : n == 2 * d + 1 ? w[d] & 0xFFFFu : 0u;
    else w[d] = n > d ? w[d] : 0u;
  }
  return w;
}

// Piece at element e of a row of `len` elements at `row` (len >= PE but for kSingle):
// where to load it, what to shift it by.  kExact: 0 or PE.
template <int DT, int MODE>
struct RowPiece {
  int64_t at;
  int shift;
  __device__ __forceinline__ RowPiece(int64_t e, int64_t len) {
    const int64_t last = len - Tile<DT>::PE;
    at = MODE == kSingle || e <= last ? e : last;
    const int64_t d = e - at;
    shift = d > Tile<DT>::PE ? Tile<DT>::PE : (int)d;
    n = MODE == kSingle ? len - e : 0;
  }
  int64_t n;  // kSingle: elements there
  __device__ __forceinline__ u32x4 raw(const uint8_t *row) const {
    if constexpr (MODE == kSingle) return ld_single<DT>(row + at * Tile<DT>::ES, n);
    return ld_frag(row + at * Tile<DT>::ES);
  }
  __device__ __forceinline__ u32x4 settled(u32x4 w) const {
    if constexpr (MODE == kSingle) return w;
    if constexpr (MODE == kExact) return shift ? u32x4{0, 0, 0, 0} : w;
    return shifted<DT>(w, shift);
  }
  __device__ __forceinline__ u32x4 load(const uint8_t *row) const { return settled(raw(row)); }
};

// The n elements (of at most PE; the others 0) at p in an array whose last 16 bytes are
// at `last`, for rows that may be shorter than a piece: the load, and what is left to do
// when the value is needed.
template <int DT, int MODE>
__device__ __forceinline__ u32x4 ld_inside(const uint8_t *p, const uint8_t *last, int n) {
  if constexpr (MODE == kSingle) return ld_single<DT>(p, n);
  return ld_frag(MODE == kCut && p > last ? last : p);
}
template <int DT, int MODE>
__device__ __forceinline__ u32x4 settle_inside(u32x4 w, const uint8_t *p, const uint8_t *last, int n) {
  if constexpr (MODE == kSingle) return w;
  if constexpr (MODE == kExact) return n > 0 ? w : u32x4{0, 0, 0, 0};
  if (p > last) {
    const int64_t d = (p - last) / Tile<DT>::ES;
    w = shifted<DT>(w, d > Tile<DT>::PE ? Tile<DT>::PE : (int)d);
  }
  return only<DT>(w, n);
}

template <int DT>
__device__ __forceinline__ void st_frag_n(uint8_t *p, u32x4 w, int64_t n) {
  if (n >= Tile<DT>::PE) {
    *reinterpret_cast<u32x4_a1 *>(p) = w;
    return;
  }
#pragma unroll
  for (int j = 0; j < Tile<DT>::PE; ++j)
    if (j < n) {
      if (DT == kBF16) reinterpret_cast<uint16_t *>(p)[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
      else reinterpret_cast<uint32_t *>(p)[j] = w[j & 3];
    }
}

// PE rows of PE elements a lane become PE fragments' lanes: fragment j holds
// element j of every row.
template <int DT>
__device__ __forceinline__ u32x4 turned(const u32x4 (&rows)[Tile<DT>::PE], int j) {
  u32x4 w;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if constexpr (DT == kBF16)
      w[d] = __builtin_amdgcn_perm(rows[2 * d + 1][j >> 1], rows[2 * d][j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
    else
      w[d] = rows[d][j];
  }
  return w;
}

// fp32 values as bf16 operands: the upper halves of two.
__device__ __forceinline__ uint32_t pack_upper(float a, float b) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
}
// The next value toward 0 (its upper half is a's next part), 0 for 0; and what that part leaves,
// which is 0 for 0 alone and has a's sign: times an infinity all parts give the same infinity (0
// for a part would give NaN).  The part of an infinity is finite, its rest the infinity.
__device__ __forceinline__ float below(float a) {
  return bits_f32(__builtin_bit_cast(uint32_t, a) - (a != 0.0f ? 1u : 0u));
}
__device__ __forceinline__ float rest(float a) {
  return a - bits_f32(__builtin_bit_cast(uint32_t, below(a)) & 0xFFFF0000u);
}
// The three parts of 8 values as a fragment's 16 bytes each.
struct Parts {
  u32x4 hi, mid, lo;
};
__device__ __forceinline__ Parts parts_of(const float (&v)[8]) {
  Parts p;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const float a = v[2 * d], b = v[2 * d + 1], ra = rest(a), rb = rest(b);
    p.hi[d] = pack_upper(below(a), below(b));
    p.mid[d] = pack_upper(below(ra), below(rb));
    p.lo[d] = pack_upper(rest(ra), rest(rb));
  }
  return p;
}

// ---- rows by adapter -----------------------------------------------------------
//
// Tokens come in any order of adapters.  A wave looks at a window of 64 rows, one
// a lane, and takes the adapters of the window one after the other: the lanes
// that share the first remaining row's adapter are found by one ballot, and one
// cross-lane move lines their rows up.  No sorted copy, no plan, no extra launch;
// a window of one adapter (a long prompt) costs a single turn.

constexpr int kWindow = 64;

// Adapter of a row, -1 for none.
__device__ __forceinline__ int row_adapter(const int32_t *ids, int64_t row, int adapters) {
  const int id = ids ? ids[row] : 0;
  return id >= 0 && id < adapters ? id : -1;
}

// Lane i gets the i-th lane of `match`; lanes from popcount(match) on the others.
__device__ __forceinline__ int lined_up(uint64_t match, int lane) {
  const uint64_t below = (1ull << lane) - 1;
  const int at = (match >> lane) & 1 ? __popcll(match & below) : __popcll(match) + __popcll(~match & below);
  return __builtin_amdgcn_ds_permute(at << 2, lane);
}

// ---- expand ----------------------------------------------------------------------
//
// A wave takes 16 PE columns (128 bf16, 64 fp32) and keeps their weights in
// registers while rows pass: u comes from the caches, base and y pass once.  Column
// PE n + j is row n of tile j, so a lane's results over the tiles are PE consecutive
// columns of a row, 16 bytes, and 16 lanes' are 256 consecutive bytes of it.
//   W [N, rank]: lane n loads the ranks of its PE columns.
//   W [rank, N] (ACROSS): a lane loads its PE columns of PE ranks and turns them.
// NF fragments of the ranks; NF 0: ranks up to 16 in bf16, whose parts hi and mid share one
// fragment (lo has both halves of another, half of it in each).

template <int DT>
constexpr int frag_count(int rank_tiles) {  // of 16-rank tiles
  return DT == kBF16 ? rank_tiles / 2 : rank_tiles;
}

template <int DT, int NF, bool ACROSS, int MODE>
struct Expand {
  using T = Tile<DT>;
  static constexpr int F = NF ? NF : 1;
  static constexpr int COLS = 16 * T::PE;
  u32x4 w[F][T::PE];

  // ranks that lane q of fragment f holds: PE from here on
  __device__ __forceinline__ static int rank0(int f, int q) {
    return NF ? f * T::KF + T::PE * q : T::PE * (q & 1);
  }

  // The weights of columns n0 to n0 + COLS - 1 of one adapter's W, loaded; settle() makes
  // the fragments of them.  Columns past the last hold anything, ranks past the last 0.
  struct From {
    const uint8_t *w;
    int64_t N, n0;
    int rank, lane;
  };
  __device__ __forceinline__ const uint8_t *row_of(const From &S, int f, int j) const {
    const int64_t col = S.n0 + T::PE * (S.lane & 15) + j;
    const int r0 = rank0(f, S.lane >> 4);  // (ranks past the last: any piece, dropped)
    return S.w + ((col < S.N ? col : S.N - 1) * S.rank + (r0 < S.rank ? r0 : 0)) * T::ES;
  }
  __device__ __forceinline__ void load(const From &S) {
    if constexpr (ACROSS) {
      const RowPiece<DT, MODE> col(S.n0 + T::PE * (S.lane & 15), S.N);
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int e = 0; e < T::PE; ++e) {
          const int r = rank0(f, S.lane >> 4) + e;
          w[f][e] = col.raw(S.w + (r < S.rank ? r : S.rank - 1) * S.N * T::ES);
        }
    } else {
      const uint8_t *last = S.w + S.N * S.rank * T::ES - 16;
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int j = 0; j < T::PE; ++j)
          w[f][j] = ld_inside<DT, MODE>(row_of(S, f, j), last, S.rank - rank0(f, S.lane >> 4));
    }
  }
  __device__ __forceinline__ void settle(const From &S) {
    if constexpr (ACROSS) {
      const RowPiece<DT, MODE> col(S.n0 + T::PE * (S.lane & 15), S.N);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        u32x4 rows[T::PE];
#pragma unroll
        for (int e = 0; e < T::PE; ++e)
          rows[e] = rank0(f, S.lane >> 4) + e < S.rank ? col.settled(w[f][e]) : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < T::PE; ++j) w[f][j] = turned<DT>(rows, j);
      }
    } else {
      const uint8_t *last = S.w + S.N * S.rank * T::ES - 16;
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int j = 0; j < T::PE; ++j)
          w[f][j] = settle_inside<DT, MODE>(w[f][j], row_of(S, f, j), last, S.rank - rank0(f, S.lane >> 4));
    }
  }

  // u's fragments: those of hi, of mid, of lo (bf16); of u (fp32)
  static constexpr int UF = DT == kF32 ? F : NF ? 3 * F : 2;
  // acc[j][v]: row 4 q + v of the tile, column n0 + PE n + h + j; u(f) gives fragment f, when it is
  // needed (all of them together cost the registers of 48 numbers at rank 128)
  template <typename U>
  __device__ __forceinline__ void product(f32x4 (&acc)[4], int h, U u) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int f = 0; f < UF; ++f) {
      const u32x4 uf = u(f);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = mma<DT>(uf, w[f % F][h + j], acc[j]);
    }
  }

  // Fragments of one row's u, given get(r, n): PE fp32 values from rank r on, those
  // from n on 0.
  template <typename G>
  __device__ __forceinline__ static void u_frags(u32x4 (&uf)[UF], int rank, int q, G get) {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int r0 = rank0(f, q);
      float v[T::PE];
      get(v, r0, rank - r0);
      if constexpr (DT == kF32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) uf[f][e] = __builtin_bit_cast(uint32_t, v[e]);
      } else {
        Parts p = parts_of(v);
        if constexpr (NF == 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = 0.5f * v[e];  // (lo of the half is half of lo)
          uf[0] = q < 2 ? p.hi : p.mid;
          uf[1] = parts_of(v).lo;
        } else {
          uf[f] = p.hi;
          uf[F + f] = p.mid;
          uf[2 * F + f] = p.lo;
        }
      }
    }
  }
};

// Columns h to h + 3 of a lane's piece: base + the products of row v, rounded once.
template <int DT>
__device__ __forceinline__ void add_products(u32x4 &piece, const f32x4 (&acc)[4], int h, int v) {
  if constexpr (DT == kBF16) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const uint32_t b = piece[h / 2 + d];
      piece[h / 2 + d] = pack_bf16(bits_f32(b << 16) + acc[2 * d][v], bits_f32(b & 0xFFFF0000u) + acc[2 * d + 1][v]);
    }
  } else {
#pragma unroll
    for (int d = 0; d < 4; ++d) piece[d] = __builtin_bit_cast(uint32_t, bits_f32(piece[d]) + acc[d][v]);
  }
}

}  // namespace mxfp4
