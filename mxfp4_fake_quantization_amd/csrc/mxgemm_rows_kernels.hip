// mxgemm_rows_kernels.hip -- the grouped MX product with its epilogue for few
// rows a group (decoding), on gfx950.
//
// A group of a few rows reads its whole weight for them: the time is the
// weights' bytes.  A workgroup takes up to 16 MT rows of one group and 16 CT
// rows of B, as v_mfma_scale_f32_16x16x128_f8f6f4 tiles: its lanes 16 apart
// hold 64 consecutive bytes of a B row, so B goes from memory to the matrix
// core without LDS, in turns of 256 along K (two steps), each loaded while the
// one before multiplies.  With few workgroups the four waves share the turns of
// one column run, read A as they read B, and their sums meet in LDS once, where
// the epilogue takes them; with many each wave has a run and the whole K of its
// own, and A passes through LDS.  Operand
// layout of the instruction (lane l: row or column l % 16, quarter q = l / 16):
// fp8 bytes 0-15 are K 16 q.., bytes 16-31 K 64 + 16 q..; fp4 nibble j is K
// 32 q + j; the scale byte is that of K-block q; result register v is row
// 4 q + v, column l % 16.
#include "moe_kernels.h"
#include "mxgemm_tile.h"

namespace mxfp4 {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kRowsCT = 2;  // 16-row tiles of B a wave takes
constexpr int kRowsWaves = 4, kRowsThreads = 64 * kRowsWaves;

// 16 bytes at any alignment of the operand's rows (16, by the checks).
__device__ __forceinline__ u32x4 ld_u4(const uint8_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

// One turn's codes and scales of a 16-row tile: two pieces of 16 bytes (E2M1)
// or four; the scale of the lane's K-block in each of the two steps.
template <int FMT>
struct Turn {
  static constexpr int N = FMT == kFmtE2M1 ? 2 : 4;
  u32x4 w[N];
  uint32_t s[2];
};

// B32: blocks of 32, a step's four scale bytes in one word (load_turn), of
// which lane quarter q takes byte q (scale_of).  Otherwise one byte a lane.
// TAIL: blocks at or past kb are zero codes with scale 2^0, read in bounds.
// SCALES false: the codes alone.
template <int FMT, bool B32, bool TAIL, bool SCALES = true>
__device__ __forceinline__ void load_turn(Turn<FMT> &T, const uint8_t *base, uint32_t at, const uint8_t *scales,
                                          uint32_t sat, int64_t c, int64_t kb, int sb, int q) {
  typedef uint32_t u32_a1 __attribute__((aligned(1)));
  constexpr int TURN = FMT == kFmtE2M1 ? 128 : 256;  // bytes of a turn
  const uint8_t *p = base + TURN * c;                // the same for the wave
#pragma unroll
  for (int i = 0; i < Turn<FMT>::N; ++i) {
    const int64_t blk = FMT == kFmtE2M1 ? 8 * c + 4 * i + q : 8 * c + 2 * i + (q >> 1);
    if (!TAIL) {
      T.w[i] = ld_u4(p + at + 64 * i);
    } else {
      const bool in = blk < kb;
      T.w[i] = ld_u4(in ? p + at + 64 * i : base + (at - 16 * q));
      if (!in) T.w[i] = u32x4{0u, 0u, 0u, 0u};
    }
  }
  if (!SCALES) return;
  if (B32 && !TAIL) {
    const uint8_t *r = scales + 8 * c + sat;
    T.s[0] = *reinterpret_cast<const u32_a1 *>(r);
    T.s[1] = *reinterpret_cast<const u32_a1 *>(r + 4);
  } else {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t blk = 8 * c + 4 * t + q;
      const uint32_t v = scales[sat + ((TAIL && blk >= kb ? 0 : blk) >> sb)];
      T.s[t] = (TAIL && blk >= kb ? 127u : v) << (B32 ? 8 * q : 0);
    }
  }
}
template <int FMT, bool B32>
__device__ __forceinline__ int scale_of(const Turn<FMT> &T, int step, int q) {
  return (int)(B32 ? T.s[step] >> (8 * q) : T.s[step]);
}

template <int FMT>
__device__ __forceinline__ v8i operand(const Turn<FMT> &T, int step) {
  if (FMT == kFmtE2M1) {
    const u32x4 v = T.w[step % Turn<FMT>::N];
    return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
  }
  const u32x4 lo = T.w[(2 * step) % Turn<FMT>::N], hi = T.w[(2 * step + 1) % Turn<FMT>::N];
  return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Row tile tm: its first row and rows (0 or less past the last), and its group.
// One group needs no walk; its count includes the row_skip rows before P.a.
template <int MLOG>
__device__ __forceinline__ int row_tile(const GemmArgs &P, int64_t tm, int64_t *m0, int64_t *mlen) {
  int g = 0;
  if (P.gl && P.G > 1) {
    block_row_uniform<false>(P.gl, P.G, P.list_type, P.M, MLOG, tm, m0, mlen, &g);
  } else {
    int64_t m = P.gl ? P.gl[0] - P.row_skip : P.M;
    m = m < P.M ? m : P.M;
    *m0 = tm << MLOG;
    *mlen = m - *m0 < (1 << MLOG) ? m - *m0 : 1 << MLOG;
  }
  return g;
}

// One 16 x 16 tile's values (and its up values) to the outputs: rows m0 ..,
// of which `rows` are there, columns oc0 .., of which `cols` are.
template <bool GATED>
__device__ __forceinline__ void put_tile(const GemmArgs &P, const ActArgs &E, int g, int64_t m0, int64_t rows,
                                         int64_t oc0, int cols, int lane, v4f z, v4f up) {
  const int l16 = lane & 15, q = lane >> 4;
  if (l16 >= cols) return;
  const int64_t oc = oc0 + l16;
  if (E.bias) {
    const float *b = E.bias + (int64_t)g * E.bias_gs + oc;
    z += b[0];
    if (GATED) up += b[P.N];
  }
  float x[4];
  with_act(E.act, [&](auto a) {
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] = act_value<decltype(a)::value>(z[v]);
  });
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (4 * q + v >= rows) break;
    const int64_t m = m0 + 4 * q + v;
    if (GATED) x[v] *= up[v];
    if (P.out_f32) {
      if (E.z) {
        float *zr = static_cast<float *>(E.z) + m * E.ldz + oc;
        zr[0] = z[v];
        if (GATED) zr[P.N] = up[v];
      }
      if (E.res) x[v] += static_cast<const float *>(E.res)[m * E.ldr + oc];
      static_cast<float *>(P.c)[m * P.ldc + oc] = x[v];
    } else {
      if (E.z) {
        uint16_t *zr = static_cast<uint16_t *>(E.z) + m * E.ldz + oc;
        zr[0] = (uint16_t)pack_bf16(z[v], 0.0f);
        if (GATED) zr[P.N] = (uint16_t)pack_bf16(up[v], 0.0f);
      }
      if (E.res) x[v] += bits_f32((uint32_t)static_cast<const uint16_t *>(E.res)[m * E.ldr + oc] << 16);
      static_cast<uint16_t *>(P.c)[m * P.ldc + oc] = (uint16_t)pack_bf16(x[v], 0.0f);
    }
  }
}

template <int AF, int BF, int MT, int CT>
struct Turns {
  Turn<AF> a[MT];
  Turn<BF> b[CT];
};

// EPI as in mxgemm_tile.h.  Gated: B tiles 0 .. CT / 2 - 1 are gate rows, the
// others the up rows of the same columns.
//
// Few waves' worth of columns: the four waves of a workgroup share the K of
// one column run (16 H columns, H tiles of output columns), in turns of 256.
//
// The waves a SIMD of both kernels are those that E2M1 weights run best with.  A
// turn of E4M3 takes twice the registers: with 16 rows (both kernels) and with 64
// (this one) its two sets do not fit and spill in the loop, 25 - 38 and 72 - 85
// scratch accesses; E2M1 with 64 rows has 4 - 6 here.  8 experts of one row, 7168
// -> 2 x 2048, take 73 us with E4M3 weights against 26 with E2M1, 32 groups of 6
// rows, 2048 -> 7168, 135 against 64 (twice the bytes each); 32 and, over the
// whole K, 64 rows do not spill: 32 groups of 25 rows 142 against 100.
template <int AF, int BF, bool B32, int MT, int CT, int EPI>
__global__ __launch_bounds__(kRowsThreads, (MT == 1 ? 4 : 2)) void mxgemm_rows_split_kernel(GemmArgs P, ActArgs E) {
  constexpr bool GATED = EPI == 2;
  constexpr int H = GATED ? CT / 2 : CT;
  constexpr int MLOG = MT == 1 ? 4 : MT == 2 ? 5 : 6;
  constexpr int KS = kRowsWaves;
  __shared__ v4f red[kRowsWaves][MT][CT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l16 = lane & 15, q = lane >> 4;

  const int64_t tm = blockIdx.x % P.tiles_m, tn = blockIdx.x / P.tiles_m;
  int64_t m0, mlen;
  const int g = row_tile<MLOG>(P, tm, &m0, &mlen);
  if (mlen <= 0) return;  // the same for the workgroup
  const int64_t n0 = tn * 16 * H;
  const int nlen = (int)(P.N - n0 < 16 * H ? P.N - n0 : 16 * H);
  const int64_t kb = P.K >> 5;

  // wave-uniform bases and 32-bit lane offsets
  const uint8_t *ab = P.a + m0 * P.lda, *asb = P.as + m0 * P.ldas;
  uint32_t ao[MT], aso[MT], bo[CT], bso[CT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = 16 * i + l16 < (int)mlen ? 16 * i + l16 : (int)mlen - 1;
    ao[i] = (uint32_t)r * (uint32_t)P.lda + 16 * q;
    aso[i] = (uint32_t)r * (uint32_t)P.ldas;
  }
  const uint8_t *bb[GATED ? 2 : 1], *bsb[GATED ? 2 : 1];
#pragma unroll
  for (int p = 0; p < (GATED ? 2 : 1); ++p) {
    bb[p] = P.b + (int64_t)g * P.b_gs + (n0 + p * P.N) * P.ldb;
    bsb[p] = P.bs + (int64_t)g * P.b_gss + (n0 + p * P.N) * P.ldbs;
  }
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    int col = 16 * (j % H) + l16;
    col = col < nlen ? col : nlen - 1;
    bo[j] = (uint32_t)col * (uint32_t)P.ldb + 16 * q;
    bso[j] = (uint32_t)col * (uint32_t)P.ldbs;
  }

  v4f acc[MT][CT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  using T = Turns<AF, BF, MT, CT>;
  auto load = [&](T &t, int64_t c, auto tail) {
    constexpr bool TAIL = decltype(tail)::value;
#pragma unroll
    for (int j = 0; j < CT; ++j)
      load_turn<BF, B32, TAIL>(t.b[j], bb[j / H], bo[j], bsb[j / H], bso[j], c, kb, P.b_sb, q);
#pragma unroll
    for (int i = 0; i < MT; ++i) load_turn<AF, B32, TAIL>(t.a[i], ab, ao[i], asb, aso[i], c, kb, P.a_sb, q);
  };
  auto multiply = [&](const T &t) {
    __builtin_amdgcn_sched_barrier(0);  // the next turn's loads stay before, the one after's behind
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        const v8i b = operand<BF>(t.b[j], s);
        const int sb = scale_of<BF, B32>(t.b[j], s, q);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand<AF>(t.a[i], s), b, acc[i][j], AF, BF, 0,
                                                                       scale_of<AF, B32>(t.a[i], s, q), 0, sb);
      }
    __builtin_amdgcn_sched_barrier(0);
  };
  // turns wave, wave + KS, ...: two sets of registers, each loaded while the
  // other multiplies (past the last turn the last one is loaded again, unused)
  const int full = (int)(kb >> 3);  // whole turns
  const int mine = (full - wave + KS - 1) / KS;
  T t0, t1;
  if (mine > 0) {
    auto turn = [&](int i) { return (int64_t)(wave + KS * (i < mine ? i : mine - 1)); };
    load(t0, turn(0), std::false_type{});
    int i = 0;
    for (; i + 1 < mine; i += 2) {
      load(t1, turn(i + 1), std::false_type{});
      multiply(t0);
      load(t0, turn(i + 2), std::false_type{});
      multiply(t1);
    }
    if (i < mine) multiply(t0);
  }
  if ((kb & 7) && full % KS == wave) {
    load(t0, full, std::true_type{});
    multiply(t0);
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) red[wave][i][j][lane] = acc[i][j];
  __syncthreads();

  // the waves take the run's (row tile, column tile) pairs in turn
  for (int u = wave; u < MT * H; u += kRowsWaves) {
    const int i = u / H, j = u % H;
    auto total = [&](int jj) {
      v4f s = red[0][i][jj][lane];
#pragma unroll
      for (int w = 1; w < kRowsWaves; ++w) s += red[w][i][jj][lane];
      return s;
    };
    put_tile<GATED>(P, E, g, m0 + 16 * i, mlen - 16 * i, n0 + 16 * j, nlen - 16 * j, lane, total(j),
                    GATED ? total((j + H) % CT) : v4f{});
  }
}

// More columns: every wave takes the whole K of a column run of its own, and
// the A rows, which the four runs share, pass through LDS in slabs of SL turns
// (double-buffered; a lane's fragment is two 16-byte reads), so that the
// memory pipeline of a CU carries B almost alone.  B's scales (blocks of 32)
// pass through LDS by the same slabs, each
// wave's its own, 16 bytes a lane (a turn's 8 bytes a row, loaded for every
// turn, read half as many lines from L2 again as the codes: 32 groups of 6
// rows, 2048 -> 7168, 70.5 us against 64.2).
template <int AF, int BF, bool B32, int MT, int CT, int SL, int EPI>
__global__ __launch_bounds__(kRowsThreads, (MT == 4 ? 2 : MT == 2 ? 3 : 4)) void mxgemm_rows_kernel(GemmArgs P, ActArgs E) {
  constexpr bool GATED = EPI == 2;
  constexpr int H = GATED ? CT / 2 : CT;
  constexpr int MLOG = MT == 1 ? 4 : MT == 2 ? 5 : 6;
  constexpr int ROWS = 16 * MT, RSTR = 256 * SL + 16;  // bytes of a slab's row in LDS: 16 rows' pieces on all banks
  constexpr int LD = ROWS * 16 * SL / kRowsThreads;     // 16-byte pieces a thread stages
  static_assert(ROWS * 16 * SL % kRowsThreads == 0 && SL % 2 == 0, "slab");
  __shared__ __align__(16) uint8_t sa[2][ROWS * RSTR];
  __shared__ __align__(16) uint8_t ss[2][ROWS * 8 * SL];
  constexpr int BSL = 8 * SL, BSTR = BSL + 8;  // blocks of a slab; bytes of a B row's scales in LDS, 16 rows on all banks
  __shared__ __align__(16) uint8_t sbs[kRowsWaves][B32 ? 16 * CT * BSTR : 8];
  static_assert(CT == 2, "two lanes a B row");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;

  const int64_t tm = blockIdx.x % P.tiles_m, tn = blockIdx.x / P.tiles_m;
  int64_t m0, mlen64;
  const int g = row_tile<MLOG>(P, tm, &m0, &mlen64);
  const int mlen = (int)mlen64;
  if (mlen <= 0) return;  // the same for the workgroup
  const int64_t n0 = (tn * kRowsWaves + wave) * 16 * H;
  const int nlen = (int)(P.N - n0 < 16 * H ? P.N - n0 : 16 * H);  // 0 or less: the wave only helps to stage
  const int64_t kb = P.K >> 5;

  const int64_t nb0 = nlen > 0 ? n0 : 0;
  const uint8_t *bb[GATED ? 2 : 1], *bsb[GATED ? 2 : 1];
  uint32_t bo[CT], bso[CT];
#pragma unroll
  for (int p = 0; p < (GATED ? 2 : 1); ++p) {
    bb[p] = P.b + (int64_t)g * P.b_gs + (nb0 + p * P.N) * P.ldb;
    bsb[p] = P.bs + (int64_t)g * P.b_gss + (nb0 + p * P.N) * P.ldbs;
  }
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    int col = 16 * (j % H) + l16;
    col = col < nlen ? col : (nlen > 0 ? nlen - 1 : 0);
    bo[j] = (uint32_t)col * (uint32_t)P.ldb + 16 * q;
    bso[j] = (uint32_t)col * (uint32_t)P.ldbs;
  }
  struct BTurn {
    Turn<BF> b[CT];
  };
  auto load_b = [&](BTurn &t, int64_t c, auto tail) {
    constexpr bool TAIL = decltype(tail)::value;
#pragma unroll
    for (int j = 0; j < CT; ++j)
      load_turn<BF, B32, TAIL, !B32>(t.b[j], bb[j / H], bo[j], bsb[j / H], bso[j], c, kb, P.b_sb, q);
  };
  // A slab's B scales: lane l holds half of row l / 2's (4 SL bytes); 2^0 past K.
  typedef uint32_t half_t __attribute__((ext_vector_type(SL)));
  typedef half_t half_a1 __attribute__((aligned(1)));
  half_t rb;
  const int brow = lane >> 1, btile = brow >> 4;
  const uint8_t *bsrow;
  {
    int col = 16 * (btile % H) + (brow & 15);
    col = col < nlen ? col : (nlen > 0 ? nlen - 1 : 0);
    bsrow = bsb[0] + (GATED && btile ? P.N * P.ldbs : 0) + (uint32_t)col * (uint32_t)P.ldbs;
  }
  auto fetch_bs = [&](int64_t s) {
    const int64_t blk = BSL * s + 4 * SL * (lane & 1);
    if (blk + 4 * SL <= kb) {
      rb = *reinterpret_cast<const half_a1 *>(bsrow + blk);
    } else {
#pragma unroll
      for (int w = 0; w < SL; ++w) {
        uint32_t v = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) v |= (blk + 4 * w + e < kb ? (uint32_t)bsrow[blk + 4 * w + e] : 127u) << (8 * e);
        rb[w] = v;
      }
    }
  };

  // A slab s (turns SL s ..): thread's pieces into registers, then into LDS.
  // Pieces past K are zero codes, blocks past K have scale 2^0; rows past the
  // tile's stay as they are (they reach only outputs that are not stored).
  u32x4 ra[LD];
  uint32_t rs[(ROWS * 2 * SL + kRowsThreads - 1) / kRowsThreads];
  constexpr int SW = ROWS * 2 * SL;  // scale words of a slab: two a row and turn
  const uint8_t *arow = P.a + m0 * P.lda, *asrow = P.as + m0 * P.ldas;
  auto fetch = [&](int64_t s) {
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int idx = tid + kRowsThreads * i, row = idx / (16 * SL), piece = idx % (16 * SL);
      const int64_t k = 256 * SL * s + 16 * piece;
      const bool in = row < mlen && k < P.K;
      ra[i] = ld_u4(arow + (in ? (int64_t)row * P.lda + k : 0));
      if (!in) ra[i] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < (SW + kRowsThreads - 1) / kRowsThreads; ++i) {
      const int idx = tid + kRowsThreads * i, row = idx / (2 * SL), word = idx % (2 * SL);
      const int64_t blk = 8 * SL * s + 4 * word;
      rs[i] = 0x7F7F7F7Fu;
      if (idx < SW && row < mlen && blk < kb) {
        const uint8_t *r = asrow + (int64_t)row * P.ldas;
        typedef uint32_t u32_a1 __attribute__((aligned(1)));
        if (B32 && blk + 4 <= kb) {
          rs[i] = *reinterpret_cast<const u32_a1 *>(r + blk);
        } else {
          uint32_t v = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) v |= (blk + e < kb ? (uint32_t)r[(blk + e) >> P.a_sb] : 127u) << (8 * e);
          rs[i] = v;
        }
      }
    }
  };
  auto stage = [&](int buf) {
    if (B32) {  // this wave read its scales before, in order
      uint32_t *r = reinterpret_cast<uint32_t *>(&sbs[wave][brow * BSTR + 4 * SL * (lane & 1)]);
#pragma unroll
      for (int w = 0; w < SL; ++w) r[w] = rb[w];
    }
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int idx = tid + kRowsThreads * i, row = idx / (16 * SL), piece = idx % (16 * SL);
      *reinterpret_cast<u32x4 *>(&sa[buf][row * RSTR + 16 * piece]) = ra[i];
    }
#pragma unroll
    for (int i = 0; i < (SW + kRowsThreads - 1) / kRowsThreads; ++i) {
      const int idx = tid + kRowsThreads * i;
      if (idx < SW) *reinterpret_cast<uint32_t *>(&ss[buf][4 * idx]) = rs[i];
    }
  };

  v4f acc[MT][CT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const BTurn &t, int buf, int u) {  // turn u of the slab in buf
    __builtin_amdgcn_sched_barrier(0);
    u32x2 sw[CT];
    if (B32) {
#pragma unroll
      for (int j = 0; j < CT; ++j) sw[j] = *reinterpret_cast<const u32x2 *>(&sbs[wave][(16 * j + l16) * BSTR + 8 * u]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      v8i a[MT];
      int sca[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint8_t *r = &sa[buf][(16 * i + l16) * RSTR + 256 * u + 128 * s + 16 * q];
        const u32x4 lo = *reinterpret_cast<const u32x4 *>(r), hi = *reinterpret_cast<const u32x4 *>(r + 64);
        a[i] = v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
        sca[i] = (int)ss[buf][(16 * i + l16) * 8 * SL + 8 * u + 4 * s + q];
      }
#pragma unroll
      for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[i], operand<BF>(t.b[j], s), acc[i][j], AF, BF, 0,
                                                                       sca[i], 0, B32 ? (int)(sw[j][s] >> (8 * q)) : (int)t.b[j].s[s]);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  const int full = (int)(kb >> 3), turns = (int)((kb + 7) >> 3);
  const int slabs = (turns + SL - 1) / SL;
  BTurn t0, t1;
  auto upto = [&](int c) { return (int64_t)(c < full ? c : full - 1); };
  fetch(0);
  if (B32) fetch_bs(0);
  if (full > 0) load_b(t0, 0, std::false_type{});
  stage(0);
  __syncthreads();
  for (int s = 0; s < slabs; ++s) {
    const int buf = s & 1;
    if (s + 1 < slabs) {
      fetch(s + 1);
      if (B32) fetch_bs(s + 1);
    }
#pragma unroll
    for (int u = 0; u < SL; u += 2) {
      const int c = SL * s + u;
      if (c < full) {
        load_b(t1, upto(c + 1), std::false_type{});
        multiply(t0, buf, u);
        if (c + 1 < full) {
          load_b(t0, upto(c + 2), std::false_type{});
          multiply(t1, buf, u + 1);
        }
      }
    }
    if (s + 1 < slabs) {
      stage(buf ^ 1);  // read last before the previous barrier
      __syncthreads();
    }
  }
  if (turns > full) {  // the partial last turn, in the last slab
    load_b(t0, full, std::true_type{});
    const int u = full - SL * (slabs - 1);
    multiply(t0, (slabs - 1) & 1, u);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < H; ++j)
      put_tile<GATED>(P, E, g, m0 + 16 * i, mlen - 16 * i, n0 + 16 * j, nlen - 16 * j, lane, acc[i][j],
                      acc[i][(j + H) % CT]);
}

template <int AF, int BF, bool B32, int MT, int EPI>
hipError_t rows_one(GemmArgs a, const ActArgs &e, hipStream_t st) {
  constexpr int CT = kRowsCT, H = EPI == 2 ? CT / 2 : CT, COLS = 16 * H, SL = MT == 1 ? 4 : 2;
  // upper bound of the row tiles: every group adds at most one partial tile,
  // and no tile is empty
  const int64_t whole = a.M / (16 * MT) + (a.gl ? a.G : (a.M % (16 * MT) ? 1 : 0));
  a.tiles_m = whole < a.M ? whole : a.M;
  const int64_t runs = (a.N + COLS - 1) / COLS;
  // Shared K below 4096 runs (4 waves a SIMD): 8 experts of one row, 7168 ->
  // 2 x 2048 (1024 runs), 26 us against 29; 32 groups, 2048 -> 7168 (about
  // 7600 runs), 127 us against 64.
  const bool split = a.tiles_m * runs < 4096;
  a.tiles_n = split ? runs : (runs + kRowsWaves - 1) / kRowsWaves;
  a.total = a.tiles_m * a.tiles_n;
  if (a.total > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 grid((unsigned)a.total), block(kRowsThreads);
  if (split)
    hipLaunchKernelGGL((mxgemm_rows_split_kernel<AF, BF, B32, MT, CT, EPI>), grid, block, 0, st, a, e);
  else
    hipLaunchKernelGGL((mxgemm_rows_kernel<AF, BF, B32, MT, CT, SL, EPI>), grid, block, 0, st, a, e);
  return hipGetLastError();
}

template <int AF, int BF, bool B32, int EPI>
hipError_t rows_mt(const GemmArgs &a, const ActArgs &e, int mt, hipStream_t st) {
  if (mt == 1) return rows_one<AF, BF, B32, 1, EPI>(a, e, st);
  if (mt == 2) return rows_one<AF, BF, B32, 2, EPI>(a, e, st);
  return rows_one<AF, BF, B32, 4, EPI>(a, e, st);
}
template <int AF, int BF, int EPI>
hipError_t rows_b32(const GemmArgs &a, const ActArgs &e, int mt, hipStream_t st) {
  return a.a_sb || a.b_sb ? rows_mt<AF, BF, false, EPI>(a, e, mt, st) : rows_mt<AF, BF, true, EPI>(a, e, mt, st);
}

template <int EPI>
hipError_t rows_any(const GemmLaunch &L, const ActArgs &e, int mt, int64_t skip, hipStream_t st) {
  GemmArgs a = gemm_args(L);
  a.row_skip = skip;
  if (L.a_fmt == kFmtE4M3)
    return L.b_fmt == kFmtE2M1 ? rows_b32<kFmtE4M3, kFmtE2M1, EPI>(a, e, mt, st) : rows_b32<kFmtE4M3, kFmtE4M3, EPI>(a, e, mt, st);
  return L.b_fmt == kFmtE2M1 ? rows_b32<kFmtE5M2, kFmtE2M1, EPI>(a, e, mt, st) : rows_b32<kFmtE5M2, kFmtE4M3, EPI>(a, e, mt, st);
}

// mt: 16-row tiles a workgroup takes; skip: rows of the (one) group before L's first.
hipError_t rows_act(const GemmLaunch &L, const ActArgs &e, bool gated, int mt, int64_t skip, hipStream_t st) {
  return gated ? rows_any<2>(L, e, mt, skip, st) : rows_any<1>(L, e, mt, skip, st);
}

}  // namespace

hipError_t launch_gemm_act(const GemmLaunch &L, const ActArgs &e, bool gated, hipStream_t st) {
  // rows an average group has, of the groups that can have any
  const int64_t groups = L.num_groups < L.M ? L.num_groups : L.M;
  const int64_t avg = (L.M + groups - 1) / groups;
  // The few-rows form up to 64: 32 groups, 2048 -> 7168, it takes 64 us with 6
  // rows a group on average, 100 with 25 and 150 with 50, the tiles 198 - 210
  // at each and 185 with 100 (this form 257); one group of 64 / 128 / 256 rows
  // 15 / 23 / 44 us against 22 / 25 / 26.  Rows a workgroup (16 / 32 / 64), us:
  //                      6 rows on average     12            25            50
  //   K = 2048 -> 7168     64 /  81 /  90   77 /  82 /  96  107 / 100 / 113  171 / 150 / 154
  //   K = 7168 -> 4096    103 / 128 / 120  138 / 145 / 130  201 / 165 / 150  340 / 251 / 209
  // (gated, 7168 -> 2 x 2048: 109 / 118 / 115 at 8, 130 / 122 / 118 at 12.)  A
  // longer K pays the larger workgroup's start and end off.
  // It also takes more rows where its pieces (64 rows by one run of columns) are
  // at most one a CU: too few tiles to fill the chip, and here four waves share
  // K.  us, the tiles and this form, by pieces: 64 (256 rows, 7168 -> 512) 43 /
  // 20, 128 (1024, 7168 -> 256) 43 / 21, 90 (1787 in 3 groups, 3200 -> 96) 24 /
  // 12, 185 (11217 in 10, 544 -> 32) 13 / 8, 256 (2048, 2048 -> 256) 18 / 19;
  // 512 (1024, 2048 -> 2 x 512) 17 / 23, 640 (2048 in 8, 2048 -> 512) 19 / 27.
  const int64_t pieces = (L.M / 64 + (L.group_list ? L.num_groups : (L.M % 64 ? 1 : 0))) *
                         (gated ? (L.N + 15) / 16 : (L.N + 31) / 32);
  if (avg <= 64 || pieces <= device_cus()) {
    const bool long_k = L.K >= 4096;
    const int mt = avg <= (long_k ? 10 : 18) ? 1 : (long_k || avg > 48 ? 4 : 2);
    return rows_act(L, e, gated, mt, 0, st);
  }
  // One group whose last row tile has few rows: a launch of its own for them,
  // where that tile would cost a share of a round (4099 x 4095 x 4096: 133 us
  // as 17 row tiles, the last 16 of them in the tail launch).
  const int64_t rest = L.M % 256, whole = L.M - rest;
  if (L.num_groups != 1 || rest == 0 || rest > 64 || whole == 0 || whole / 256 * ((L.N + 255) / 256) > 1024)
    return gated ? launch_gated_tiles(L, e, st) : launch_act_tiles(L, e, st);
  GemmLaunch T = L;
  T.M = whole;
  const hipError_t r = gated ? launch_gated_tiles(T, e, st) : launch_act_tiles(T, e, st);
  if (r != hipSuccess) return r;
  const int64_t es = L.out_f32 ? 4 : 2;
  T.M = rest;
  T.a += whole * L.lda;
  T.as += whole * L.ldas;
  T.c = static_cast<uint8_t *>(L.c) + whole * L.ldc * es;
  ActArgs t = e;
  if (e.res) t.res = static_cast<const uint8_t *>(e.res) + whole * e.ldr * es;
  if (e.z) t.z = static_cast<uint8_t *>(e.z) + whole * e.ldz * es;
  return rows_act(T, t, gated, rest <= 16 ? 1 : rest <= 32 ? 2 : 4, whole, st);
}

}  // namespace mxfp4
