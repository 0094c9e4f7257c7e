// mxgemm_rows_kernels.hip -- the grouped MX product with its epilogue for few
// rows a group (decoding), on gfx950.
//
// A group of a few rows reads its whole weight for them: the time is the
// weights' bytes.  A workgroup takes up to 16 MT rows of one group and 16 CT
// rows of B, as v_mfma_scale_f32_16x16x128_f8f6f4 tiles: its lanes 16 apart
// hold 64 consecutive bytes of a B row, so B and A go from memory to the
// matrix core without LDS.  K is split over the four waves in turns of 256
// (two steps); a wave loads its next turn while the current one multiplies, and
// the waves' sums meet in LDS once, where the epilogue takes them.  Operand
// layout of the instruction (lane l: row or column l % 16, quarter q = l / 16):
// fp8 bytes 0-15 are K 16 q.., bytes 16-31 K 64 + 16 q..; fp4 nibble j is K
// 32 q + j; the scale byte is that of K-block q; result register v is row
// 4 q + v, column l % 16.
#include "moe_kernels.h"
#include "mxgemm_tile.h"

namespace mxfp4 {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kRowsWaves = 4, kRowsThreads = 64 * kRowsWaves;

// 16 bytes at any alignment of the operand's rows (16, by the checks).
__device__ __forceinline__ u32x4 ld_u4(const uint8_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

// One turn's codes and scales of a 16-row tile: T4 two pieces (E2M1), else four.
template <int FMT>
struct Turn {
  static constexpr int N = FMT == kFmtE2M1 ? 2 : 4;
  u32x4 w[N];
  uint32_t s[2];  // scale bytes of the two steps' four blocks
};

// The 8 scale bytes of blocks 8 c .. 8 c + 7 of a row (128-element blocks: one
// byte stands for four), bytes of blocks at or past kb replaced by 2^0.
template <bool TAIL>
__device__ __forceinline__ void load_scales(const uint8_t *row, int64_t c, int64_t kb, int sb, uint32_t (&s)[2]) {
  typedef uint32_t u32_a1 __attribute__((aligned(1)));
  if (!TAIL) {
    if (!sb) {
      s[0] = *reinterpret_cast<const u32_a1 *>(row + 8 * c);
      s[1] = *reinterpret_cast<const u32_a1 *>(row + 8 * c + 4);
    } else {
      s[0] = row[2 * c] * 0x01010101u;
      s[1] = row[2 * c + 1] * 0x01010101u;
    }
    return;
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    s[t] = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int64_t blk = 8 * c + 4 * t + b;
      s[t] |= (blk < kb ? (uint32_t)row[blk >> sb] : 127u) << (8 * b);
    }
  }
}

template <int FMT, bool TAIL>
__device__ __forceinline__ void load_turn(Turn<FMT> &T, const uint8_t *codes, const uint8_t *scales, int64_t c,
                                          int64_t kb, int sb, int q) {
#pragma unroll
  for (int i = 0; i < Turn<FMT>::N; ++i) {
    // piece i: its K offset in the turn's 256, and its block
    const int64_t k = FMT == kFmtE2M1 ? 256 * c + 128 * i + 32 * q : 256 * c + 64 * i + 16 * q;
    const bool in = !TAIL || (k >> 5) < kb;
    const int64_t at = FMT == kFmtE2M1 ? k >> 1 : k;
    T.w[i] = ld_u4(codes + (in ? at : 0));
    if (TAIL && !in) T.w[i] = u32x4{0u, 0u, 0u, 0u};
  }
  load_scales<TAIL>(scales, c, kb, sb, T.s);
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

template <int AF, int BF, int MT, int CT>
struct Turns {
  Turn<AF> a[MT];
  Turn<BF> b[CT];
};

// EPI as in mxgemm_tile.h.  Gated: B tiles 0 .. CT / 2 - 1 are gate rows, the
// others the up rows of the same columns.
template <int AF, int BF, int MT, int CT, int EPI>
__global__ __launch_bounds__(kRowsThreads) void mxgemm_rows_kernel(GemmArgs P, ActArgs E) {
  constexpr bool GATED = EPI == 2;
  constexpr int H = GATED ? CT / 2 : CT;  // tiles of output columns
  constexpr int MLOG = MT == 1 ? 4 : MT == 2 ? 5 : 6;
  __shared__ v4f red[kRowsWaves][MT][CT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, q = lane >> 4;

  const int64_t tm = blockIdx.x % P.tiles_m, tn = blockIdx.x / P.tiles_m;
  int64_t m0, mlen;
  int g = 0;
  if (P.gl) {
    block_row_uniform<false>(P.gl, P.G, P.list_type, P.M, MLOG, tm, &m0, &mlen, &g);
  } else {
    m0 = tm << MLOG;
    mlen = P.M - m0 < 16 * MT ? P.M - m0 : 16 * MT;
  }
  if (mlen <= 0) return;  // the same for the workgroup
  const int64_t n0 = tn * 16 * H;
  const int nlen = (int)(P.N - n0 < 16 * H ? P.N - n0 : 16 * H);
  const int64_t kb = P.K >> 5;

  const uint8_t *ac[MT], *as[MT], *bc[CT], *bs[CT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = 16 * i + l16 < (int)mlen ? 16 * i + l16 : (int)mlen - 1;
    ac[i] = P.a + (m0 + r) * P.lda;
    as[i] = P.as + (m0 + r) * P.ldas;
  }
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const int col = 16 * (j % H) + l16 < nlen ? 16 * (j % H) + l16 : nlen - 1;
    const int64_t r = n0 + col + (j >= H ? P.N : 0);
    bc[j] = P.b + (int64_t)g * P.b_gs + r * P.ldb;
    bs[j] = P.bs + (int64_t)g * P.b_gss + r * P.ldbs;
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
    for (int j = 0; j < CT; ++j) load_turn<BF, TAIL>(t.b[j], bc[j], bs[j], c, kb, P.b_sb, q);
#pragma unroll
    for (int i = 0; i < MT; ++i) load_turn<AF, TAIL>(t.a[i], ac[i], as[i], c, kb, P.a_sb, q);
  };
  auto multiply = [&](const T &t) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        const v8i b = operand<BF>(t.b[j], s);
        const int sb = (int)(t.b[j].s[s] >> (8 * q));
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              operand<AF>(t.a[i], s), b, acc[i][j], AF, BF, 0, (int)(t.a[i].s[s] >> (8 * q)), 0, sb);
      }
  };
  const int64_t full = kb >> 3;  // whole turns
  T cur, next;
  int64_t c = wave;
  if (c < full) load(cur, c, std::false_type{});
  for (; c < full; c += kRowsWaves) {
    if (c + kRowsWaves < full) load(next, c + kRowsWaves, std::false_type{});
    multiply(cur);
    cur = next;
  }
  if ((kb & 7) && full % kRowsWaves == wave) {
    load(cur, full, std::true_type{});
    multiply(cur);
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) red[wave][i][j][lane] = acc[i][j];
  __syncthreads();

  // Wave w takes the (row tile, column tile) pairs w, w + 4, ...
  auto total = [&](int i, int j) {
    v4f s = red[0][i][j][lane];
#pragma unroll
    for (int w = 1; w < kRowsWaves; ++w) s += red[w][i][j][lane];
    return s;
  };
  for (int u = wave; u < MT * H; u += kRowsWaves) {
    const int i = u / H, j = u % H;
    const int col = 16 * j + l16;
    if (col >= nlen) continue;
    const int64_t oc = n0 + col;
    v4f z = total(i, j), up = GATED ? total(i, (j + H) % CT) : v4f{};
    if (E.bias) {
      const float *b = E.bias + (int64_t)g * E.bias_gs + oc;
      z += b[0];
      if (GATED) up += b[P.N];
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 16 * i + 4 * q + v;
      if (row >= mlen) break;
      const int64_t m = m0 + row;
      if (E.z) {
        if (P.out_f32) {
          float *zr = static_cast<float *>(E.z) + m * E.ldz + oc;
          zr[0] = z[v];
          if (GATED) zr[P.N] = up[v];
        } else {
          uint16_t *zr = static_cast<uint16_t *>(E.z) + m * E.ldz + oc;
          zr[0] = f32_to_bf16_rne(z[v]);
          if (GATED) zr[P.N] = f32_to_bf16_rne(up[v]);
        }
      }
      float x = 0.0f;
      with_act(E.act, [&](auto a) { x = act_value<decltype(a)::value>(z[v]); });
      if (GATED) x *= up[v];
      if (P.out_f32) {
        if (E.res) x += static_cast<const float *>(E.res)[m * E.ldr + oc];
        static_cast<float *>(P.c)[m * P.ldc + oc] = x;
      } else {
        if (E.res) x += bits_f32((uint32_t)static_cast<const uint16_t *>(E.res)[m * E.ldr + oc] << 16);
        static_cast<uint16_t *>(P.c)[m * P.ldc + oc] = f32_to_bf16_rne(x);
      }
    }
  }
}

template <int AF, int BF, int MT, int EPI>
hipError_t rows_one(const GemmArgs &a0, const ActArgs &e, hipStream_t st) {
  constexpr int CT = 2, H = EPI == 2 ? CT / 2 : CT;
  GemmArgs a = a0;
  // upper bound of the row tiles: every group adds at most one partial tile,
  // and no tile is empty
  const int64_t whole = a.M / (16 * MT) + (a.gl ? a.G : (a.M % (16 * MT) ? 1 : 0));
  a.tiles_m = whole < a.M ? whole : a.M;
  a.tiles_n = (a.N + 16 * H - 1) / (16 * H);
  a.total = a.tiles_m * a.tiles_n;
  if (a.total > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mxgemm_rows_kernel<AF, BF, MT, CT, EPI>), dim3((unsigned)a.total), dim3(kRowsThreads), 0, st, a, e);
  return hipGetLastError();
}

template <int AF, int BF, int EPI>
hipError_t rows_mt(const GemmArgs &a, const ActArgs &e, int mt, hipStream_t st) {
  if (mt == 1) return rows_one<AF, BF, 1, EPI>(a, e, st);
  if (mt == 2) return rows_one<AF, BF, 2, EPI>(a, e, st);
  return rows_one<AF, BF, 4, EPI>(a, e, st);
}

template <int EPI>
hipError_t rows_any(const GemmLaunch &L, const ActArgs &e, int mt, hipStream_t st) {
  const GemmArgs a = gemm_args(L);
  if (L.a_fmt == kFmtE4M3)
    return L.b_fmt == kFmtE2M1 ? rows_mt<kFmtE4M3, kFmtE2M1, EPI>(a, e, mt, st) : rows_mt<kFmtE4M3, kFmtE4M3, EPI>(a, e, mt, st);
  return L.b_fmt == kFmtE2M1 ? rows_mt<kFmtE5M2, kFmtE2M1, EPI>(a, e, mt, st) : rows_mt<kFmtE5M2, kFmtE4M3, EPI>(a, e, mt, st);
}

}  // namespace

hipError_t launch_gemm_act(const GemmLaunch &L, const ActArgs &e, bool gated, hipStream_t st) {
  // rows an average group has, of the groups that can have any
  const int64_t groups = L.num_groups < L.M ? L.num_groups : L.M;
  const int64_t avg = (L.M + groups - 1) / groups;
  if (avg > 64) return gated ? launch_gated_tiles(L, e, st) : launch_act_tiles(L, e, st);
  const int mt = avg <= 8 ? 1 : avg <= 24 ? 2 : 4;
  return gated ? rows_any<2>(L, e, mt, st) : rows_any<1>(L, e, mt, st);
}

}  // namespace mxfp4
