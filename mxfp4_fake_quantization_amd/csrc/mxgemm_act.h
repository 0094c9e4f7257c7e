// mxgemm_act.h -- activations, and the epilogue of the grouped MX product:
// bias, pre-activation output, activation (gated or not), residual.
#pragma once

#include "mxfp4_rows8.h"

namespace mxfp4 {

enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

// Arguments of the epilogue; res and z are of the output's type.
struct ActArgs {
  const float *bias;  // [groups, columns of B] or NULL
  int64_t bias_gs;    // elements between groups (0: one row for all)
  const void *res;    // [M, ldr] or NULL
  int64_t ldr;
  void *z;            // [M, ldz]: A B^T + bias, or NULL
  int64_t ldz;
  int act;
};

// 1 / (1 + exp(-x)) on the hardware 2^x and reciprocal (1 ulp each): the
// product with log2 e rounds the exponent, a relative error of |x| 2^-24.
__device__ __forceinline__ float sigmoid_f(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}

// Phi(x) of the normal distribution, and exp(-x^2 / 2), without a branch: with w =
// 3 |x| / (8 sqrt 2) and u = w / (1 + w), Phi(-|x|) = exp(-x^2 / 2) Q(u).  Q, of degree
// 9 with Q(0) = 1/2, was fitted in 64 bits (least squares, weighted towards equal
// ripple, its coefficients rounded to fp32 from the lowest): within 1.3e-8 of the
// quotient for |x| up to 13, where exp(-x^2 / 2) reaches 2^-126.  In u, unlike in 1 -
// u, the roundings of a small |x| stay small.  So the tail is good to (2.2 x^2 + 9)
// 2^-24 of itself; over normal arguments gelu's error is 3.4e-8 of its norm and the
// slope's 3.8e-8, as with 32-bit erf (3.8e-8, 4.0e-8).
__device__ __forceinline__ float normal_cdf(float x, float *gauss) {
  const float w = fminf(fabsf(x) * 0.265165043f, 1e30f);  // an infinite x keeps u = 1
  const float u = w * __builtin_amdgcn_rcpf(1.0f + w);
  float q = fmaf(u, -0.0303070173f, 0.131572232f);
  q = fmaf(u, q, -0.171980724f);
  q = fmaf(u, q, -0.0414950512f);
  q = fmaf(u, q, 0.180597797f);
  q = fmaf(u, q, 0.411485612f);
  q = fmaf(u, q, -1.52645111f);
  q = fmaf(u, q, 2.05108619f);
  q = fmaf(u, q, -1.50450635f);
  q = fmaf(u, q, 0.5f);
  *gauss = __builtin_amdgcn_exp2f(-0.72134752f * (x * x));
  const float tail = q * *gauss;
  return x > 0.0f ? 1.0f - tail : tail;
}

// Act(x): x, max(x, 0), x sigmoid(x), x Phi(x).
template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  float gauss;
  if (ACT == kActRelu) return x < 0.0f ? 0.0f : x;
  if (ACT == kActSilu) return x * sigmoid_f(x);
  if (ACT == kActGelu) return x * normal_cdf(x, &gauss);
  return x;
}

// Calls f with the activation as a compile-time number.
template <int V>
struct ActT {
  static constexpr int value = V;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {  // the same for the whole launch
    case kActRelu: f(ActT<kActRelu>{}); break;
    case kActSilu: f(ActT<kActSilu>{}); break;
    case kActGelu: f(ActT<kActGelu>{}); break;
    default: f(ActT<kActNone>{}); break;
  }
}

// The first n < 8 elements of a 16-byte bf16 piece, as one 8-, one 4- and one
// 2-byte access (element by element the last column tile of an odd row took
// 15 us longer than the others).
__device__ __forceinline__ u32x4 load_part(const uint16_t *p, int n) {
  typedef uint64_t u64_a2 __attribute__((aligned(2)));
  typedef uint32_t u32_a2 __attribute__((aligned(2)));
  const uint64_t four = n & 4 ? *reinterpret_cast<const u64_a2 *>(p) : 0;
  const uint32_t two = n & 2 ? *reinterpret_cast<const u32_a2 *>(p + (n & 4)) : 0;
  const uint32_t one = n & 1 ? p[n & 6] : 0;
  const uint64_t rest = n & 2 ? two | ((uint64_t)one << 32) : one;
  const uint64_t lo = n & 4 ? four : rest, hi = n & 4 ? rest : 0;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
__device__ __forceinline__ void store_part(uint16_t *p, u32x4 w, int n) {
  typedef uint64_t u64_a2 __attribute__((aligned(2)));
  typedef uint32_t u32_a2 __attribute__((aligned(2)));
  if (n & 4) *reinterpret_cast<u64_a2 *>(p) = (uint64_t)w.x | ((uint64_t)w.y << 32);
  const uint32_t t = n & 4 ? w.z : w.x, o = n & 4 ? w.w : w.y;
  if (n & 2) *reinterpret_cast<u32_a2 *>(p + (n & 4)) = t;
  if (n & 1) p[n & 6] = (uint16_t)(n & 2 ? o : t);
}

// The accumulators of a tile of mxgemm_tile.h (row 8(v/4) + 4h + v%4, column
// l32 of each 32 x 32) to the outputs.  bf16 outputs are staged in LDS, the
// first half of the rows in the A buffers, the second in the B buffers, and
// leave in 16-byte row pieces (any alignment of elements); the residual comes
// in through the same places, so that its sum with the activation is rounded
// once.  fp32 outputs are written as they lie, 128 bytes a half-wave.
template <int EPI, int BM, int BN, int NT, int WM, int WN, int RS, typename ACC>
__device__ __forceinline__ void act_epilogue(void *c, int64_t ldc, int out_f32, const ActArgs &E, ACC &acc,
                                             uint8_t *bufa, uint8_t *bufb, int64_t m0, int64_t mlen, int64_t n0,
                                             int64_t nlen, int64_t N, int g, int wr0, int wc0, int lane, int tid) {
  constexpr bool GATED = EPI == 2;
  constexpr int H = GATED ? WN / 2 : WN;          // MFMA tiles of output columns
  constexpr int BNO = GATED ? BN / 2 : BN;
  typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
  const int h = lane >> 5, l32 = lane & 31;
  const int oc0 = GATED ? wc0 / 2 : wc0;           // the wave's first output column

  // without a bias 0 is added: a branch around it would have to merge the
  // accumulators' register tuples, which spilled
  const float *b = E.bias + (E.bias ? (int64_t)g * E.bias_gs + n0 : 0);
#pragma unroll
  for (int j = 0; j < WN; ++j) {
    const int col = oc0 + 32 * (j % H) + l32;
    const float bj = E.bias && col < nlen ? b[col + (j >= H ? N : 0)] : 0.0f;
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] += bj;
    __builtin_amdgcn_sched_barrier(0);
  }

  constexpr int OS = 2 * BN + 16, HR = BM / 2;
  static_assert(HR * OS <= 2 * BM * RS && HR * OS <= 2 * BN * RS, "output staging");
  auto lds_row = [&](int r) { return (r < HR ? bufa : bufb) + (r & (HR - 1)) * OS; };
  // row of a lane's value v of MFMA tile i, without the wave's and half's part
  auto tile_row = [&](int i, int v) { return 32 * i + 8 * (v >> 2) + (v & 3); };
  const int row0 = wr0 + 4 * h;
  // the lane's places in the stage: a wave's rows lie in one half
  static_assert(HR % (32 * WM) == 0, "a wave's rows in one half");
  uint8_t *const mine = (wr0 < HR ? bufa : bufb) + ((wr0 & (HR - 1)) + 4 * h) * OS + 2 * l32;

  // Pieces of 8 columns of the staged rows, W columns wide; f(row, column in
  // the stage, valid elements).
  auto pieces = [&](auto width, auto f) {
    constexpr int W = decltype(width)::value, CH = W / 8, RPI = NT / CH;
    const int ch = tid % CH;
#pragma unroll 4
    for (int k = 0; k < BM / RPI; ++k) {
      const int row = tid / CH + RPI * k;
      if (row < mlen) f(row, 8 * ch);
    }
  };
  auto put = [&](void *dst, int64_t ld, int row, int stage_col, int64_t out_col, int left) {
    if (left <= 0) return;
    const uint8_t *src = lds_row(row) + 2 * stage_col;
    uint16_t *d = static_cast<uint16_t *>(dst) + (m0 + row) * ld + out_col;
    if (left >= 8) {
      __builtin_nontemporal_store(*reinterpret_cast<const u32x4 *>(src), reinterpret_cast<u32x4_a2 *>(d));
    } else {
      store_part(d, *reinterpret_cast<const u32x4 *>(src), left);
    }
  };

  if (E.z) {
    if (!out_f32) {
      __syncthreads();  // every wave is past its last fragment read
#pragma unroll
      for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int j = 0; j < WN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            *reinterpret_cast<uint16_t *>(mine + 2 * wc0 + tile_row(i, v) * OS + 64 * j) = (uint16_t)pack_bf16(acc[i][j][v], 0.0f);
            if ((v & 3) == 3) __builtin_amdgcn_sched_barrier(0);
          }
      __syncthreads();
      pieces(ActT<BN>{}, [&](int row, int sc) {
        const int q = sc >> 5, j = q % WN;
        const int col = GATED ? q / WN * (16 * WN) + 32 * (j % H) + (sc & 31) : sc;
        put(E.z, E.ldz, row, sc, n0 + col + (GATED && j >= H ? N : 0), (int)(nlen - col));
      });
    } else {
#pragma unroll
      for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int j = 0; j < WN; ++j) {
          const int col = oc0 + 32 * (j % H) + l32;
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int row = row0 + tile_row(i, v);
            if (row < mlen && col < nlen)
              static_cast<float *>(E.z)[(m0 + row) * E.ldz + n0 + col + (j >= H ? N : 0)] = acc[i][j][v];
            __builtin_amdgcn_sched_barrier(0);
          }
        }
    }
  }

  if (E.res && !out_f32) {
    // 8 pieces in flight a lane (2 were 5 us slower on a 4096 x 4096 product);
    // pieces past the edge read the tile's first ones and are not used
    constexpr int CH = BNO / 8, RPI = NT / CH, AHEAD = BM / RPI < 8 ? BM / RPI : 8;
    const int sc = 8 * (tid % CH), left = (int)(nlen - sc);
    const uint16_t *src = static_cast<const uint16_t *>(E.res) + m0 * E.ldr + n0;
    __syncthreads();
    for (int k = 0; k < BM / RPI; k += AHEAD) {
      u32x4 w[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int row = tid / CH + RPI * (k + u);
        const bool in = row < mlen && left > 0;
        const uint16_t *p = src + (in ? row * E.ldr + sc : 0);
        if (left >= 8 || !in) {
          if (nlen >= 8) w[u] = *reinterpret_cast<const u32x4_a2 *>(p);
        } else {
          w[u] = load_part(p, left);
        }
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int row = tid / CH + RPI * (k + u);
        if (row < mlen && left > 0) *reinterpret_cast<u32x4 *>(lds_row(row) + 2 * sc) = w[u];
      }
    }
  }
  __syncthreads();
  with_act(E.act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const int col = oc0 + 32 * j + l32;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          float x = act_value<ACT>(acc[i][j][v]);
          if (GATED) x *= acc[i][(j + H) % WN][v];
          if (!out_f32) {
            uint16_t *at = reinterpret_cast<uint16_t *>(mine + 2 * oc0 + tile_row(i, v) * OS + 64 * j);
            // places past the tile's edge hold what was there before, and are not stored
            if (E.res) x += bits_f32((uint32_t)*at << 16);
            *at = (uint16_t)pack_bf16(x, 0.0f);
          } else {
            const int row = row0 + tile_row(i, v);
            if (row < mlen && col < nlen) {
              if (E.res) x += static_cast<const float *>(E.res)[(m0 + row) * E.ldr + n0 + col];
              static_cast<float *>(c)[(m0 + row) * ldc + n0 + col] = x;
            }
          }
          if ((v & 3) == 3) __builtin_amdgcn_sched_barrier(0);  // few temporaries beside the accumulators
        }
      }
  });
  if (out_f32) return;
  __syncthreads();
  pieces(ActT<BNO>{}, [&](int row, int sc) { put(c, ldc, row, sc, n0 + sc, (int)(nlen - sc)); });
}

}  // namespace mxfp4
