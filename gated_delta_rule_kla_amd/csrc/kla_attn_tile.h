// kla_attn_tile.h -- a wave's share of a tile of keys in attention (kla_attn.hip,
// kla_kv4_chunk.hip): 32 queries against 32 or 64 keys and values in LDS, both products on
// v_mfma_f32_32x32x16_bf16 and transposed (see kla_attn.hip).
#pragma once

#include "kla_common.h"

namespace kla {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// The left operand V^T, channels 32 j + r against the slots of keys 16 kk .. 16 kk + 15, from a
// tile of rows of V: two transposing reads of 4 keys x 16 channels.
template <int D>
__device__ __forceinline__ bf16x8 v_operand(const bf16 *tile, int kk, int j, int lane) {
  constexpr int PPR = D / 8;
  bf16x4 w[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = 16 * kk + 8 * e + 4 * (lane >> 5) + ((lane >> 2) & 3);
    const int col = 32 * j + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    const bf16 *a = tile + row * D + 8 * ((col >> 3) ^ ((row & 3) << 2 & (PPR - 1))) + (col & 7);
    w[e] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)a);
  }
  return bf16x8{w[0][0], w[0][1], w[0][2], w[0][3], w[1][0], w[1][1], w[1][2], w[1][3]};
}

// The left operand K, keys 32 kb + r against channels 16 j + 8 h and up, from a tile of rows.
template <int D>
__device__ __forceinline__ bf16x8 k_operand(const bf16 *tile, int kb, int j, int lane) {
  const int row = 32 * kb + (lane & 31);
  return *reinterpret_cast<const bf16x8 *>(tile + row * D + 8 * ((2 * j + (lane >> 5)) ^ (row & (D / 8 - 1))));
}

// The larger of a lane's value and its neighbour's in the other half of the wave.  The two results
// are copied first: the compiler's bit cast of a vector's element is one of its first element,
// which is the lower half's value alone.
__device__ __forceinline__ float both_halves_max(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto w = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned lower = w[0], upper = w[1];
  return fmaxf(__builtin_bit_cast(float, lower), __builtin_bit_cast(float, upper));
}

// One tile's softmax: scores x[kb][i] (key 32 kb + 8 (i / 4) + 4 h + i % 4 against query r) to
// weights, with the running maximum m, this half's sum l and the output so far.  The maximum
// only moves when a score exceeds it by 2^LAG: weights up to 2^LAG cost no precision (they are
// floating point, and the sum too), and most tiles leave the output as it is.
constexpr float LAG = 8.f;
template <int DB, int KB>
__device__ __forceinline__ void softmax_tile(const f32x16 *x, float c, float &m, float &l, f32x16 *acc, bf16x8 *pt) {
  float t4[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t4[i] = x[0][i];
#pragma unroll
  for (int k = 4; k < 16 * KB; k += 4)
#pragma unroll
    for (int i = 0; i < 4; ++i) t4[i] = fmaxf(t4[i], x[k / 16][k % 16 + i]);
  float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
  top = both_halves_max(top) * c;
  if (__any(top > m + LAG)) {
    const float mn = top > m + LAG ? top : m;
    const float al = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
    l *= al;
#pragma unroll
    for (int j = 0; j < DB; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[j][i] *= al;
    m = mn;
  }
  const float base = m == -INFINITY ? 0.f : m;
  float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float e = __builtin_amdgcn_exp2f(fmaf(x[kb][i], c, -base));
      s4[i % 4] += e;
      pt[2 * kb + i / 8][i % 8] = (bf16)e;
    }
  l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
}

}  // namespace

}  // namespace kla
