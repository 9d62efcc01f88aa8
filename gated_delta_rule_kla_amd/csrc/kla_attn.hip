// kla_attn.hip -- causal softmax attention over whole prompts (gfx950).
//
// o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j) over the keys j that query i
// sees: j <= i + (lk - lq) of its own sequence (include/kla.h, kla_attn_fwd).
//
// One pass over the keys with a running maximum and sum.  Each wave of a workgroup holds 32
// queries of one head, their 32 x D output and statistics in registers, and all waves share
// tiles of 64 (or 32) keys and values in LDS, two of them: while one is used, the next arrives
// by direct global-to-LDS loads.  Both products run transposed on v_mfma_f32_32x32x16_bf16: S^T =
// K Q^T puts one query in each lane (pair), so maxima and sums need one exchange between the
// two halves of a wave, and S^T's registers, rounded to bf16, are the right operand P^T of
// O^T = V^T P^T as they stand: its contraction slots are taken in the order in which the
// accumulator holds the keys (slot 8h + e of 16 keys is key 4h + e, or 8 + 4h + e - 4).  V^T
// comes out of the row-major tile by transposing LDS reads.
//
// Measured: 16,384 tokens, 16 heads of 128 over 2: 0.91 to 0.98 ms, up to 1.2 PFLOP/s, where a bf16 product
// of 8192^3 reaches 1.38 and the clock falls below 2.0 GHz under either.  The matrix cores are
// busy 60% of the cycles and the vector ALU 54%.  Tried on the way, at 0.98: two groups of
// waves half a tile apart with a barrier between their phases 1.06 ms; three or four tiles in
// LDS 0.99; the next tile's scores beside this tile's weights within a wave spilled (8,192
// tokens, 32 heads: 0.99 ms against 0.49) and lost with tiles of 32 keys too, where nothing
// did (0.63 against 0.53).
//
// LDS rows are D values long without padding (the direct loads write 1 KB runs); 16-byte
// pieces are exchanged within a row instead, K's by the row's low bits, V's by its low two
// bits in steps of 64 bytes, so that the reads of a wave spread over the banks.
#include <algorithm>
#include <cmath>

#include "kla_common.h"
#include "kla_internal.h"

namespace kla {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

struct AttnParams {
  const void *q, *k, *v;
  void *o;
  float *lse;
  const int32_t *cu_q, *cu_k;  // device, or nullptr (dense)
  float c;                     // |scale| log2(e)
  int flip;                    // scale < 0: q is negated; scale == 0: q is zero
  int N, B, Hq, Hkv, Tq, Tk;
  int slots;                   // query tiles of a head, at most
};

// Query tile `slot` of a head: its sequence's queries and keys, and its first query.
struct Span {
  int q0, lq, k0, lk, first;
};
template <int BM>
__device__ __forceinline__ bool find_span(const AttnParams &p, int slot, int b, Span *s) {
  if (!p.cu_q) {
    *s = Span{0, p.Tq, 0, p.Tk, slot * BM};
    return s->first < s->lq;
  }
  // sequence n has the slots cu[n] / BM + n and up: never another's
  int lo = 0, hi = p.N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_q[mid] / BM + mid <= slot) lo = mid; else hi = mid;
  }
  const int a = min(max(p.cu_q[lo], 0), p.Tq), z = min(max(p.cu_q[lo + 1], a), p.Tq);
  const int ka = min(max(p.cu_k[lo], 0), p.Tk), kz = min(max(p.cu_k[lo + 1], ka), p.Tk);
  *s = Span{a, z - a, ka, kz - ka, (slot - (p.cu_q[lo] / BM + lo)) * BM};
  return s->first >= 0 && s->first < s->lq;
}

// Head (with its batch row) and query tile of a workgroup.  Workgroup ids go round the eight
// XCDs, each with its own L2: the heads that share keys stay on one, and the longest tiles (a
// sequence's last) start first.
__device__ __forceinline__ void place(const AttnParams &p, unsigned id, int *bh, int *slot) {
  const int heads = p.B * p.Hq;
  if (heads % 8 == 0) {
    const int per = heads / 8;
    const unsigned s = id >> 3;
    *bh = (id & 7) * per + s % per;
    *slot = p.slots - 1 - s / per;
  } else {
    *bh = id % heads;
    *slot = p.slots - 1 - id / heads;
  }
}

// 1 KB straight from global memory, at a scalar address and each lane's byte offset, into LDS
// at byte `at`: lane i's 16 bytes land 16 i behind.  In asm, since the compiler makes the next
// LDS read wait for the builtin's load, also where it goes to the other buffer; the kernel
// itself waits (vmcnt) before the barrier that ends a tile.  It has no output register.  m0 is
// listed so that no value which the compiler keeps there lives across it; the compiler warns of
// every reserved register in such a list.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds(const bf16 *src, unsigned lane_at, unsigned at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(lane_at), "s"(src)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// One query against keys 0 .. n-1 by one wave, key by key.
template <typename E, int D>
__device__ void attend_one(const E *q, const E *k, const E *v, int n, const AttnParams &p, E *o, float *lse) {
  constexpr int CPL = D / 64;  // channels of a lane
  const int lane = threadIdx.x & 63;
  const float sign = p.flip == 0 ? 1.f : (p.flip == 1 ? -1.f : 0.f);
  float m = -INFINITY, l = 0.f, acc[CPL] = {};
  for (int j0 = 0; j0 < n; j0 += 64) {
    float x = 0.f;
    const E *kr = k + (size_t)min(j0 + lane, n - 1) * D;
#pragma unroll 4
    for (int d = 0; d < D; d += 16 / (int)sizeof(E)) {
      const uint4 a = ldg16(q + d), b = ldg16(kr + d);
      E ea[16 / sizeof(E)], eb[16 / sizeof(E)];
      __builtin_memcpy(ea, &a, 16);
      __builtin_memcpy(eb, &b, 16);
#pragma unroll
      for (unsigned i = 0; i < 16 / sizeof(E); ++i) x = fmaf(Elem<E>::to_f32(ea[i]) * sign, Elem<E>::to_f32(eb[i]), x);
    }
    x = j0 + lane < n ? x * p.c : -INFINITY;
    float top = x;
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) top = fmaxf(top, __shfl_xor(top, w));
    const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
    const float al = __builtin_amdgcn_exp2f(m - base), e = __builtin_amdgcn_exp2f(x - base);
    m = mn;
    l = l * al + e;
#pragma unroll
    for (int i = 0; i < CPL; ++i) acc[i] *= al;
    for (int j = 0; j < min(64, n - j0); ++j) {
      const float w = Elem<E>::to_f32(Elem<E>::from_f32(__shfl(e, j)));
      const E *vr = v + (size_t)(j0 + j) * D + CPL * lane;
#pragma unroll
      for (int i = 0; i < CPL; ++i) acc[i] = fmaf(w, Elem<E>::to_f32(vr[i]), acc[i]);
    }
  }
#pragma unroll
  for (int w = 32; w >= 1; w >>= 1) l += __shfl_xor(l, w);
#pragma unroll
  for (int i = 0; i < CPL; ++i) o[CPL * lane + i] = Elem<E>::from_f32(l == 0.f ? 0.f : acc[i] / l);
  if (lse && lane == 0) *lse = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.693147181f;
}

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

// q's row as the right operand.  The running maximum is taken of the unscaled scores, so the
// scale's sign goes to q.  The values are here when this returns: a wait for them in the loop
// would also wait for the tile in flight.
template <int D>
__device__ __forceinline__ void load_q(const AttnParams &p, const bf16 *row, int h, bf16x8 *q) {
#pragma unroll
  for (int j = 0; j < D / 16; ++j) q[j] = __builtin_bit_cast(bf16x8, ldg16(row + 16 * j + 8 * h));
  if (p.flip) {
    const float sign = p.flip == 1 ? -1.f : 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) q[j][i] = (bf16)((float)q[j][i] * sign);
  }
#pragma unroll
  for (int j = 0; j < D / 16; ++j) asm volatile("" : "+v"(q[j]));
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
  {  // the other half's
    const auto w = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, top), __builtin_bit_cast(unsigned, top), false, false);
    top = fmaxf(__builtin_bit_cast(float, w[0]), __builtin_bit_cast(float, w[1])) * c;
  }
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

// A wave's results: lane (r, h) holds query qw + r, channels 32 j + 8 (i / 4) + 4 h + i % 4.
template <typename E, int D>
__device__ __forceinline__ void finish(const AttnParams &p, const Span &s, int bh, int qw, const f32x16 *acc, float m,
                                       float l, const E *K, const E *V) {
  constexpr int DB = D / 32;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5, off = s.lk - s.lq;
  l += __shfl_xor(l, 32);
  const bool mine = qw + r < s.lq;
  float worst = l;  // not finite if any of this lane's results is not
#pragma unroll
  for (int j = 0; j < DB; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) worst = fmaf(acc[j][i], 0.f, worst);
  const unsigned long long odd = __ballot(mine && !(fabsf(worst) < INFINITY));
  const unsigned again = (unsigned)odd | (unsigned)(odd >> 32);
  if (mine && !(again >> r & 1)) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    E *O = (E *)p.o + ((size_t)bh * p.Tq + s.q0 + qw + r) * D;
#pragma unroll
    for (int j = 0; j < DB; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        if constexpr (sizeof(E) == 2) {
          // channels 2 i + 4 h and 2 i + 8 + 4 h, four each: the halves change pieces, so that
          // each stores eight in a row
          u32x4 w;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bf16x2 lo = {(bf16)(acc[j][i + 2 * e] * inv), (bf16)(acc[j][i + 2 * e + 1] * inv)};
            const bf16x2 hi = {(bf16)(acc[j][i + 4 + 2 * e] * inv), (bf16)(acc[j][i + 4 + 2 * e + 1] * inv)};
            const auto c = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, lo),
                                                            __builtin_bit_cast(unsigned, hi), false, false);
            w[e] = c[0];
            w[2 + e] = c[1];
          }
          *reinterpret_cast<u32x4 *>(O + 32 * j + 2 * i + 8 * h) = w;
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 4)
            *reinterpret_cast<f32x4 *>(O + 32 * j + 2 * (i + e) + 4 * h) =
                f32x4{acc[j][i + e] * inv, acc[j][i + e + 1] * inv, acc[j][i + e + 2] * inv, acc[j][i + e + 3] * inv};
        }
      }
    if (p.lse && h == 0)
      p.lse[(size_t)bh * p.Tq + s.q0 + qw + r] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.693147181f;
  }
  // A value that is not finite, times the zero weight of a query that does not see it, is NaN
  // in the matrix product: such queries are computed again from the keys that they see alone, one
  // by one, also where they do see it (4,096 tokens of 16 heads, an infinity in an early value of
  // eight: 21 ms against 0.08; 16,384: 0.27 s against 0.96 ms).
  for (unsigned left = again; left; left &= left - 1) {
    const int i = qw + __builtin_ctz(left);
    const size_t row = (size_t)bh * p.Tq + s.q0 + i;
    attend_one<E, D>((const E *)p.q + row * D, K, V, i + off + 1, p, (E *)p.o + row * D, p.lse ? p.lse + row : nullptr);
  }
}

// KS groups of NW / KS waves share the queries and take every KS-th tile of BN keys, and join at
// the end, so that a workgroup's chain of tiles is as much shorter.
template <int D, int NW, int KS, int BN>
__global__ __launch_bounds__(64 * NW, 2) void kla_attn_kernel(AttnParams p) {
  constexpr int BM = 32 * NW / KS, KB = BN / 32;  // queries, tiles of 32 keys
  constexpr int PPR = D / 8;         // 16-byte pieces of a row
  constexpr int RPI = 64 / PPR;      // rows of one direct load
  constexpr int KJ = D / 16, DB = D / 32;
  __shared__ __attribute__((aligned(1024))) bf16 s_kv[2][2][KS * BN * D];  // K and V, two buffers each

  int bh, slot;
  place(p, blockIdx.x, &bh, &slot);
  const int b = bh / p.Hq, hq = bh % p.Hq, hk = hq / (p.Hq / p.Hkv);
  Span s;
  if (!find_span<BM>(p, slot, b, &s)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5, group = KS == 1 ? 0 : wave / (NW / KS);
  const int off = s.lk - s.lq;
  const bf16 *Q = (const bf16 *)p.q + ((size_t)bh * p.Tq + s.q0) * D;
  const bf16 *K = (const bf16 *)p.k + (((size_t)b * p.Hkv + hk) * p.Tk + s.k0) * D;
  const bf16 *V = (const bf16 *)p.v + (((size_t)b * p.Hkv + hk) * p.Tk + s.k0) * D;

  const int qw = s.first + 32 * (wave % (NW / KS));  // this wave's first query
  const int qi = min(qw + r, s.lq - 1);              // this lane's (queries past the end repeat the last)
  f32x16 acc[DB];
#pragma unroll
  for (int j = 0; j < DB; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  // keys up to the last that the workgroup's, and this wave's, last query sees
  const int seen = min(s.first + BM, s.lq) + off;
  const int steps = seen > 0 ? (seen + KS * BN - 1) / (KS * BN) : 0;
  const int first_key = qw + off, last_key = min(qw + 31, s.lq - 1) + off;  // of the wave's first and last query

  // Each wave brings NP pieces of 1 KB of K and of V.  In a whole tile their places are a scalar
  // address and lane offsets that stay: worked out per load, they took a tenth of a tile's time.
  constexpr int NP = KS * BN / RPI / NW;
  static_assert(NP * RPI * NW == KS * BN, "pieces");
  unsigned ko[NP], vo[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int row = (wave * NP + i) * RPI + lane / PPR, pc = lane % PPR;
    ko[i] = 2 * (row * D + 8 * (pc ^ (row & (PPR - 1))));
    vo[i] = 2 * (row * D + 8 * (pc ^ ((row & 3) << 2 & (PPR - 1))));
  }
  const unsigned lds = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)&s_kv[0][0][0] + wave * NP * 1024;
  auto fetch = [&](int t, int buf) {
    const bf16 *const kt = K + (size_t)t * KS * BN * D, *const vt = V + (size_t)t * KS * BN * D;
    const int left = s.lk - t * KS * BN;
    const unsigned to = lds + buf * KS * BN * D * 2;
    if (left >= KS * BN) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        load_lds(kt, ko[i], to + i * 1024);
        load_lds(vt, vo[i], to + 2 * KS * BN * D * 2 + i * 1024);
      }
    } else {  // past the end: the last key, masked below
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int row = (wave * NP + i) * RPI + lane / PPR, over = 2 * D * max(row - (left - 1), 0);
        load_lds(kt, ko[i] - over, to + i * 1024);
        load_lds(vt, vo[i] - over, to + 2 * KS * BN * D * 2 + i * 1024);
      }
    }
  };

  if (steps > 0) fetch(0, 0);
  bf16x8 q[KJ];
  load_q<D>(p, Q + (size_t)qi * D, h, q);
  for (int t = 0; t < steps; ++t) {
    const int buf = t & 1;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (t + 1 < steps) fetch(t + 1, buf ^ 1);
    const int key0 = (t * KS + group) * BN;
    if (key0 > last_key || qw >= s.lq) continue;
    const bf16 *kt = s_kv[0][buf] + group * BN * D, *vt = s_kv[1][buf] + group * BN * D;

    f32x16 x[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[kb][i] = 0.f;
#pragma unroll
    for (int j = 0; j < KJ; ++j)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        x[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k_operand<D>(kt, kb, j, lane), q[j], x[kb], 0, 0, 0);
    // eight operands are read ahead of the products, and the first of V's ahead of the softmax:
    // left to the compiler, each product waits for its own read
    constexpr int AHEAD = KJ * KB < 8 ? KJ * KB : 8, VA = KB == 1 ? 2 : 1;
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
    for (int j = 0; j < KJ * KB - AHEAD; ++j) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, AHEAD, 0);
    bf16x8 va[VA][DB];
#pragma unroll
    for (int kk = 0; kk < VA; ++kk)
#pragma unroll
      for (int j = 0; j < DB; ++j) va[kk][j] = v_operand<D>(vt, kk, j, lane);
    if (key0 + BN - 1 > first_key) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (key0 + 32 * kb + 8 * (i / 4) + 4 * h + i % 4 > qi + off) x[kb][i] = -INFINITY;
    }
    bf16x8 pt[2 * KB];
    softmax_tile<DB, KB>(x, p.c, m, l, acc, pt);
#pragma unroll
    for (int kk = 0; kk < 2 * KB; ++kk)
#pragma unroll
      for (int j = 0; j < DB; ++j)
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kk < VA ? va[kk][j] : v_operand<D>(vt, kk, j, lane), pt[kk], acc[j], 0, 0, 0);
  }
  if constexpr (KS > 1) {
    // the other groups' results through LDS, lane to lane: the layouts are the same
    constexpr int WG = NW / KS, SIZE = (4 * DB + 1) * 64;  // waves of a group, f32x4 of a wave
    static_assert((KS - 1) * WG * SIZE * 16 <= 4 * KS * BN * D * 2, "exchange");
    f32x4 *const ex = reinterpret_cast<f32x4 *>(s_kv) + lane;
    __syncthreads();
    if (group > 0) {
      f32x4 *const to = ex + (wave - WG) * SIZE;
#pragma unroll
      for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[(4 * j + i) * 64] = f32x4{acc[j][4 * i], acc[j][4 * i + 1], acc[j][4 * i + 2], acc[j][4 * i + 3]};
      to[4 * DB * 64] = f32x4{m, l, 0.f, 0.f};
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < KS; ++g) {
      const f32x4 *const from = ex + (wave + (g - 1) * WG) * SIZE;
      const f32x4 ml = from[4 * DB * 64];
      const float mn = fmaxf(m, ml[0]), base = mn == -INFINITY ? 0.f : mn;
      const float f0 = __builtin_amdgcn_exp2f(m - base), f1 = __builtin_amdgcn_exp2f(ml[0] - base);
      m = mn;
      l = l * f0 + ml[1] * f1;
#pragma unroll
      for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][i] = acc[j][i] * f0 + from[(4 * j + i / 4) * 64][i % 4] * f1;
    }
  }
  finish<bf16, D>(p, s, bh, qw, acc, m, l, K, V);
}

// fp32: the same two products with every operand split into three bf16 terms (24 bits), the
// six products of terms that reach 2^-24 summed in fp32: 6 / 16 of the fp32 matrix
// instructions' cycles for the same sums.  A term ends at 2^-133, so numbers below 2^-109 keep
// fewer bits.  Tiles of 32 keys, split on their way from registers (the next tile's loads in
// flight) into one LDS buffer; the split of each tile, by every workgroup that reads it, and the two
// barriers stand between the products.  4,096 tokens of 16 heads over 2: 443 us (six products at
// a bf16 product's rate: 299), 64 channels 255; 16,384 tokens 6.5 ms (4.8).
template <int D>
__global__ __launch_bounds__(256, 1) void kla_attn_f32_kernel(AttnParams p) {
  constexpr int NW = 4, BM = 32 * NW, BN = 32;
  constexpr int PPR = D / 8, KJ = D / 16, DB = D / 32;
  constexpr int NP = BN * PPR / 256;  // pieces of 8 values a thread moves
  __shared__ __attribute__((aligned(1024))) bf16 s_k[3][BN * D], s_v[3][BN * D];

  int bh, slot;
  place(p, blockIdx.x, &bh, &slot);
  const int b = bh / p.Hq, hq = bh % p.Hq, hk = hq / (p.Hq / p.Hkv);
  Span s;
  if (!find_span<BM>(p, slot, b, &s)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int off = s.lk - s.lq;
  const float *Q = (const float *)p.q + ((size_t)bh * p.Tq + s.q0) * D;
  const float *K = (const float *)p.k + (((size_t)b * p.Hkv + hk) * p.Tk + s.k0) * D;
  const float *V = (const float *)p.v + (((size_t)b * p.Hkv + hk) * p.Tk + s.k0) * D;
  const int qw = s.first + 32 * wave, qi = min(qw + r, s.lq - 1);
  const float sign = p.flip == 0 ? 1.f : (p.flip == 1 ? -1.f : 0.f);

  bf16x8 q[KJ][3];
#pragma unroll
  for (int j = 0; j < KJ; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f = Q[(size_t)qi * D + 16 * j + 8 * h + i] * sign;
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        q[j][u][i] = (bf16)f;
        f -= (float)q[j][u][i];
      }
    }
  f32x16 acc[DB];
#pragma unroll
  for (int j = 0; j < DB; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  const int seen = min(s.first + BM, s.lq) + off;
  const int tiles = seen > 0 ? (seen + BN - 1) / BN : 0;
  const int first_key = qw + off, last_key = min(qw + 31, s.lq - 1) + off;

  f32x4 nk[NP][2], nv[NP][2];
  auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pc = tid + 256 * i, row = pc / PPR;
      const size_t at = (size_t)min(t * BN + row, s.lk - 1) * D + 8 * (pc % PPR);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        nk[i][w] = *reinterpret_cast<const f32x4 *>(K + at + 4 * w);
        nv[i][w] = *reinterpret_cast<const f32x4 *>(V + at + 4 * w);
      }
    }
  };
  auto put = [&](bf16 (*dst)[BN * D], int i, const f32x4 *f, int swz) {
    const int pc = tid + 256 * i, row = pc / PPR;
    float x[8] = {f[0][0], f[0][1], f[0][2], f[0][3], f[1][0], f[1][1], f[1][2], f[1][3]};
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      bf16x8 w;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = (bf16)x[e];
        x[e] -= (float)w[e];
      }
      *reinterpret_cast<bf16x8 *>(dst[u] + row * D + 8 * (pc % PPR ^ swz)) = w;
    }
  };
  if (tiles > 0) load(0);
  for (int t = 0; t < tiles; ++t) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int row = (tid + 256 * i) / PPR;
      put(s_k, i, nk[i], row & (PPR - 1));
      put(s_v, i, nv[i], (row & 3) << 2 & (PPR - 1));
    }
    __syncthreads();
    if (t + 1 < tiles) load(t + 1);
    const int key0 = t * BN;
    if (key0 > last_key || qw >= s.lq) continue;

    f32x16 x;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      bf16x8 a[3];
#pragma unroll
      for (int u = 0; u < 3; ++u)
        a[u] = *reinterpret_cast<const bf16x8 *>(s_k[u] + r * D + 8 * ((2 * j + h) ^ (r & (PPR - 1))));
#pragma unroll
      for (int u = 2; u >= 0; --u)
#pragma unroll
        for (int w = 2 - u; w >= 0; --w) x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[u], q[j][w], x, 0, 0, 0);
    }
    if (key0 + BN - 1 > first_key) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (key0 + 8 * (i / 4) + 4 * h + i % 4 > qi + off) x[i] = -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
    top = fmaxf(top, __shfl_xor(top, 32)) * p.c;
    if (__any(top > m)) {
      const float mn = fmaxf(m, top);
      const float al = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
      l *= al;
#pragma unroll
      for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][i] *= al;
      m = mn;
    }
    const float base = m == -INFINITY ? 0.f : m;
    bf16x8 pt[2][3];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float e = __builtin_amdgcn_exp2f(fmaf(x[i], p.c, -base));
      l += e;
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        pt[i / 8][u][i % 8] = (bf16)e;
        e -= (float)pt[i / 8][u][i % 8];
      }
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int j = 0; j < DB; ++j) {
        bf16x8 va[3];
#pragma unroll
        for (int u = 0; u < 3; ++u) va[u] = v_operand<D>(s_v[u], kk, j, lane);
#pragma unroll
        for (int u = 2; u >= 0; --u)
#pragma unroll
          for (int w = 2 - u; w >= 0; --w)
            acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va[u], pt[kk][w], acc[j], 0, 0, 0);
      }
  }
  finish<float, D>(p, s, bh, qw, acc, m, l, K, V);
}

// p.slots and the workgroups of tiles of BM queries
unsigned attn_grid(AttnParams *p, int BM) {
  p->slots = p->cu_q ? p->Tq / BM + p->N : (p->Tq + BM - 1) / BM;
  return (unsigned)((long long)p->slots * p->B * p->Hq);
}

template <int D, int NW, int KS, int BN>
hipError_t launch_attn_t(AttnParams p, hipStream_t st) {
  const unsigned grid = attn_grid(&p, 32 * NW / KS);
  hipLaunchKernelGGL((kla_attn_kernel<D, NW, KS, BN>), dim3(grid), dim3(64 * NW), 0, st, p);
  return hipGetLastError();
}

template <int D>
hipError_t launch_attn_f32(AttnParams p, hipStream_t st) {
  const unsigned grid = attn_grid(&p, 128);
  hipLaunchKernelGGL((kla_attn_f32_kernel<D>), dim3(grid), dim3(256), 0, st, p);
  return hipGetLastError();
}

// Which tiling, by the workgroups that tiles of 128 queries make:
// - 32 queries, keys in four groups, where those are at most a quarter of the CUs (100 queries,
//   3,000 keys, 16 heads: 33 us, with two groups 38; 1,000 tokens, 8 heads: 15.5, 16.1; at 128
//   of them, 1,000 tokens of 16 heads, 21.5, 16.5);
// - 64 queries, keys in two groups, where those are at most half the CUs (1,000 tokens, 16
//   heads: 16.5 us, 128 queries 19.0), and up to one a CU for dense batches whose later queries
//   see most keys, so that their work is uneven (2,048 tokens, 16 heads: 30.7 us, 128 queries
//   32.8; 8 times 128 queries of 2,000 keys: 42.1, 37.7).  Two groups' tiles make 16 KB each of
//   K and V: 32 keys of 128 channels (64: 17.7 us for 1,000 tokens), 64 of 64 (2,048 tokens
//   19.1 us, 32 keys 19.9);
// - 128 queries, keys in two groups, for dense batches of at most two of them a CU (4,096
//   tokens, 16 heads: 74 us against 83); packed sequences are uneven, and lose (8 of 1,000 to
//   8,000 tokens: 163 us against 140);
// - 256 queries where that still makes two workgroups a CU and sequences are long (16,384
//   tokens, 16 heads: 937 us against 978; 4,096 tokens, 32 heads: 128, 139);
// - 128 queries else (12 packed sequences of 200 to 4,096 tokens, 16 heads: 88 us, with 256
//   queries 90, with two groups 99).
template <int D>
hipError_t launch_attn_d(const AttnParams &p, hipStream_t st) {
  const long long seqs = p.cu_q ? p.N : 1, heads = (long long)p.B * p.Hq;
  const long long wgs = heads * (p.cu_q ? p.Tq / 128 + p.N : (p.Tq + 127) / 128);
  if (wgs <= 64) return launch_attn_t<D, 4, 4, 32>(p, st);
  if (wgs <= 128 || (!p.cu_q && wgs <= 256 && p.Tk < 2 * p.Tq)) return launch_attn_t<D, 4, 2, 4096 / D>(p, st);
  if (!p.cu_q && wgs <= 512) return launch_attn_t<D, 8, 2, 64>(p, st);
  if (heads * p.Tq >= 512 * 256 && p.Tq >= 2048 * seqs) return launch_attn_t<D, 8, 1, 64>(p, st);
  return launch_attn_t<D, 4, 1, 64>(p, st);
}

}  // namespace

bool attn_supported(int dtype, int D) { return (dtype == 0 || dtype == 1) && (D == 64 || D == 128); }

// Tiles of 128 queries, 256 threads each; finer ones are for few of them, tiles of 256 are as
// many threads.
bool attn_grid_fits(const AttnArgs &a) {
  const double slots = (a.cu_q ? a.num_seqs : 1) + a.Tq / 128;
  return launch_fits(slots * a.B * a.Hq, 512);
}

hipError_t launch_attn(const AttnArgs &a, hipStream_t st) {
  AttnParams p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.o = a.o;
  p.lse = a.lse;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.c = (a.scale == 0.f ? 1.f : std::fabs(a.scale)) * 1.44269504f;
  p.flip = a.scale > 0.f ? 0 : (a.scale < 0.f ? 1 : 2);
  p.N = a.num_seqs;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.Tq = a.Tq;
  p.Tk = a.Tk;
  if (a.dtype == 1) return a.D == 128 ? launch_attn_f32<128>(p, st) : launch_attn_f32<64>(p, st);
  return a.D == 128 ? launch_attn_d<128>(p, st) : launch_attn_d<64>(p, st);
}

}  // namespace kla
