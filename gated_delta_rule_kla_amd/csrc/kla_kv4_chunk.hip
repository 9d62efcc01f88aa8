// kla_kv4_chunk.hip -- attention of each sequence's newest tokens over the 4-bit cache, and the
// weight that they give to every cached token (gfx950).
//
// kla_attn_kv4_chunk_fwd: o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = exp(scale q_i . k_j) over the
// cached tokens j <= i + len - new, the new tokens' own among them (include/kla.h).
//
// The queries that share a key head are rows of one product: row G i + g is query head g of the
// group's G, token i.  A workgroup takes a tile of a sequence's rows and a run of its keys; its
// waves hold 32 rows each and share tiles of keys and values in LDS, converted to bf16 on the
// way (exact: four significand bits and a power of two), 32 channels and their scale to a
// thread.  The products, the running maximum and sum, and the layouts are kla_attn.hip's.  Keys are split
// over workgroups where the rows alone leave CUs idle: each run then leaves its maximum, sum and
// unnormalised output, which a second kernel joins.
#include <algorithm>
#include <cmath>

#include "kla_attn_tile.h"
#include "kla_common.h"
#include "kla_internal.h"
#include "kla_kv4.h"
#include "kla_ops.h"

namespace kla {

namespace {

struct KvChunkParams {
  KvParams kv;
  const void *q;
  void *o;
  float *lse;
  const int32_t *lens, *cu;  // device; cu: or nullptr (dense)
  float c;                   // |scale| log2(e)
  float sign;                // of the scale; 0 for 0
  int N, B, Hq, G, T;
  int max_len, splits, per;  // runs of `per` keys
  int slots;                 // row tiles of a key head, at most
  float *part_o, *part_ml;   // [B Hq T, splits, D], [B Hq T, splits, 2] where splits > 1
};

// A row tile: its sequence, the sequence's rows, first query row of the batch and batch row, and
// the tile's first row.
struct RowTile {
  int n, b, t0, first;
  long long rows;
};
template <int BM>
__device__ __forceinline__ bool row_tile(const int32_t *cu, int N, int T, int G, int slot, RowTile *r) {
  if (!cu) {
    const int per = (int)(((long long)T * G + BM - 1) / BM);
    *r = RowTile{slot / per, slot / per, 0, slot % per * BM, (long long)T * G};
    return true;
  }
  // sequence n has the slots cu[n] G / BM + n and up: never another's
  auto base = [&](int n) { return (long long)min(max(cu[n], 0), T) * G / BM + n; };
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (base(mid) <= slot) lo = mid; else hi = mid;
  }
  const int a = min(max(cu[lo], 0), T), z = min(max(cu[lo + 1], a), T);
  const long long first = (slot - base(lo)) * BM;
  *r = RowTile{lo, 0, a, (int)first, (long long)(z - a) * G};
  return first >= 0 && first < r->rows;
}

// Cached tokens of sequence n that the call may read, and how many there are in all.
__device__ __forceinline__ int readable(const KvParams &kv, int len, int max_len) {
  const long long room = (long long)kv.max_pages * kv.page;
  return (int)min((long long)min(len, max_len), room);
}

// The 16-byte operand of eight channels of a query in NT bf16 terms, its sign that of the scale.
template <typename E, int NT>
__device__ __forceinline__ void q_terms(const E *p, float sign, bf16x8 *q) {
  float f[8];
  ld8(p, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x = f[i] * sign;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      q[u][i] = (bf16)x;
      x -= (float)q[u][i];
    }
  }
}

// One row against keys lo .. hi-1 by one wave, key by key: maximum (base two), sum, and the
// wave's channels of the unnormalised output.
template <typename E, int D>
__device__ void attend_row(const KvChunkParams &p, const E *q, int n, int head, int lo, int hi, float *m_, float *l_,
                           float *acc) {
  constexpr int CPL = D / 64;
  const int lane = threadIdx.x & 63;
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < CPL; ++i) acc[i] = 0.f;
  for (int j0 = lo; j0 < hi; j0 += 64) {
    const int pos = j0 + lane;
    const long long row = pos < hi ? kv_row(p.kv, n, pos, 0, head) : -1;
    float x = -INFINITY;
    if (row >= 0) {
      x = 0.f;
      for (int d = 0; d < D; d += 8) {
        const float s = __builtin_bit_cast(float, (unsigned)p.kv.scales[row * (D / 32) + d / 32] << 23);
        unsigned w[4];
        cvt8(*reinterpret_cast<const unsigned *>(p.kv.codes + row * (D / 2) + d / 2), s, w);
        float f[8];
        ld8(q + d, f);
        bf16x8 k;
        __builtin_memcpy(&k, w, 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) x = fmaf(f[i] * p.sign, (float)k[i], x);
      }
      x *= p.c;
    }
    float top = x;
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) top = fmaxf(top, __shfl_xor(top, w));
    const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
    const float al = __builtin_amdgcn_exp2f(m - base), e = row < 0 ? 0.f : __builtin_amdgcn_exp2f(x - base);
    m = mn;
    l = l * al + e;
#pragma unroll
    for (int i = 0; i < CPL; ++i) acc[i] *= al;
    for (int j = 0; j < min(64, hi - j0); ++j) {
      const float w = __shfl(e, j);
      const long long vr = kv_row(p.kv, n, j0 + j, 1, head);
      if (vr < 0) continue;
      const int at = CPL * lane;  // a byte holds two channels
      const float s = __builtin_bit_cast(float, (unsigned)p.kv.scales[vr * (D / 32) + at / 32] << 23);
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p.kv.codes[vr * (D / 2) + at / 2], s, 0);
      if constexpr (CPL == 2) {
        acc[0] = fmaf(w, v[0], acc[0]);
        acc[1] = fmaf(w, v[1], acc[1]);
      } else {
        acc[0] = fmaf(w, lane & 1 ? v[1] : v[0], acc[0]);
      }
    }
  }
#pragma unroll
  for (int w = 32; w >= 1; w >>= 1) l += __shfl_xor(l, w);
  *m_ = m;
  *l_ = l;
}

// KS groups of NW / KS waves share the rows and take every KS-th part of BN keys of a tile.
template <typename E, int D, int NW, int KS, int BN>
__global__ __launch_bounds__(64 * NW, 1) void kla_kv4_chunk_kernel(KvChunkParams p) {
  constexpr int NT = sizeof(E) == 2 ? 1 : 3;           // bf16 terms of q and of the weights
  constexpr int BM = 32 * NW / KS, KT = KS * BN, KB = BN / 32;
  constexpr int KJ = D / 16, DB = D / 32, PPR = D / 8, PPK = D / 32;  // PPK: blocks of 32 channels
  constexpr int NP = 2 * KT * PPK / (64 * NW);         // blocks of a thread, keys before values
  constexpr int NBUF = KT * D * 8 <= 65536 ? 2 : 1;
  static_assert(NP * 64 * NW == 2 * KT * PPK, "blocks");
  __shared__ __attribute__((aligned(1024))) bf16 s_kv[2][NBUF][KT * D];
  __shared__ int s_none[NBUF][KT / 16];                // 16 keys of a missing page

  unsigned id = blockIdx.x;
  const int head = id % p.kv.Hkv;
  id /= p.kv.Hkv;
  const int slot = id % p.slots, split = id / p.slots;
  RowTile rt;
  if (!row_tile<BM>(p.cu, p.N, p.T, p.G, slot, &rt)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5, group = KS == 1 ? 0 : wave / (NW / KS);
  const int n = rt.n, lq = (int)(rt.rows / p.G);
  const int len = max(p.lens[n], 0), off = len - lq;
  const int lo = split * p.per, hi = (int)min((long long)readable(p.kv, len, p.max_len), (long long)lo + p.per);
  // the row of this lane (past the end: the last one) and the last key that it sees
  const int w0 = rt.first + 32 * (wave % (NW / KS));
  auto last_seen = [&](long long row) { return min((int)(min(row, rt.rows - 1) / p.G) + off, hi - 1); };
  const long long mine = w0 + r;
  const int row = (int)min(mine, rt.rows - 1), ti = row / p.G;
  const size_t qrow = ((size_t)rt.b * p.Hq + head * p.G + row % p.G) * p.T + rt.t0 + ti;
  const int lim = last_seen(row), wfirst = last_seen(w0), wlast = last_seen(w0 + 31);
  const int end = last_seen(rt.first + BM - 1) + 1;    // keys of the workgroup

  f32x16 acc[DB];
#pragma unroll
  for (int j = 0; j < DB; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  const int steps = end > lo ? (end - lo + KT - 1) / KT : 0;
  // codes and scales of a tile as they are loaded; pages a tile ahead of them
  u32x4 code[NP];
  unsigned scale[NP];
  int page[NP];
  auto find = [&](int t) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pos = lo + t * KT + (tid + 64 * NW * i) % (KT * PPK) / PPK;
      page[i] = pos < end ? p.kv.table[(size_t)n * p.kv.max_pages + pos / p.kv.page] : -1;
    }
  };
  auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pc = tid + 64 * NW * i, j = pc / (KT * PPK), b = pc % PPK, pos = lo + t * KT + pc % (KT * PPK) / PPK;
      const bool there = page[i] >= 0 && page[i] < p.kv.num_pages;
      code[i] = u32x4{0, 0, 0, 0};
      scale[i] = 127;
      if (there) {
        const size_t at = (((size_t)page[i] * 2 + j) * p.kv.Hkv + head) * p.kv.page + pos % p.kv.page;
        code[i] = *reinterpret_cast<const u32x4 *>(p.kv.codes + at * (D / 2) + 16 * b);
        scale[i] = p.kv.scales[at * (D / 32) + b];
      } else if (pos < end) {
        scale[i] = 0x100 | 127;  // missing
      }
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pc = tid + 64 * NW * i, j = pc / (KT * PPK), key = pc % (KT * PPK) / PPK, b = pc % PPK;
      const int swz = j ? (key & 3) << 2 & (PPR - 1) : key & (PPR - 1);
      const float s = __builtin_bit_cast(float, (scale[i] & 255) << 23);
      bf16 *const to = s_kv[j][buf] + key * D;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        unsigned w[4];
        cvt8(code[i][k], s, w);
        *reinterpret_cast<u32x4 *>(to + 8 * ((4 * b + k) ^ swz)) = u32x4{w[0], w[1], w[2], w[3]};
      }
      if (j == 0 && b == 0 && key % 16 == 0) s_none[buf][key / 16] = scale[i] >> 8;
    }
  };

  if (steps > 0) {
    find(0);
    load(0);
    if (steps > 1) find(1);
  }
  bf16x8 q[KJ][NT];
#pragma unroll
  for (int j = 0; j < KJ; ++j) q_terms<E, NT>((const E *)p.q + qrow * D + 16 * j + 8 * h, p.sign, q[j]);
  if (NBUF == 2 && steps > 0) {
    put(0);
    if (steps > 1) load(1);
    if (steps > 2) find(2);
  }
  for (int t = 0; t < steps; ++t) {
    const int buf = NBUF == 2 ? t & 1 : 0;
    lds_barrier();
    if constexpr (NBUF == 2) {
      if (t + 1 < steps) put(buf ^ 1);
      if (t + 2 < steps) load(t + 2);
      if (t + 3 < steps) find(t + 3);
    } else {
      put(0);
      if (t + 1 < steps) load(t + 1);
      if (t + 2 < steps) find(t + 2);
      lds_barrier();
    }
    const int key0 = lo + t * KT + group * BN;
    if (key0 > wlast || w0 >= rt.rows) continue;
    const bf16 *const kt = s_kv[0][buf] + group * BN * D, *const vt = s_kv[1][buf] + group * BN * D;
    f32x16 x[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[kb][i] = 0.f;
#pragma unroll
    for (int j = 0; j < KJ; ++j)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const bf16x8 a = k_operand<D>(kt, kb, j, lane);
#pragma unroll
        for (int u = NT - 1; u >= 0; --u) x[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[j][u], x[kb], 0, 0, 0);
      }
    int none = 0;  // bit i: keys 16 i .. 16 i + 15 of the part are missing
#pragma unroll
    for (int i = 0; i < 2 * KB; ++i) none |= s_none[buf][group * 2 * KB + i] << i;
    if (key0 + BN - 1 > wfirst || none) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (key0 + 32 * kb + 8 * (i / 4) + 4 * h + i % 4 > lim || (none >> (2 * kb + i / 8) & 1)) x[kb][i] = -INFINITY;
    }
    if constexpr (NT == 1) {
      bf16x8 pt[2 * KB];
      softmax_tile<DB, KB>(x, p.c, m, l, acc, pt);
#pragma unroll
      for (int kk = 0; kk < 2 * KB; ++kk)
#pragma unroll
        for (int j = 0; j < DB; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v_operand<D>(vt, kk, j, lane), pt[kk], acc[j], 0, 0, 0);
    } else {
      float top = -INFINITY;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, x[kb][i]);
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
#pragma unroll
      for (int kk = 0; kk < 2 * KB; ++kk) {
        bf16x8 pt[NT];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float e = __builtin_amdgcn_exp2f(fmaf(x[kk / 2][8 * (kk & 1) + i], p.c, -base));
          l += e;
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            pt[u][i] = (bf16)e;
            e -= (float)pt[u][i];
          }
        }
#pragma unroll
        for (int j = 0; j < DB; ++j) {
          const bf16x8 v = v_operand<D>(vt, kk, j, lane);
#pragma unroll
          for (int u = NT - 1; u >= 0; --u) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, pt[u], acc[j], 0, 0, 0);
        }
      }
    }
  }
  l += __shfl_xor(l, 32);
  if constexpr (KS > 1) {
    // the other groups' results through LDS, lane to lane: the layouts are the same
    constexpr int WG = NW / KS, SIZE = (4 * DB + 1) * 64;  // waves of a group, f32x4 of a wave
    static_assert((KS - 1) * WG * SIZE * 16 <= 4 * NBUF * KT * D, "exchange");
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

  // Results: lane (r, h) holds row w0 + r, channels 32 j + 8 (i / 4) + 4 h + i % 4.  A value that
  // is not finite, times the zero weight of a row that does not see it, is NaN in the matrix
  // product: rows whose results are not finite are computed again from the keys they see, one by one.
  const bool valid = mine < rt.rows;
  float worst = l;
#pragma unroll
  for (int j = 0; j < DB; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) worst = fmaf(acc[j][i], 0.f, worst);
  const unsigned long long odd = __ballot(valid && !(fabsf(worst) < INFINITY));
  const unsigned again = (unsigned)odd | (unsigned)(odd >> 32);
  const size_t part = qrow * p.splits + split;
  if (valid && !(again >> r & 1)) {
    const float inv = p.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
    const bool some = p.splits == 1 || l != 0.f;
#pragma unroll
    for (int j = 0; j < DB; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const f32x4 v = {acc[j][i] * inv, acc[j][i + 1] * inv, acc[j][i + 2] * inv, acc[j][i + 3] * inv};
        const int ch = 32 * j + 2 * i + 4 * h;
        if (p.splits > 1) {
          if (some) *reinterpret_cast<f32x4 *>(p.part_o + part * D + ch) = v;
        } else if constexpr (sizeof(E) == 2) {
          *reinterpret_cast<bf16x4 *>((bf16 *)p.o + qrow * D + ch) = bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
        } else {
          *reinterpret_cast<f32x4 *>((float *)p.o + qrow * D + ch) = v;
        }
      }
    if (h == 0) {
      if (p.splits > 1) {
        p.part_ml[part * 2] = m;
        p.part_ml[part * 2 + 1] = l;
      } else if (p.lse) {
        p.lse[qrow] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.693147181f;
      }
    }
  }
  for (unsigned left = again; left; left &= left - 1) {
    const int i = __builtin_ctz(left);
    const size_t qr = ((size_t)__builtin_amdgcn_readlane((int)(qrow >> 32), i) << 32) | (unsigned)__builtin_amdgcn_readlane((int)qrow, i);
    constexpr int CPL = D / 64;
    float rm, rl, a[CPL];
    attend_row<E, D>(p, (const E *)p.q + qr * D, n, head, lo, __builtin_amdgcn_readlane(lim, i) + 1, &rm, &rl, a);
    const float inv = rl == 0.f ? 0.f : 1.f / rl;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
      if (p.splits > 1) p.part_o[(qr * p.splits + split) * D + CPL * lane + k] = a[k];
      else ((E *)p.o)[qr * D + CPL * lane + k] = Elem<E>::from_f32(rl == 0.f ? 0.f : a[k] * inv);
    }
    if (lane == 0) {
      if (p.splits > 1) {
        p.part_ml[(qr * p.splits + split) * 2] = rm;
        p.part_ml[(qr * p.splits + split) * 2 + 1] = rl;
      } else if (p.lse) {
        p.lse[qr] = rl == 0.f ? -INFINITY : (rm + __builtin_amdgcn_logf(rl)) * 0.693147181f;
      }
    }
  }
}

// The runs of one query: D / 4 lanes to a row.
template <typename E, int D>
__global__ __launch_bounds__(256) void kla_kv4_chunk_join_kernel(KvChunkParams p) {
  constexpr int LPR = D / 4;
  const size_t row = (size_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (row >= (size_t)p.B * p.Hq * p.T) return;
  const int t = row % p.T, ch = threadIdx.x % LPR * 4;
  if (p.cu && (t < p.cu[0] || t >= p.cu[p.N])) return;  // a row of no sequence
  const float *const ml = p.part_ml + row * p.splits * 2, *const po = p.part_o + row * p.splits * D + ch;
  float m = -INFINITY;
  for (int s = 0; s < p.splits; ++s)
    if (ml[2 * s + 1] != 0.f) m = fmaxf(m, ml[2 * s]);
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.splits; ++s) {
    const float ls = ml[2 * s + 1];
    if (ls == 0.f) continue;  // a run of which the query sees nothing: its output is not there
    const float f = __builtin_amdgcn_exp2f(ml[2 * s] - base);
    const f32x4 v = *reinterpret_cast<const f32x4 *>(po + (size_t)s * D);
    l = fmaf(ls, f, l);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(v[i], f, o[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) ((E *)p.o)[row * D + ch + i] = Elem<E>::from_f32(l == 0.f ? 0.f : o[i] / l);
  if (ch == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.693147181f;
}

// ---- the weight that queries give to cached tokens -------------------------------------------------
//
// w_j += sum over the rows that see key j of exp(scale q . k_j - lse).  Each wave owns KPW keys, their
// channels as left operands in registers (lane (r, h): channels h D/2 and up of key r, eight to a
// product, q's taken in the same order), and goes over the rows 32 at a time: one product, one
// exponential and an addition a score, the sums in registers with rows along the lanes until the
// end.  A key's sum is made by one wave in one order.
struct KvWeighParams {
  KvParams kv;
  const void *q;
  const float *lse;
  const int32_t *lens, *cu;
  float c, sign;
  float *w;
  int N, B, Hq, G, T, W;
  int max_len, blocks;  // key blocks of a sequence
};

template <typename E, int D>
__global__ __launch_bounds__(256) void kla_kv4_weigh_kernel(KvWeighParams p) {
  constexpr int NT = sizeof(E) == 2 ? 1 : 3, KJ = D / 16, KB = 2, KPW = 32 * KB;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  unsigned id = blockIdx.x;
  const int head = id % p.kv.Hkv;
  id /= p.kv.Hkv;
  const int n = id % p.N, block = id / p.N;
  const int t0 = p.cu ? min(max(p.cu[n], 0), p.T) : 0;
  const int lq = p.cu ? min(max(p.cu[n + 1], t0), p.T) - t0 : p.T;
  const int len = max(p.lens[n], 0), off = len - lq, end = readable(p.kv, len, p.max_len);
  const int key0 = (block * 4 + wave) * KPW;
  if (key0 >= end || lq == 0) return;

  // the wave's keys: 32 kb + r
  bf16x8 k[KB][KJ];
  bool there[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int pos = key0 + 32 * kb + r;
    const long long row = pos < end ? kv_row(p.kv, n, pos, 0, head) : -1;
    there[kb] = row >= 0;
    unsigned code[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; i += 4) {
      u32x4 u = {0, 0, 0, 0};
      if (row >= 0) u = ld16<false>(p.kv.codes + row * (D / 2) + h * (D / 4) + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) code[i + e] = u[e];
    }
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      const unsigned s = row >= 0 ? p.kv.scales[row * (D / 32) + (h * (D / 2) + 8 * j) / 32] : 127u;
      unsigned w[4];
      cvt8(code[j], __builtin_bit_cast(float, s << 23), w);
      __builtin_memcpy(&k[kb][j], w, 16);
    }
  }
  float sum[KB][16];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[kb][i] = 0.f;

  // from the first token that sees the wave's first key
  const long long rows = (long long)lq * p.G;
  const int first = max(key0 - off, 0);
  for (long long r0 = (long long)first * p.G; r0 < rows; r0 += 32) {
    const long long row = min(r0 + r, rows - 1);
    const int ti = (int)(row / p.G);
    const size_t qrow = ((size_t)p.B == 1 && p.cu ? 0 : (size_t)n) * p.Hq * p.T + (size_t)(head * p.G + (int)(row % p.G)) * p.T + t0 + ti;
    float lse = p.lse[qrow];
    // a query that sees nothing gives nothing, nor does a row past the end
    lse = lse == -INFINITY || r0 + r >= rows ? INFINITY : lse;
    const float base = lse * 1.44269504f;
    f32x16 x[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[kb][i] = 0.f;
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      bf16x8 q[NT];
      q_terms<E, NT>((const E *)p.q + qrow * D + h * (D / 2) + 8 * j, p.sign, q);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int u = NT - 1; u >= 0; --u) x[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[kb][j], q[u], x[kb], 0, 0, 0);
    }
    const int lim = ti + off;  // the last key that the row sees
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e = __builtin_amdgcn_exp2f(fmaf(x[kb][i], p.c, -base));
        const int key = key0 + 32 * kb + 8 * (i / 4) + 4 * h + i % 4;
        sum[kb][i] += key <= lim && base < INFINITY ? e : 0.f;
      }
  }
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) sum[kb][i] += __shfl_xor(sum[kb][i], w);
    }
  // lane (r, h) writes key 8 (r / 4 % 4) + 4 h + r % 4 of part r / 16: register r % 16 of either half
  const unsigned long long ok[KB] = {__ballot(there[0]), __ballot(there[1])};
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int at = 8 * (i / 4) + 4 * h + i % 4, key = key0 + 32 * kb + at;
      if (r == i && key < end && (ok[kb] >> at & 1)) {
        float *const to = p.w + ((size_t)n * p.kv.Hkv + head) * p.W + key;
        *to += sum[kb][i];
      }
    }
}

// How a chunk call runs: tiles of 32, 128 or 256 rows by the rows of a sequence (the host's mean),
// and runs of keys as many as make about 512 workgroups, of 512 keys at least.
struct ChunkPlan {
  int BM, slots, splits, per;
};
ChunkPlan chunk_plan(const Kv4ChunkArgs &a) {
  const long long G = a.Hq / a.c.Hkv, seqs = std::max(a.N, 1);
  const long long rows = (long long)a.B * a.T * G, mean = (rows + seqs - 1) / seqs;
  ChunkPlan p;
  p.BM = mean <= 64 ? 32 : mean <= 512 || a.dtype != 0 ? 128 : 256;
  const long long tiles = a.cu ? (long long)a.T * G / p.BM + a.N : seqs * (((long long)a.T * G + p.BM - 1) / p.BM);
  p.slots = (int)std::min<long long>(tiles, 0x7fffffff);
  const long long busy = seqs * ((mean + p.BM - 1) / p.BM) * a.c.Hkv;
  long long want = std::max<long long>(1, 512 / std::max<long long>(1, busy));
  want = std::min(want, std::max<long long>(1, a.max_len / 512));
  const long long len = (a.max_len + want - 1) / want;
  p.per = (int)std::max<long long>(128, (len + 127) / 128 * 128);
  p.splits = (int)std::max<long long>(1, ((long long)a.max_len + p.per - 1) / p.per);
  return p;
}

template <typename E, int D, int NW, int KS, int BN>
hipError_t launch_chunk_t(const KvChunkParams &p, hipStream_t st) {
  const long long grid = (long long)p.slots * p.kv.Hkv * p.splits;
  hipLaunchKernelGGL((kla_kv4_chunk_kernel<E, D, NW, KS, BN>), dim3((unsigned)grid), dim3(64 * NW), 0, st, p);
  if (p.splits > 1) {
    const size_t rows = (size_t)p.B * p.Hq * p.T, per = 256 / (D / 4);
    hipLaunchKernelGGL((kla_kv4_chunk_join_kernel<E, D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, st, p);
  }
  return hipGetLastError();
}
template <typename E, int D>
hipError_t launch_chunk(const KvChunkParams &p, int BM, hipStream_t st) {
  if (BM == 32) return launch_chunk_t<E, D, 4, 4, 32>(p, st);
  if constexpr (sizeof(E) == 2) {
    if (BM == 256) return launch_chunk_t<E, D, 8, 1, 8192 / D>(p, st);
    return launch_chunk_t<E, D, 4, 1, 64>(p, st);
  } else {
    return launch_chunk_t<E, D, 4, 1, 4096 / D>(p, st);
  }
}

int weigh_blocks(const Kv4ChunkArgs &a) { return (a.max_len + 255) / 256; }

}  // namespace

size_t kv4_chunk_workspace_bytes(const Kv4ChunkArgs &a) {
  const ChunkPlan p = chunk_plan(a);
  return p.splits == 1 ? 0 : (size_t)a.B * a.Hq * a.T * p.splits * (a.D + 2) * sizeof(float);
}

bool kv4_chunk_grid_fits(const Kv4ChunkArgs &a) {
  const ChunkPlan p = chunk_plan(a);
  const double rows = (double)a.T * (a.Hq / a.c.Hkv);
  const double tiles = a.cu ? rows / p.BM + a.N : (double)a.N * (rows / p.BM + 1);
  return rows <= 2147418112.0 && launch_fits(tiles * a.c.Hkv * p.splits, p.BM == 256 ? 512 : 256) &&
         launch_fits((double)a.B * a.Hq * a.T / 8 + 1, 256);
}

bool kv4_weigh_grid_fits(const Kv4ChunkArgs &a) {
  return (double)a.T * (a.Hq / a.c.Hkv) <= 2147418112.0 && launch_fits((double)weigh_blocks(a) * a.N * a.c.Hkv, 256);
}

hipError_t launch_attn_kv4_chunk(const Kv4ChunkArgs &a, void *workspace, hipStream_t st) {
  const ChunkPlan plan = chunk_plan(a);
  KvChunkParams p{};
  p.kv = kv_params(a.c);
  p.q = a.q;
  p.o = a.o;
  p.lse = a.lse;
  p.lens = a.lens;
  p.cu = a.cu;
  p.c = (a.scale == 0.f ? 1.f : std::fabs(a.scale)) * 1.44269504f;
  p.sign = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
  p.N = a.N;
  p.B = a.B;
  p.Hq = a.Hq;
  p.G = a.Hq / a.c.Hkv;
  p.T = a.T;
  p.max_len = a.max_len;
  p.splits = plan.splits;
  p.per = plan.per;
  p.slots = plan.slots;
  p.part_o = (float *)workspace;
  p.part_ml = p.part_o + (size_t)a.B * a.Hq * a.T * p.splits * a.D;
  if (a.dtype == 0) return a.D == 128 ? launch_chunk<bf16, 128>(p, plan.BM, st) : launch_chunk<bf16, 64>(p, plan.BM, st);
  return a.D == 128 ? launch_chunk<float, 128>(p, plan.BM, st) : launch_chunk<float, 64>(p, plan.BM, st);
}

hipError_t launch_attn_kv4_weigh(const Kv4ChunkArgs &a, float *weights, int W, hipStream_t st) {
  KvWeighParams p{};
  p.kv = kv_params(a.c);
  p.q = a.q;
  p.lse = a.lse;
  p.lens = a.lens;
  p.cu = a.cu;
  p.c = (a.scale == 0.f ? 1.f : std::fabs(a.scale)) * 1.44269504f;
  p.sign = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
  p.w = weights;
  p.N = a.N;
  p.B = a.B;
  p.Hq = a.Hq;
  p.G = a.Hq / a.c.Hkv;
  p.T = a.T;
  p.W = W;
  p.max_len = a.max_len;
  p.blocks = weigh_blocks(a);
  const dim3 grid((unsigned)((long long)p.blocks * p.N * a.c.Hkv));
  if (a.max_len == 0) return hipSuccess;
  if (a.dtype == 0) {
    if (a.D == 128) hipLaunchKernelGGL((kla_kv4_weigh_kernel<bf16, 128>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((kla_kv4_weigh_kernel<bf16, 64>), grid, dim3(256), 0, st, p);
  } else {
    if (a.D == 128) hipLaunchKernelGGL((kla_kv4_weigh_kernel<float, 128>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((kla_kv4_weigh_kernel<float, 64>), grid, dim3(256), 0, st, p);
  }
  return hipGetLastError();
}

}  // namespace kla
