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
// thread.  The products, the running maximum and sum, and the layouts are kla_attn.hip's.  Keys are
// split over workgroups where the rows alone leave CUs idle: each run then leaves its maximum, sum
// and unnormalised output, which a second kernel joins.
#include <algorithm>
#include <cmath>

#include "kla_attn_tile.h"
#include "kla_common.h"
#include "kla_index.h"
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
  int n, b, t0, first, rows;
};
template <int BM>
__device__ __forceinline__ bool row_tile(const int32_t *cu, int N, int T, int G, int slot, RowTile *r) {
  if (!cu) {
    const int per = (int)(((long long)T * G + BM - 1) / BM);
    *r = RowTile{slot / per, slot / per, 0, slot % per * BM, T * G};
    return true;
  }
  // sequence n has the slots cu[n] G / BM + n and up: never another's
  auto base = [&](int n) { return (long long)min(max(cu[n], 0), T) * G / BM + n; };
  const int lo = wave_last_where(N, [&](int n) { return base(n) <= slot; });
  const int a = min(max(cu[lo], 0), T), z = min(max(cu[lo + 1], a), T);
  const long long first = (slot - base(lo)) * BM;
  *r = RowTile{lo, 0, a, (int)first, (z - a) * G};
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

// Tiles of BN keys, 32 rows to a wave.  2,048 new tokens behind 60,000, 16 heads over 2: 971 to
// 1,004 us, 1.02 to 1.06 PFLOP/s.  Bound: the vector ALU (softmax, conversions and addresses, about
// as many issue cycles as the matrix products take) beside a clock that falls with the matrix
// cores' use.
template <typename E, int D, int NW, int BN>
__global__ __launch_bounds__(64 * NW, 1) void kla_kv4_chunk_kernel(KvChunkParams p) {
  constexpr int NT = sizeof(E) == 2 ? 1 : 3;           // bf16 terms of q and of the weights
  constexpr int BM = 32 * NW, KB = BN / 32;
  constexpr int KJ = D / 16, DB = D / 32, PPR = D / 8, PPK = D / 32;  // PPK: blocks of 32 channels
  constexpr int NP = 2 * BN * PPK / (64 * NW);         // blocks of a thread, keys before values
  static_assert(NP * 64 * NW == 2 * BN * PPK, "blocks");
  __shared__ __attribute__((aligned(1024))) bf16 s_kv[2][2][BN * D];
  __shared__ int s_none[2][BN / 16];                // 16 keys of a missing page

  unsigned id = blockIdx.x;
  const int head = id % p.kv.Hkv;
  id /= p.kv.Hkv;
  const int slot = id % p.slots, split = id / p.slots;
  RowTile rt;
  if (!row_tile<BM>(p.cu, p.N, p.T, p.G, slot, &rt)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int n = rt.n, lq = rt.rows / p.G;
  const int len = max(p.lens[n], 0), off = len - lq;
  const int lo = split * p.per, hi = (int)min((long long)readable(p.kv, len, p.max_len), (long long)lo + p.per);
  // the row of this lane (past the end: the last one) and the last key that it sees
  const int w0 = rt.first + 32 * wave;
  auto last_seen = [&](int row) { return min((int)((unsigned)min(row, rt.rows - 1) / (unsigned)p.G) + off, hi - 1); };
  const int mine = w0 + r, row = min(mine, rt.rows - 1);
  const unsigned ti = (unsigned)row / (unsigned)p.G;
  const size_t qrow = ((size_t)rt.b * p.Hq + head * p.G + (row - ti * p.G)) * p.T + rt.t0 + ti;
  const int lim = last_seen(row), wfirst = last_seen(w0), wlast = last_seen(w0 + 31);
  const int end = last_seen(rt.first + BM - 1) + 1;    // keys of the workgroup

  f32x16 acc[DB];
#pragma unroll
  for (int j = 0; j < DB; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  const int steps = end > lo ? (end - lo + BN - 1) / BN : 0;
  // Codes and scales of a tile as they are loaded; pages a tile ahead of them.  Every load is made,
  // from the first page where there is none: behind a branch the compiler waits for it there.
  u32x4 code[NP];
  unsigned scale[NP];
  int page[NP];
  int state[NP];  // of a block: 0 cached, 1 past the end, 2 missing
  // a block's place in the table and in its page move on by a tile each time (one box: 971 us; with
  // two divisions and three products of 64 bits a tile instead 1,005)
  int at_page[NP], at_row[NP], row_[NP];
  size_t first[NP];  // of page 0
  const size_t stride = (size_t)2 * p.kv.Hkv * p.kv.page;
  const int by_page = BN / p.kv.page, by_row = BN % p.kv.page, last_page = (end - 1) / p.kv.page;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int pos = lo + (tid + 64 * NW * i) % (BN * PPK) / PPK;
    at_page[i] = pos / p.kv.page;
    at_row[i] = pos % p.kv.page;
    first[i] = ((size_t)((tid + 64 * NW * i) / (BN * PPK)) * p.kv.Hkv + head) * p.kv.page;
  }
  auto find = [&] {  // the next tile's
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      page[i] = p.kv.table[(size_t)n * p.kv.max_pages + min(at_page[i], last_page)];
      row_[i] = at_row[i];
      at_page[i] += by_page;
      at_row[i] += by_row;
      if (at_row[i] >= p.kv.page) {
        at_row[i] -= p.kv.page;
        ++at_page[i];
      }
    }
  };
  auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pc = tid + 64 * NW * i, b = pc % PPK;
      const unsigned pos = (unsigned)lo + t * BN + pc % (BN * PPK) / PPK, last = end - 1;
      const bool there = page[i] >= 0 && page[i] < p.kv.num_pages;
      state[i] = pos > last ? 1 : there ? 0 : 2;
      const size_t at = (unsigned)(there ? page[i] : 0) * stride + first[i] + row_[i];
      code[i] = *reinterpret_cast<const u32x4 *>(p.kv.codes + at * (D / 2) + 16 * b);
      scale[i] = p.kv.scales[at * (D / 32) + b];
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pc = tid + 64 * NW * i, j = pc / (BN * PPK), key = pc % (BN * PPK) / PPK, b = pc % PPK;
      const int swz = j ? (key & 3) << 2 & (PPR - 1) : key & (PPR - 1);
      asm volatile("" : "+v"(code[i]));
      const float s = __builtin_bit_cast(float, state[i] ? 0x3f800000u : scale[i] << 23);
      bf16 *const to = s_kv[j][buf] + key * D;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        unsigned w[4];
        cvt8(state[i] ? 0u : code[i][k], s, w);
        *reinterpret_cast<u32x4 *>(to + 8 * ((4 * b + k) ^ swz)) = u32x4{w[0], w[1], w[2], w[3]};
      }
      if (j == 0 && b == 0 && key % 16 == 0) s_none[buf][key / 16] = state[i] >> 1;
    }
  };

  if (steps > 0) {
    find();
    load(0);
    find();
  }
  bf16x8 q[KJ][NT];
#pragma unroll
  for (int j = 0; j < KJ; ++j) q_terms<E, NT>((const E *)p.q + qrow * D + 16 * j + 8 * h, p.sign, q[j]);
  if (steps > 0) {
    put(0);
    load(1);
    find();
  }
  for (int t = 0; t < steps; ++t) {
    const int buf = t & 1;
    lds_barrier();
    put(buf ^ 1);
    load(t + 2);
    find();
    const int key0 = lo + t * BN;
    if (key0 > wlast || w0 >= rt.rows) continue;
    const bf16 *const kt = s_kv[0][buf], *const vt = s_kv[1][buf];
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
    int none = 0;  // bit i: keys 16 i .. 16 i + 15 of the tile are missing
#pragma unroll
    for (int i = 0; i < 2 * KB; ++i) none |= s_none[buf][i] << i;
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

// Few rows (a draft's tokens, single tokens): 16 RB rows of a sequence and key head to a workgroup,
// and a run of keys, of which its four waves take tiles of 32 in turn, each with its own running
// maximum, sum and output; nothing is shared until the end.  Layouts are those of the single-token
// kernel (kla_kv4.hip): K's codes become operands as they arrive, lane (r, c) holding channels c
// D/4 and up of key r; the scores have keys 4 c + i of the two 16-key halves in a lane's registers
// and rows along the lanes, and so are the second product's operand as they stand; V goes through
// the wave's own LDS in 4 bits.  64 sequences of 4,096 to 16,384 cached tokens (326 MB) and five
// new ones, 16 heads over 4: 109 to 117 us, 3.0 TB/s.  Bound: the vector ALU, about 270
// instructions per tile of 32 keys, the conversions 64 of them, which all row blocks share; the
// softmax over tiles that the new tokens fill to five eighths.
template <typename E, int D, int RB, bool ONCE>
__global__ __launch_bounds__(256, 2) void kla_kv4_rows_kernel(KvChunkParams p) {
  constexpr int NT = sizeof(E) == 2 ? 1 : 3;  // bf16 terms of q and of the weights
  constexpr int KJ = D / 32, DW = D / 16, BM = 16 * RB;
  // what the tiles need, and what joining the waves needs behind them
  struct Tiles {
    uint8_t v[4][32 * D / 2];
    unsigned sc[4][64];
    int page[KV_MAX_PER / 16];
  };
  struct Joined {
    float o[4][16][D / 2 + 4], ml[4][16][2], f[4][16], m[16], l[16];
  };
  union Lds {
    Tiles t;
    Joined j;
  };
  __shared__ __attribute__((aligned(16))) Lds lds;
  int *const s_page = lds.t.page;
  __shared__ unsigned s_bad;
  __shared__ size_t s_row[BM];  // places of the tile's rows among the queries

  unsigned id = blockIdx.x;
  const int head = id % p.kv.Hkv;
  id /= p.kv.Hkv;
  const int slot = id % p.slots, split = id / p.slots;
  RowTile rt;
  if (!row_tile<BM>(p.cu, p.N, p.T, p.G, slot, &rt)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, c = lane >> 4, n = rt.n, lq = rt.rows / p.G;
  const int len = max(p.lens[n], 0), off = len - lq;
  const int lo = split * p.per, hi = (int)min((long long)readable(p.kv, len, p.max_len), (long long)lo + p.per);
  auto last_seen = [&](int row) { return min((int)((unsigned)min(row, rt.rows - 1) / (unsigned)p.G) + off, hi - 1); };
  auto q_row = [&](int row) {
    const unsigned ti = (unsigned)row / (unsigned)p.G;
    return ((size_t)rt.b * p.Hq + head * p.G + (row - ti * p.G)) * p.T + rt.t0 + ti;
  };
  const int gn = min(BM, rt.rows - rt.first);  // rows of the tile
  const int end = last_seen(rt.first + BM - 1) + 1, all = last_seen(rt.first);  // keys of the tile, of its first row
  if (tid == 0) s_bad = 0;
  if (tid < gn) s_row[tid] = q_row(rt.first + tid);
  for (int i = tid; i < (max(end - lo, 0) + 31) / 32 * 2; i += 256) {
    const int t = lo + 16 * i;
    int page = -1;
    if (t < end) {
      page = p.kv.table[(size_t)n * p.kv.max_pages + t / p.kv.page];
      if (page >= p.kv.num_pages) page = -1;
    }
    s_page[i] = page;
  }
  bf16x8 q[RB][KJ][NT];
  int lim[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int row = min(rt.first + 16 * b + r, rt.rows - 1);
    lim[b] = last_seen(row);
    const E *const qp = (const E *)p.q + q_row(row) * D;
#pragma unroll
    for (int j = 0; j < KJ; ++j) q_terms<E, NT>(qp + c * (D / 4) + 8 * j, p.sign, q[b][j]);
  }
  __syncthreads();

  f32x4 acc[RB][DW];
  float m[RB], l[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    m[b] = -INFINITY;
    l[b] = 0.f;
#pragma unroll
    for (int j = 0; j < DW; ++j) acc[b][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  constexpr int VP = D / 64, LPR = D / 32;  // pieces of V a lane loads, lanes of a row of V
  struct Tile {
    unsigned k[2][KJ];
    u32x4 v[VP];
    unsigned sc;
    int id0, id1;
  } next;
  auto load = [&](Tile &x, int t) {
    x.id0 = __builtin_amdgcn_readfirstlane(s_page[(t - lo) >> 4]);
    x.id1 = __builtin_amdgcn_readfirstlane(s_page[((t - lo) >> 4) + 1]);
    const size_t pg = (size_t)p.kv.Hkv * p.kv.page;
    // rows of the two 16-token blocks (page 0 where there is none: masked below)
    const size_t r0 = (size_t)max(x.id0, 0) * 2 * pg + (size_t)head * p.kv.page + t % p.kv.page;
    const size_t r1 = (size_t)max(x.id1, 0) * 2 * pg + (size_t)head * p.kv.page + (t + 16) % p.kv.page;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t *a = p.kv.codes + ((h ? r1 : r0) + r) * (D / 2) + c * (D / 8);
      if constexpr (D == 128) {
        const u32x4 u = ld16<ONCE>(a);
        x.k[h][0] = u[0], x.k[h][1] = u[1], x.k[h][2] = u[2], x.k[h][3] = u[3];
      } else {
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 u = *reinterpret_cast<const u32x2 *>(a);
        x.k[h][0] = u[0], x.k[h][1] = u[1];
      }
    }
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int key = lane / LPR + 64 / LPR * i;
      x.v[i] = ld16<ONCE>(p.kv.codes + ((key < 16 ? r0 : r1) + pg + key % 16) * (D / 2) + 16 * (lane % LPR));
    }
    const uint8_t *a = p.kv.scales + ((lane & 16 ? r1 : r0) + (lane & 15) + (lane & 32 ? pg : 0)) * (D / 32);
    if constexpr (D == 128) x.sc = *reinterpret_cast<const unsigned *>(a);
    else x.sc = *reinterpret_cast<const unsigned short *>(a);
  };

  int t = lo + 32 * wave;
  if (t < end) load(next, t);
  for (; t < end; t += 128) {
    const Tile x0 = next;
    if (t + 128 < end) load(next, t + 128);
    // V and the scales through the wave's own LDS; key 16 h + 4 c + e at slot 16 h + 4 e + c
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int key = lane / LPR + 64 / LPR * i, slot_ = (key & 16) + 4 * (key & 3) + ((key >> 2) & 3);
      *reinterpret_cast<u32x4 *>(lds.t.v[wave] + slot_ * (D / 2) + 16 * (lane % LPR)) = x0.v[i];
    }
    lds.t.sc[wave][lane] = x0.sc;
    const uint8_t *sc8 = reinterpret_cast<const uint8_t *>(lds.t.sc[wave]);
    const int id0 = x0.id0, id1 = x0.id1;
    // scores of keys t + 16 h + 4 c + i against rows 16 b + r
    float x[RB][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 s[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b) s[b] = f32x4{0.f, 0.f, 0.f, 0.f};
      const float sc = __builtin_bit_cast(float, (unsigned)sc8[4 * (16 * h + r) + (D == 128 ? c : c / 2)] << 23);
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        unsigned w[4];
        cvt8(x0.k[h][j], sc, w);
        bf16x8 a;
        __builtin_memcpy(&a, w, 16);
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int u = 0; u < NT; ++u) s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q[b][j][u], s[b], 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[b][4 * h + i] = s[b][i];
    }
    unsigned va[8];
    float vf[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t *a = lds.t.v[wave] + ((e & 4) * 4 + 4 * (e & 3) + c) * (D / 2);
      unsigned short half;
      if constexpr (D == 128) __builtin_memcpy(&va[e], __builtin_assume_aligned(a + 4 * r, 4), 4);
      else __builtin_memcpy(&half, __builtin_assume_aligned(a + 2 * r, 2), 2), va[e] = half;
      vf[e] = __builtin_bit_cast(float, (unsigned)sc8[4 * (32 + 16 * (e >> 2) + 4 * c + (e & 3)) + r * DW / 32] << 23);
    }
    if (id0 < 0 || id1 < 0 || t + 31 > all) {
      // keys that a row does not see have no score; those of no row, and of missing pages, a value
      // of zero whatever the memory behind them holds
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int key = t + 16 * (e >> 2) + 4 * c + (e & 3);
        const bool none = (e < 4 ? id0 : id1) < 0 || key >= end;
#pragma unroll
        for (int b = 0; b < RB; ++b) x[b][e] = none || key > lim[b] ? -INFINITY : x[b][e];
        va[e] = none ? 0u : va[e];
        vf[e] = none ? 1.f : vf[e];
      }
    }
    bf16x8 pt[RB][NT];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      float top = x[b][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, x[b][e]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32)) * p.c;
      // the maximum moves by 2^LAG at least, as in kla_attn_tile.h
      if (__any(top > m[b] + LAG)) {
        const float mn = top > m[b] + LAG ? top : m[b];
        const float al = __builtin_amdgcn_exp2f(m[b] - (mn == -INFINITY ? 0.f : mn));
        l[b] *= al;
#pragma unroll
        for (int j = 0; j < DW; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[b][j][i] *= al;
        m[b] = mn;
      }
      const float base = m[b] == -INFINITY ? 0.f : m[b];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = __builtin_amdgcn_exp2f(fmaf(x[b][e], p.c, -base));
        l[b] += v;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          pt[b][u][e] = (bf16)v;
          v -= (float)pt[b][u][e];
        }
      }
    }
    // V: pairs of channels of each key, then pairs of keys of each channel
    unsigned w[8][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) cvt8(va[e], vf[e], w[e]);
#pragma unroll
    for (int j = 0; j < DW; ++j) {
      unsigned a[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        a[e] = __builtin_amdgcn_perm(w[2 * e + 1][j / 2], w[2 * e][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
      bf16x8 av;
      __builtin_memcpy(&av, a, 16);
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int u = 0; u < NT; ++u) acc[b][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, pt[b][u], acc[b][j], 0, 0, 0);
    }
  }

  // join the waves, 16 rows at a time and half of the channels (DW / 2 of each lane's)
  constexpr int DH = DW / 2;
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    l[b] += __shfl_xor(l[b], 16);
    l[b] += __shfl_xor(l[b], 32);
    const int rows = min(gn - 16 * b, 16);
    __syncthreads();
    if (c == 0) {
      lds.j.ml[wave][r][0] = m[b];
      lds.j.ml[wave][r][1] = l[b];
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half) __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < DH; ++j) lds.j.o[wave][r][(4 * c + i) * DH + j] = acc[b][half * DH + j][i];
      __syncthreads();
      if (half == 0) {
        if (tid < 16) {
          float mm = lds.j.ml[0][tid][0], ll = 0.f;
#pragma unroll
          for (int w = 1; w < 4; ++w) mm = fmaxf(mm, lds.j.ml[w][tid][0]);
          const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float f = __builtin_amdgcn_exp2f(lds.j.ml[w][tid][0] - base);
            lds.j.f[w][tid] = f;
            ll = fmaf(lds.j.ml[w][tid][1], f, ll);
          }
          lds.j.m[tid] = mm;
          lds.j.l[tid] = ll;
        }
        __syncthreads();
      }
      for (int i = tid; i < rows * (D / 2); i += 256) {
        const int g = i / (D / 2), e = i % (D / 2), d = e / DH * DW + half * DH + e % DH;
        const float mm = lds.j.m[g], ll = lds.j.l[g];
        float oo = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) oo = fmaf(lds.j.o[w][g][e], lds.j.f[w][g], oo);
        if (!(fabsf(fmaf(oo, 0.f, ll)) < INFINITY)) atomicOr(&s_bad, 1u << (16 * b + g));
        const size_t qr = s_row[16 * b + g], part = qr * p.splits + split;
        if (p.splits == 1) {
          ((E *)p.o)[qr * D + d] = Elem<E>::from_f32(ll == 0.f ? 0.f : oo / ll);
          if (d == 0 && p.lse) p.lse[qr] = ll == 0.f ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * 0.693147181f;
        } else {
          p.part_o[part * D + d] = oo;
          if (d == 0) {
            p.part_ml[part * 2] = mm;
            p.part_ml[part * 2 + 1] = ll;
          }
        }
      }
    }
  }
  // rows whose results are not finite, again from the keys that they see alone, one by one
  __syncthreads();
  int i = 0;
  each_bit((unsigned)__builtin_amdgcn_readfirstlane((int)s_bad), [&](int at) {
    if (i++ % 4 != wave) return;
    const size_t qr = s_row[at], part = qr * p.splits + split;
    constexpr int CPL = D / 64;
    float rm, rl, a[CPL];
    attend_row<E, D>(p, (const E *)p.q + qr * D, n, head, lo, last_seen(rt.first + at) + 1, &rm, &rl, a);
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
      if (p.splits > 1) p.part_o[part * D + CPL * lane + k] = a[k];
      else ((E *)p.o)[qr * D + CPL * lane + k] = Elem<E>::from_f32(rl == 0.f ? 0.f : a[k] / rl);
    }
    if (lane == 0) {
      if (p.splits > 1) {
        p.part_ml[part * 2] = rm;
        p.part_ml[part * 2 + 1] = rl;
      } else if (p.lse) {
        p.lse[qr] = rl == 0.f ? -INFINITY : (rm + __builtin_amdgcn_logf(rl)) * 0.693147181f;
      }
    }
  });
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
// w_j += sum over the rows that see key j of exp(scale q . k_j - lse).  One product, one
// exponential and an addition a score; a key's sum is made by one workgroup in one order.
struct KvWeighParams {
  KvParams kv;
  const void *q;
  const float *lse;
  const int32_t *lens, *cu;
  float c;  // scale log2(e)
  float *w;
  int N, Hq, G, T, W;
  int max_len, per;  // keys of a workgroup
};

// A sequence's queries and keys.
struct WeighSpan {
  int t0, lq, off, end;
  size_t q0;  // row of the batch's first query of query head 0
};
__device__ __forceinline__ WeighSpan weigh_span(const KvWeighParams &p, int n) {
  const int t0 = p.cu ? min(max(p.cu[n], 0), p.T) : 0;
  const int lq = p.cu ? min(max(p.cu[n + 1], t0), p.T) - t0 : p.T;
  const int len = max(p.lens[n], 0);
  return {t0, lq, len - lq, readable(p.kv, len, p.max_len), (p.cu ? 0 : (size_t)n) * p.Hq * p.T + t0};
}
// log2(e) lse of a row, infinite where it gives nothing: past the end, or with a query that sees
// nothing
__device__ __forceinline__ float weigh_base(float lse, bool there) {
  return there && fabsf(lse) < INFINITY ? lse * 1.44269504f : INFINITY;
}

// Many rows: 64 keys to a workgroup, in each of its four waves as left operands in registers
// (lane (r, h): channels h D/2 and up of key r, eight to a product, q's taken in the same
// order).  The waves take the rows in turn, 32 at a time, the next ones' loads ahead, and keep sums
// with rows along the lanes until the end.
// Bound: latency: the keys' operands are made once for all rows, by every wave.
template <typename E, int D>
__global__ __launch_bounds__(256) void kla_kv4_weigh_kernel(KvWeighParams p) {
  constexpr int NT = sizeof(E) == 2 ? 1 : 3, KJ = D / 16, KB = 2;
  constexpr int QP = D / 2 * (int)sizeof(E) / 16;  // 16-byte pieces of half a query
  __shared__ float s_sum[4][32 * KB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  unsigned id = blockIdx.x;
  const int head = id % p.kv.Hkv;
  id /= p.kv.Hkv;
  const int n = id % p.N, key0 = (int)(id / p.N) * 32 * KB;
  const WeighSpan s = weigh_span(p, n);
  if (key0 >= s.end || s.lq == 0) return;

  bf16x8 k[KB][KJ];  // keys 32 kb + r
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int pos = key0 + 32 * kb + r;
    const long long row = pos < s.end ? kv_row(p.kv, n, pos, 0, head) : -1;
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
      const unsigned sc = row >= 0 ? p.kv.scales[row * (D / 32) + (h * (D / 2) + 8 * j) / 32] : 127u;
      unsigned w[4];
      cvt8(code[j], __builtin_bit_cast(float, sc << 23), w);
      __builtin_memcpy(&k[kb][j], w, 16);
    }
  }
  float sum[KB][16];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[kb][i] = 0.f;

  // rows from the first token that sees the first key on
  const long long rows = (long long)s.lq * p.G;
  const size_t h0 = s.q0 + (size_t)head * p.G * p.T;
  struct Query {
    u32x4 q[QP];
    float lse;
    int lim;  // the last key that it sees
    bool there;
  };
  auto load = [&](Query &x, long long r0) {
    const long long row = min(r0 + r, rows - 1);
    const int ti = (int)(row / p.G);
    const size_t at = h0 + (size_t)(row - (long long)ti * p.G) * p.T + ti;
#pragma unroll
    for (int i = 0; i < QP; ++i) x.q[i] = *reinterpret_cast<const u32x4 *>((const E *)p.q + at * D + h * (D / 2) + i * (16 / (int)sizeof(E)));
    x.lse = p.lse[at];
    x.lim = ti + s.off;
    x.there = r0 + r < rows;
  };
  long long r0 = (long long)max(key0 - s.off, 0) * p.G + 32 * wave;
  Query next;
  load(next, r0);
  for (; r0 < rows; r0 += 128) {
    const Query cur = next;
    load(next, r0 + 128);
    const float base = weigh_base(cur.lse, cur.there);
    f32x16 x[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[kb][i] = 0.f;
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      bf16x8 q[NT];
      if constexpr (NT == 1) {
        q[0] = __builtin_bit_cast(bf16x8, cur.q[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const unsigned bits = cur.q[2 * j + i / 4][i % 4];
          float f = __builtin_bit_cast(float, bits);
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            q[u][i] = (bf16)f;
            f -= (float)q[u][i];
          }
        }
      }
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int u = NT - 1; u >= 0; --u) x[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[kb][j], q[u], x[kb], 0, 0, 0);
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e = __builtin_amdgcn_exp2f(fmaf(x[kb][i], p.c, -base));
        const int key = key0 + 32 * kb + 8 * (i / 4) + 4 * h + i % 4;
        sum[kb][i] += key <= cur.lim && base < INFINITY ? e : 0.f;
      }
  }
  // over the rows of a wave; lane (r, h) of the first 16 keeps key 8 (r / 4) + 4 h + r % 4
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = sum[kb][i];
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) v += __shfl_xor(v, w);
      mine = r == i ? v : mine;
    }
    if (r < 16) s_sum[wave][32 * kb + 8 * (r / 4) + 4 * h + r % 4] = mine;
  }
  __syncthreads();
  if (threadIdx.x < 32 * KB) {
    const int key = key0 + threadIdx.x;
    if (key < s.end && kv_row(p.kv, n, key, 0, head) >= 0) {
      float v = s_sum[0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < 4; ++w) v += s_sum[w][threadIdx.x];
      p.w[((size_t)n * p.kv.Hkv + head) * p.W + key] += v;
    }
  }
}

// Few rows: 16 RB of them stay in registers as left operands and the keys stream past, 32 at a
// time to each of four waves (lane (r, c): channels c D/4 and up of keys r and 16 + r).  A score
// tile has a row in each register and keys along the lanes, so a key's sum is additions within
// a lane and two exchanges.  More rows than that: the keys again for the next ones.  64 sequences
// of 4,096 to 16,384 cached tokens, one new one: 50 to 53 us.  Bound: HBM (K's codes and the weights in
// and out, 3.4 TB/s) and the latency of a wave's few tiles.
template <typename E, int D, int RB>
__global__ __launch_bounds__(256) void kla_kv4_weigh_few_kernel(KvWeighParams p) {
  constexpr int NT = sizeof(E) == 2 ? 1 : 3, KJ = D / 32, BM = 16 * RB;
  __shared__ int s_page[KV_MAX_PER / 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  unsigned id = blockIdx.x;
  const int head = id % p.kv.Hkv;
  id /= p.kv.Hkv;
  const int n = id % p.N, lo = (int)(id / p.N) * p.per;
  const WeighSpan s = weigh_span(p, n);
  const int hi = (int)min((long long)s.end, (long long)lo + p.per);
  if (lo >= hi || s.lq == 0) return;
  for (int i = threadIdx.x; i < (hi - lo + 31) / 32 * 2; i += 256) {
    const int t = lo + 16 * i;
    int page = -1;
    if (t < hi) {
      page = p.kv.table[(size_t)n * p.kv.max_pages + t / p.kv.page];
      if (page >= p.kv.num_pages) page = -1;
    }
    s_page[i] = page;
  }
  __syncthreads();
  const long long rows = (long long)s.lq * p.G;
  const size_t h0 = s.q0 + (size_t)head * p.G * p.T;
  float *const weights = p.w + ((size_t)n * p.kv.Hkv + head) * p.W;
  for (long long row0 = 0; row0 < rows; row0 += BM) {
    bf16x8 q[RB][KJ][NT];
    float base[RB][4];
    int lim[RB][4];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      auto at = [&](long long row, int *ti) {
        *ti = (int)(row / p.G);
        return h0 + (size_t)(row - (long long)*ti * p.G) * p.T + *ti;
      };
      int ti;
      const E *const qp = (const E *)p.q + at(min(row0 + 16 * b + r, rows - 1), &ti) * D;
#pragma unroll
      for (int j = 0; j < KJ; ++j) q_terms<E, NT>(qp + c * (D / 4) + 8 * j, 1.f, q[b][j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long row = row0 + 16 * b + 4 * c + i;
        const size_t a = at(min(row, rows - 1), &ti);
        base[b][i] = weigh_base(p.lse[a], row < rows);
        lim[b][i] = base[b][i] < INFINITY ? ti + s.off : -1;
      }
    }
    struct Tile {
      unsigned k[2][KJ];
      unsigned sc[2];
      float w;
      int id0, id1;
    } next;
    auto load = [&](Tile &x, int t) {
      x.id0 = __builtin_amdgcn_readfirstlane(s_page[(t - lo) >> 4]);
      x.id1 = __builtin_amdgcn_readfirstlane(s_page[((t - lo) >> 4) + 1]);
      const size_t pg = (size_t)p.kv.Hkv * p.kv.page;
      const size_t b0 = (size_t)max(x.id0, 0) * 2 * pg + (size_t)head * p.kv.page + t % p.kv.page;
      const size_t b1 = (size_t)max(x.id1, 0) * 2 * pg + (size_t)head * p.kv.page + (t + 16) % p.kv.page;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const size_t row = (h ? b1 : b0) + r;
        const uint8_t *a = p.kv.codes + row * (D / 2) + c * (D / 8);
        if constexpr (D == 128) {
          const u32x4 u = ld16<false>(a);
          x.k[h][0] = u[0], x.k[h][1] = u[1], x.k[h][2] = u[2], x.k[h][3] = u[3];
        } else {
          typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
          const u32x2 u = *reinterpret_cast<const u32x2 *>(a);
          x.k[h][0] = u[0], x.k[h][1] = u[1];
        }
        x.sc[h] = p.kv.scales[row * (D / 32) + (D == 128 ? c : c / 2)];
      }
      x.w = weights[min(t + (lane & 31), hi - 1)];
    };
    int t = lo + 32 * wave;
    if (t < hi) load(next, t);
    for (; t < hi; t += 128) {
      const Tile x0 = next;
      if (t + 128 < hi) load(next, t + 128);
      float sum[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4 x[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) x[b] = f32x4{0.f, 0.f, 0.f, 0.f};
        const float sc = __builtin_bit_cast(float, x0.sc[h] << 23);
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          unsigned w[4];
          cvt8(x0.k[h][j], sc, w);
          bf16x8 a;
          __builtin_memcpy(&a, w, 16);
#pragma unroll
          for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int u = NT - 1; u >= 0; --u) x[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[b][j][u], a, x[b], 0, 0, 0);
        }
        const int key = t + 16 * h + r;
        float v = 0.f;
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = __builtin_amdgcn_exp2f(fmaf(x[b][i], p.c, -base[b][i]));
            v += key <= lim[b][i] ? e : 0.f;
          }
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        sum[h] = v;
      }
      const int key = t + (lane & 31);
      if (lane < 32 && key < hi && (lane < 16 ? x0.id0 : x0.id1) >= 0) weights[key] = x0.w + (lane < 16 ? sum[0] : sum[1]);
    }
  }
}

// How a chunk call runs, by the rows of a sequence (the host's mean).  Up to 128 rows go in tiles
// of 16 or 32, more in tiles of 256, whose waves without rows only bring keys; fp32 operands are
// three terms, and the registers hold 128 rows.  64 sequences of 4,096 to 16,384 cached tokens, 16
// heads over 4, in tiles of 32 and of 256 rows (us; of 128 rows no count is the fastest):
//   24 new tokens each 311 and 354, 40 new 427 and 501, 64 new 621 and 845, 100 new 905 and 894,
//   200 new 1,695 and 1,442; 8 such sequences 75 and 72, 81 and 90, 103 and 133, 153 and 132, 215
//   and 232.
// So from 128 rows to some 300 the smaller tiles would be the better ones yet.  fp32, 8 sequences,
// in tiles of 16 and of 128 rows: 5 new 50 and 123, 24 new 80 and 133, 64 new 152 and 218.  One
// sequence of 60,000 and 2,048 new ones takes 1,004, in tiles of 128 rows 1,620.  A batch whose
// lengths differ much is planned by its mean all the same: 63 single tokens beside 1,000 and beside
// 2,048 new ones of one sequence take 264 and 517, where the single tokens alone take 75 and the
// others 145 and 277.
// Keys go in runs, as many as make about 512 workgroups (that sequence of
// 60,000, 128 tiles: 256 workgroups 946 us, 512: 958 to 1,004, 1,024: 984; those 64 sequences with
// five new tokens, 1,024: 116, 512: 112, 256: 117; with few rows 1,024), of 512 keys at least.
struct ChunkPlan {
  int BM, slots, splits, per;
};
ChunkPlan chunk_plan(const Kv4ChunkArgs &a) {
  const long long G = a.Hq / a.c.Hkv, seqs = std::max(a.N, 1);
  const long long rows = (long long)a.B * a.T * G, mean = (rows + seqs - 1) / seqs;
  ChunkPlan p;
  p.BM = mean <= 16 || (mean <= 128 && a.dtype != 0) ? 16 : mean <= 128 ? 32 : a.dtype != 0 ? 128 : 256;
  const long long tiles = a.cu ? (long long)a.T * G / p.BM + a.N : seqs * (((long long)a.T * G + p.BM - 1) / p.BM);
  p.slots = (int)std::min<long long>(tiles, 0x7fffffff);
  const long long busy = seqs * ((mean + p.BM - 1) / p.BM) * a.c.Hkv;
  long long want = std::max<long long>(1, (p.BM <= 32 ? 1024 : 512) / std::max<long long>(1, busy));
  want = std::min(want, std::max<long long>(1, a.max_len / (p.BM <= 32 ? 384 : 512)));
  const long long len = (a.max_len + want - 1) / want;
  p.per = (int)std::max<long long>(128, (len + 127) / 128 * 128);
  if (p.BM <= 32) p.per = std::min(p.per, KV_MAX_PER);
  p.splits = (int)std::max<long long>(1, ((long long)a.max_len + p.per - 1) / p.per);
  return p;
}

template <typename E, int D>
hipError_t launch_chunk(const KvChunkParams &p, int BM, hipStream_t st) {
  const dim3 grid((unsigned)((long long)p.slots * p.kv.Hkv * p.splits));
  auto go = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, st, p); };
  // few rows: codes past the caches where those do not keep them from call to call anyway, by the
  // single-token step's rule (kla_kv4.hip), which wins there what it does not win here (326 MB of
  // codes and five new tokens 117 us, through the caches 116); two row blocks of fp32 queries would not
  // fit the registers
  const bool once = (double)p.N * p.kv.Hkv * p.max_len * (D + D / 16) >= 96 << 20;
  if (BM == 16) {
    if (once) go(kla_kv4_rows_kernel<E, D, 1, true>, 256);
    else go(kla_kv4_rows_kernel<E, D, 1, false>, 256);
  } else if constexpr (sizeof(E) == 2) {
    if (BM == 32) {
      if (once) go(kla_kv4_rows_kernel<E, D, 2, true>, 256);
      else go(kla_kv4_rows_kernel<E, D, 2, false>, 256);
    } else {
      go(kla_kv4_chunk_kernel<E, D, 8, 8192 / D>, 512);
    }
  } else {
    go(kla_kv4_chunk_kernel<E, D, 4, 4096 / D>, 256);
  }
  if (p.splits > 1) {
    const size_t rows = (size_t)p.B * p.Hq * p.T, per = 256 / (D / 4);
    hipLaunchKernelGGL((kla_kv4_chunk_join_kernel<E, D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, st, p);
  }
  return hipGetLastError();
}

// How the weights are made: rows of a sequence (the host's mean) that a wave holds, in blocks of
// 16, with keys streaming past in runs; 0: more, with 64 keys to a workgroup.  Up to 384 rows the
// keys pass by for every 32.  64 sequences of 4,096 to 16,384 cached tokens, 16 heads over 4, with
// rows and with 64 keys to a workgroup (us):
//   one new token each 43 and 661, 24 new 159 and 704, 40 new 257 and 810, 64 new 400 and 885, 100
//   new 641 and 1,118, 200 new 1,207 and 1,744; 8 such sequences 13 and 96, 41 and 101, 64 and 119,
//   99 and 128, 151 and 162, 281 and 234; 12 sequences of up to 1,000 new ones behind 200 to 4,000
//   246 and 42.
// So with many sequences the rows would be the better ones at 400 and 800 too.  The mean serves
// batches badly whose lengths differ much: 63 single tokens beside 1,000 and beside 2,048 new ones
// of one sequence take 3,793 and 7,748 us, where the single tokens alone take 44 and the others 115
// and 231.  fp32 rows are three terms, 16 of them at a time up to 128 (8 sequences, 5 new 29 and
// 104, 24 new 77 and 122, 64 new 183 and 175).
struct WeighPlan {
  int RB, blocks, per;
};
WeighPlan weigh_plan(const Kv4ChunkArgs &a) {
  const long long G = a.Hq / a.c.Hkv, seqs = std::max(a.N, 1);
  const long long mean = ((long long)a.B * a.T * G + seqs - 1) / seqs;
  WeighPlan p;
  p.RB = a.dtype == 0 ? mean <= 16 ? 1 : mean <= 384 ? 2 : 0 : mean <= 128 ? 1 : 0;
  p.per = 64;
  if (p.RB) {
    const long long want = std::max<long long>(1, 2048 / (seqs * a.c.Hkv)), len = (a.max_len + want - 1) / want;
    p.per = (int)std::min<long long>(KV_MAX_PER, std::max<long long>(256, (len + 127) / 128 * 128));
  }
  p.blocks = (int)(((long long)a.max_len + p.per - 1) / p.per);
  return p;
}

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
  return (double)a.T * (a.Hq / a.c.Hkv) <= 2147418112.0 && launch_fits((double)weigh_plan(a).blocks * a.N * a.c.Hkv, 256);
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
  p.c = a.scale * 1.44269504f;
  p.w = weights;
  p.N = a.N;
  p.Hq = a.Hq;
  p.G = a.Hq / a.c.Hkv;
  p.T = a.T;
  p.W = W;
  p.max_len = a.max_len;
  const WeighPlan plan = weigh_plan(a);
  p.per = plan.per;
  if (a.max_len == 0) return hipSuccess;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((long long)plan.blocks * p.N * a.c.Hkv)), dim3(256), 0, st, p);
    return hipGetLastError();
  };
  if (a.dtype == 0) {
    if (plan.RB == 1) return a.D == 128 ? go(kla_kv4_weigh_few_kernel<bf16, 128, 1>) : go(kla_kv4_weigh_few_kernel<bf16, 64, 1>);
    if (plan.RB == 2) return a.D == 128 ? go(kla_kv4_weigh_few_kernel<bf16, 128, 2>) : go(kla_kv4_weigh_few_kernel<bf16, 64, 2>);
    return a.D == 128 ? go(kla_kv4_weigh_kernel<bf16, 128>) : go(kla_kv4_weigh_kernel<bf16, 64>);
  }
  if (plan.RB == 1) return a.D == 128 ? go(kla_kv4_weigh_few_kernel<float, 128, 1>) : go(kla_kv4_weigh_few_kernel<float, 64, 1>);
  return a.D == 128 ? go(kla_kv4_weigh_kernel<float, 128>) : go(kla_kv4_weigh_kernel<float, 64>);
}

}  // namespace kla
