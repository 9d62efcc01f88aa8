// kla_kv4.hip -- a paged key/value cache held in 4 bits, and attention of single tokens over
// it (gfx950).
//
// Format (include/kla.h, kla_kv4_append): per token, head and K or V, blocks of 32 channels
// share a power-of-two scale 2^(s - 127) (one byte, E8M0), and every channel is one E2M1 code
// (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), the even channel in a byte's low half:
// D/2 + D/32 bytes for D channels, 68 for D = 128 against 256 in bf16.  With
// s - 127 = floor(log2 max|x|) - 2 every step is exact but the one rounding to a code (to the
// nearest, ties to the even code, beyond 6 to 6), which gfx950's v_cvt_scalef32_pk_fp4_f32
// does; the values read back are exact in bf16.
//
// Bound: all three kernels by HBM.  kla_kv4_append and kla_kv4_read give four lanes to a block
// of 32 channels (16 bytes of bf16 and 4 of codes each).  The decode kernel is described below.
#include <algorithm>

#include "kla_common.h"
#include "kla_internal.h"

namespace kla {

namespace {

struct KvParams {
  uint8_t *codes, *scales;
  const int32_t *table;
  int num_pages, page, max_pages, Hkv;
};

// Row (in units of a token's codes or scales) of position pos of sequence n in K (j = 0) or V
// (j = 1) of a head; -1 where the table does not lead to a page of the cache.
__device__ __forceinline__ long long kv_row(const KvParams &p, int n, int pos, int j, int head) {
  if (pos < 0 || pos / p.page >= p.max_pages) return -1;
  const int id = p.table[(size_t)n * p.max_pages + pos / p.page];
  if (id < 0 || id >= p.num_pages) return -1;
  return (((long long)id * 2 + j) * p.Hkv + head) * p.page + pos % p.page;
}

template <int CTRL>
__device__ __forceinline__ unsigned quad_max(unsigned v) {
  return max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}

struct KvMoveParams {
  KvParams kv;
  void *k, *v;                // [B, Hkv, T, D]
  const int32_t *start, *cu;  // device
  int N, T;
  long long rows;             // B * Hkv * T
};

// 16 bytes; ONCE: with the non-temporal hint, for what is not used again soon
template <bool ONCE>
__device__ __forceinline__ u32x4 ld16(const void *p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
  else return *reinterpret_cast<const u32x4 *>(p);
}

// eight channels as fp32
template <typename E, bool ONCE = false>
__device__ __forceinline__ void ld8(const E *p, float *f) {
  constexpr int PER = 16 / sizeof(E);
#pragma unroll
  for (int i = 0; i < 8; i += PER) {
    const u32x4 u = ld16<ONCE>(p + i);
    E e[PER];
    __builtin_memcpy(e, &u, 16);
#pragma unroll
    for (int j = 0; j < PER; ++j) f[i + j] = Elem<E>::to_f32(e[j]);
  }
}
template <typename E, bool ONCE>
__device__ __forceinline__ void st8(E *p, const float *f) {
  constexpr int PER = 16 / sizeof(E);
#pragma unroll
  for (int i = 0; i < 8; i += PER) {
    E e[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) e[j] = Elem<E>::from_f32(f[i + j]);
    u32x4 u;
    __builtin_memcpy(&u, e, 16);
    if constexpr (ONCE) __builtin_nontemporal_store(u, reinterpret_cast<u32x4 *>(p + i));
    else *reinterpret_cast<u32x4 *>(p + i) = u;
  }
}

// A workgroup moves TOKENS consecutive tokens of one head's keys or values: as many threads find
// their places (sequence, position, page) while the other loads are in flight, then D / 8 lanes
// move a row.  A token that the device's offsets give to no sequence (a padded batch) is not
// moved.  Many tokens: 256 to a workgroup, and their rows past the caches (ONCE).
constexpr int KV_CU = 1024;  // offsets searched in LDS

template <typename E, int D, bool READ, int TOKENS, bool ONCE>
__global__ __launch_bounds__(256) void kla_kv4_move_kernel(KvMoveParams p) {
  constexpr int LPR = D / 8, RPT = TOKENS * LPR / 256;  // lanes of a row, rows of a thread
  __shared__ long long s_row[TOKENS];
  __shared__ int s_cu[KV_CU];
  const int tid = threadIdx.x, lane = tid % LPR;
  const unsigned jh = blockIdx.x % (2 * p.kv.Hkv);
  const int j = jh / p.kv.Hkv, head = jh % p.kv.Hkv;
  const long long tok0 = (long long)(blockIdx.x / (2 * p.kv.Hkv)) * TOKENS, toks = p.rows / p.kv.Hkv;  // B * T
  E *const base = (E *)(j ? p.v : p.k);

  auto x_of = [&](int i) {  // row i of the workgroup (the last one's again past the end)
    const long long tok = min(tok0 + i, toks - 1), b = p.cu ? 0 : tok / p.T;  // packed: one row of the batch
    return base + ((b * p.kv.Hkv + head) * p.T + (tok - b * p.T)) * D + 8 * lane;
  };
  float f[RPT][8];
  if constexpr (!READ) {
#pragma unroll
    for (int r = 0; r < RPT; ++r) ld8<E, ONCE>((const E *)x_of(tid / LPR + 256 / LPR * r), f[r]);
  }
  const bool near = p.cu && p.N < KV_CU;
  if (near) {
    for (int i = tid; i <= p.N; i += 256) s_cu[i] = p.cu[i];
    __syncthreads();
  }
  // The workgroup's tokens that belong to sequences; a read writes no other rows.  Their bounds
  // are compared, not kept with each place: a flag read back per row took fp32 reads of 131,000
  // tokens from 147 to 172 us.
  auto within = [&](long long tok) { return (int)max(min(tok - tok0, (long long)TOKENS), 0LL); };
  int from = 0, to = within(toks);
  if (p.cu) {
    from = within(near ? s_cu[0] : p.cu[0]);
    to = min(to, within(near ? s_cu[p.N] : p.cu[p.N]));
  }
  if (tid < TOKENS) {
    const long long tok = tok0 + tid;
    long long row = -1;
    if (tid >= from && tid < to) {
      int n = p.cu ? 0 : (int)(tok / p.T), at = (int)(tok - (long long)n * p.T);
      if (p.cu) {
        // the last sequence that starts at or before the token (its offsets not decreasing)
        int lo = 0, hi = p.N;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if ((near ? s_cu[mid] : p.cu[mid]) <= at) lo = mid; else hi = mid;
        }
        n = lo;
        at -= max(near ? s_cu[n] : p.cu[n], 0);
      }
      // a negative start: all of the sequence is padding
      const int start = p.start[n];
      const long long pos = (long long)start + at;
      if (start >= 0 && pos <= 0x7fffffffLL) row = kv_row(p.kv, n, (int)pos, j, head);
    }
    s_row[tid] = row;
  }
  __syncthreads();
  if constexpr (READ) {
    unsigned u[RPT];
    uint8_t sc[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const long long row = s_row[tid / LPR + 256 / LPR * r];
      // a token without a place: zero codes
      u[r] = row >= 0 ? *reinterpret_cast<const unsigned *>(p.kv.codes + row * (D / 2) + 4 * lane) : 0u;
      sc[r] = row >= 0 ? p.kv.scales[row * (D / 32) + lane / 4] : 127;
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const float s = __builtin_bit_cast(float, (unsigned)sc[r] << 23);
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u[r], s, 0);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u[r], s, 1);
      const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u[r], s, 2);
      const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u[r], s, 3);
      const float y[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
      const int i = tid / LPR + 256 / LPR * r;
      if (i >= from && i < to) st8<E, ONCE>(x_of(i), y);
    }
  } else {
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      unsigned top = 0;  // |x| as bits: NaN above infinity above every number
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(unsigned, f[r][i]) & 0x7fffffffu);
      top = quad_max<0xB1>(top);
      top = quad_max<0x4E>(top);
      const unsigned e = top >> 23, s = e == 255 ? 255u : (e > 3 ? e - 2 : 1u);
      const float sc = __builtin_bit_cast(float, s << 23);
      unsigned u = 0;
      u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(u, f[r][0], f[r][1], sc, 0);
      u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(u, f[r][2], f[r][3], sc, 1);
      u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(u, f[r][4], f[r][5], sc, 2);
      u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(u, f[r][6], f[r][7], sc, 3);
      const long long row = s_row[tid / LPR + 256 / LPR * r];
      if (row >= 0) {
        *reinterpret_cast<unsigned *>(p.kv.codes + row * (D / 2) + 4 * lane) = u;
        if (lane % 4 == 0) p.kv.scales[row * (D / 32) + lane / 4] = (uint8_t)s;
      }
    }
  }
}

// ---- attention of one token per sequence ------------------------------------------------------
//
// o = softmax(scale q K^T) V over the sequence's cached tokens.  A workgroup (four waves) owns
// one (sequence, key head, up to 16 of its query heads, run of `per` tokens); its waves take
// tiles of 32 tokens in turn, each with its own running maximum, sum and output, joined in LDS
// at the end, and the runs of one head are joined by a second kernel.
//
// K's codes become MFMA operands as they are loaded.  Lane (r = lane & 15, c = lane >> 4) holds a
// quarter of key r's row, channels c D/4 and up; its j-th eight channels are its slots of the
// j-th v_mfma_f32_16x16x32_bf16, q being laid out the same.  The scores S^T come with heads
// along the lanes and keys 4c .. 4c+3 in each, so that two 16-key tiles are the left-over
// operand P^T of the second product as they stand: slots 8c + e are the keys 4c + e and
// 16 + 4c + e - 4.  V goes through LDS, still in 4 bits, into lanes that hold channels r D/16
// and up of those eight keys; they convert pairs of channels (v_cvt_scalef32_pk_bf16_fp4
// applies the scale too) and exchange halves (v_perm) into pairs of keys, and MFMA j takes
// channel r D/16 + j of every lane.
//
// Measured (64 sequences of 4,096 to 16,384 tokens, 16 heads over 4, D = 128, 326 MB): 66 us a
// step, 4.9 TB/s, where 4 KB reads in any order reach 5.8; of it the joining kernel is 5.  With
// V's dwords and scale bytes loaded straight into that layout, and the runs of a sequence side
// by side in the grid, it took 107, with the codes through the caches 74; a second tile in
// flight, or two or four workgroups on a CU for three, change nothing: what is left is spread
// over the conversions (37% of the issue slots), the latency of one tile's chain and the
// lengths' unevenness.
//
// Queries in fp32 run the same products with q and P split into three bf16 terms (24 bits),
// exact against the cache's values.
struct KvDecodeParams {
  KvParams kv;
  const void *q;
  void *o;
  const int32_t *lens;
  float scale_log2;    // scale * log2(e)
  int N, Hq, G, GB;    // G query heads to a key head, in GB blocks of 16
  int max_len, splits, per;
  float *part_o, *part_ml;  // [N Hq, splits, D], [N Hq, splits, 2] where splits > 1
};

constexpr int KV_MAX_PER = 8192;  // tokens of a run

typedef bf16 bf16x8v __attribute__((ext_vector_type(8)));

// eight channels in a dword as four bf16 pairs
__device__ __forceinline__ void cvt8(unsigned u, float s, unsigned *r) {
  r[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, s, 0));
  r[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, s, 1));
  r[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, s, 2));
  r[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, s, 3));
}

template <typename E, int D, bool ONCE>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 3 : 2) void kla_kv4_decode_kernel(KvDecodeParams p) {
  constexpr int NT = sizeof(E) == 2 ? 1 : 3;  // bf16 terms of q and P
  constexpr int KJ = D / 32;                  // products over the channels, 8 channels a lane
  constexpr int DW = D / 16;                  // channels of V a lane holds
  __shared__ int s_page[KV_MAX_PER / 16];
  __shared__ float s_o[4][16][D + 4];
  __shared__ float s_ml[4][16][2];
  __shared__ __attribute__((aligned(16))) uint8_t s_v[4][32 * D / 2];
  __shared__ unsigned s_sc[4][64];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, c = lane >> 4;
  // runs slowest: workgroups go round the eight XCDs, and with the runs of a sequence side by
  // side the first ones, which every sequence has, met on a few of them
  unsigned b = blockIdx.x;
  const int gb = b % p.GB;
  b /= p.GB;
  const int head = b % p.kv.Hkv;
  b /= p.kv.Hkv;
  const int n = b % p.N, split = b / p.N;
  const int g0 = gb * 16, gn = min(p.G - g0, 16);  // query heads of this workgroup
  const int hq0 = head * p.G + g0;
  // tokens of the sequence, of this run
  const long long room = (long long)p.kv.max_pages * p.kv.page;
  const int len = (int)min((long long)min(max(p.lens[n], 0), p.max_len), room);
  const int lo = split * p.per, hi = (int)min((long long)len, (long long)lo + p.per);

  if (hi > lo) {
    for (int i = tid; i < (hi - lo + 31) / 32 * 2; i += 256) {
      const int t = lo + 16 * i;
      int id = -1;
      if (t < hi) {
        id = p.kv.table[(size_t)n * p.kv.max_pages + t / p.kv.page];
        if (id >= p.kv.num_pages) id = -1;
      }
      s_page[i] = id;
    }
  }
  // q: slots 8c + e of product j are channels c D/4 + 8j + e
  bf16x8v q[NT][KJ];
#pragma unroll
  for (int j = 0; j < KJ; ++j) {
    float f[8] = {};
    if (r < gn) ld8((const E *)p.q + ((size_t)n * p.Hq + hq0 + r) * D + c * (D / 4) + 8 * j, f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bf16 h = (bf16)f[i];
        q[t][j][i] = h;
        f[i] -= (float)h;
      }
  }
  __syncthreads();

  f32x4 acc[DW];
#pragma unroll
  for (int j = 0; j < DW; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  // A tile's codes and scales as they are loaded: K in operand layout, V in 16-byte pieces of
  // rows, and the 32 keys' scales, then the values', a row to a lane.
  constexpr int VP = D / 64;           // pieces of V a lane loads
  constexpr int LPR = D / 32;          // lanes of a row of V
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
        u32x2 u;
        if constexpr (ONCE) u = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(a));
        else u = *reinterpret_cast<const u32x2 *>(a);
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
  if (t < hi) load(next, t);
  for (; t < hi; t += 128) {
    const Tile x0 = next;
    if (t + 128 < hi) load(next, t + 128);
    // V and the scales through the wave's own LDS; key 16 h + 4 c + e at slot 16 h + 4 e + c,
    // so that the four keys of a read fill the banks
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int key = lane / LPR + 64 / LPR * i, slot = (key & 16) + 4 * (key & 3) + ((key >> 2) & 3);
      *reinterpret_cast<u32x4 *>(s_v[wave] + slot * (D / 2) + 16 * (lane % LPR)) = x0.v[i];
    }
    s_sc[wave][lane] = x0.sc;
    const uint8_t *sc8 = reinterpret_cast<const uint8_t *>(s_sc[wave]);
    const int id0 = x0.id0, id1 = x0.id1;
    // scores of keys t + 16h + 4c + i against head r
    float x[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
      const float sc = __builtin_bit_cast(float, (unsigned)sc8[4 * (16 * h + r) + (D == 128 ? c : c / 2)] << 23);
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        unsigned w[4];
        cvt8(x0.k[h][j], sc, w);
        bf16x8v a;
        __builtin_memcpy(&a, w, 16);
#pragma unroll
        for (int u = 0; u < NT; ++u) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q[u][j], s, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * h + i] = s[i] * p.scale_log2;
    }
    unsigned va[8];
    float vf[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t *a = s_v[wave] + ((e & 4) * 4 + 4 * (e & 3) + c) * (D / 2);
      unsigned short half;
      if constexpr (D == 128) __builtin_memcpy(&va[e], __builtin_assume_aligned(a + 4 * r, 4), 4);
      else __builtin_memcpy(&half, __builtin_assume_aligned(a + 2 * r, 2), 2), va[e] = half;
      vf[e] = __builtin_bit_cast(float, (unsigned)sc8[4 * (32 + 16 * (e >> 2) + 4 * c + (e & 3)) + r * DW / 32] << 23);
    }
    if (id0 < 0 || id1 < 0 || t + 32 > hi) {
      // tokens past the end and tokens of missing pages: no score, and a value of zero
      // whatever the memory behind them holds
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool none = (e < 4 ? id0 : id1) < 0 || t + 16 * (e >> 2) + 4 * c + (e & 3) >= hi;
        x[e] = none ? -INFINITY : x[e];
        va[e] = none ? 0u : va[e];
        vf[e] = none ? 1.f : vf[e];
      }
    }

    float top = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float mn = fmaxf(m, top);
    const float base = mn == -INFINITY ? 0.f : mn;
    if (__any(mn > m)) {
      const float al = __builtin_amdgcn_exp2f(m - base);
      l *= al;
#pragma unroll
      for (int j = 0; j < DW; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] *= al;
      m = mn;
    }
    bf16x8v pt[NT];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = __builtin_amdgcn_exp2f(x[e] - base);
      l += v;
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const bf16 h = (bf16)v;  // P in bf16 terms: one has half a step of 2^-8, as the output's rounding
        pt[u][e] = h;
        v -= (float)h;
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
      bf16x8v av;
      __builtin_memcpy(&av, a, 16);
#pragma unroll
      for (int u = 0; u < NT; ++u) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, pt[u], acc[j], 0, 0, 0);
    }
  }

  // join the waves
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (c == 0) {
    s_ml[wave][r][0] = m;
    s_ml[wave][r][1] = l;
  }
#pragma unroll
  for (int j = 0; j < DW; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_o[wave][r][(4 * c + i) * DW + j] = acc[j][i];
  __syncthreads();
  for (int i = tid; i < gn * D; i += 256) {
    const int g = i / D, d = i % D;
    float mm = s_ml[0][g][0];
#pragma unroll
    for (int w = 1; w < 4; ++w) mm = fmaxf(mm, s_ml[w][g][0]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, oo = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = __builtin_amdgcn_exp2f(s_ml[w][g][0] - base);
      ll = fmaf(s_ml[w][g][1], f, ll);
      oo = fmaf(s_o[w][g][d], f, oo);
    }
    const size_t row = (size_t)n * p.Hq + hq0 + g;
    if (p.splits == 1) {
      ((E *)p.o)[row * D + d] = Elem<E>::from_f32(ll == 0.f ? 0.f : oo / ll);
    } else {
      p.part_o[(row * p.splits + split) * D + d] = oo;
      if (d == 0) {
        p.part_ml[(row * p.splits + split) * 2] = mm;
        p.part_ml[(row * p.splits + split) * 2 + 1] = ll;
      }
    }
  }
}

// The runs of one (sequence, query head): GROUPS groups of threads take every GROUPS-th run,
// four channels to a thread, and meet in LDS.  Few runs: 8 groups over all channels; many: 32
// groups over 32 channels of them (16 heads of 256 runs: 4.7 us against 5.9 with 8 groups,
// and 19 run by run).
template <typename E, int D, int GROUPS, int CH>
__global__ __launch_bounds__(GROUPS *CH / 4) void kla_kv4_join_kernel(KvDecodeParams p) {
  constexpr int LPG = CH / 4, PARTS = D / CH;  // lanes of a group, workgroups of a row
  __shared__ f32x4 s_o[GROUPS][LPG];
  __shared__ float s_l[GROUPS];
  const size_t row = blockIdx.x / PARTS;
  const int g = threadIdx.x / LPG, lane = threadIdx.x % LPG, ch = (blockIdx.x % PARTS) * CH + 4 * lane;
  const float *ml = p.part_ml + row * p.splits * 2;
  float m = -INFINITY;
  for (int s = threadIdx.x % 64; s < p.splits; s += 64) m = fmaxf(m, ml[2 * s]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  const float *po = p.part_o + row * p.splits * D + ch;
#pragma unroll 4
  for (int s = g; s < p.splits; s += GROUPS) {
    const float f = __builtin_amdgcn_exp2f(ml[2 * s] - base);
    const f32x4 v = *reinterpret_cast<const f32x4 *>(po + (size_t)s * D);
    l = fmaf(ml[2 * s + 1], f, l);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(v[i], f, o[i]);
  }
  s_o[g][lane] = o;
  if (lane == 0) s_l[g] = l;
  __syncthreads();
  if (g) return;
#pragma unroll
  for (int k = 1; k < GROUPS; ++k) {
    l += s_l[k];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] += s_o[k][lane][i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    ((E *)p.o)[row * D + ch + i] = Elem<E>::from_f32(l == 0.f ? 0.f : o[i] / l);
}

template <typename E, int D, bool READ, int TOKENS, bool ONCE>
hipError_t launch_move_t(const KvMoveParams &p, hipStream_t st) {
  const long long groups = (p.rows / p.kv.Hkv + TOKENS - 1) / TOKENS;
  hipLaunchKernelGGL((kla_kv4_move_kernel<E, D, READ, TOKENS, ONCE>), dim3((unsigned)(groups * 2 * p.kv.Hkv)), dim3(256), 0,
                     st, p);
  return hipGetLastError();
}

// Tokens of a workgroup, and whether the rows go past the caches, by the bytes of k and v.  From
// 96 MB on (what the caches keep between calls) more tokens hide the search for their places,
// and bf16 rows, written in whole lines, leave the caches to the codes: 131,000 tokens of 4 heads
// of 128 (268 MB) append 64 us against 75 with 64 tokens, 96,000 49 against 55; 32,000 the other
// way 19.8 against 18.6.  A thread of a read holds eight rows: 128 tokens of 128 channels (96,000
// tokens read in 41 us, with 256 tokens 46; 131,000 in 53, 60, with 64 tokens 104; 256,000 in 95,
// 103), 256 tokens of 64 channels (8 heads: 96,000 in 41 us either way; 131,000 in 51, with 128
// tokens 54; 256,000 in 95, 99; 400,000 in 145, 155).  fp32 rows are written in half lines, which
// must meet in the caches (64,000 tokens past them 108 us, 63 to 69 with 256 tokens and 83 with
// 64; 131,000 147, with 128 tokens 159); their appends take the same time either way.
template <typename E, int D, bool READ>
hipError_t launch_move(const KvMoveParams &p, hipStream_t st) {
  constexpr bool ONCE = sizeof(E) == 2;
  constexpr int MANY = READ && ONCE ? 16384 / D : 256;
  const long long mb = p.rows * D * 2 * (long long)sizeof(E) >> 20;
  if constexpr (READ || ONCE)
    if (mb >= 96) return launch_move_t<E, D, READ, MANY, ONCE>(p, st);
  return launch_move_t<E, D, READ, 64, false>(p, st);
}

template <typename E, int D>
hipError_t launch_kv4_decode(const KvDecodeParams &p, hipStream_t st) {
  const long long grid = (long long)p.N * p.kv.Hkv * p.GB * p.splits;
  // The codes go past the caches where the cache is larger than what those keep from step to step
  // (64 sequences, 326 MB: 66 us, 74 through them; 32 of 30,000 tokens: 100, 113; 16 of 4,000
  // with 8 heads, 70 MB: 23.1, 22.3).
  if ((double)p.N * p.kv.Hkv * p.max_len * (D + D / 16) >= 96 << 20)
    hipLaunchKernelGGL((kla_kv4_decode_kernel<E, D, true>), dim3((unsigned)grid), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((kla_kv4_decode_kernel<E, D, false>), dim3((unsigned)grid), dim3(256), 0, st, p);
  const long long rows = (long long)p.N * p.Hq;
  if (p.splits > 32)
    hipLaunchKernelGGL((kla_kv4_join_kernel<E, D, 32, 32>), dim3((unsigned)(rows * (D / 32))), dim3(256), 0, st, p);
  else if (p.splits > 1)
    hipLaunchKernelGGL((kla_kv4_join_kernel<E, D, 8, D>), dim3((unsigned)rows), dim3(2 * D), 0, st, p);
  return hipGetLastError();
}

KvParams kv_params(const Kv4Cache &c) {
  return KvParams{(uint8_t *)c.codes, (uint8_t *)c.scales, c.table, c.num_pages, c.page, c.max_pages, c.Hkv};
}

// Runs of the sequences: as many as bring about 1,024 workgroups.  That is for sequences of
// uneven lengths, 4 heads of D = 128: 64 of 4,096 to 16,384 tokens 66 us (with 512 workgroups 84,
// with 768 78, with 1,536 77, with 2,048 73), 64 of 1,000 to 8,000 37 (768: 44, 1,536: 42), 24 of
// 2,000 to 40,000 62 (71, 64); 10 of 8,000 to 60,000 with 8 heads 65 (64, 62).  Sequences that all
// reach max_len do better with 768, one round, by 3 to 9%: 32 of 30,000 tokens 95 us against 92, 64
// of 8,000 54 against 50, 8 of 8,000 with 8 heads 21.8 against 20.1; but the lengths are the
// device's.  A run has 384 tokens at least (three tiles a wave; one sequence of 131,072 tokens,
// 2 heads: 16.6 us, with 256 tokens 19.0, with 512 18.2) and KV_MAX_PER at most.
void kv4_runs(const Kv4DecodeArgs &a, int *splits, int *per) {
  const long long GB = (a.Hq / a.c.Hkv + 15) / 16, base = (long long)a.N * a.c.Hkv * GB;
  long long want = std::max<long long>(1, 1024 / std::max<long long>(1, base));
  want = std::min(want, std::max<long long>(1, a.max_len / 384));
  long long len = (a.max_len + want - 1) / want;
  len = std::min<long long>(KV_MAX_PER, std::max<long long>(128, (len + 127) / 128 * 128));
  *per = (int)len;
  *splits = (int)std::max<long long>(1, (a.max_len + len - 1) / len);
}

}  // namespace

size_t kv4_decode_workspace_bytes(const Kv4DecodeArgs &a) {
  int splits, per;
  kv4_runs(a, &splits, &per);
  return splits == 1 ? 0 : (size_t)a.N * a.Hq * splits * (a.D + 2) * sizeof(float);
}

bool kv4_decode_grid_fits(const Kv4DecodeArgs &a) {
  int splits, per;
  kv4_runs(a, &splits, &per);
  return launch_fits((double)a.N * a.c.Hkv * ((a.Hq / a.c.Hkv + 15) / 16) * splits, 256) &&
         launch_fits((double)a.N * a.Hq * (a.D / 32), 256);
}

bool kv4_move_grid_fits(int B, int Hkv, int T, int D, int dtype, bool read) {
  // a large batch's tokens to a workgroup: launch_move
  const int tokens = read && dtype == 0 ? 16384 / D : (read || dtype == 0 ? 256 : 64);
  return launch_fits(((double)B * T / tokens + 1) * 2 * Hkv, 256);
}

hipError_t launch_kv4_move(const Kv4Cache &c, void *k, void *v, const int32_t *start, const int32_t *cu, int N, int B,
                           int T, int D, int dtype, bool read, hipStream_t st) {
  const KvMoveParams p{kv_params(c), k, v, start, cu, N, T, (long long)B * c.Hkv * T};
  if (p.rows == 0) return hipSuccess;
  if (dtype == 0) {
    if (D == 128) return read ? launch_move<bf16, 128, true>(p, st) : launch_move<bf16, 128, false>(p, st);
    return read ? launch_move<bf16, 64, true>(p, st) : launch_move<bf16, 64, false>(p, st);
  }
  if (D == 128) return read ? launch_move<float, 128, true>(p, st) : launch_move<float, 128, false>(p, st);
  return read ? launch_move<float, 64, true>(p, st) : launch_move<float, 64, false>(p, st);
}

hipError_t launch_attn_kv4_decode(const Kv4DecodeArgs &a, void *workspace, hipStream_t st) {
  KvDecodeParams p{};
  p.kv = kv_params(a.c);
  p.q = a.q;
  p.o = a.o;
  p.lens = a.lens;
  p.scale_log2 = a.scale * 1.44269504f;
  p.N = a.N;
  p.Hq = a.Hq;
  p.G = a.Hq / a.c.Hkv;
  p.GB = (p.G + 15) / 16;
  p.max_len = a.max_len;
  kv4_runs(a, &p.splits, &p.per);
  p.part_o = (float *)workspace;
  p.part_ml = p.part_o + (size_t)a.N * a.Hq * p.splits * a.D;
  if (a.dtype == 0) return a.D == 128 ? launch_kv4_decode<bf16, 128>(p, st) : launch_kv4_decode<bf16, 64>(p, st);
  return a.D == 128 ? launch_kv4_decode<float, 128>(p, st) : launch_kv4_decode<float, 64>(p, st);
}

}  // namespace kla
