// kla_glr.hip -- gated linear recurrence per channel (gfx950): forward, backward, one step.
//
// Per sequence, head and channel (include/kla.h, kla_glr_chunk_fwd):
//   a_t = exp(g_t),  h_t = a_t h_{t-1} + x_t,  o_t = h_t
// and backwards, with e_t = a_t dh_t the gradient that reaches h_{t-1}:
//   dx_t = dh_t = do_t + e_{t+1},  e_t = a_t dh_t,  dg_t = e_t h_{t-1},  dh_0 = e_1
// Both are scans of affine maps (A, C): y -> A y + C, composed in order: (A1, C1) then
// (A2, C2) is (A1 A2, A2 C1 + C2).  The forward's map of token t is (a_t, x_t); the
// backward's, in reverse order, is (a_t, a_t do_t).  Maps are composed in fp32 in an order
// that depends on the sizes alone, so results repeat bit for bit.
//
// The forward reads x and g and writes o once (6 bytes per element in bf16), the backward
// reads g, o and do and writes dx and dg (10 bytes): both are bound by HBM.  One workgroup of
// eight waves owns a slice of 64 (or 32, or 128) bytes of the rows of one (sequence, head) and
// walks its tokens in tiles of 512 rows (1,024 with 32 bytes, 256 with 128; 256 or 64 by four
// waves or one for short sequences), the next tile's 16-byte loads in flight in registers.  A tile
// goes through LDS from the loads' order (consecutive lanes along a row) to the scan's (a wave's
// lanes are 4 groups of V channels times 16 row groups; with 128 bytes 8 times 8): each lane
// composes R consecutive rows of its V channels, DPP row shifts compose the row groups of a wave
// (two instructions a step and channel), the waves' maps meet in LDS behind the one barrier of a
// tile, and the outputs go back through LDS into whole row pieces.  Every byte is read once and no
// workgroup waits for another.  Measured on B=4 H=16 T=4096 d=128: forward 45 to 49 us (4.1 to 4.5
// TB/s; a copy of 1 GiB reaches 5.2), 32 packed sequences of 268 M elements backward 564 us (4.8
// TB/s); a first form with the scan's steps as lane shuffles in the loads' order took 56 and 790 us.
//
// Where few channels leave most CUs idle, sequences are cut into segments: a first pass forms
// each segment's map, and the second starts every segment from the maps of those before it; it
// reads x and g twice (glr_plan has the rule).  Plans go by the host's lengths, tokens by the
// device's: where those differ, results are the device's and only time is lost.
#include <algorithm>

#include "kla_common.h"
#include "kla_internal.h"
#include "kla_ops.h"

namespace kla {

namespace {

constexpr int GLR_ORDER = 64;  // sequences that are put in order

struct GlrParams {
  const void *x, *g;         // x: the forward's input, the backward's do
  const void *h;             // backward: the forward's output o
  const float *y0;           // [N,H,d] start of the scan (initial state / dfinal), or nullptr
  const float *h0;           // backward: [N,H,d] initial state, or nullptr
  void *o, *dg;              // outputs (o: forward output / dx)
  float *yend;               // [N,H,d] end of the scan (final state / dinitial), or nullptr
  const int32_t *cu;         // device, or nullptr (dense)
  int N, H, T, d;
  int lines, inner;          // 128-byte lines of a head's channels, slices of one
  int segs, nseg, seg_rows;  // segments of a sequence at most, of this launch, tokens in one
  float *maps;               // [N,H,segs,2,d]: the segments' maps (A then C)
  int ordered;               // the sequences start in `order`, the longest first
  int order[GLR_ORDER];
};

// exp of the log-decay: one base-2 exponential for bf16 gates, whose own spacing is 2^-8 of
// their value; the library's exp for fp32, where the product's rounding would show.
__device__ __forceinline__ float decay(float g, const bf16 *) { return __builtin_amdgcn_exp2f(g * 1.44269504f); }
__device__ __forceinline__ float decay(float g, const float *) { return expf(g); }

template <typename E, int V>
struct Vec {
  E v[V];
};
// V elements at a multiple of their size (V divides d)
template <typename E, int V>
__device__ __forceinline__ Vec<E, V> ld(const E *p) {
  Vec<E, V> r;
  __builtin_memcpy(&r, __builtin_assume_aligned(p, V * sizeof(E)), V * sizeof(E));
  return r;
}
template <typename E, int V>
__device__ __forceinline__ void st(E *p, const float *f) {
  Vec<E, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = Elem<E>::from_f32(f[i]);
  __builtin_memcpy(__builtin_assume_aligned(p, V * sizeof(E)), &r, V * sizeof(E));
}

// V floats; V > 1 divides d, so rows of floats are 16-byte aligned
template <int V>
__device__ __forceinline__ void ldf(float *r, const float *p) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<f32x4 *>(r + i) = *reinterpret_cast<const f32x4 *>(p + i);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = p[i];
  }
}

// 16 bytes; ONCE: with the non-temporal hint, for whole lines, which no other workgroup wants
template <bool ONCE>
__device__ __forceinline__ uint4 ldq(const void *p) {
  if constexpr (ONCE) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p)));
  else return ldg16(p);
}
enum { GLR_WHOLE = 0, GLR_MAPS = 1, GLR_CARRIED = 2 };

// v of the lane S before this one in its row of 16; the row's first S lanes keep `old`.
template <int S>
__device__ __forceinline__ float row_shr(float old, float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v),
                                                               0x110 + S, 0xF, 0xF, false));
}
// the same among GW lanes, this one number gw of them
template <int S, int GW>
__device__ __forceinline__ float group_shr(float old, float v, int gw) {
  const float x = row_shr<S>(old, v);
  return GW == 16 || gw >= S ? x : old;
}
template <int S, int V, int GW>
__device__ __forceinline__ void scan_step(float *A, float *C, int gw) {
  if (S >= GW) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    // the map S lanes before, then this one; in front of the group's first lanes the identity
    C[i] = fmaf(group_shr<S, GW>(0.f, C[i], gw), A[i], C[i]);
    A[i] = group_shr<S, GW>(1.f, A[i], gw) * A[i];
  }
}

// LDS of a workgroup: per wave its rows of the tensors it reads, and a row set on its way out.
template <typename E, int V, int NW, int R, bool BWD, int MODE, bool PIECES, int CG>
struct GlrLds {
  static constexpr int CW = CG * V, GW = 64 / CG;
  static constexpr int NT = BWD && MODE != GLR_MAPS ? 3 : 2;
  static constexpr int ROWB = CW * (int)sizeof(E), P = CG == 8 ? 1 : 64 / (ROWB < 64 ? ROWB : 64);  // row sets to 1 KB
  static constexpr int STAGE = PIECES ? R * GW * ROWB : 16;
  float map[2][NW][2][CW], carry[2][2][CW];
  __attribute__((aligned(1024))) char in[NW][NT][STAGE];
  __attribute__((aligned(1024))) char out[NW][BWD ? 2 : 1][PIECES ? 1024 : 16];
};

template <typename E, int V, int NW, int R, bool BWD, int MODE, bool PIECES, int CG>
__global__ __launch_bounds__(64 * NW) void kla_glr_kernel(GlrParams p) {
  using Lds = GlrLds<E, V, NW, R, BWD, MODE, PIECES, CG>;
  constexpr int GW = 64 / CG;         // CG channel groups, GW row groups of a wave
  constexpr int ROWS = NW * GW * R;   // rows of a tile
  constexpr int CW = CG * V, P = Lds::P, NT = Lds::NT;
  constexpr bool HV = NT == 3;
  __shared__ Lds s;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cg = lane / GW, gw = lane % GW;
  // workgroups go round the eight XCDs: the slices of one 128-byte line stay on one, side by
  // side in time, so that its L2 reads the line once
  const unsigned u = blockIdx.x / (8 * p.inner) * 8 + blockIdx.x % 8, in = blockIdx.x / 8 % p.inner;
  unsigned b = u / p.lines;
  const int slice = (u % p.lines) * p.inner + in;
  const int head = b % p.H;
  b /= p.H;
  int seq = b % p.N;
  const int seg = b / p.N;
  if (seg >= p.nseg || slice * CW >= p.d) return;
  if (MODE == GLR_WHOLE && p.ordered) seq = p.order[seq];

  // the tokens of this sequence (device cu_seqlens clamped to [0, T]), then of the segment
  int t0 = 0, t1 = p.T;
  size_t row0 = (size_t)head * p.T;
  if (p.cu) {
    t0 = min(max(p.cu[seq], 0), p.T);
    t1 = min(max(p.cu[seq + 1], t0), p.T);
  } else {
    row0 += (size_t)seq * p.H * p.T;
  }
  const int len_seq = t1 - t0;
  const int skip = MODE == GLR_WHOLE ? 0 : seg * p.seg_rows;  // scan steps before this segment
  if (MODE != GLR_WHOLE && seg > 0 && skip >= len_seq) return;
  // the last segment takes the rest: the host's lengths set the segments, the device's may be longer
  const bool rest = MODE == GLR_WHOLE || (MODE == GLR_CARRIED && seg == p.nseg - 1);
  const int len = rest ? len_seq - skip : min(len_seq - skip, p.seg_rows);
  const bool last_seg = skip + len == len_seq;

  const int c = slice * CW + cg * V;
  const bool live = c < p.d;  // V divides d
  const int cc = live ? c : 0;
  const size_t sh = ((size_t)seq * p.H + head) * p.d + cc;  // states, at this thread's channels

  float carry[V];  // the scan's value before the tile
#pragma unroll
  for (int i = 0; i < V; ++i) carry[i] = MODE == GLR_WHOLE && p.y0 ? p.y0[sh + i] : 0.f;
  float total[V];  // MAPS: the segment's A
#pragma unroll
  for (int i = 0; i < V; ++i) total[i] = 1.f;
  const size_t mrow = (((size_t)seq * p.H + head) * p.segs) * 2 * p.d + cc;
  // yend may be y0: with segments the start goes through the slot of the last segment, whose
  // own map nothing needs
  float *const start = p.maps + mrow + (size_t)(p.segs - 1) * 2 * p.d;
  if (MODE == GLR_MAPS && seg == 0 && live && !wave && !gw) {
#pragma unroll
    for (int i = 0; i < V; ++i) start[i] = p.y0 ? p.y0[sh + i] : 0.f;
  }
  if (MODE == GLR_CARRIED) {
    ldf<V>(carry, start);
#pragma unroll 4
    for (int q = 0; q < seg; ++q) {
      float ma[V], mc[V];
      ldf<V>(ma, p.maps + mrow + (size_t)q * 2 * p.d);
      ldf<V>(mc, p.maps + mrow + (size_t)q * 2 * p.d + p.d);
#pragma unroll
      for (int i = 0; i < V; ++i) carry[i] = fmaf(ma[i], carry[i], mc[i]);
    }
  }

  // Scan step j of the segment is token t0 + skip + j, backwards t1 - 1 - skip - j.  A tile's n
  // steps from base are the n rows from token `low` on, row k of them being step k, backwards
  // n - 1 - k.
  const int pitch = p.d * (int)sizeof(E);
  auto low = [&](int base, int n) { return BWD ? t1 - skip - base - n : t0 + skip + base; };
  // PIECES: this lane's 16 bytes of a row, row set and row group (P row sets to a load)
  constexpr int LPR = PIECES ? Lds::ROWB / 16 : 1;
  const int piece = lane % LPR, slot = lane / LPR, dgw = slot % GW, dr = slot / GW;
  const int dc = slice * CW + piece * (16 / (int)sizeof(E));
  const bool dlive = dc < p.d;
  const unsigned dcol = (dlive ? dc : 0) * (unsigned)sizeof(E);
  const int dj = (wave * GW + dgw) * R + dr, j0 = (wave * GW + gw) * R;

  // the next tile
  uint4 pre[NT][PIECES ? R / P : 1];
  Vec<E, V> nx[R], ng[R], nh[HV ? R : 1];  // not PIECES
  auto fetch = [&](int base) {
    const int n = min(ROWS, len - base), lo = low(base, n);
    const size_t first = (row0 + lo) * p.d;
    const int back = BWD && lo > t0 ? 0 : 1;  // h_{t-1} is a row up, where the sequence has one
    if constexpr (PIECES) {
      const E *x = (const E *)p.x + first, *g = (const E *)p.g + first;
      const E *h = HV ? (const E *)p.h + first - (back ? 0 : p.d) : nullptr;
#pragma unroll
      for (int i = 0; i < R / P; ++i) {
        const int j = min(dj + i * P, n - 1), k = BWD ? n - 1 - j : j;  // past the end: the last
        const unsigned off = (unsigned)k * pitch + dcol;
        pre[0][i] = ldq<CG == 8>((const char *)x + off);
        pre[1][i] = ldq<CG == 8>((const char *)g + off);
        if constexpr (HV) pre[2][i] = ldq<CG == 8>((const char *)h + ((unsigned)max(k - back, 0) * pitch + dcol));
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int j = min(j0 + r, n - 1), k = BWD ? n - 1 - j : j;
        const size_t at = first + (size_t)k * p.d + cc;
        nx[r] = ld<E, V>((const E *)p.x + at);
        ng[r] = ld<E, V>((const E *)p.g + at);
        if constexpr (HV) nh[r] = ld<E, V>((const E *)p.h + at - (k > 0 || !back ? p.d : 0));
      }
    }
  };
  // this lane's row r of a tensor in the stage
  auto staged = [&](int t, int r) {
    return s.in[wave][t] + (r / P) * 1024 + ((r % P) * GW + gw) * Lds::ROWB + cg * V * (int)sizeof(E);
  };
  // A wave has rows in the tile from base on, but in a sequence's last tile.  The branch pays
  // where sequences may be short; in tiles of 1,024 rows, for long ones, it cost 4%.
  const int w0 = R == 8 ? 0 : wave * GW * R;
  if (w0 < len) fetch(0);

  int buf = 0;
  for (int base = 0; base < len; base += ROWS, buf ^= 1) {
    float a[R][V], A[V], C[V];
    Vec<E, V> xv[R], hv[HV ? R : 1];
    const int left = len - base - j0;
    const bool full = base + ROWS <= len;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      A[i] = 1.f;
      C[i] = 0.f;
    }
    if (R == 8 || base + w0 < len) {
      if constexpr (PIECES) {
#pragma unroll
        for (int i = 0; i < R / P; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t) *reinterpret_cast<uint4 *>(s.in[wave][t] + 1024 * i + 16 * lane) = pre[t][i];
        Vec<E, V> gv[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          __builtin_memcpy(&xv[r], __builtin_assume_aligned(staged(0, r), V * sizeof(E)), V * sizeof(E));
          __builtin_memcpy(&gv[r], __builtin_assume_aligned(staged(1, r), V * sizeof(E)), V * sizeof(E));
          if constexpr (HV) __builtin_memcpy(&hv[r], __builtin_assume_aligned(staged(2, r), V * sizeof(E)), V * sizeof(E));
        }
        if (base + ROWS + w0 < len) fetch(base + ROWS);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < V; ++i) a[r][i] = decay(Elem<E>::to_f32(gv[r].v[i]), (const E *)nullptr);
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          xv[r] = nx[r];
          if constexpr (HV) hv[r] = nh[r];
#pragma unroll
          for (int i = 0; i < V; ++i) a[r][i] = decay(Elem<E>::to_f32(ng[r].v[i]), (const E *)nullptr);
        }
        if (base + ROWS + w0 < len) fetch(base + ROWS);
      }
      if (!full) {
        // rows past the end: the identity
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (r >= left) {
              a[r][i] = 1.f;
              xv[r].v[i] = Elem<E>::from_f32(0.f);
            }
          }
      }

      // this thread's rows as one map, then all maps of the wave up to it
#pragma unroll
      for (int i = 0; i < V; ++i) {
        A[i] = a[0][i];
        C[i] = BWD ? a[0][i] * Elem<E>::to_f32(xv[0].v[i]) : Elem<E>::to_f32(xv[0].v[i]);
      }
#pragma unroll
      for (int r = 1; r < R; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float x = Elem<E>::to_f32(xv[r].v[i]);
          C[i] = BWD ? a[r][i] * (C[i] + x) : fmaf(a[r][i], C[i], x);
          A[i] *= a[r][i];
        }
      scan_step<1, V, GW>(A, C, gw);
      scan_step<2, V, GW>(A, C, gw);
      scan_step<4, V, GW>(A, C, gw);
      scan_step<8, V, GW>(A, C, gw);
    }
    if (gw == GW - 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s.map[buf][wave][0][cg * V + i] = A[i];
        s.map[buf][wave][1][cg * V + i] = C[i];
      }
    }
    lds_barrier();
    // the value before this wave; the last wave's goes on to the next tile (two buffers: a wave
    // is at most one barrier ahead of another)
    float y[V];
    if (MODE != GLR_MAPS || wave == NW - 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = base == 0 ? carry[i] : s.carry[buf][0][cg * V + i];
      if (MODE == GLR_MAPS && base > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) total[i] = s.carry[buf][1][cg * V + i];
      }
#pragma unroll
      for (int w = 0; w < NW - 1; ++w) {
        if (w < wave) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float ma = s.map[buf][w][0][cg * V + i];
            y[i] = fmaf(ma, y[i], s.map[buf][w][1][cg * V + i]);
            if (MODE == GLR_MAPS) total[i] *= ma;
          }
        }
      }
      if (wave == NW - 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          carry[i] = fmaf(A[i], y[i], C[i]);
          if (MODE == GLR_MAPS) total[i] *= A[i];
          if (gw == GW - 1) {
            s.carry[buf ^ 1][0][cg * V + i] = carry[i];
            if (MODE == GLR_MAPS) s.carry[buf ^ 1][1][cg * V + i] = total[i];
          }
        }
      }
    }
    if (MODE != GLR_MAPS && (R == 8 || base + w0 < len)) {
      // the value before this thread's rows
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = fmaf(group_shr<1, GW>(1.f, A[i], gw), y[i], group_shr<1, GW>(0.f, C[i], gw));
      const int n = min(ROWS, len - base);
      const size_t first = (row0 + low(base, n)) * p.d;
      // rows r of all lanes: through LDS into whole rows (PIECES), or each lane its own piece
      auto put = [&](E *dst, int t, int r, const float *f) {
        if constexpr (PIECES) {
          Vec<E, V> w;
#pragma unroll
          for (int i = 0; i < V; ++i) w.v[i] = Elem<E>::from_f32(f[i]);
          char *at = s.out[wave][t] + ((r % P) * GW + gw) * Lds::ROWB + cg * V * (int)sizeof(E);
          __builtin_memcpy(__builtin_assume_aligned(at, V * sizeof(E)), &w, V * sizeof(E));
          if (r % P == P - 1) {
            const uint4 q = *reinterpret_cast<const uint4 *>(s.out[wave][t] + 16 * lane);
            const int j = dj + r / P * P, k = BWD ? n - 1 - j : j;
            if (full ? dlive : dlive && j < n) stg16((char *)(dst + first) + (unsigned)k * (size_t)pitch + dcol, q);
          }
        } else {
          const int j = j0 + r, k = BWD ? n - 1 - j : j;
          if (live && r < left) st<E, V>(dst + first + (size_t)k * p.d + cc, f);
        }
      };
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float out[V], dg[V];
        if constexpr (BWD) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            out[i] = y[i] + Elem<E>::to_f32(xv[r].v[i]);
            y[i] = a[r][i] * out[i];
            dg[i] = y[i] * Elem<E>::to_f32(hv[r].v[i]);
          }
          if (skip + base + j0 + r + 1 == len_seq) {  // the sequence's first token: h_{t-1} = h0
#pragma unroll
            for (int i = 0; i < V; ++i) dg[i] = y[i] * (p.h0 ? p.h0[sh + i] : 0.f);
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            y[i] = fmaf(a[r][i], y[i], Elem<E>::to_f32(xv[r].v[i]));
            out[i] = y[i];
          }
        }
        put((E *)p.o, 0, r, out);
        if constexpr (BWD) put((E *)p.dg, 1, r, dg);
      }
    }
  }
  if (!live || wave != NW - 1 || gw != GW - 1) return;
  // where there was no token, carry is what the segment started from
  if (MODE == GLR_MAPS) {
    float *m = p.maps + mrow + (size_t)seg * 2 * p.d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      m[i] = total[i];
      m[p.d + i] = carry[i];
    }
  } else if (p.yend && last_seg) {
#pragma unroll
    for (int i = 0; i < V; ++i) p.yend[sh + i] = carry[i];
  }
}

// One token of N sequences: N * H * d independent channels.
template <typename E, int V>
__global__ __launch_bounds__(256) void kla_glr_step_kernel(const E *__restrict__ x, const E *__restrict__ g,
                                                           float *__restrict__ state, E *__restrict__ o, size_t n) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (i >= n) return;  // V divides n
  const Vec<E, V> xv = ld<E, V>(x + i), gv = ld<E, V>(g + i);
  float h[V];
  if constexpr (V >= 4) {
#pragma unroll
    for (int j = 0; j < V; j += 4) *reinterpret_cast<f32x4 *>(h + j) = *reinterpret_cast<const f32x4 *>(state + i + j);
  } else {
    h[0] = state[i];
  }
#pragma unroll
  for (int j = 0; j < V; ++j) h[j] = fmaf(decay(Elem<E>::to_f32(gv.v[j]), (const E *)nullptr), h[j], Elem<E>::to_f32(xv.v[j]));
  if constexpr (V >= 4) {
#pragma unroll
    for (int j = 0; j < V; j += 4) *reinterpret_cast<f32x4 *>(state + i + j) = *reinterpret_cast<f32x4 *>(h + j);
  } else {
    state[i] = h[0];
  }
  st<E, V>(o + i, h);
}

template <typename E, int V, int NW, int R, bool BWD, bool PIECES, int CG = 4>
struct GlrShape {
  static constexpr int CW = CG * V;
  static constexpr int INNER = 128 / (CW * (int)sizeof(E)) > 1 ? 128 / (CW * (int)sizeof(E)) : 1;
  template <int MODE>
  static void go(GlrParams p, long long segs, hipStream_t st) {
    p.nseg = (int)segs;
    p.inner = INNER;
    p.lines = (p.d + CW * p.inner - 1) / (CW * p.inner);
    const long long units = (long long)p.N * p.H * p.lines * segs;
    const long long grid = (units + 7) / 8 * 8 * p.inner;
    hipLaunchKernelGGL((kla_glr_kernel<E, V, NW, R, BWD, MODE, PIECES, CG>), dim3((unsigned)grid), dim3(64 * NW), 0, st, p);
  }
  static hipError_t whole(const GlrParams &p, hipStream_t st) {
    go<GLR_WHOLE>(p, 1, st);
    return hipGetLastError();
  }
  static hipError_t launch(const GlrParams &p, long long segs, hipStream_t st) {
    if (segs <= 1) {
      go<GLR_WHOLE>(p, 1, st);
    } else {
      go<GLR_MAPS>(p, segs - 1, st);  // the last segment's map is not needed
      go<GLR_CARRIED>(p, segs, st);
    }
    return hipGetLastError();
  }
};

// How a call runs: slices of 64 or 32 bytes of a row, sequences whole or in segments.
//
// A CU keeps a limited number of lines in flight (about 21 GB/s where it takes 64 bytes of
// each, half that at 32), so it takes all 256 CUs to fill HBM's rate.  Slices of 64 bytes where
// they make 256 workgroups (8,192 channels, T = 4096: 46 us against 59 with 32 bytes); slices
// of 32 where that makes them 256 (4,096 channels, T = 65536: 442 us against 595, and 575 with
// segments, which read x and g twice); segments below (2,048 channels, T = 32768: 148 us
// against 181 with 32 bytes and 273 whole; 256 channels, T = 65536: 44 against 222 and 444).
// Short sequences do not pay for a second pass (512 channels, 3,000 tokens: 15 us with 32
// bytes, 19 with segments), nor for tiles of 1,024 rows (5,000 channels, 1,500 tokens: 19 us
// whole, 25 with 32 bytes).
//
// Slices of a whole line (8 channel groups for 4, a wave's rows half as many) where they fill the
// CUs: no other workgroup wants their lines, which then go past the caches.  A workgroup takes
// most of a CU's LDS, so the last round must not be much emptier than the others: dense batches
// whose lines fill five sixths of their rounds (128 sequences and heads of d=128, T=4096: backward
// 120 us against 148 with 64 bytes, 256 forward 143 against 174, in fp32 138 against 197; 192:
// 136 against 129), packed ones from 640 lines on (20 of 300 to 3,000 tokens, 16 heads: 55 us
// against 69; 16 of 512 to 16,384 tokens 171 against 139).
//
// Tiles fit the longest sequence: one wave's 64 rows, four waves' 256 or eight waves' 512 (19
// sequences of 2 to 7 tokens, 16 heads of 2,560 channels: 37 us against 393 with 512 rows).
struct GlrPlan {
  bool pieces, narrow, line;
  int waves;
  int segs, seg_rows;
};

GlrPlan glr_plan(const GlrArgs &a) {
  const int e = a.dtype == 0 ? 2 : 4;
  // rows of 16-byte pieces whose tile offsets fit 32 bits; others element by element
  const bool pieces = a.d * (long long)e % 16 == 0 && (long long)a.d * e <= (1 << 20);
  const int V = pieces ? 16 / e : (a.d % (8 / e) == 0 ? 8 / e : 1);
  const long long wide = (long long)a.num_seqs * a.H * ((a.d + 4 * V - 1) / (4 * V));
  GlrPlan r{pieces, false, false, a.longest <= 64 ? 1 : (a.longest <= 256 ? 4 : 8), 1, 0};
  const long long lines = (long long)a.num_seqs * a.H * a.d * e / 128;
  r.line = pieces && (long long)a.d * e % 128 == 0 && r.waves == 8 &&
           (a.cu_seqlens ? lines >= 640 : lines >= 256 && (lines + 255) / 256 * 256 * 5 <= lines * 6);
  if (r.line) return r;
  if (wide == 0 || wide >= 256 || a.longest <= 2048) return r;
  if (pieces && (wide >= 128 || a.longest <= 3584)) {
    r.narrow = true;
    return r;
  }
  const long long want = std::min<long long>((256 + wide - 1) / wide, (a.longest + 511) / 512);
  const long long rows = ((a.longest + want - 1) / want + 511) / 512 * 512;
  r.seg_rows = (int)rows;
  r.segs = (int)((a.longest + rows - 1) / rows);
  return r;
}

template <typename E, int V, bool BWD, bool PIECES>
hipError_t launch_glr_v(const GlrParams &p, const GlrPlan &plan, hipStream_t st) {
  if (plan.waves == 1) return GlrShape<E, V, 1, 4, BWD, PIECES>::whole(p, st);
  if (plan.waves == 4) return GlrShape<E, V, 4, 4, BWD, PIECES>::whole(p, st);
  return GlrShape<E, V, 8, 4, BWD, PIECES>::launch(p, plan.segs, st);
}

template <typename E, bool BWD>
hipError_t launch_glr(const GlrParams &p, const GlrPlan &plan, hipStream_t st) {
  constexpr int V = 16 / sizeof(E);
  if (plan.line) return GlrShape<E, V, 8, 4, BWD, true, 8>::whole(p, st);
  if (plan.narrow) return GlrShape<E, V / 2, 8, 8, BWD, true>::whole(p, st);
  if (plan.pieces) return launch_glr_v<E, V, BWD, true>(p, plan, st);
  if (p.d % (V / 2) == 0) return launch_glr_v<E, V / 2, BWD, false>(p, plan, st);
  return launch_glr_v<E, 1, BWD, false>(p, plan, st);
}

}  // namespace

bool glr_grid_fits(const GlrArgs &a) {
  const GlrPlan plan = glr_plan(a);
  const int e = a.dtype == 0 ? 2 : 4, V = plan.pieces ? (plan.narrow ? 8 : 16) / e : (a.d % (8 / e) == 0 ? 8 / e : 1);
  const int inner = plan.line ? 1 : std::max(1, 128 / (4 * V * e)), lines = (a.d - 1) / ((plan.line ? 8 : 4) * V * inner) + 1;
  return launch_fits(((double)a.num_seqs * a.H * lines * plan.segs + 7) * inner, 64 * plan.waves);
}

size_t glr_workspace_bytes(const GlrArgs &a) {
  const long long segs = glr_plan(a).segs;
  return segs <= 1 ? 0 : (size_t)a.num_seqs * a.H * segs * 2 * a.d * sizeof(float);
}

hipError_t launch_glr_chunk(const GlrArgs &a, bool bwd, hipStream_t st) {
  const GlrPlan plan = glr_plan(a);
  GlrParams p{};
  p.x = a.x;
  p.g = a.g;
  p.h = a.h;
  p.y0 = a.y0;
  p.h0 = a.h0;
  p.o = a.o;
  p.dg = a.dg;
  p.yend = a.yend;
  p.cu = a.cu_seqlens;
  p.N = a.num_seqs;
  p.H = a.H;
  p.T = a.T;
  p.d = a.d;
  p.segs = plan.segs;
  p.seg_rows = plan.seg_rows;
  p.maps = (float *)a.workspace;
  // Packed sequences of several tiles start in the order of their lengths, the longest first (32
  // of 512 to 16,384 tokens, 16 heads of d=128, backward: 564 us against 627 as they come).  The
  // order is the host's lengths'; other lengths on the device cost time alone.
  p.ordered = a.cu_seqlens && a.num_seqs > 1 && a.num_seqs <= GLR_ORDER && plan.waves == 8 && plan.segs == 1;
  if (p.ordered) {
    for (int n = 0; n < a.num_seqs; ++n) p.order[n] = n;
    const int32_t *cu = a.cu_seqlens_host;
    std::stable_sort(p.order, p.order + a.num_seqs, [cu](int i, int j) { return cu[i + 1] - cu[i] > cu[j + 1] - cu[j]; });
  }
  if (a.dtype == 0) return bwd ? launch_glr<bf16, true>(p, plan, st) : launch_glr<bf16, false>(p, plan, st);
  return bwd ? launch_glr<float, true>(p, plan, st) : launch_glr<float, false>(p, plan, st);
}

bool glr_step_fits(size_t n, int dtype) {
  const int V = dtype == 0 ? 8 : 4;
  return launch_fits((double)n / (n % V == 0 ? V : 1) / 256 + 1, 256);
}

template <typename E>
static hipError_t launch_step(const void *x, const void *g, float *state, void *o, size_t n, hipStream_t st) {
  constexpr int V = 16 / sizeof(E);
  if (n % V == 0)
    hipLaunchKernelGGL((kla_glr_step_kernel<E, V>), dim3((unsigned)((n / V + 255) / 256)), dim3(256), 0, st, (const E *)x,
                       (const E *)g, state, (E *)o, n);
  else
    hipLaunchKernelGGL((kla_glr_step_kernel<E, 1>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, (const E *)x,
                       (const E *)g, state, (E *)o, n);
  return hipGetLastError();
}

hipError_t launch_glr_step(const void *x, const void *g, float *state, void *o, size_t n, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_step<bf16>(x, g, state, o, n, st) : launch_step<float>(x, g, state, o, n, st);
}

}  // namespace kla
