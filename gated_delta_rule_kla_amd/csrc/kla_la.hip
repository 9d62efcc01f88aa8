// kla_la.hip -- linear attention with a decay per head (gfx950): prompts, gradients, single tokens.
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t      (include/kla.h, kla_la_chunk_fwd)
//
// In chunks of C tokens, with c_t the sum of the chunk's log-decays up to token t, S the state at
// the chunk's start and tot = c_{C-1}:
//
//   o_t = exp(c_t) S^T q_t + sum_{s <= t} exp(c_t - c_s) (q_t . k_s) v_s
//   S'  = exp(tot) S + sum_s exp(tot - c_s) k_s v_s^T
//
// Log-decays are summed in 64 bits and kept as two floats in base two, so that c_t - c_s is as
// exact behind a token that forgets everything (g = -inf counts as 2^-65536) as elsewhere.
// Operands of the products are in the element type: the scores and the state (where outputs are
// read from it) are rounded to it once, as the outputs are; the state itself is fp32, and the
// scaled v_s that enter it are three bf16 terms (24 bits), since a final state is fp32 as well.
//
// Backward, with M the gradient of the state at a chunk's end (dL/dS_final at the last):
//
//   dq_t = exp(c_t) S do_t + sum_{s <= t} D_ts (do_t . v_s) k_s        D_ts = exp(c_t - c_s)
//   dk_s = exp(tot - c_s) M v_s + sum_{t >= s} D_ts (do_t . v_s) q_t
//   dv_s = exp(tot - c_s) M^T k_s + sum_{t >= s} D_ts (q_t . k_s) do_t
//   M'   = exp(tot) M + sum_t exp(c_t) q_t do_t^T                      (at the chunk's start)
//   dg_t = what passes token t: from the writes before it to the reads from it on,
//          sum_{i >= t > j} D_ij (q_i . k_j)(do_i . v_j) + sum_{i >= t} (the state's part of q_i . dq_i)
//          + sum_{j < t} (the later chunks' part of k_j . dk_j) + exp(tot) <M, S>
//
// The S and M of the chunks are kept in fp16 with powers of two, and rounded on to bf16 for the
// products; <M, S>, which is most of dg where decays are weak, takes the fp16 values: from bf16
// ones dg was off by 1.8 times what its own rounding to bf16 makes (16 heads, 26,339 tokens).
//
// (in dg every term is a sum of products that belong to it; the shorter form, q . dq - k . dk
// summed from t to the sequence's end, loses what the terms have in common, and with operands of
// eight bits little is left of it).
#include <algorithm>
#include <type_traits>

#include "kla_common.h"
#include "kla_internal.h"
#include "kla_ops.h"

namespace kla {

namespace {

constexpr int LA_NV = 32;         // state columns of the smaller slices
constexpr float LA_FORGET = -65536.f;  // log2 of the smallest decay

// Chunks and operands by element type.  A 16-byte operand holds VL contraction values of a row
// (or column), four of them (KG values) make a product.
template <typename E> struct La;
template <> struct La<bf16> {
  static constexpr int C = 64, KG = 32, VL = 8, TERMS = 3;
  typedef bf16x8 Op;
  typedef _Float16 Stored;
  static __device__ __forceinline__ void store(_Float16 *p, f32x4 v, float unit) {
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<f16x4 *>(p) =
        f16x4{(_Float16)(v[0] * unit), (_Float16)(v[1] * unit), (_Float16)(v[2] * unit), (_Float16)(v[3] * unit)};
  }
  static __device__ __forceinline__ Op nat(const bf16 *row, int kb, int g) {
    return *reinterpret_cast<const bf16x8 *>(row + kb + 8 * g);
  }
  static __device__ __forceinline__ Op grp(const bf16 *row, int kb, int g) { return Ops<bf16>::ldg_grp(row, kb, g); }
  // column c16 + (lane & 15) of rows kb .. kb + 31, in the order of accumulator tiles
  static __device__ __forceinline__ Op tr(const bf16 *M, int ld, int kb, int c16, int lane) {
    const int g = lane >> 4, x = (lane >> 2) & 3, a = lane & 3;
    const bf16 *p = M + (kb + 4 * g + x) * ld + c16 + 4 * a;
    const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)p);
    const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)(p + 16 * ld));
    return Op{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }
  static __device__ __forceinline__ Op cvt(uint4 v) { return __builtin_bit_cast(Op, v); }
};
template <> struct La<float> {
  static constexpr int C = 32, KG = 16, VL = 4, TERMS = 1;
  typedef f32x4 Op;
  typedef float Stored;
  static __device__ __forceinline__ void store(float *p, f32x4 v, float) { *reinterpret_cast<f32x4 *>(p) = v; }
  static __device__ __forceinline__ Op nat(const float *row, int kb, int g) {
    return *reinterpret_cast<const f32x4 *>(row + kb + 4 * g);
  }
  static __device__ __forceinline__ Op grp(const float *row, int kb, int g) { return nat(row, kb, g); }
  static __device__ __forceinline__ Op tr(const float *M, int ld, int kb, int c16, int lane) {
    const float *p = M + (kb + 4 * (lane >> 4)) * ld + c16 + (lane & 15);
    return Op{p[0], p[ld], p[2 * ld], p[3 * ld]};
  }
  static __device__ __forceinline__ Op cvt(uint4 v) { return __builtin_bit_cast(Op, v); }
};

// four consecutive elements of a row as fp32
__device__ __forceinline__ f32x4 load4(const bf16 *p) {
  const bf16x4 v = *reinterpret_cast<const bf16x4 *>(p);
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

// Inclusive prefix sum of doubles over the lanes of a wave (row shifts, then the rows' totals).
template <int CTRL>
__device__ __forceinline__ double dpp_shr(double v) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
  const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, 0xF, 0xF, false);
  const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
__device__ __forceinline__ double lane_double(double v, int src) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
  const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)u, src);
  const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(u >> 32), src);
  return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
// *rest: what the sum over the lane's row of 16 still adds behind it
__device__ __forceinline__ double scan_double(double v, double *rest) {
  v += dpp_shr<0x111>(v);
  v += dpp_shr<0x112>(v);
  v += dpp_shr<0x114>(v);
  v += dpp_shr<0x118>(v);
  const double r0 = lane_double(v, 15), r1 = lane_double(v, 31), r2 = lane_double(v, 47), r3 = lane_double(v, 63);
  const int row = (threadIdx.x & 63) >> 4;
  *rest = (row == 0 ? r0 : row == 1 ? r1 : row == 2 ? r2 : r3) - v;
  return v + ((row >= 1 ? r0 : 0.0) + (row >= 2 ? r1 : 0.0) + (row >= 3 ? r2 : 0.0));
}

// A chunk's decays: c_t in base two as hi + lo, exp(c_t), exp(tot - c_t), the decay from a token
// to the last of its 16, exp(tot), tot.
template <int C>
struct Decays {
  float hi[C], lo[C], out[C], left[C], near[C];
  float all;
  double tot;
};

// by one wave; g: the lane's log-decay (0 past the chunk's tokens)
template <int C>
__device__ __forceinline__ void scan_decays(Decays<C> *d, float g) {
  const int lane = threadIdx.x & 63;
  double x = (double)g * 1.4426950408889634, rest;
  x = x < LA_FORGET ? LA_FORGET : x;  // a NaN stays
  if (lane >= C) x = 0.0;
  const double c = scan_double(x, &rest), tot = lane_double(c, 63);
  if (lane < C) {
    const float hi = (float)c;
    d->hi[lane] = hi;
    d->lo[lane] = (float)(c - (double)hi);
    d->out[lane] = __builtin_amdgcn_exp2f((float)c);
    d->left[lane] = __builtin_amdgcn_exp2f((float)(tot - c));
    d->near[lane] = __builtin_amdgcn_exp2f((float)rest);
  }
  if (lane == 0) {
    d->all = __builtin_amdgcn_exp2f((float)tot);
    d->tot = tot;
  }
}

// The largest of a wave's numbers, in all lanes.
__device__ __forceinline__ unsigned wave_max(unsigned v) {
  auto step = [&](auto ctrl) { v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF, false)); };
  step(std::integral_constant<int, 0x111>{});
  step(std::integral_constant<int, 0x112>{});
  step(std::integral_constant<int, 0x114>{});
  step(std::integral_constant<int, 0x118>{});
  const unsigned a = max((unsigned)__builtin_amdgcn_readlane((int)v, 15), (unsigned)__builtin_amdgcn_readlane((int)v, 31));
  const unsigned b = max((unsigned)__builtin_amdgcn_readlane((int)v, 47), (unsigned)__builtin_amdgcn_readlane((int)v, 63));
  return max(a, b);
}

// One direction of a scan: the factors of the state's updates (k, v; reverse: q, dout), the state
// at the first processed chunk and behind the last.
struct LaDir {
  const void *x, *y;
  const float *s0;  // or nullptr
  float *send;      // or nullptr
  void *states;     // [H, slots, dv, dk] fp32, or fp16 for bf16 elements
  float *units;     // [H, slots, slices, 4] of the fp16 states: a power of two to each slice and wave
  float *seg_s;     // [N H segs, dk, dv] states behind all segments but the last; in the last's
                    // place the initial state (final_state may be the same memory)
  double *seg_g;    // [N H segs] log2 of their decays
};

struct LaParams {
  LaDir dir[2];               // forward, reverse
  const void *q, *g;
  const float *gfix;          // [H] log-decays in place of g, or nullptr
  void *o;
  const int32_t *cu;          // device offsets, or nullptr
  int N, H, T, dk, dv;
  int slices, segs, seg_chunks;
  unsigned half;              // workgroups of a direction
  int slots;                  // chunk slots of a head (states)
};

// Sequence n: its first row among a head's, its length, and its first slot of C tokens.
__device__ __forceinline__ void la_span(const int32_t *cu, int n, int T, int C, int *t0, int *len, int *slot0) {
  if (!cu) {
    *t0 = 0, *len = T, *slot0 = n * ((T + C - 1) / C);
    return;
  }
  const int a = min(max(cu[n], 0), T), z = min(max(cu[n + 1], a), T);
  *t0 = a, *len = z - a, *slot0 = a / C + n;
}

// The scan over a sequence's chunks.  A workgroup holds NV columns of the state.  Four waves
// own the state, a quarter of its rows each, in fp32: they bring x and y to LDS a chunk ahead of
// their use (from registers that hold the chunks after that), with y's scaled copy, update the
// state, and leave a copy of it in the element type in LDS.  Beside them four waves compute the
// outputs from those copies, 16 rows each (fp32, 32 tokens to a chunk: half of the columns);
// the first, which has the fewest scores, also sums the decays of the chunk after next.  One
// barrier per chunk.  B=4 H=16 T=4096 dk=dv=128: 90 to 107 us; H=16 T=65536 dv=256, in segments of
// 256 chunks with the pass for their ends: 825 to 840 us (1.9 TB/s).
// Bound: a chunk's chain, 1.5 us: LDS takes 1,370 cycles of it (the state's operands of every wave),
// and the vector ALU, matrix products and the exchange behind the barrier hide little of each other
// with one workgroup to a CU.
//
// OUT: outputs and the final state.  ENDS: a segment's end state only, where few sequences leave
// CUs idle and are cut: all segments but the last are scanned once for that, and the other modes
// start each from those before it.  STORE: the state at every chunk's start, and of the
// reverse direction the state's gradient at its end, for the gradients.
enum { LA_OUT, LA_ENDS, LA_STORE };
constexpr int la_threads(int mode) { return mode == LA_OUT ? 512 : 320; }

template <typename E, int DK, int MODE, int NV>
__global__ __launch_bounds__(la_threads(MODE)) void kla_la_scan_kernel(LaParams p) {
  using L = La<E>;
  using Op = typename L::Op;
  constexpr int C = L::C, KG = L::KG, VL = L::VL;
  constexpr int PAD = LdsPad<E>::V, LDX = DK + PAD, LDY = NV + PAD;
  constexpr int XP = C * DK / VL / 256, YP = C * NV / VL / 256;  // 16-byte pieces of a thread
  constexpr int RT = DK / 64;                                  // row tiles of a wave
  constexpr int NC = NV / 16, NS = C / 16, CT = NC * NS / 4;   // column tiles, strips, a wave's output tiles
  constexpr int KS = DK / KG;
  constexpr int AHEAD = 3;  // chunks that loads run ahead
  static_assert(XP * 256 * VL == C * DK && YP * 256 * VL == C * NV && CT * 4 == NC * NS, "tiles");
  __shared__ __attribute__((aligned(16))) E s_x[2][C * LDX];
  __shared__ __attribute__((aligned(16))) E s_y[MODE == LA_OUT ? 2 : 1][MODE == LA_OUT ? C * LDY : 8];
  __shared__ __attribute__((aligned(16))) E s_w[2][L::TERMS][C * LDY];  // y scaled
  __shared__ __attribute__((aligned(16))) E s_s[MODE == LA_OUT ? 2 : 1][MODE == LA_OUT ? NV * LDX : 8];  // S^T
  __shared__ Decays<C> s_d[3];

  const bool rev = MODE != LA_OUT && blockIdx.x >= p.half;
  const LaDir &dir = p.dir[rev];
  // workgroup ids go round the eight XCDs: the slices of a sequence and head, which read the
  // same rows, stay on one
  const unsigned id = blockIdx.x - (rev ? p.half : 0), rest = id >> 3;
  const int slice = rest % p.slices;
  const long long pair = (long long)(rest / p.slices) * 8 + (id & 7);
  if (pair >= (long long)p.N * p.H * p.segs) return;
  const int seg = pair % p.segs;
  const long long nh = pair / p.segs;
  const int n = nh / p.H, h = nh % p.H;
  int t0, len, slot0;
  la_span(p.cu, n, p.T, C, &t0, &len, &slot0);
  const int nch = (len + C - 1) / C;
  // the chunks in processed order
  const int c0 = seg * p.seg_chunks, c1 = seg == p.segs - 1 ? nch : min(nch, c0 + p.seg_chunks);
  if (seg > 0 && c0 >= nch) return;
  if (MODE == LA_ENDS && c1 >= nch) return;
  const size_t row0 = ((size_t)(p.cu ? 0 : n) * p.H + h) * p.T + t0;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, li = lane & 15;
  const int col0 = slice * NV;
  auto first_token = [&](int j) { return (rev ? nch - 1 - j : j) * C; };
  // loads ahead go past the last chunk as loads of it: under a condition the compiler would wait
  // for them where they are issued
  auto within = [&](int j) { return min(j, c1 - 1); };

  if (wave >= 4) {  // decays and outputs
    const int strip = (wave - 4) % NS, ct0 = (wave - 4) / NS * CT;
    if (c0 >= c1) return;
    const float fixed = p.gfix ? p.gfix[h] : 0.f;
    const E *const gp = p.gfix ? (const E *)p.q : (const E *)p.g + row0;
    auto load_g = [&](int j) {  // the lane's log-decay as it stands in memory (0 past the end)
      const int t = first_token(j);
      const __amdgpu_buffer_rsrc_t r = buffer_rsrc(gp + t, p.gfix ? 0 : min(C, len - t) * (int)sizeof(E));
      return (unsigned)buffer_ld_elem(r, lane, gp);
    };
    auto decay = [&](unsigned u, int j) {
      asm volatile("" : "+v"(u));  // not where the load is issued, which would wait for it
      if (p.gfix) return lane < len - first_token(j) ? fixed : 0.f;
      if constexpr (sizeof(E) == 2) return elem_bits_to_f32((unsigned short)u);
      else return elem_bits_to_f32(u);
    };
    typedef Op Query[MODE == LA_OUT ? KS : 1];
    const E *const qp = (const E *)p.q + row0 * p.dk;
    auto load_q = [&](Query &q, int j) {
      if constexpr (MODE == LA_OUT) {
        const int t = first_token(j), rows = min(C, len - t);
        const __amdgpu_buffer_rsrc_t rq = buffer_rsrc(qp + (size_t)t * p.dk, rows * p.dk * (int)sizeof(E));
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int c = k * KG + VL * g;
          q[k] = L::cvt(buffer_ld16(rq, c < p.dk ? ((16 * strip + li) * p.dk + c) * (int)sizeof(E) : 0x40000000));
        }
      }
    };
    unsigned gn[AHEAD];
    Query qs[AHEAD];
    const unsigned g0 = load_g(c0), g1 = load_g(within(c0 + 1));
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) gn[i] = load_g(within(c0 + 2 + i));
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load_q(qs[i], within(c0 + i));
    if (wave == 4) {
      scan_decays<C>(&s_d[c0 % 3], decay(g0, c0));
      scan_decays<C>(&s_d[(c0 + 1) % 3], decay(g1, within(c0 + 1)));
    }
    lds_barrier();
    // A strip's code is its own: its scores and their keys are as many as its number says, and in
    // one run of instructions.
    auto run = [&](auto which) {
      constexpr int ST = decltype(which)::value;
      auto step = [&](int j, Query &q, unsigned &gj) {  // gj: the decay of chunk j + 2
        lds_barrier();
        if (ST == 0 && wave == 4) {
          const float x = decay(gj, within(j + 2));
          gj = load_g(within(j + 2 + AHEAD));
          scan_decays<C>(&s_d[(j + 2) % 3], x);  // behind the last chunk: nobody reads it
        }
        if constexpr (MODE == LA_OUT) {
          const E *const X = s_x[j & 1], *const Y = s_y[j & 1], *const S = s_s[j & 1];
          const Decays<C> &d = s_d[j % 3];
          // P^T: keys 16 kt + 4 g + e against the strip's query li
          f32x4 pt[NS];
#pragma unroll
          for (int kt = 0; kt < NS; ++kt) {
            pt[kt] = zero4();
            if (kt > ST) continue;
#pragma unroll
            for (int k = 0; k < KS; ++k)
              pt[kt] = Ops<E>::mma_grp(L::nat(X + (16 * kt + li) * LDX, k * KG, g), q[k], pt[kt]);
          }
          f32x4 o[CT];  // o^T: columns 4 g + e of query li
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            o[c] = zero4();
#pragma unroll
            for (int k = 0; k < KS; ++k)
              o[c] = Ops<E>::mma_grp(L::nat(S + (16 * (ct0 + c) + li) * LDX, k * KG, g), q[k], o[c]);
          }
          load_q(q, within(j + AHEAD));
          // earlier keys: the decay to the end of their 16, and from there
          const float th = d.hi[16 * ST + li], tl = d.lo[16 * ST + li], f = d.out[16 * ST + li];
#pragma unroll
          for (int kt = 0; kt < ST; ++kt) {
            const f32x4 near = *reinterpret_cast<const f32x4 *>(&d.near[16 * kt + 4 * g]);
            const float far = __builtin_amdgcn_exp2f((th - d.hi[16 * kt + 15]) + (tl - d.lo[16 * kt + 15]));
#pragma unroll
            for (int e = 0; e < 4; ++e) pt[kt][e] *= near[e] * far;
          }
          {
            const f32x4 sh = *reinterpret_cast<const f32x4 *>(&d.hi[16 * ST + 4 * g]);
            const f32x4 sl = *reinterpret_cast<const f32x4 *>(&d.lo[16 * ST + 4 * g]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              pt[ST][e] = 4 * g + e <= li ? pt[ST][e] * __builtin_amdgcn_exp2f((th - sh[e]) + (tl - sl[e])) : 0.f;
          }
#pragma unroll
          for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[c][e] *= f;
#pragma unroll
          for (int kb = 0; kb < C; kb += KG) {
            if (kb / 16 > ST) continue;
            const Op w = Ops<E>::b_from_d(&pt[kb / 16]);
#pragma unroll
            for (int c = 0; c < CT; ++c)
              o[c] = Ops<E>::mma_grp(L::tr(Y, LDY, kb, 16 * (ct0 + c), lane), w, o[c]);
          }
          const int t = first_token(j) + 16 * ST + li;
          if (t < len) {
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              const int col = col0 + 16 * (ct0 + c) + 4 * g;
              if (col < p.dv) store4((E *)p.o + (row0 + t) * p.dv + col, o[c]);
            }
          }
        }
      };
      int j = c0;
      for (; j + AHEAD <= c1; j += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) step(j + i, qs[i], gn[i]);
      }
#pragma unroll
      for (int i = 0; i < AHEAD - 1; ++i)
        if (j + i < c1) step(j + i, qs[i], gn[i]);
    };
    if (strip == 0) run(std::integral_constant<int, 0>{});
    else if (strip == 1) run(std::integral_constant<int, 1>{});
    if constexpr (NS > 2) {
      if (strip == 2) run(std::integral_constant<int, 2>{});
      else if (strip == 3) run(std::integral_constant<int, 3>{});
    }
    return;
  }

  // the state
  const int tid = threadIdx.x;
  struct Rows {
    u32x4 x[XP], y[YP];
  } ahead[AHEAD];
  const E *const xp = (const E *)(rev ? p.dir[1].x : p.dir[0].x) + row0 * p.dk;
  const E *const yp = (const E *)(rev ? p.dir[1].y : p.dir[0].y) + row0 * p.dv;
  auto load = [&](Rows &to, int j) {
    const int t = first_token(j), rows = min(C, len - t);
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(xp + (size_t)t * p.dk, rows * p.dk * (int)sizeof(E));
    const __amdgpu_buffer_rsrc_t ry = buffer_rsrc(yp + (size_t)t * p.dv, rows * p.dv * (int)sizeof(E));
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int pc = tid + 256 * i, r = pc / (DK / VL), c = pc % (DK / VL) * VL;
      to.x[i] = __builtin_bit_cast(u32x4, buffer_ld16(rx, c < p.dk ? (r * p.dk + c) * (int)sizeof(E) : 0x40000000));
    }
#pragma unroll
    for (int i = 0; i < YP; ++i) {
      const int pc = tid + 256 * i, r = pc / (NV / VL), c = col0 + pc % (NV / VL) * VL;
      to.y[i] = __builtin_bit_cast(u32x4, buffer_ld16(ry, c < p.dv ? (r * p.dv + c) * (int)sizeof(E) : 0x40000000));
    }
  };
  typedef float Scale[YP];
  auto scales = [&](int j, Scale &f) {  // y's, of chunk j
    const Decays<C> &d = s_d[j % 3];
#pragma unroll
    for (int i = 0; i < YP; ++i) f[i] = (rev ? d.out : d.left)[(tid + 256 * i) / (NV / VL)];
  };
  auto put = [&](const Rows &from, int j, const Scale &f) {  // chunk j's rows from registers
    E *const dx = s_x[j & 1];
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int pc = tid + 256 * i;
      *reinterpret_cast<u32x4 *>(dx + pc / (DK / VL) * LDX + pc % (DK / VL) * VL) = from.x[i];
    }
#pragma unroll
    for (int i = 0; i < YP; ++i) {
      const int pc = tid + 256 * i, r = pc / (NV / VL), at = r * LDY + pc % (NV / VL) * VL;
      E e[VL], w[L::TERMS][VL];
      u32x4 y = from.y[i];
      // taken apart here: the compiler would do so, and wait for the load, where it is issued
      asm volatile("" : "+v"(y));
      __builtin_memcpy(e, &y, 16);
      if constexpr (MODE == LA_OUT) *reinterpret_cast<u32x4 *>(s_y[j & 1] + at) = y;
#pragma unroll
      for (int u = 0; u < VL; ++u) {
        float v = Elem<E>::to_f32(e[u]) * f[i];
#pragma unroll
        for (int k = 0; k < L::TERMS; ++k) {
          w[k][u] = Elem<E>::from_f32(v);
          v -= Elem<E>::to_f32(w[k][u]);
        }
      }
#pragma unroll
      for (int k = 0; k < L::TERMS; ++k) {
        uint4 v;
        __builtin_memcpy(&v, w[k], 16);
        *reinterpret_cast<uint4 *>(s_w[j & 1][k] + at) = v;
      }
    }
  };

  // this wave's rows of the state: tile i, element e is row 16 (wave RT + i) + 4 g + e
  f32x4 acc[RT][NC];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[i][c] = zero4();
  auto each = [&](auto f) {  // element = f(element, offset in a [dk, dv] state)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * (wave * RT + i) + 4 * g + e, col = col0 + 16 * c + li;
          if (r < p.dk && col < p.dv) acc[i][c][e] = f(acc[i][c][e], (size_t)r * p.dv + col);
        }
  };
  const size_t ssize = (size_t)p.dk * p.dv;
  if (c0 < c1) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(ahead[i], within(c0 + i));
  }
  if (seg == 0) {
    const bool copied = MODE != LA_ENDS && p.segs > 1 && c1 < nch;
    const float *s0 = dir.s0 ? (copied ? dir.seg_s + (nh * p.segs + p.segs - 1) * ssize : dir.s0 + nh * ssize) : nullptr;
    if (s0) each([&](float, size_t at) { return s0[at]; });
    if (MODE == LA_ENDS && s0) {
      float *const copy = dir.seg_s + (nh * p.segs + p.segs - 1) * ssize;
      each([&](float a, size_t at) { return copy[at] = a; });
    }
  } else if (MODE != LA_ENDS) {
    for (int i = 0; i < seg; ++i) {  // the segments before this one, in order
      const float f = __builtin_amdgcn_exp2f((float)dir.seg_g[nh * p.segs + i]);
      const float *const d = dir.seg_s + (nh * p.segs + i) * ssize;
      each([&](float a, size_t at) { return (i ? f * a : 0.f) + d[at]; });
    }
  }
  auto publish = [&](int j) {  // the state in front of chunk j
    if constexpr (MODE == LA_OUT) {
      E *const d = s_s[j & 1];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) store4(d + (16 * c + li) * LDX + 16 * (wave * RT + i) + 4 * g, acc[i][c]);
    }
    if constexpr (MODE == LA_STORE) {
      const size_t place = (size_t)h * p.slots + slot0 + first_token(j) / C;
      typedef typename L::Stored St;
      St *const to = (St *)dir.states + place * ssize;
      float unit = 1.f;
      if constexpr (sizeof(E) == 2) {  // the largest finite magnitude becomes 2^14 to 2^15
        unsigned top = 0;
        auto largest = [&](bool finite) {
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float x = acc[i][c][e];
                const unsigned b = __builtin_bit_cast(unsigned, x) & 0x7fffffffu;
                top = max(top, finite && b >= 0x7f800000u ? 0u : b);
              }
          top = wave_max(top);
        };
        largest(false);
        if (top >= 0x7f800000u) {
          top = 0;
          largest(true);
        }
        const unsigned x = min(268u - (top >> 23), 253u);
        unit = __builtin_bit_cast(float, x << 23);
        if (lane == 0) dir.units[(place * p.slices + slice) * 4 + wave] = __builtin_bit_cast(float, (254u - x) << 23);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int r = 16 * (wave * RT + i) + 4 * g, col = col0 + 16 * c + li;
          if (r < p.dk && col < p.dv) L::store(to + (size_t)col * p.dk + r, acc[i][c], unit);
        }
    }
  };
  double total = 0.0;
  if (c0 < c1) {
    lds_barrier();
    Scale f;
    scales(c0, f);
    put(ahead[0], c0, f);
    publish(c0);
    load(ahead[0], within(c0 + AHEAD));
  }

  auto step = [&](int j, Rows &next) {  // next: chunk j + 1's rows
    lds_barrier();
    // all that is read from LDS first: its operations stay in order
    const E *const X = s_x[j & 1];
    const Decays<C> &d = s_d[j % 3];
    const float f = d.all;
    Scale fs;
    scales(within(j + 1), fs);
    constexpr int CW = NC < 2 ? NC : 2;  // column tiles whose operands are held at a time
    Op w[L::TERMS][CW], a[RT];
    auto scaled = [&](int kb, int c0) {
#pragma unroll
      for (int k = 0; k < L::TERMS; ++k)
#pragma unroll
        for (int c = 0; c < CW; ++c) w[k][c] = L::tr(s_w[j & 1][k], LDY, kb, 16 * (c0 + c), lane);
    };
    auto rows = [&](int kb) {
#pragma unroll
      for (int i = 0; i < RT; ++i) a[i] = L::tr(X, LDX, kb, 16 * (wave * RT + i), lane);
    };
    scaled(0, 0);
    rows(0);
    if (MODE == LA_ENDS) total += d.tot;
    __builtin_amdgcn_sched_barrier(0);
    put(next, j + 1, fs);  // behind the last chunk: into a buffer that nobody reads
    load(next, within(j + 1 + AHEAD));
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][c][e] *= f;
#pragma unroll
    for (int kb = 0; kb < C; kb += KG) {
      if (kb) rows(kb);
#pragma unroll
      for (int cc = 0; cc < NC; cc += CW) {
        if (kb || cc) scaled(kb, cc);
#pragma unroll
        for (int k = 0; k < L::TERMS; ++k)
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int c = 0; c < CW; ++c) acc[i][cc + c] = Ops<E>::mma_grp(a[i], w[k][c], acc[i][cc + c]);
      }
    }
    if (j + 1 < c1) publish(j + 1);
  };
  int j = c0;
  for (; j + AHEAD <= c1; j += AHEAD) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) step(j + i, ahead[(i + 1) % AHEAD]);
  }
#pragma unroll
  for (int i = 0; i < AHEAD - 1; ++i)
    if (j + i < c1) step(j + i, ahead[(i + 1) % AHEAD]);
  if constexpr (MODE == LA_ENDS) {
    float *const to = dir.seg_s + (nh * p.segs + seg) * ssize;
    each([&](float a, size_t at) { return to[at] = a; });
    if (tid == 0 && slice == 0) dir.seg_g[nh * p.segs + seg] = total;
  } else if (dir.send && c1 >= nch) {
    float *const to = dir.send + nh * ssize;
    each([&](float a, size_t at) { return to[at] = a; });
  }
}

// The gradients of one chunk and head from its rows, the state at its start and the state's
// gradient at its end.  Wave w owns 16 tokens, as queries (dq) and as keys (dk, dv); the
// products' accumulators hold gradients transposed (channels in a lane, tokens along lanes), and
// the scores that the second products take are accumulator tiles as they stand: (do . v)
// transposed for dq, (do . v) and (q . k) for dk and dv.  The values' channels come in slices of
// LA_NV.  16 packed documents (26,339 tokens, 16 heads, dk=dv=128): 316 of the backward's 620 us.
// Bound: latency, with two workgroups to a CU (70 KB of LDS; beyond 128 registers it takes 470 us).
struct LaGradParams {
  const void *q, *k, *v, *g, *dout, *states, *dstates;
  const float *units, *dunits;
  const float *gfix;
  void *dq, *dk_, *dv_, *dg;
  float *dg_chunk;  // [H, slots] sums over a chunk's tokens, where decays are fixed
  const int32_t *cu;
  int N, H, T, dk, dv, slots;
};

// Eight fp16 values and their unit as bf16; the sum of eight products of such values.
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x4 restored(u32x4 s, float unit) {
  const f16x8 a = __builtin_bit_cast(f16x8, s);
  bf16x8 x;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (bf16)((float)a[e] * unit);
  return __builtin_bit_cast(u32x4, x);
}
__device__ __forceinline__ float dot8(u32x4 a, u32x4 b) {
  float x = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const unsigned u = a[e], w = b[e];
    x = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, u), __builtin_bit_cast(f16x2, w), x, false);
  }
  return x;
}

template <typename E, int DK>
__global__ __launch_bounds__(La<E>::C * 4) void kla_la_grad_kernel(LaGradParams p) {
  using L = La<E>;
  using Op = typename L::Op;
  constexpr int C = L::C, KG = L::KG, VL = L::VL, NV = LA_NV, NS = C / 16, NT = 64 * NS;
  constexpr int PAD = LdsPad<E>::V, LDX = DK + PAD, LDY = NV + PAD;
  constexpr int KS = DK / KG, RB = DK / 16, NC = NV / 16;
  __shared__ __attribute__((aligned(16))) E s_q[C * LDX], s_k[C * LDX], s_v[C * LDY], s_o[C * LDY], s_s[NV * LDX], s_m[NV * LDX];
  __shared__ Decays<C> s_d;
  __shared__ float s_row[NS][C], s_read[C], s_write[C], s_dot[NS];

  const int h = blockIdx.x % p.H, slot = blockIdx.x / p.H;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, li = lane & 15;
  int n = 0;
  if (p.cu) {
    n = wave_last_where(p.N, [&](int i) { return min(max(p.cu[i], 0), p.T) / C + i <= slot; });
  } else {
    n = slot / ((p.T + C - 1) / C);
  }
  int t0, len, slot0;
  la_span(p.cu, n, p.T, C, &t0, &len, &slot0);
  const int first = (slot - slot0) * C, rows = min(C, len - first);
  if (first < 0 || rows <= 0) {
    if (p.dg_chunk && tid == 0) p.dg_chunk[(size_t)h * p.slots + slot] = 0.f;
    return;
  }
  const size_t row0 = ((size_t)(p.cu ? 0 : n) * p.H + h) * p.T + t0 + first;

  {
    const __amdgpu_buffer_rsrc_t rq = buffer_rsrc((const E *)p.q + row0 * p.dk, rows * p.dk * (int)sizeof(E));
    const __amdgpu_buffer_rsrc_t rk = buffer_rsrc((const E *)p.k + row0 * p.dk, rows * p.dk * (int)sizeof(E));
    constexpr int NP = C * DK / VL / NT;
    uint4 a[NP], b[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pc = tid + NT * i, r = pc / (DK / VL), c = pc % (DK / VL) * VL;
      const int at = c < p.dk ? (r * p.dk + c) * (int)sizeof(E) : 0x40000000;
      a[i] = buffer_ld16(rq, at);
      b[i] = buffer_ld16(rk, at);
    }
    if (wave == 0) {
      const float gl = lane >= rows ? 0.f : p.gfix ? p.gfix[h] : Elem<E>::to_f32(((const E *)p.g)[row0 + lane]);
      scan_decays<C>(&s_d, gl);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pc = tid + NT * i, at = pc / (DK / VL) * LDX + pc % (DK / VL) * VL;
      *reinterpret_cast<uint4 *>(s_q + at) = a[i];
      *reinterpret_cast<uint4 *>(s_k + at) = b[i];
    }
  }

  f32x4 dq[RB], dk[RB];  // transposed: channels 16 i + 4 g + e of token 16 wave + li
#pragma unroll
  for (int i = 0; i < RB; ++i) dq[i] = dk[i] = zero4();
  f32x4 w[NS], wt[NS];  // do . v: tokens 16 i + 4 g + e against key li; keys 16 i + 4 g + e against query li
  f32x4 sc[NS];         // q . k as w
#pragma unroll
  for (int i = 0; i < NS; ++i) w[i] = wt[i] = sc[i] = zero4();
  Op pv[C / KG];        // the decayed scores for dv
  float dot = 0.f;
  const int me = 16 * wave + li;

  // a slice's rows and states: in registers while the one before it is in use
  constexpr int YP = C * NV / VL / NT, XT = NV * DK / VL, XP = (XT + NT - 1) / NT;
  u32x4 rv[YP], ro[YP], rs[XP], rm[XP];
  float us[XP], um[XP];  // units of the states
  const size_t place = (size_t)h * p.slots + slot;
  const int slices = (p.dv + NV - 1) / NV;
  auto load = [&](int c0) {
    const int cols = min(NV, p.dv - c0);
    const __amdgpu_buffer_rsrc_t bv = buffer_rsrc((const E *)p.v + row0 * p.dv, rows * p.dv * (int)sizeof(E));
    const __amdgpu_buffer_rsrc_t bo = buffer_rsrc((const E *)p.dout + row0 * p.dv, rows * p.dv * (int)sizeof(E));
    const size_t at0 = place * p.dk * p.dv + (size_t)c0 * p.dk;
    const __amdgpu_buffer_rsrc_t bs = buffer_rsrc((const E *)p.states + at0, cols * p.dk * (int)sizeof(E));
    const __amdgpu_buffer_rsrc_t bm = buffer_rsrc((const E *)p.dstates + at0, cols * p.dk * (int)sizeof(E));
#pragma unroll
    for (int i = 0; i < YP; ++i) {
      const int pc = tid + NT * i, r = pc / (NV / VL), c = c0 + pc % (NV / VL) * VL;
      const int at = c < p.dv ? (r * p.dv + c) * (int)sizeof(E) : 0x40000000;
      rv[i] = __builtin_bit_cast(u32x4, buffer_ld16(bv, at));
      ro[i] = __builtin_bit_cast(u32x4, buffer_ld16(bo, at));
    }
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int pc = tid + NT * i, r = pc / (DK / VL), c = pc % (DK / VL) * VL;
      const int at = pc < XT && c < p.dk ? (r * p.dk + c) * (int)sizeof(E) : 0x40000000;
      rs[i] = __builtin_bit_cast(u32x4, buffer_ld16(bs, at));
      rm[i] = __builtin_bit_cast(u32x4, buffer_ld16(bm, at));
      if constexpr (sizeof(E) == 2) {
        const size_t u = (place * slices + c0 / NV) * 4 + c / (DK / 4);
        us[i] = p.units[u];
        um[i] = p.dunits[u];
      }
    }
  };
  load(0);
  for (int c0 = 0; c0 < p.dv; c0 += NV) {
    lds_barrier();
#pragma unroll
    for (int i = 0; i < YP; ++i) {
      const int pc = tid + NT * i, at = pc / (NV / VL) * LDY + pc % (NV / VL) * VL;
      *reinterpret_cast<u32x4 *>(s_v + at) = rv[i];
      *reinterpret_cast<u32x4 *>(s_o + at) = ro[i];
    }
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int pc = tid + NT * i, at = pc / (DK / VL) * LDX + pc % (DK / VL) * VL;
      u32x4 x = rs[i], y = rm[i];
      asm volatile("" : "+v"(x), "+v"(y));  // taken apart here, not where the loads are issued
      if constexpr (sizeof(E) == 2) {
        dot = fmaf(dot8(x, y) * us[i], um[i], dot);
        x = restored(x, us[i]);
        y = restored(y, um[i]);
      } else {
#pragma unroll
        for (int e = 0; e < VL; ++e) {
          const unsigned a = x[e], b = y[e];
          dot = fmaf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b), dot);
        }
      }
      if (XT % NT == 0 || pc < XT) {
        *reinterpret_cast<u32x4 *>(s_s + at) = x;
        *reinterpret_cast<u32x4 *>(s_m + at) = y;
      }
    }
    load(c0 + NV < p.dv ? c0 + NV : c0);  // (not under a condition: it would be waited for)
    lds_barrier();
    if (c0 == 0) {  // the scores of the wave's keys, once
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i >= wave) {
#pragma unroll
          for (int k = 0; k < KS; ++k)
            sc[i] = Ops<E>::mma_grp(L::nat(s_q + (16 * i + li) * LDX, k * KG, g), L::nat(s_k + me * LDX, k * KG, g), sc[i]);
          const f32x4 th = *reinterpret_cast<const f32x4 *>(&s_d.hi[16 * i + 4 * g]);
          const f32x4 tl = *reinterpret_cast<const f32x4 *>(&s_d.lo[16 * i + 4 * g]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[i][e] = i > wave || 4 * g + e >= li
                           ? sc[i][e] * __builtin_amdgcn_exp2f((th[e] - s_d.hi[me]) + (tl[e] - s_d.lo[me])) : 0.f;
        }
#pragma unroll
      for (int kb = 0; kb < C; kb += KG) pv[kb / KG] = Ops<E>::b_from_d(&sc[kb / 16]);
    }
    // do . v, both ways round
#pragma unroll
    for (int kb = 0; kb < NV; kb += KG) {
      const Op v = L::nat(s_v + me * LDY, kb, g), o = L::nat(s_o + me * LDY, kb, g);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (i >= wave) w[i] = Ops<E>::mma_grp(L::nat(s_o + (16 * i + li) * LDY, kb, g), v, w[i]);
        if (i <= wave) wt[i] = Ops<E>::mma_grp(L::nat(s_v + (16 * i + li) * LDY, kb, g), o, wt[i]);
      }
    }
    // the states' parts of dq and dk
#pragma unroll
    for (int kb = 0; kb < NV; kb += KG) {
      const Op v = L::grp(s_v + me * LDY, kb, g), o = L::grp(s_o + me * LDY, kb, g);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        dq[i] = Ops<E>::mma_grp(L::tr(s_s, LDX, kb, 16 * i, lane), o, dq[i]);
        dk[i] = Ops<E>::mma_grp(L::tr(s_m, LDX, kb, 16 * i, lane), v, dk[i]);
      }
    }
    // dv, whole for these channels
    f32x4 dv[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      dv[c] = zero4();
#pragma unroll
      for (int k = 0; k < KS; ++k)
        dv[c] = Ops<E>::mma_grp(L::nat(s_m + (16 * c + li) * LDX, k * KG, g), L::nat(s_k + me * LDX, k * KG, g), dv[c]);
      const float f = s_d.left[me];
#pragma unroll
      for (int e = 0; e < 4; ++e) dv[c][e] *= f;
#pragma unroll
      for (int kb = 0; kb < C; kb += KG)
        if (kb + KG > 16 * wave) dv[c] = Ops<E>::mma_grp(L::tr(s_o, LDY, kb, 16 * c, lane), pv[kb / KG], dv[c]);
      const int col = c0 + 16 * c + 4 * g;
      if (me < rows && col < p.dv) store4((E *)p.dv_ + (row0 + me) * p.dv + col, dv[c]);
    }
  }

  // what the states' parts give to the decays' gradient, then the chunk's own parts
  const float fo = s_d.out[me], fl = s_d.left[me];
  float read = 0.f, write = 0.f;
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const f32x4 a = load4(s_q + me * LDX + 16 * i + 4 * g), b = load4(s_k + me * LDX + 16 * i + 4 * g);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dq[i][e] *= fo;
      dk[i][e] *= fl;
      read = fmaf(a[e], dq[i][e], read);
      write = fmaf(b[e], dk[i][e], write);
    }
  }
  read += __shfl_xor(read, 16);
  read += __shfl_xor(read, 32);
  write += __shfl_xor(write, 16);
  write += __shfl_xor(write, 32);
  float col = 0.f;  // the products of the wave's keys with later queries
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    f32x4 r = zero4();
    if (i >= wave) {
      const f32x4 th = *reinterpret_cast<const f32x4 *>(&s_d.hi[16 * i + 4 * g]);
      const f32x4 tl = *reinterpret_cast<const f32x4 *>(&s_d.lo[16 * i + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool seen = i > wave || 4 * g + e >= li;
        r[e] = i > wave || 4 * g + e > li ? sc[i][e] * w[i][e] : 0.f;  // sc has its decay
        col += r[e];
        w[i][e] = seen ? w[i][e] * __builtin_amdgcn_exp2f((th[e] - s_d.hi[me]) + (tl[e] - s_d.lo[me])) : 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[e] += __shfl_xor(r[e], 1);
      r[e] += __shfl_xor(r[e], 2);
      r[e] += __shfl_xor(r[e], 4);
      r[e] += __shfl_xor(r[e], 8);
    }
    if (li == 0) *reinterpret_cast<f32x4 *>(&s_row[wave][16 * i + 4 * g]) = r;
    if (i <= wave) {
      const f32x4 sh = *reinterpret_cast<const f32x4 *>(&s_d.hi[16 * i + 4 * g]);
      const f32x4 sl = *reinterpret_cast<const f32x4 *>(&s_d.lo[16 * i + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        wt[i][e] = i < wave || 4 * g + e <= li
                       ? wt[i][e] * __builtin_amdgcn_exp2f((s_d.hi[me] - sh[e]) + (s_d.lo[me] - sl[e])) : 0.f;
    }
  }
  col += __shfl_xor(col, 16);
  col += __shfl_xor(col, 32);
  if (g == 0) {
    s_read[me] = read - col;
    s_write[me] = write;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) dot += __shfl_xor(dot, off);
  if (lane == 0) s_dot[wave] = dot;
#pragma unroll
  for (int kb = 0; kb < C; kb += KG) {
    if (kb <= 16 * wave) {  // keys up to the queries
      const Op b = Ops<E>::b_from_d(&wt[kb / 16]);
#pragma unroll
      for (int i = 0; i < RB; ++i) dq[i] = Ops<E>::mma_grp(L::tr(s_k, LDX, kb, 16 * i, lane), b, dq[i]);
    }
    if (kb + KG > 16 * wave) {  // queries from the keys on
      const Op b = Ops<E>::b_from_d(&w[kb / 16]);
#pragma unroll
      for (int i = 0; i < RB; ++i) dk[i] = Ops<E>::mma_grp(L::tr(s_q, LDX, kb, 16 * i, lane), b, dk[i]);
    }
  }
  if (me < rows) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int c = 16 * i + 4 * g;
      if (c < p.dk) {
        store4((E *)p.dq + (row0 + me) * p.dk + c, dq[i]);
        store4((E *)p.dk_ + (row0 + me) * p.dk + c, dk[i]);
      }
    }
  }
  __syncthreads();
  if (wave == 0) {
    // lane l: token C - 1 - l, so that sums from a token on are prefix sums
    const int t = C - 1 - lane;
    float ahead = 0.f, before = 0.f, x = 0.f;
    if (t >= 0) {
      ahead = s_read[t];
      before = s_write[t];
#pragma unroll
      for (int i = 0; i < NS; ++i) ahead += s_row[i][t];
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) x += s_dot[i];
    const float sum = wave_inclusive_scan(ahead), behind = wave_inclusive_scan(before);
    // writes in front of t: all of them less those from t on
    const float dg = sum + (lane_value(behind, 63) - behind) + s_d.all * x;
    if (p.dg_chunk) {
      float v = t >= 0 && t < rows ? dg : 0.f;
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
      if (lane == 0) p.dg_chunk[(size_t)h * p.slots + slot] = v;
    } else if (t >= 0 && t < rows) {
      ((E *)p.dg)[row0 + t] = Elem<E>::from_f32(dg);
    }
  }
}

// The fixed decays' gradient: a head's chunks, in 64 bits and in an order of their own.
__global__ __launch_bounds__(256) void kla_la_sum_kernel(const float *part, float *out, int slots) {
  __shared__ double s[256];
  double a = 0.0;
  for (int i = threadIdx.x; i < slots; i += 256) a += part[(size_t)blockIdx.x * slots + i];
  s[threadIdx.x] = a;
  __syncthreads();
  for (int w = 128; w >= 1; w >>= 1) {
    if ((int)threadIdx.x < w) s[threadIdx.x] += s[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) out[blockIdx.x] = (float)s[0];
}

// One token.  A workgroup owns 4 CG columns of one state, CG threads to a row and 256 / CG rows
// at a time; each thread's rows are loaded together.  256 sequences of 16 heads, dk=dv=128 (537 MB
// in and out): 87 us on one state, 112 to 117 on several in turn (4.6 to 4.8 TB/s).  Bound: HBM.
struct LaStepParams {
  const void *q, *k, *v, *g;
  const float *gfix;
  float *state;
  void *o;
  int H, dk, dv, slices;
};

template <typename E, int CG>
__global__ __launch_bounds__(256) void kla_la_step_kernel(LaStepParams p) {
  constexpr int RG = 256 / CG, RPT = 256 / RG < 16 ? 256 / RG : 16;  // rows at a time
  __shared__ float s_k[256], s_q[256];
  __shared__ f32x4 s_o[4][CG];
  const size_t nh = blockIdx.x / p.slices;
  const int slice = blockIdx.x % p.slices, tid = threadIdx.x;
  const int cg = tid % CG, rg = tid / CG, col = (slice * CG + cg) * 4;
  const bool mine = col < p.dv;
  float *const S = p.state + nh * p.dk * p.dv + col;
  f32x4 s[RPT];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = r0 + rg + RG * i;
      s[i] = mine && r < p.dk ? *reinterpret_cast<const f32x4 *>(S + (size_t)r * p.dv) : zero4();
    }
  };
  load(0);
  if (tid < p.dk) {
    s_k[tid] = Elem<E>::to_f32(((const E *)p.k)[nh * p.dk + tid]);
    s_q[tid] = Elem<E>::to_f32(((const E *)p.q)[nh * p.dk + tid]);
  }
  const float g = p.gfix ? p.gfix[nh % p.H] : Elem<E>::to_f32(((const E *)p.g)[nh]);
  const float a = __expf(g);
  f32x4 v = zero4(), o = zero4();
  if (mine) v = load4((const E *)p.v + nh * p.dv + col);
  __syncthreads();
  for (int r0 = 0; r0 < p.dk; r0 += RG * RPT) {
    if (r0) load(r0);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = r0 + rg + RG * i;
      if (r < p.dk) {
        const float k = s_k[r], q = s_q[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][e] = fmaf(a, s[i][e], k * v[e]);
          o[e] = fmaf(q, s[i][e], o[e]);
        }
        if (mine) *reinterpret_cast<f32x4 *>(S + (size_t)r * p.dv) = s[i];
      }
    }
  }
#pragma unroll
  for (int off = CG; off < 64; off <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], off);
  if ((tid & 63) < CG) s_o[tid >> 6][cg] = o;
  __syncthreads();
  if (tid < CG && mine) {
    o = s_o[0][cg];
#pragma unroll
    for (int w = 1; w < 4; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += s_o[w][cg][e];
    store4((E *)p.o + nh * p.dv + col, o);
  }
}

// Workgroups of a scan's direction, in slices of NV columns.
long long la_workgroups(long long seqs, int H, int segs, int dv, int NV) {
  return (seqs * H * segs + 7) / 8 * 8 * ((dv + NV - 1) / NV);
}

template <typename E, int DK, int MODE, int NV>
hipError_t launch_scan_t(LaParams p, int dirs, hipStream_t st) {
  p.slices = (p.dv + NV - 1) / NV;
  p.half = (unsigned)la_workgroups(p.N, p.H, p.segs, p.dv, NV);
  hipLaunchKernelGGL((kla_la_scan_kernel<E, DK, MODE, NV>), dim3(dirs * p.half), dim3(la_threads(MODE)), 0, st, p);
  return hipGetLastError();
}
// Slices of 64 columns, which read x half as often, where they still make a workgroup to a CU and
// where their rows, states and scaled values fit LDS (T=65536 dv=256 of 16 heads: 840 us, with 32
// columns 1,026).  Not where states are stored, for which the registers do not suffice (when that was
// tried, 16 packed documents backward took 685 us, with 32 columns 610).
template <typename E, int MODE>
hipError_t launch_scan(const LaParams &p, int dirs, hipStream_t st) {
  if constexpr (sizeof(E) == 2 && MODE != LA_STORE) {
    if (p.dk <= 128 && p.dv > LA_NV && dirs * la_workgroups(p.N, p.H, p.segs, p.dv, 2 * LA_NV) >= 256) {
      if (p.dk <= 64) return launch_scan_t<E, 64, MODE, 2 * LA_NV>(p, dirs, st);
      return launch_scan_t<E, 128, MODE, 2 * LA_NV>(p, dirs, st);
    }
  }
  if (p.dk <= 64) return launch_scan_t<E, 64, MODE, LA_NV>(p, dirs, st);
  if (p.dk <= 128) return launch_scan_t<E, 128, MODE, LA_NV>(p, dirs, st);
  return launch_scan_t<E, 256, MODE, LA_NV>(p, dirs, st);
}

int la_chunk(int dtype) { return dtype == 0 ? La<bf16>::C : La<float>::C; }

int la_slots(const LaArgs &a) {
  const int C = la_chunk(a.dtype);
  return a.cu_seqlens ? a.T / C + a.num_seqs : a.num_seqs * ((a.T + C - 1) / C);
}

// Segments of the scans, where their workgroups leave CUs idle: as many as make two rounds of
// workgroups, each of 8 chunks at least (T=65536 dv=256 of 16 heads, 128 workgroups unsplit: 840
// us, in one segment 1,182, for 256 workgroups 1,001, for 1,024 918).  All sequences count as work:
// one of 65,536 tokens packed beside fifteen of 256 is not cut and takes 1,803, alone 877.
void la_segments(const LaArgs &a, int *segs, int *chunks) {
  const int C = la_chunk(a.dtype), nch = (a.longest + C - 1) / C;
  const long long wgs = (long long)a.num_seqs * a.H * ((a.dv + LA_NV - 1) / LA_NV);
  *segs = 1;
  *chunks = std::max(nch, 1);
  if (wgs > 128 || wgs == 0 || nch < 32) return;
  const int want = (int)std::min<long long>({512 / wgs, nch / 8, 32});
  *chunks = (nch + want - 1) / want;
  *segs = (nch + *chunks - 1) / *chunks;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// The workspace: the segments' states and decays (backward: of both directions); the backward's
// states and gradients of states of all chunks with their units, and the fixed decays' partial
// sums.
struct LaSpace {
  size_t seg_s[2], seg_g[2], states[2], units[2], dg, total;
};
LaSpace la_space(const LaArgs &a, bool bwd) {
  int segs, chunks;
  la_segments(a, &segs, &chunks);
  const size_t pairs = (size_t)a.num_seqs * a.H * segs, state = (size_t)a.dk * a.dv;
  LaSpace s{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t was = at;
    at += up(n);
    return was;
  };
  for (int i = 0; i <= (int)bwd; ++i) {
    s.seg_s[i] = take(segs > 1 ? pairs * state * sizeof(float) : 0);
    s.seg_g[i] = take(segs > 1 ? pairs * sizeof(double) : 0);
  }
  if (bwd) {
    const size_t n = (size_t)la_slots(a) * a.H;
    for (int i = 0; i < 2; ++i) {
      s.states[i] = take(n * state * (a.dtype == 0 ? 2 : 4));
      s.units[i] = take(a.dtype == 0 ? n * ((a.dv + LA_NV - 1) / LA_NV) * 4 * sizeof(float) : 0);
    }
    s.dg = take(n * sizeof(float));
  }
  s.total = at;
  return s;
}

LaParams la_params(const LaArgs &a, const LaSpace &s) {
  LaParams p{};
  char *const ws = (char *)a.workspace;
  p.q = a.q;
  p.g = a.g;
  p.gfix = a.gfix;
  p.o = a.o;
  p.cu = a.cu_seqlens;
  p.N = a.num_seqs;
  p.H = a.H;
  p.T = a.T;
  p.dk = a.dk;
  p.dv = a.dv;
  la_segments(a, &p.segs, &p.seg_chunks);
  for (int i = 0; i < 2; ++i) {
    p.dir[i].seg_s = (float *)(ws + s.seg_s[i]);
    p.dir[i].seg_g = (double *)(ws + s.seg_g[i]);
    p.dir[i].states = ws + s.states[i];
    p.dir[i].units = (float *)(ws + s.units[i]);
  }
  p.dir[0].x = a.k;
  p.dir[0].y = a.v;
  p.dir[0].s0 = a.initial_state;
  return p;
}

template <typename E>
hipError_t la_fwd_t(const LaArgs &a, hipStream_t st) {
  LaParams p = la_params(a, la_space(a, false));
  p.dir[0].send = a.final_state;
  if (p.segs > 1)
    if (const hipError_t e = launch_scan<E, LA_ENDS>(p, 1, st); e != hipSuccess) return e;
  return launch_scan<E, LA_OUT>(p, 1, st);
}

template <typename E, int DK>
hipError_t launch_grad_t(const LaGradParams &p, hipStream_t st) {
  hipLaunchKernelGGL((kla_la_grad_kernel<E, DK>), dim3((unsigned)((long long)p.slots * p.H)), dim3(La<E>::C * 4), 0, st, p);
  return hipGetLastError();
}
template <typename E>
hipError_t launch_grad(const LaGradParams &p, hipStream_t st) {
  if (p.dk <= 64) return launch_grad_t<E, 64>(p, st);
  if (p.dk <= 128) return launch_grad_t<E, 128>(p, st);
  return launch_grad_t<E, 256>(p, st);
}

template <typename E>
hipError_t la_bwd_t(const LaArgs &a, const LaGrads &b, hipStream_t st) {
  const LaSpace s = la_space(a, true);
  char *const ws = (char *)a.workspace;
  if (a.num_seqs == 0) {  // nothing but the fixed decays' gradient, which is zero
    if (a.gfix) hipLaunchKernelGGL(kla_la_sum_kernel, dim3((unsigned)a.H), dim3(256), 0, st, nullptr, (float *)b.dg, 0);
    return hipGetLastError();
  }
  LaParams p = la_params(a, s);
  p.slots = la_slots(a);
  p.dir[1].x = a.q;
  p.dir[1].y = b.dout;
  p.dir[1].s0 = b.dfinal_state;
  p.dir[1].send = b.dinitial_state;
  hipError_t e;
  if (p.segs > 1 && (e = launch_scan<E, LA_ENDS>(p, 2, st)) != hipSuccess) return e;
  if ((e = launch_scan<E, LA_STORE>(p, 2, st)) != hipSuccess) return e;
  LaGradParams gp{};
  gp.q = a.q;
  gp.k = a.k;
  gp.v = a.v;
  gp.g = a.g;
  gp.gfix = a.gfix;
  gp.dout = b.dout;
  gp.states = p.dir[0].states;
  gp.dstates = p.dir[1].states;
  gp.units = p.dir[0].units;
  gp.dunits = p.dir[1].units;
  gp.dq = b.dq;
  gp.dk_ = b.dk;
  gp.dv_ = b.dv;
  gp.dg = b.dg;
  gp.dg_chunk = a.gfix ? (float *)(ws + s.dg) : nullptr;
  gp.cu = a.cu_seqlens;
  gp.N = a.num_seqs;
  gp.H = a.H;
  gp.T = a.T;
  gp.dk = a.dk;
  gp.dv = a.dv;
  gp.slots = p.slots;
  if (gp.slots > 0 && (e = launch_grad<E>(gp, st)) != hipSuccess) return e;
  if (a.gfix) {
    hipLaunchKernelGGL(kla_la_sum_kernel, dim3((unsigned)a.H), dim3(256), 0, st, gp.dg_chunk, (float *)b.dg, gp.slots);
    return hipGetLastError();
  }
  return hipSuccess;
}

template <typename E, int CG>
hipError_t launch_step_t(LaStepParams p, long long nh, hipStream_t st) {
  p.slices = (p.dv + 4 * CG - 1) / (4 * CG);
  hipLaunchKernelGGL((kla_la_step_kernel<E, CG>), dim3((unsigned)(nh * p.slices)), dim3(256), 0, st, p);
  return hipGetLastError();
}
template <typename E>
hipError_t launch_step(const LaStepParams &p, long long nh, hipStream_t st) {
  // few states: narrow pieces, for more workgroups (16 states 9.4 us either way, since the host
  // bounds the call; 4,096 states 140 against 117)
  if (nh * ((p.dv + 127) / 128) < 512) return launch_step_t<E, 4>(p, nh, st);
  return launch_step_t<E, 32>(p, nh, st);
}

}  // namespace

bool la_supported(int dk, int dv) { return dk % 16 == 0 && dk <= 256 && dv % 16 == 0 && dv <= 256; }

bool la_grid_fits(const LaArgs &a) {
  int segs, chunks;
  la_segments(a, &segs, &chunks);
  const int C = la_chunk(a.dtype);
  const double slots = a.cu_seqlens ? (double)a.T / C + a.num_seqs + 1 : (double)a.num_seqs * ((a.T + C - 1) / C);
  return launch_fits(2.0 * ((double)a.num_seqs * a.H * segs + 8) * ((a.dv + LA_NV - 1) / LA_NV), 512) &&
         launch_fits(slots * a.H, 256);
}

size_t la_workspace_bytes(const LaArgs &a, bool bwd) { return la_space(a, bwd).total; }

hipError_t launch_la_fwd(const LaArgs &a, hipStream_t st) {
  return a.dtype == 0 ? la_fwd_t<bf16>(a, st) : la_fwd_t<float>(a, st);
}
hipError_t launch_la_bwd(const LaArgs &a, const LaGrads &b, hipStream_t st) {
  return a.dtype == 0 ? la_bwd_t<bf16>(a, b, st) : la_bwd_t<float>(a, b, st);
}

bool la_step_fits(long long nh, int dv) { return launch_fits((double)nh * ((dv + 15) / 16), 256); }

hipError_t launch_la_step(const void *q, const void *k, const void *v, const void *g, const float *gfix, float *state,
                          void *o, int N, int H, int dk, int dv, int dtype, hipStream_t st) {
  const LaStepParams p{q, k, v, g, gfix, state, o, H, dk, dv, 1};
  return dtype == 0 ? launch_step<bf16>(p, (long long)N * H, st) : launch_step<float>(p, (long long)N * H, st);
}

}  // namespace kla
