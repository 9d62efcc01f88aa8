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
// reads g, o and do and writes dx and dg: both are bound by HBM.  One workgroup owns a
// slice of CG * V channels of one (sequence, head) and walks its tokens in tiles of
// RG * R rows: thread (row group rg, channel group cg) holds R consecutive rows of V
// channels (16-byte loads, the next tile's in flight while this one is computed), composes
// them, a shuffle scan composes the row groups of a wave, and the waves' maps meet in LDS,
// one barrier per tile.  Every byte is read once and no workgroup waits for another.
//
// Where few channels leave most CUs idle, sequences are cut into segments (SEG): a first
// pass forms each segment's map, and the second starts every segment from the maps of those
// before it; it reads x and g twice.
#include "kla_common.h"
#include "kla_internal.h"

namespace kla {

namespace {

struct GlrParams {
  const void *x, *g;         // x: the forward's input, the backward's do
  const void *h;             // backward: the forward's output o
  const float *y0;           // [N,H,d] start of the scan (initial state / dfinal), or nullptr
  const float *h0;           // backward: [N,H,d] initial state, or nullptr
  void *o, *dg;              // outputs (o: forward output / dx)
  float *yend;               // [N,H,d] end of the scan (final state / dinitial), or nullptr
  const int32_t *cu;         // device, or nullptr (dense)
  int N, H, T, d;
  int slices;                // channel slices of a head
  int segs, seg_rows;        // segments of a sequence at most, tokens in one
  float *maps;               // [N,H,segs,2,d]: the segments' maps (A then C)
};

// exp of the log-decay: one base-2 exponential for bf16 gates, whose own spacing is 2^-8 of
// their value; the library's exp for fp32, where the product's rounding would show.
__device__ __forceinline__ float decay(float g, const bf16 *) { return __builtin_amdgcn_exp2f(g * 1.44269504f); }
__device__ __forceinline__ float decay(float g, const float *) { return expf(g); }

template <typename E, int V>
struct Vec {
  E v[V];
};
template <typename E, int V>
__device__ __forceinline__ Vec<E, V> ld(const E *p) {
  Vec<E, V> r;
  if constexpr (V * sizeof(E) == 16) {
    const uint4 u = ldg16(p);
    __builtin_memcpy(&r, &u, 16);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = p[i];
  }
  return r;
}
template <typename E, int V>
__device__ __forceinline__ void st(E *p, const float *f) {
  Vec<E, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = Elem<E>::from_f32(f[i]);
  if constexpr (V * sizeof(E) == 16) {
    uint4 u;
    __builtin_memcpy(&u, &r, 16);
    stg16(p, u);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = r.v[i];
  }
}

enum { GLR_WHOLE = 0, GLR_MAPS = 1, GLR_CARRIED = 2 };

template <typename E, int V, int CG, int NW, int R, bool BWD, int MODE>
__global__ __launch_bounds__(64 * NW) void kla_glr_kernel(GlrParams p) {
  constexpr int GW = 64 / CG;       // row groups of a wave
  constexpr int ROWS = NW * GW * R; // rows of a tile
  constexpr int CW = CG * V;
  __shared__ float s_map[2][NW][2][CW];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cg = lane % CG, gw = lane / CG;
  // workgroups: slice fastest, then head and sequence; segments slowest
  unsigned b = blockIdx.x;
  const int slice = b % p.slices;
  b /= p.slices;
  const int head = b % p.H;
  b /= p.H;
  const int seq = b % p.N, seg = b / p.N;

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
  const int len = MODE == GLR_WHOLE ? len_seq : min(len_seq - skip, p.seg_rows);
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
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = start[i];
    for (int s = 0; s < seg; ++s) {
      const float *m = p.maps + mrow + (size_t)s * 2 * p.d;
#pragma unroll
      for (int i = 0; i < V; ++i) carry[i] = fmaf(m[i], carry[i], m[p.d + i]);
    }
  }

  // scan step j of the segment is token t0 + skip + j, backwards t1 - 1 - skip - j
  const E *px = (const E *)p.x + (row0 + (BWD ? t1 - 1 - skip : t0 + skip)) * p.d + cc;
  const E *pg = (const E *)p.g + (row0 + (BWD ? t1 - 1 - skip : t0 + skip)) * p.d + cc;
  const E *ph = BWD ? (const E *)p.h + (row0 + (t1 - 1 - skip)) * p.d + cc : nullptr;
  const long long step = BWD ? -(long long)p.d : p.d;

  Vec<E, V> nx[R], ng[R], nh[BWD && MODE != GLR_MAPS ? R : 1];
  const int j0 = (wave * GW + gw) * R;  // this thread's first step in a tile
  auto load = [&](int base) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int j = min(base + j0 + r, len - 1);  // rows past the end repeat the last one
      nx[r] = ld<E, V>(px + j * step);
      ng[r] = ld<E, V>(pg + j * step);
      if constexpr (BWD && MODE != GLR_MAPS) {
        // h_{t-1}: the output of the token before, which the sequence's first does not have
        const int jh = min(skip + j + 1, len_seq - 1) - skip;
        nh[r] = ld<E, V>(ph + jh * step);
      }
    }
  };
  if (len > 0) load(0);

  int buf = 0;
  for (int base = 0; base < len; base += ROWS, buf ^= 1) {
    float a[R][V], x[R][V];
    Vec<E, V> hv[BWD && MODE != GLR_MAPS ? R : 1];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = base + j0 + r < len;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[r][i] = in ? decay(Elem<E>::to_f32(ng[r].v[i]), (const E *)nullptr) : 1.f;
        x[r][i] = in ? Elem<E>::to_f32(nx[r].v[i]) : 0.f;
      }
      if constexpr (BWD && MODE != GLR_MAPS) hv[r] = nh[r];
    }
    if (base + ROWS < len) load(base + ROWS);

    // this thread's rows as one map
    float A[V], C[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      A[i] = 1.f;
      C[i] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        C[i] = BWD ? a[r][i] * (C[i] + x[r][i]) : fmaf(a[r][i], C[i], x[r][i]);
        A[i] *= a[r][i];
      }
    // inclusive scan over the wave's row groups
#pragma unroll
    for (int s = 1; s < GW; s <<= 1)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float pa = __shfl_up(A[i], s * CG), pc = __shfl_up(C[i], s * CG);
        if (gw >= s) {
          C[i] = fmaf(A[i], pc, C[i]);
          A[i] *= pa;
        }
      }
    if (gw == GW - 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s_map[buf][wave][0][cg * V + i] = A[i];
        s_map[buf][wave][1][cg * V + i] = C[i];
      }
    }
    __syncthreads();
    // the value before this wave, and before the next tile (two buffers: a wave can be at
    // most one barrier ahead of another)
    float y[V];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (w == wave) y[i] = carry[i];
        const float ma = s_map[buf][w][0][cg * V + i], mc = s_map[buf][w][1][cg * V + i];
        carry[i] = fmaf(ma, carry[i], mc);
        if (MODE == GLR_MAPS) total[i] *= ma;
      }
    }
    if constexpr (MODE != GLR_MAPS) {
      // the value before this thread's rows
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float pa = __shfl_up(A[i], CG), pc = __shfl_up(C[i], CG);
        if (gw > 0) y[i] = fmaf(pa, y[i], pc);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int j = base + j0 + r;
        float out[V], dg[V];
        if constexpr (BWD) {
          const bool first = skip + j + 1 >= len_seq;  // the sequence's first token: h_{t-1} = h0
#pragma unroll
          for (int i = 0; i < V; ++i) {
            out[i] = y[i] + x[r][i];
            y[i] = a[r][i] * out[i];
            const float hp = first ? (p.h0 ? p.h0[sh + i] : 0.f) : Elem<E>::to_f32(hv[r].v[i]);
            dg[i] = y[i] * hp;
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            y[i] = fmaf(a[r][i], y[i], x[r][i]);
            out[i] = y[i];
          }
        }
        if (live && j < len) {
          const size_t at = (row0 + (BWD ? t1 - 1 - skip - j : t0 + skip + j)) * p.d + c;
          st<E, V>((E *)p.o + at, out);
          if constexpr (BWD) st<E, V>((E *)p.dg + at, dg);
        }
      }
    }
  }
  if (!live || wave || gw) return;
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

template <typename E, int V, int CG, int NW, int R, bool BWD>
struct GlrShape {
  static constexpr int ROWS = NW * (64 / CG) * R, CW = CG * V;
  static long long slices(int d) { return (d + CW - 1) / CW; }
  static hipError_t launch(GlrParams p, long long segs, hipStream_t st) {
    p.slices = (int)slices(p.d);
    const long long grid = (long long)p.N * p.H * p.slices;
    if (segs <= 1) {
      hipLaunchKernelGGL((kla_glr_kernel<E, V, CG, NW, R, BWD, GLR_WHOLE>), dim3((unsigned)grid), dim3(64 * NW), 0, st, p);
    } else {
      // the last segment's map is not needed
      hipLaunchKernelGGL((kla_glr_kernel<E, V, CG, NW, R, BWD, GLR_MAPS>), dim3((unsigned)(grid * (segs - 1))),
                         dim3(64 * NW), 0, st, p);
      hipLaunchKernelGGL((kla_glr_kernel<E, V, CG, NW, R, BWD, GLR_CARRIED>), dim3((unsigned)(grid * segs)), dim3(64 * NW),
                         0, st, p);
    }
    return hipGetLastError();
  }
};

constexpr int GLR_SEG_ROWS = 1024;  // a multiple of every shape's tile rows

template <typename E, bool BWD>
hipError_t launch_glr(const GlrParams &p, long long segs, hipStream_t st) {
  constexpr int V = 16 / sizeof(E);
  if (p.d % V == 0) return GlrShape<E, V, 4, 4, 4, BWD>::launch(p, segs, st);
  return GlrShape<E, 1, 16, 4, 4, BWD>::launch(p, segs, st);
}

}  // namespace

// Workgroups of one segment, and segments of the longest sequence: 1 unless few channels
// leave CUs idle.
static long long glr_groups(const GlrArgs &a) {
  const int V = a.dtype == 0 ? 8 : 4;
  const long long cw = a.d % V == 0 ? 4 * V : 16;
  return (long long)a.num_seqs * a.H * ((a.d + cw - 1) / cw);
}
static long long glr_segments(const GlrArgs &a) {
  const long long segs = ((long long)a.longest + GLR_SEG_ROWS - 1) / GLR_SEG_ROWS;
  return glr_groups(a) >= 256 || segs < 2 ? 1 : segs;
}

bool glr_grid_fits(const GlrArgs &a) { return glr_groups(a) * glr_segments(a) <= 0x7fffffffLL; }

size_t glr_workspace_bytes(const GlrArgs &a) {
  const long long segs = glr_segments(a);
  return segs <= 1 ? 0 : (size_t)a.num_seqs * a.H * segs * 2 * a.d * sizeof(float);
}

hipError_t launch_glr_chunk(const GlrArgs &a, bool bwd, hipStream_t st) {
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
  const long long segs = glr_segments(a);
  p.segs = (int)segs;
  p.seg_rows = GLR_SEG_ROWS;
  p.maps = (float *)a.workspace;
  if (a.dtype == 0) return bwd ? launch_glr<bf16, true>(p, segs, st) : launch_glr<bf16, false>(p, segs, st);
  return bwd ? launch_glr<float, true>(p, segs, st) : launch_glr<float, false>(p, segs, st);
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
