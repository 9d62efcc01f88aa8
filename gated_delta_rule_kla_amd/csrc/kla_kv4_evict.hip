// kla_kv4_evict.hip -- a 4-bit cache cut to a budget by the weight its tokens got (gfx950).
//
// Per sequence of more than `budget` tokens and key head: the newest `recent` tokens stay, and of
// the others the `budget - recent` of the largest weight, the earlier of two that are equal; they
// move to the front in their order (include/kla.h, kla_kv4_evict).
//
// Three kernels.  Choice, a workgroup to a (sequence, head): a radix selection finds the smallest
// weight that stays, eleven bits of the weights' order at a time (a histogram in LDS per pass;
// integer counts, so the order of the atomics changes nothing; the first pass's bins are a weight's
// sign, exponent and two more bits, so weights of like size meet in one and are added in turn);
// then each wave goes over its part of the tokens and writes the positions that stay, at places
// counted ahead.  Few (sequence, head)s: the same in parts, over four launches.  Then the rows that
// change place go to a workspace and from there to their places: kept rows move towards the front
// over rows that others still have to read.
// Bound: the choice by its passes over the weights (from L2), the moves by HBM and the memory-side
// cache, which holds the workspace in between: 64 sequences of 4,096 to 16,384 tokens and four heads
// cut to 4,096 tokens, choice 30 us, rows out 34 (200 MB read) and in 25; one sequence of 131,071
// and two heads cut to 32,768, choice 39 in four launches (the first 7, the others 10 to 12: each of
// their workgroups adds up the histograms of all parts, 8 KB each), rows 5 and 5.
#include <algorithm>

#include "kla_common.h"
#include "kla_index.h"
#include "kla_internal.h"
#include "kla_kv4.h"

namespace kla {

namespace {

struct KvEvictParams {
  KvParams kv;
  const int32_t *lens;
  int32_t *new_lens, *kept;  // kept [N, Hkv, budget]
  float *w;                  // [N, Hkv, W]
  int N, D, W, budget, recent;
  u32x4 *rows;               // [N Hkv, budget] rows of a token: K's codes, V's, K's scales, V's, weight
  int row_bytes;
  // a choice in parts: [N Hkv, 3, parts, EV_BINS] histograms, [N Hkv, 3, 2] prefix and rest behind
  // each, [N Hkv, 2, parts] tokens of a part above it
  unsigned *hist, *state, *above;
  int parts;
};

__device__ __forceinline__ int evict_len(const KvEvictParams &p, int n) {
  const long long room = (long long)p.kv.max_pages * p.kv.page;
  return (int)min((long long)max(p.lens[n], 0), room);
}

// Weights in their order as unsigned numbers: both zeros are one, every NaN is above all numbers.
__device__ __forceinline__ unsigned order_of(float w) {
  if (w != w) return 0xffffffffu;
  const unsigned u = __builtin_bit_cast(unsigned, w + 0.f);
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

constexpr int EV_T = 1024, EV_W = EV_T / 64;
constexpr int EV_BITS = 11, EV_BINS = 1 << EV_BITS;

// Each wave owns a part of the tokens, 256 of them at a time, four in a row to a lane.  CACHED:
// the weights' order stays in registers (up to EV_CACHE tokens), else every pass reads them again.
constexpr int EV_STEPS = 8, EV_CACHE = EV_T * 4 * EV_STEPS;

template <bool CACHED>
__device__ void choose(const KvEvictParams &p, const float *w, int32_t *kept, int len, unsigned *s_hist, int *s_more,
                       int *s_same, unsigned *s_pick) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int free = len - p.recent, want = p.budget - p.recent;  // free > want
  const bool vec = p.W % 4 == 0;
  const int per = ((free + EV_W - 1) / EV_W + 255) / 256 * 256, lo = min(wave * per, free), hi = min(lo + per, free);
  auto read = [&](int i, unsigned *u) {  // tokens i + 4 lane and up
    // (past the end: the last ones again, which nobody counts; free tokens are more than none)
    const int at = i + 4 * lane;
    f32x4 v;
    if (vec) {  // rows of whole 16 bytes: the load ends within the row
      v = *reinterpret_cast<const f32x4 *>(w + min(at, (free - 1) & ~3));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = w[min(at + e, free - 1)];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = order_of(v[e]);
  };
  unsigned u[EV_STEPS][4];
  auto fill = [&](int first) {
#pragma unroll
    for (int k = 0; k < EV_STEPS; ++k) read(first + 256 * k, u[k]);
  };
  if constexpr (CACHED) fill(lo);
  auto each = [&](auto f) {  // f(first token, orders): by all lanes of the wave
    for (int i = lo; i < hi; i += 256 * EV_STEPS) {
      if constexpr (!CACHED) fill(i);
#pragma unroll
      for (int k = 0; k < EV_STEPS; ++k)
        if (i + 256 * k < hi) f(i + 256 * k, u[k]);
    }
  };
  // the want-th largest of the free tokens' orders, from the top bits down
  unsigned prefix = 0, left = want;
  for (int top = 32; want > 0 && top > 0;) {
    // bits [shift, top) of those whose bits from `top` on are the prefix's
    const int shift = max(top - EV_BITS, 0);
    const unsigned known = top == 32 ? 0u : ~0u << top, bins = (1u << (top - shift)) - 1;
    for (int i = tid; i < EV_BINS; i += EV_T) s_hist[i] = 0;
    __syncthreads();
    each([&](int i, const unsigned *u) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + 4 * lane + e < hi && ((u[e] ^ prefix) & known) == 0) atomicAdd(&s_hist[u[e] >> shift & bins], 1u);
    });
    __syncthreads();
    // thread t: the bins 2 t and 2 t + 1 from the top; the bin in which the count reaches `left`
    const unsigned c0 = s_hist[EV_BINS - 1 - 2 * tid], c1 = s_hist[EV_BINS - 2 - 2 * tid];
    unsigned upto = c0 + c1;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const unsigned v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 63) s_more[wave] = (int)upto;
    __syncthreads();
    unsigned above = upto - c0 - c1;
    for (int i = 0; i < wave; ++i) above += (unsigned)s_more[i];
    if (above < left && above + c0 >= left) s_pick[0] = EV_BINS - 1 - 2 * tid, s_pick[1] = left - above;
    else if (above + c0 < left && above + c0 + c1 >= left) s_pick[0] = EV_BINS - 2 - 2 * tid, s_pick[1] = left - above - c0;
    __syncthreads();
    prefix |= s_pick[0] << shift;
    left = s_pick[1];
    __syncthreads();
    top = shift;
  }
  // tokens above `prefix` stay, and the first `left` that equal it: places in front of a wave's part
  int more = 0, same = 0;
  if (want > 0)
    each([&](int i, const unsigned *u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = i + 4 * lane + e < hi;
        more += __popcll(__ballot(in && u[e] > prefix));
        same += __popcll(__ballot(in && u[e] == prefix));
      }
    });
  if (lane == 0) {
    s_more[wave] = more;
    s_same[wave] = same;
  }
  __syncthreads();
  more = same = 0;
  for (int i = 0; i < wave; ++i) {
    more += s_more[i];
    same += s_same[i];
  }
  const unsigned long long below = (1ull << lane) - 1;
  if (want > 0)
    each([&](int i, const unsigned *u) {
      bool top[4], tie[4];
      int a = more, b = same;  // in front of this lane's tokens
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = i + 4 * lane + e < hi;
        top[e] = in && u[e] > prefix;
        tie[e] = in && u[e] == prefix;
        const unsigned long long x = __ballot(top[e]), y = __ballot(tie[e]);
        a += __popcll(x & below);
        b += __popcll(y & below);
        more += __popcll(x);
        same += __popcll(y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // (within the row also where another stream changes the weights meanwhile)
        const int to = a + min(b, (int)left);
        if ((top[e] || (tie[e] && b < (int)left)) && to < want) kept[to] = i + 4 * lane + e;
        a += top[e];
        b += tie[e];
      }
    });
  for (int i = tid; i < p.recent; i += EV_T) kept[want + i] = free + i;
}

__global__ __launch_bounds__(EV_T) void kla_kv4_choose_kernel(KvEvictParams p) {
  __shared__ unsigned s_hist[EV_BINS], s_pick[2];
  __shared__ int s_more[EV_W], s_same[EV_W];
  const int n = blockIdx.x / p.kv.Hkv, tid = threadIdx.x;
  const int len = evict_len(p, n);
  int32_t *const kept = p.kept + (size_t)blockIdx.x * p.budget;
  if (blockIdx.x % p.kv.Hkv == 0 && tid == 0) p.new_lens[n] = min(len, p.budget);
  if (len <= p.budget) {
    for (int i = tid; i < p.budget; i += EV_T) kept[i] = i < len ? i : -1;
    return;
  }
  const float *const w = p.w + (size_t)blockIdx.x * p.W;
  if (len - p.recent <= EV_CACHE) choose<true>(p, w, kept, len, s_hist, s_more, s_same, s_pick);
  else choose<false>(p, w, kept, len, s_hist, s_more, s_same, s_pick);
}

// The same choice with a (sequence, head)'s tokens in parts, a workgroup to each, where there are
// few of them: a launch per histogram, each of which first finds the bits that the one before it
// decides, from all parts' counts, and a last one that writes.
constexpr int EV_PT = 256, EV_PART = 4096;  // threads, tokens of a part
static_assert(EV_BINS == EV_PT * 8 && EV_PART == EV_PT * 16, "parts");

template <int STAGE>
__global__ __launch_bounds__(EV_PT) void kla_kv4_choose_part_kernel(KvEvictParams p) {
  __shared__ unsigned s_hist[EV_BINS], s_pick[3], s_sum[EV_PT / 64];
  const int pair = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const int n = pair / p.kv.Hkv, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int len = evict_len(p, n);
  int32_t *const kept = p.kept + (size_t)pair * p.budget;
  if (STAGE == 3 && part == 0 && pair % p.kv.Hkv == 0 && tid == 0) p.new_lens[n] = min(len, p.budget);
  if (len <= p.budget) {
    if (STAGE == 3)
      for (int i = part * EV_PT + tid; i < p.budget; i += p.parts * EV_PT) kept[i] = i < len ? i : -1;
    return;
  }
  const int free = len - p.recent, want = p.budget - p.recent;
  unsigned *const state = p.state + (size_t)pair * 6, *const above = p.above + (size_t)pair * 2 * p.parts;
  if (STAGE == 3)
    for (int i = part * EV_PT + tid; i < p.recent; i += p.parts * EV_PT) kept[want + i] = free + i;
  if (want == 0) return;
  constexpr int TOP = STAGE == 0 ? 32 : STAGE == 1 ? 21 : STAGE == 2 ? 10 : 0;  // bits from here on are known
  constexpr int SHIFT = STAGE == 0 ? 21 : STAGE == 1 ? 10 : 0;                  // the histogram's
  static_assert(EV_BITS == 11, "bits");
  unsigned prefix = 0, left = want, more = 0, same = 0;  // more, same: of the parts before this one (STAGE 3)
  auto block_sum = [&](unsigned v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if (lane == 0) s_sum[wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < EV_PT / 64; ++i) v += s_sum[i];
    return v;
  };
  if constexpr (STAGE > 0) {
    if (STAGE > 1) prefix = state[2 * (STAGE - 2)], left = state[2 * (STAGE - 2) + 1];
    // thread t: the bins 8 t .. 8 t + 7 from the top, of all parts, of this one, of those before it
    const unsigned *const h = p.hist + ((size_t)pair * 3 + STAGE - 1) * p.parts * EV_BINS + (EV_BINS - 8 * tid - 8);
    unsigned all[8] = {}, own[8] = {}, before[8] = {};
#pragma unroll 8
    for (int g = 0; g < p.parts; ++g) {
      unsigned c[8];
      __builtin_memcpy(c, h + (size_t)g * EV_BINS, 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        all[i] += c[i];
        if (g == part) own[i] = c[i];
        if (STAGE == 3 && g < part) before[i] += c[i];
      }
    }
    unsigned mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += all[i];
    unsigned upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const unsigned v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 63) s_sum[wave] = upto;
    __syncthreads();
    unsigned over = upto - mine;
    for (int i = 0; i < wave; ++i) over += s_sum[i];
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      if (over < left && over + all[i] >= left) {
        s_pick[0] = EV_BINS - 8 * tid - 8 + i;
        s_pick[1] = left - over;
      }
      over += all[i];
    }
    __syncthreads();
    const unsigned pick = s_pick[0];
    left = s_pick[1];
    unsigned a = 0, b = 0, c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned bin = EV_BINS - 8 * tid - 8 + i;
      if (bin > pick) a += own[i], b += before[i];
      if (bin == pick) c += before[i];
    }
    prefix |= pick << (STAGE == 1 ? 21 : STAGE == 2 ? 10 : 0);
    if constexpr (STAGE < 3) {
      a = block_sum(a);
      if (tid == 0) {
        above[(STAGE - 1) * p.parts + part] = a;
        if (part == 0) state[2 * (STAGE - 1)] = prefix, state[2 * (STAGE - 1) + 1] = left;
      }
    } else {
      for (int g = tid; g < part; g += EV_PT) b += above[g] + above[p.parts + g];
      more = block_sum(b);
      same = block_sum(c);
    }
  }
  // the part's tokens, 16 in a row to a thread
  const float *const w = p.w + (size_t)pair * p.W;
  const int i0 = part * EV_PART + 16 * tid;
  unsigned u[16];
  if (p.W % 4 == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x4 v = *reinterpret_cast<const f32x4 *>(w + min(i0 + 4 * k, (free - 1) & ~3));
#pragma unroll
      for (int e = 0; e < 4; ++e) u[4 * k + e] = order_of(v[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) u[e] = order_of(w[min(i0 + e, free - 1)]);
  }
  if constexpr (STAGE < 3) {
    for (int i = tid; i < EV_BINS; i += EV_PT) s_hist[i] = 0;
    __syncthreads();
    constexpr unsigned KNOWN = TOP == 32 ? 0u : ~0u << (TOP & 31), BINS = (1u << (TOP - SHIFT)) - 1;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (i0 + e < free && ((u[e] ^ prefix) & KNOWN) == 0) atomicAdd(&s_hist[u[e] >> SHIFT & BINS], 1u);
    __syncthreads();
    unsigned *const to = p.hist + (((size_t)pair * 3 + STAGE) * p.parts + part) * EV_BINS;
    for (int i = tid; i < EV_BINS; i += EV_PT) to[i] = s_hist[i];
  } else {
    unsigned a = 0, b = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      a += i0 + e < free && u[e] > prefix;
      b += i0 + e < free && u[e] == prefix;
    }
    // in front of this thread's: both counts in one number (a part has 2^12 tokens)
    unsigned upto = a << 16 | b;
    const unsigned mine = upto;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const unsigned v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    __syncthreads();
    if (lane == 63) s_sum[wave] = upto;
    __syncthreads();
    upto -= mine;
    for (int i = 0; i < wave; ++i) upto += s_sum[i];
    a = more + (upto >> 16);
    b = same + (upto & 0xffff);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const bool in = i0 + e < free, top = in && u[e] > prefix, tie = in && u[e] == prefix;
      const unsigned to = a + min(b, left);
      if ((top || (tie && b < left)) && to < (unsigned)want) kept[to] = i0 + e;
      a += top;
      b += tie;
    }
  }
}

// Rows of 64 kept tokens to the workspace (TAKE) or from it to their places; a token's row is
// row_bytes / 16 pieces.  The places behind the kept ones get weight zero.
template <int D, bool TAKE>
__global__ __launch_bounds__(256) void kla_kv4_shift_kernel(KvEvictParams p, int blocks) {
  constexpr int CP = D / 32, PIECES = 2 * CP;  // 16-byte pieces of K's (V's) codes, of both
  const int pair = blockIdx.x / blocks, block = blockIdx.x % blocks;
  const int n = pair / p.kv.Hkv, head = pair % p.kv.Hkv;
  const int len = evict_len(p, n);
  if (len <= p.budget) return;
  const int32_t *const kept = p.kept + (size_t)pair * p.budget;
  float *const w = p.w + (size_t)pair * p.W;
  const int r0 = block * 64, r1 = min(r0 + 64, p.budget);
  for (int i = threadIdx.x; i < (r1 - r0) * PIECES; i += 256) {
    const int at = r0 + i / PIECES, pc = i % PIECES, j = pc / CP, b = pc % CP;
    const int from = kept[at];
    if (from == at || (unsigned)from >= (unsigned)len) continue;
    uint8_t *const ws = (uint8_t *)p.rows + ((size_t)pair * p.budget + at) * p.row_bytes;
    const long long row = kv_row(p.kv, n, TAKE ? from : at, j, head);
    u32x4 *const wc = reinterpret_cast<u32x4 *>(ws + 16 * pc);
    uint8_t *const wsc = ws + D + pc;
    if constexpr (TAKE) {
      // a token of a missing page reads as zero
      *wc = row >= 0 ? *reinterpret_cast<const u32x4 *>(p.kv.codes + row * (D / 2) + 16 * b) : u32x4{0, 0, 0, 0};
      *wsc = row >= 0 ? p.kv.scales[row * (D / 32) + b] : 1;
      if (pc == 0) *reinterpret_cast<float *>(ws + D + 16) = w[from];
    } else {
      if (row >= 0) {
        *reinterpret_cast<u32x4 *>(p.kv.codes + row * (D / 2) + 16 * b) = *wc;
        p.kv.scales[row * (D / 32) + b] = *wsc;
      }
      if (pc == 0) w[at] = *reinterpret_cast<float *>(ws + D + 16);
    }
  }
  if constexpr (!TAKE) {
    each_position(p.budget, len, block, blocks, threadIdx.x, [&](long long i) { w[i] = 0.f; });
  }
}

int row_bytes(int D) { return D + 32; }  // codes, 2 D / 32 scales, the weight

// Parts of a choice: one workgroup for all tokens of a (sequence, head), unless those are few
// enough that parts of 4,096 tokens do not make more than 256 (one sequence of 131,071 tokens and
// two heads 60 us, in one piece 184; a batch of 64 sequences and four heads 261 us in one piece
// each, in parts 299; each with what is left read back).
int evict_parts(int N, int Hkv, long long room) {
  const long long pairs = (long long)N * Hkv, parts = (room + EV_PART - 1) / EV_PART;
  return parts > 2 && pairs * parts <= 256 ? (int)parts : 1;
}
size_t up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t kv4_evict_workspace_bytes(int N, int Hkv, int D, int budget, long long room) {
  if (budget >= room) return 0;  // nothing can be cut
  const size_t pairs = (size_t)N * Hkv, parts = evict_parts(N, Hkv, room);
  return up(pairs * budget * row_bytes(D)) + (parts > 1 ? pairs * (3 * parts * EV_BINS + 6 + 2 * parts) * sizeof(unsigned) : 0);
}

bool kv4_evict_grid_fits(int N, int Hkv, int budget) {
  return launch_fits((double)N * Hkv, EV_T) && launch_fits((double)N * Hkv * (budget / 64 + 1), 256);
}

hipError_t launch_kv4_evict(const Kv4Cache &c, const int32_t *lens, int32_t *new_lens, int32_t *kept, float *weights,
                            int N, int D, int W, int budget, int recent, void *workspace, hipStream_t st) {
  const long long room = (long long)c.max_pages * c.page;
  const size_t pairs = (size_t)N * c.Hkv;
  KvEvictParams p{kv_params(c), lens, new_lens, kept, weights, N, D, W, budget, recent, (u32x4 *)workspace,
                  row_bytes(D)};
  p.parts = evict_parts(N, c.Hkv, room);
  const bool cut = budget < room;  // else the choice only says what is there
  if (p.parts > 1) {
    const dim3 grid((unsigned)(pairs * p.parts));
    if (cut) {
      p.hist = (unsigned *)((char *)workspace + up(pairs * budget * row_bytes(D)));
      p.state = p.hist + pairs * 3 * p.parts * EV_BINS;
      p.above = p.state + pairs * 6;
      hipLaunchKernelGGL((kla_kv4_choose_part_kernel<0>), grid, dim3(EV_PT), 0, st, p);
      hipLaunchKernelGGL((kla_kv4_choose_part_kernel<1>), grid, dim3(EV_PT), 0, st, p);
      hipLaunchKernelGGL((kla_kv4_choose_part_kernel<2>), grid, dim3(EV_PT), 0, st, p);
    }
    hipLaunchKernelGGL((kla_kv4_choose_part_kernel<3>), grid, dim3(EV_PT), 0, st, p);
  } else {
    hipLaunchKernelGGL(kla_kv4_choose_kernel, dim3((unsigned)pairs), dim3(EV_T), 0, st, p);
  }
  if (!cut) return hipGetLastError();
  const int blocks = (budget + 63) / 64;
  const dim3 grid((unsigned)(pairs * blocks));
  if (D == 128) {
    hipLaunchKernelGGL((kla_kv4_shift_kernel<128, true>), grid, dim3(256), 0, st, p, blocks);
    hipLaunchKernelGGL((kla_kv4_shift_kernel<128, false>), grid, dim3(256), 0, st, p, blocks);
  } else {
    hipLaunchKernelGGL((kla_kv4_shift_kernel<64, true>), grid, dim3(256), 0, st, p, blocks);
    hipLaunchKernelGGL((kla_kv4_shift_kernel<64, false>), grid, dim3(256), 0, st, p, blocks);
  }
  return hipGetLastError();
}

}  // namespace kla
