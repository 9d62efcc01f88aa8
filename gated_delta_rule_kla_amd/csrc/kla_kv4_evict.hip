// kla_kv4_evict.hip -- a 4-bit cache cut to a budget by the weight its tokens got (gfx950).
//
// Per sequence of more than `budget` tokens and key head: the newest `recent` tokens stay, and of
// the others the `budget - recent` of the largest weight, the earlier of two that are equal; they
// move to the front in their order (include/kla.h, kla_kv4_evict).
//
// Three kernels.  Choice, a workgroup to a (sequence, head): a radix selection finds the smallest
// weight that stays, eight bits of the weights' order at a time (a histogram in LDS per pass; integer counts, so
// the order of the atomics changes nothing); then each wave goes over its part of the tokens and
// writes the positions that stay, at places counted ahead.  Then the rows that change place go
// to a workspace and from there to their places: kept rows move towards the front over rows that
// others still have to read.
// Bound: the choice by its passes over the weights (from L2), the moves by HBM.
#include <algorithm>

#include "kla_common.h"
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

__global__ __launch_bounds__(EV_T) void kla_kv4_choose_kernel(KvEvictParams p) {
  __shared__ unsigned s_hist[256], s_pick, s_left;
  __shared__ int s_more[EV_W], s_same[EV_W];
  const int n = blockIdx.x / p.kv.Hkv, head = blockIdx.x % p.kv.Hkv;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int len = evict_len(p, n);
  int32_t *const kept = p.kept + (size_t)blockIdx.x * p.budget;
  if (head == 0 && tid == 0) p.new_lens[n] = min(len, p.budget);
  if (len <= p.budget) {
    for (int i = tid; i < p.budget; i += EV_T) kept[i] = i < len ? i : -1;
    return;
  }
  const float *const w = p.w + (size_t)blockIdx.x * p.W;
  const int free = len - p.recent, want = p.budget - p.recent;  // free > want
  // the want-th largest of the free tokens' weights, from the top byte down
  unsigned prefix = 0, left = want;
  for (int shift = 24; want > 0 && shift >= 0; shift -= 8) {
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < free; i += EV_T) {
      const unsigned u = order_of(w[i]);
      if (shift == 24 || (u ^ prefix) >> (shift + 8) == 0) atomicAdd(&s_hist[u >> shift & 255], 1u);
    }
    __syncthreads();
    if (wave == 0) {
      // lane l: bins 255 - 4 l and down; the bin in which the count from the top reaches `left`
      unsigned c[4], mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) mine += c[i] = s_hist[255 - 4 * lane - i];
      unsigned upto = mine;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const unsigned v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
      }
      unsigned above = upto - mine;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < left && above + c[i] >= left) {
          s_pick = 255 - 4 * lane - i;
          s_left = left - above;
        }
        above += c[i];
      }
    }
    __syncthreads();
    prefix |= s_pick << shift;
    left = s_left;
    __syncthreads();
  }
  // tokens above `prefix` stay, and the first `left` that equal it; each wave a part of the tokens
  const int per = ((free + EV_W - 1) / EV_W + 63) / 64 * 64, lo = min(wave * per, free), hi = min(lo + per, free);
  int more = 0, same = 0;
  for (int i = lo; i < hi && want > 0; i += 64) {
    const unsigned u = i + lane < hi ? order_of(w[i + lane]) : 0;
    more += __popcll(__ballot(i + lane < hi && u > prefix));
    same += __popcll(__ballot(i + lane < hi && u == prefix));
  }
  if (lane == 0) {
    s_more[wave] = more;
    s_same[wave] = same;
  }
  __syncthreads();
  more = same = 0;  // before this wave's part
  for (int i = 0; i < wave; ++i) {
    more += s_more[i];
    same += s_same[i];
  }
  const unsigned long long below = (1ull << lane) - 1;
  for (int i = lo; i < hi && want > 0; i += 64) {
    const unsigned u = i + lane < hi ? order_of(w[i + lane]) : 0;
    const bool top = i + lane < hi && u > prefix, tie = i + lane < hi && u == prefix;
    const unsigned long long a = __ballot(top), b = __ballot(tie);
    const int before = same + __popcll(b & below);  // equal ones in front of this token
    if (top || (tie && before < (int)left)) kept[more + __popcll(a & below) + min(before, (int)left)] = i + lane;
    more += __popcll(a);
    same += __popcll(b);
  }
  for (int i = tid; i < p.recent; i += EV_T) kept[want + i] = free + i;
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
    if (from == at) continue;
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
    for (int i = p.budget + block * 256 + threadIdx.x; i < len; i += blocks * 256) w[i] = 0.f;
  }
}

int row_bytes(int D) { return D + 32; }  // codes, 2 D / 32 scales, the weight

}  // namespace

size_t kv4_evict_workspace_bytes(int N, int Hkv, int D, int budget) {
  return (size_t)N * Hkv * budget * row_bytes(D);
}

bool kv4_evict_grid_fits(int N, int Hkv, int budget) {
  return launch_fits((double)N * Hkv, EV_T) && launch_fits((double)N * Hkv * (budget / 64 + 1), 256);
}

hipError_t launch_kv4_evict(const Kv4Cache &c, const int32_t *lens, int32_t *new_lens, int32_t *kept, float *weights,
                            int N, int D, int W, int budget, int recent, void *workspace, hipStream_t st) {
  const KvEvictParams p{kv_params(c), lens, new_lens, kept, weights, N, D, W, budget, recent, (u32x4 *)workspace,
                        row_bytes(D)};
  const unsigned pairs = (unsigned)(N * c.Hkv);
  hipLaunchKernelGGL(kla_kv4_choose_kernel, dim3(pairs), dim3(EV_T), 0, st, p);
  const int blocks = (budget + 63) / 64;
  const dim3 grid(pairs * blocks);
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
