// kla_api.cpp -- the C ABI declared in include/kla.h.
//
// Every argument is validated on the host before the first HIP call, so the
// error paths run (and are tested) on machines without a GPU.  After
// validation the call only enqueues kernels on the caller's stream.
#include <cmath>
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <vector>

#include "../../include/kla.h"
#include "kla_internal.h"

namespace {

bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }  // int32 arrays

// Enum-typed arguments come from C callers as plain ints and may hold any value; their
// bytes are read as an int (a read as the C++ enum type is undefined outside the range
// of its enumerators), and everything below works on that int.
template <typename E>
int raw(const E &e) {
  static_assert(sizeof(E) == sizeof(int), "the enums of the C ABI are int-sized");
  int v;
  std::memcpy(&v, &e, sizeof v);
  return v;
}

bool bad_eps(float eps) { return !std::isfinite(eps) || eps < 0.f; }

kla_status_t from_hip(hipError_t e) { return e == hipSuccess ? KLA_OK : KLA_ERR_HIP; }

// Shape, dtype, eps and cu_seqlens checks shared by kla_chunk_fwd and
// kla_chunk_workspace_bytes.
// Heads index the second dimension of the prep, backward and PGDN launch grids, which
// the device caps at 65,536 workgroups.
constexpr int kMaxHeads = 65536;

kla_status_t check_chunk_shapes(float eps, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                                int num_seqs, int B, int H, int T, int dk, int dv, int chunk,
                                int dtype) {
  if (dtype != KLA_DT_BF16 && dtype != KLA_DT_F32) return KLA_ERR_DTYPE;
  if (B < 0 || H <= 0 || T < 0 || dk <= 0 || dv <= 0 || chunk <= 0 || num_seqs < 0)
    return KLA_ERR_SHAPE;
  if (H > kMaxHeads) return KLA_ERR_SHAPE;
  if (bad_eps(eps)) return KLA_ERR_EPS;
  if (!kla::chunk_supported(dtype, dk, dv, chunk)) return KLA_ERR_UNSUPPORTED;
  if (cu_seqlens == nullptr) {
    if (cu_seqlens_host != nullptr) return KLA_ERR_NULL;
    if (num_seqs != B) return KLA_ERR_SHAPE;
  } else {
    if (cu_seqlens_host == nullptr) return KLA_ERR_NULL;
    if (B != 1) return KLA_ERR_SHAPE;
    if (cu_seqlens_host[0] != 0 || cu_seqlens_host[num_seqs] != T) return KLA_ERR_SEQLENS;
    for (int n = 0; n < num_seqs; ++n)
      if (cu_seqlens_host[n + 1] < cu_seqlens_host[n]) return KLA_ERR_SEQLENS;
    if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return KLA_ERR_ALIGN;
  }
  if ((long long)num_seqs * H * ((dv + 15) / 16) > 0x7fffffffLL) return KLA_ERR_SHAPE;
  if ((long long)B * H * T > (1LL << 40)) return KLA_ERR_SHAPE;
  // workspace slots per head (see kla_chunk.hip): a grid dimension and int-indexed
  const long long slots = cu_seqlens ? (long long)T / chunk + num_seqs + 1
                                     : (long long)B * ((T + (long long)chunk - 1) / chunk);
  if (slots > 0x7fffffffLL) return KLA_ERR_SHAPE;
  return KLA_OK;
}

kla::ChunkArgs chunk_args(const void *q, const void *k, const void *v, const void *g, const void *eta,
                          float eps, const float *initial_state, void *o, float *final_state,
                          const int32_t *cu_seqlens, int num_seqs, int B, int H, int T, int dk, int dv,
                          int chunk, int dtype, void *workspace, int beta_direct) {
  return kla::ChunkArgs{q,          k,        v, g, eta, eps, initial_state, o,     final_state,
                        cu_seqlens, num_seqs, B, H, T,   dk,  dv,            chunk, dtype,
                        workspace,  beta_direct};
}

kla_status_t decode_impl(const void *q, const void *k, const void *v, const void *g, const void *eta,
                         float eps, int beta_direct, float *state, void *o, int N, int H, int dk, int dv,
                         int dtype, void *stream) {
  if (dtype != KLA_DT_BF16 && dtype != KLA_DT_F32) return KLA_ERR_DTYPE;
  if (N < 0 || H <= 0 || dk <= 0 || dv <= 0) return KLA_ERR_SHAPE;
  if (bad_eps(eps)) return KLA_ERR_EPS;
  if (!kla::decode_supported(dtype, dk, dv)) return KLA_ERR_UNSUPPORTED;
  if (N == 0) return KLA_OK;
  if (!q || !k || !v || !g || !eta || !state || !o) return KLA_ERR_NULL;
  if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(g) || misaligned(eta) ||
      misaligned(state) || misaligned(o))
    return KLA_ERR_ALIGN;
  if ((long long)N * H > 0x7fffffffLL) return KLA_ERR_SHAPE;
  kla::DecodeArgs a{q, k, v, g, eta, eps, state, o, N, H, dk, dv, dtype, beta_direct};
  return from_hip(kla::launch_decode(a, reinterpret_cast<hipStream_t>(stream)));
}

// Segments of a forward call: seg_req < 0 the library's choice (0 where it keeps one
// segment per sequence), 0 none, > 0 that many chunks each.  KLA_ERR_UNSUPPORTED for a
// requested length on shapes the segmented scan does not run; KLA_ERR_SHAPE when the
// segment grid would not fit its int indices.  *L = 0: one segment per sequence.
kla_status_t seg_length(const kla::ChunkArgs &a, const int32_t *cu_seqlens_host, int seg_req, int *L) {
  *L = 0;
  if (seg_req == 0) return KLA_OK;
  const bool chosen = seg_req < 0;
  if (!kla::chunk_seg_supported(a.dtype, a.dk, a.dv, a.chunk)) return chosen ? KLA_OK : KLA_ERR_UNSUPPORTED;
  const int len = chosen ? kla::chunk_auto_seg_chunks(a, cu_seqlens_host) : seg_req;
  if (len <= 0) return KLA_OK;
  const long long nseg = kla::chunk_seg_count(a, cu_seqlens_host, len);
  if (nseg * a.H * (a.dv / 16 + a.dk / 16) > 0x7fffffffLL) return chosen ? KLA_OK : KLA_ERR_SHAPE;
  *L = len;
  return KLA_OK;
}

// static_scratch: take the workspace from the library's fixed per-GPU buffer
// (kla_chunk_fwd_noalloc) instead of the caller's.  seg_req: as seg_length; with the
// library's choice, a workspace (or scratch) too small for the segments' buffers
// runs the call unsegmented.
kla_status_t chunk_fwd_impl(const void *q, const void *k, const void *v, const void *g, const void *eta,
                            float eps, int beta_direct, const float *initial_state, void *o,
                            float *final_state, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                            int num_seqs, int B, int H, int T, int dk, int dv, int chunk, void *workspace,
                            size_t workspace_bytes, int dtype, void *stream,
                            bool static_scratch = false, int seg_req = -1) {
  const kla_status_t st =
      check_chunk_shapes(eps, cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dk, dv, chunk, dtype);
  if (st != KLA_OK) return st;
  if (seg_req > 0 && !kla::chunk_seg_supported(dtype, dk, dv, chunk)) return KLA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return KLA_OK;
  // token tensors are only dereferenced when there are tokens
  if ((long long)B * T > 0 && (!q || !k || !v || !g || !eta || !o)) return KLA_ERR_NULL;
  if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(g) || misaligned(eta) ||
      misaligned(o) || misaligned(initial_state) || misaligned(final_state) || misaligned(workspace))
    return KLA_ERR_ALIGN;
  kla::ChunkArgs a = chunk_args(q, k, v, g, eta, eps, initial_state, o, final_state, cu_seqlens, num_seqs,
                                B, H, T, dk, dv, chunk, dtype, workspace, beta_direct);
  int L = 0;
  const kla_status_t sst = seg_length(a, cu_seqlens_host, seg_req, &L);
  if (sst != KLA_OK) return sst;
  size_t need = (long long)B * T > 0 ? kla::chunk_workspace_bytes(a) : 0;
  if (L > 0) {
    const size_t seg_need = kla::chunk_seg_workspace_bytes(a, cu_seqlens_host, L);
    const size_t have = static_scratch ? kla::static_scratch_bytes() : (workspace ? workspace_bytes : 0);
    if (seg_req < 0 && have < seg_need)
      L = 0;  // the library's choice falls back to one segment per sequence
    else
      need = seg_need;
  }
  if (static_scratch) {
    // every check above and this one run before the first HIP call
    if (need > kla::static_scratch_bytes()) return KLA_ERR_SCRATCH;
    if (need > 0) {
      void *p = nullptr;
      if (kla::static_scratch(&p) != hipSuccess) return KLA_ERR_HIP;
      a.workspace = p;
    }
  } else if (need > 0 && (workspace == nullptr || workspace_bytes < need)) {
    return KLA_ERR_WORKSPACE;
  }
  if (L > 0) return from_hip(kla::launch_chunk_fwd_seg(a, cu_seqlens_host, L, reinterpret_cast<hipStream_t>(stream)));
  return from_hip(kla::launch_chunk_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t chunk_ws_impl(const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B, int H, int T,
                     int dk, int dv, int chunk, int dtype, int seg_req) {
  if (check_chunk_shapes(0.f, cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dk, dv, chunk, dtype) != KLA_OK)
    return 0;
  if (seg_req > 0 && !kla::chunk_seg_supported(dtype, dk, dv, chunk)) return 0;
  if (num_seqs == 0) return 0;
  const kla::ChunkArgs a = chunk_args(nullptr, nullptr, nullptr, nullptr, nullptr, 0.f, nullptr, nullptr, nullptr,
                                      cu_seqlens, num_seqs, B, H, T, dk, dv, chunk, dtype, nullptr, 0);
  int L = 0;
  if (seg_length(a, cu_seqlens_host, seg_req, &L) != KLA_OK) return 0;
  if (L > 0) return kla::chunk_seg_workspace_bytes(a, cu_seqlens_host, L);
  return (long long)B * T == 0 ? 0 : kla::chunk_workspace_bytes(a);
}

kla_status_t chunk_bwd_impl(const void *q, const void *k, const void *v, const void *g, const void *eta,
                            float eps, int beta_direct, const float *initial_state, const void *dout,
                            const float *dfinal_state, void *dq, void *dk, void *dv, float *dg, float *deta,
                            float *dinitial_state, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                            int num_seqs, int B, int H, int T, int dkk, int dvv, int chunk, void *workspace,
                            size_t workspace_bytes, int dtype, void *stream) {
  const kla_status_t st =
      check_chunk_shapes(eps, cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dkk, dvv, chunk, dtype);
  if (st != KLA_OK) return st;
  if (!kla::chunk_bwd_supported(dtype, dkk, dvv, chunk)) return KLA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return KLA_OK;
  if ((long long)B * T > 0 &&
      (!q || !k || !v || !g || !eta || !dout || !dq || !dk || !dv || !dg || !deta))
    return KLA_ERR_NULL;
  if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(g) || misaligned(eta) ||
      misaligned(initial_state) || misaligned(dout) || misaligned(dfinal_state) || misaligned(dq) ||
      misaligned(dk) || misaligned(dv) || misaligned(dg) || misaligned(deta) || misaligned(dinitial_state) ||
      misaligned(workspace))
    return KLA_ERR_ALIGN;
  const kla::ChunkArgs a = chunk_args(q, k, v, g, eta, eps, initial_state, nullptr, nullptr, cu_seqlens,
                                      num_seqs, B, H, T, dkk, dvv, chunk, dtype, workspace, beta_direct);
  const size_t need = (long long)B * T > 0 ? kla::chunk_bwd_workspace_bytes(a) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KLA_ERR_WORKSPACE;
  const kla::ChunkBwdArgs b{dout, dfinal_state, dq, dk, dv, dg, deta, dinitial_state};
  return from_hip(kla::launch_chunk_bwd(a, b, reinterpret_cast<hipStream_t>(stream)));
}

kla_status_t check_pgdn(int gain, float band, float eps) {
  if (gain != KLA_GAIN_GIVEN && gain != KLA_GAIN_KACZMARZ) return KLA_ERR_PARAM;
  if (!std::isfinite(band) || band < 1.f) return KLA_ERR_PARAM;
  if (gain == KLA_GAIN_KACZMARZ && bad_eps(eps)) return KLA_ERR_EPS;
  return KLA_OK;
}

// Layout of a packed or dense batch of sequences: num_seqs, cu_seqlens and its host mirror
// against B and T.  *longest: tokens of the longest sequence.
kla_status_t check_seqs(const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B, int T,
                        int *longest) {
  *longest = T;
  if (cu_seqlens == nullptr) {
    if (cu_seqlens_host != nullptr) return KLA_ERR_NULL;
    return num_seqs == B ? KLA_OK : KLA_ERR_SHAPE;
  }
  if (cu_seqlens_host == nullptr) return KLA_ERR_NULL;
  if (B != 1) return KLA_ERR_SHAPE;
  if (cu_seqlens_host[0] != 0 || cu_seqlens_host[num_seqs] != T) return KLA_ERR_SEQLENS;
  *longest = 0;
  for (int n = 0; n < num_seqs; ++n) {
    if (cu_seqlens_host[n + 1] < cu_seqlens_host[n]) return KLA_ERR_SEQLENS;
    *longest = std::max(*longest, cu_seqlens_host[n + 1] - cu_seqlens_host[n]);
  }
  return (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) ? KLA_ERR_ALIGN : KLA_OK;
}

// Tokens of a sequence dimension: tile arithmetic in ints may run one tile past the end.
constexpr int kMaxTokens = 0x7fffffff - 65536;

kla_status_t check_glr(const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B, int H, int T,
                       int d, int dtype, kla::GlrArgs *a) {
  if (dtype != KLA_DT_BF16 && dtype != KLA_DT_F32) return KLA_ERR_DTYPE;
  if (B < 0 || H <= 0 || T < 0 || T > kMaxTokens || d <= 0 || d > (1 << 24) || num_seqs < 0) return KLA_ERR_SHAPE;
  if ((long long)B * H > 0x7fffffffLL || (double)B * H * T > (double)(1LL << 40)) return KLA_ERR_SHAPE;
  *a = kla::GlrArgs{};
  const kla_status_t st = check_seqs(cu_seqlens, cu_seqlens_host, num_seqs, B, T, &a->longest);
  if (st != KLA_OK) return st;
  a->cu_seqlens = cu_seqlens;
  a->cu_seqlens_host = cu_seqlens_host;
  a->num_seqs = num_seqs;
  a->H = H;
  a->T = T;
  a->d = d;
  a->dtype = dtype;
  return kla::glr_grid_fits(*a) ? KLA_OK : KLA_ERR_SHAPE;
}

kla_status_t run_glr(kla::GlrArgs &a, bool bwd, void *workspace, size_t workspace_bytes, void *stream) {
  const size_t need = kla::glr_workspace_bytes(a);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KLA_ERR_WORKSPACE;
  a.workspace = workspace;
  return from_hip(kla::launch_glr_chunk(a, bwd, reinterpret_cast<hipStream_t>(stream)));
}

// The 4-bit cache's own arguments.
kla_status_t check_kv4(int Hkv, int D, int num_pages, int page_size, int max_pages, int N, int dtype) {
  if (dtype != KLA_DT_BF16 && dtype != KLA_DT_F32) return KLA_ERR_DTYPE;
  if (N < 0 || Hkv <= 0 || Hkv > (1 << 20) || D <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0)
    return KLA_ERR_SHAPE;
  if ((D != 64 && D != 128) || page_size % 16 != 0 || page_size > (1 << 20)) return KLA_ERR_UNSUPPORTED;
  return KLA_OK;
}

kla_status_t kv4_move(void *k, void *v, const void *codes, const void *scales, const int32_t *table,
                      const int32_t *start, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs,
                      int B, int Hkv, int T, int D, int num_pages, int page_size, int max_pages, int dtype, bool read,
                      void *stream) {
  kla_status_t st = check_kv4(Hkv, D, num_pages, page_size, max_pages, num_seqs, dtype);
  if (st != KLA_OK) return st;
  if (B < 0 || T < 0 || T > kMaxTokens) return KLA_ERR_SHAPE;
  int longest;
  st = check_seqs(cu_seqlens, cu_seqlens_host, num_seqs, B, T, &longest);
  if (st != KLA_OK) return st;
  if ((double)B * Hkv * T > (double)0x7fffffff || !kla::kv4_move_grid_fits(B, Hkv, T, D, dtype, read)) return KLA_ERR_SHAPE;
  if (num_seqs == 0 || (long long)B * T == 0) return KLA_OK;
  if (!k || !v || !codes || !scales || !table || !start) return KLA_ERR_NULL;
  if (misaligned(k) || misaligned(v) || misaligned(codes) || misaligned(scales) || misaligned4(table) ||
      misaligned4(start))
    return KLA_ERR_ALIGN;
  const kla::Kv4Cache c{const_cast<void *>(codes), const_cast<void *>(scales), table, num_pages, page_size, max_pages,
                        Hkv};
  return from_hip(kla::launch_kv4_move(c, k, v, start, cu_seqlens, num_seqs, B, T, D, dtype, read,
                                       reinterpret_cast<hipStream_t>(stream)));
}

// The decode step's sizes; a's sizes are set where they are fine.
kla_status_t check_kv4_decode(int N, int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages, int max_len,
                              int dtype, kla::Kv4DecodeArgs *a) {
  const kla_status_t st = check_kv4(Hkv, D, num_pages, page_size, max_pages, N, dtype);
  if (st != KLA_OK) return st;
  if (Hq <= 0 || Hq > (1 << 20) || Hq % Hkv != 0 || max_len < 0 || max_len > kMaxTokens) return KLA_ERR_SHAPE;
  *a = kla::Kv4DecodeArgs{};
  a->c.num_pages = num_pages;
  a->c.page = page_size;
  a->c.max_pages = max_pages;
  a->c.Hkv = Hkv;
  a->N = N;
  a->Hq = Hq;
  a->D = D;
  a->max_len = max_len;
  a->dtype = dtype;
  return kla::kv4_decode_grid_fits(*a) ? KLA_OK : KLA_ERR_SHAPE;
}

// Attention's scale, also as the kernels take it: times log2(e).
bool good_scale(float scale) { return std::isfinite(scale * 1.44269504f); }

float band_log(float band) { return band == 1.f ? 0.f : std::log(band); }

}  // namespace

extern "C" {

size_t kla_pgdn_chunk_workspace_bytes(const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs,
                                      int B, int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_) {
  const int dtype = raw(dtype_);
  if (check_chunk_shapes(0.f, cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dk, dv, chunk, dtype) != KLA_OK)
    return 0;
  if (num_seqs == 0 || (long long)B * T == 0) return 0;
  return kla::pgdn_workspace_bytes(chunk_args(nullptr, nullptr, nullptr, nullptr, nullptr, 0.f, nullptr, nullptr,
                                              nullptr, cu_seqlens, num_seqs, B, H, T, dk, dv, chunk, dtype,
                                              nullptr, 0));
}

kla_status_t kla_pgdn_chunk_fwd(const void *q, const void *k, const void *v, const void *g, const void *coef,
                                float eps, kla_gain_t gain_, float band, const float *initial_state,
                                const float *initial_acc, void *o, float *final_state, float *final_acc,
                                const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B,
                                int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_, void *workspace,
                                size_t workspace_bytes, void *stream) {
  const int dtype = raw(dtype_), gain = raw(gain_);
  if (dtype != KLA_DT_BF16 && dtype != KLA_DT_F32) return KLA_ERR_DTYPE;
  kla_status_t st = check_pgdn(gain, band, eps);
  if (st != KLA_OK) return st;
  const float e = gain == KLA_GAIN_KACZMARZ ? eps : 0.f;
  st = check_chunk_shapes(e, cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dk, dv, chunk, dtype);
  if (st != KLA_OK) return st;
  if (!kla::general_supported(dtype, dk, dv, chunk)) return KLA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return KLA_OK;
  if ((long long)B * T > 0 && (!q || !k || !v || !g || !coef || !o)) return KLA_ERR_NULL;
  if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(g) || misaligned(coef) || misaligned(o) ||
      misaligned(initial_state) || misaligned(final_state) || misaligned(initial_acc) || misaligned(final_acc) ||
      misaligned(workspace))
    return KLA_ERR_ALIGN;
  const kla::ChunkArgs a = chunk_args(q, k, v, g, coef, e, initial_state, o, final_state, cu_seqlens, num_seqs, B,
                                      H, T, dk, dv, chunk, dtype, workspace, gain == KLA_GAIN_GIVEN ? 1 : 0);
  const kla::GenExtra x{1, band_log(band), initial_acc, final_acc};
  if (kla::pgdn_fast_supported(dtype, dk, dv, chunk)) {
    const size_t need = (long long)B * T > 0 ? kla::pgdn_workspace_bytes(a) : 0;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KLA_ERR_WORKSPACE;
    return from_hip(kla::launch_pgdn_fast(a, x, reinterpret_cast<hipStream_t>(stream)));
  }
  return from_hip(kla::launch_chunk_general(a, x, reinterpret_cast<hipStream_t>(stream)));
}

kla_status_t kla_pgdn_decode_step(const void *q, const void *k, const void *v, const void *g, const void *coef,
                                  float eps, kla_gain_t gain_, float band, float *state, float *acc, void *o,
                                  int N, int H, int dk, int dv, kla_dtype_t dtype_, void *stream) {
  const int dtype = raw(dtype_), gain = raw(gain_);
  if (dtype != KLA_DT_BF16 && dtype != KLA_DT_F32) return KLA_ERR_DTYPE;
  if (N < 0 || H <= 0 || dk <= 0 || dv <= 0) return KLA_ERR_SHAPE;
  const kla_status_t st = check_pgdn(gain, band, eps);
  if (st != KLA_OK) return st;
  if (!kla::pgdn_decode_supported(dtype, dk, dv)) return KLA_ERR_UNSUPPORTED;
  if (N == 0) return KLA_OK;
  if (!q || !k || !v || !g || !coef || !state || !acc || !o) return KLA_ERR_NULL;
  if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(g) || misaligned(coef) || misaligned(state) ||
      misaligned(acc) || misaligned(o))
    return KLA_ERR_ALIGN;
  if ((long long)N * H > 0x7fffffffLL) return KLA_ERR_SHAPE;
  const float e = gain == KLA_GAIN_KACZMARZ ? eps : 0.f;
  kla::DecodeArgs a{q, k, v, g, coef, e, state, o, N, H, dk, dv, dtype, gain == KLA_GAIN_GIVEN ? 1 : 0};
  return from_hip(kla::launch_pgdn_decode(a, band_log(band), acc, reinterpret_cast<hipStream_t>(stream)));
}

int kla_abi_version(void) { return KLA_ABI_VERSION; }

const char *kla_status_str(kla_status_t s) {
  switch (raw(s)) {
    case KLA_OK: return "ok";
    case KLA_ERR_NULL: return "a required pointer is NULL";
    case KLA_ERR_SHAPE: return "invalid or inconsistent sizes";
    case KLA_ERR_DTYPE: return "unknown dtype";
    case KLA_ERR_UNSUPPORTED: return "shape/dtype/chunk combination not compiled";
    case KLA_ERR_SEQLENS: return "cu_seqlens must be non-decreasing from 0 to T";
    case KLA_ERR_EPS: return "eps must be finite and >= 0";
    case KLA_ERR_ALIGN: return "data pointers must be 16-byte aligned";
    case KLA_ERR_WORKSPACE: return "workspace missing or smaller than the entry point's _workspace_bytes function says";
    case KLA_ERR_HIP: return "HIP runtime error";
    case KLA_ERR_PARAM: return "gain must be a kla_gain_t and band finite and >= 1; an attention scale finite, up to 2.3e38";
    case KLA_ERR_SCRATCH: return "the call needs more scratch than kla_chunk_fwd_noalloc's fixed buffer holds";
  }
  return "unknown status";
}

size_t kla_chunk_workspace_bytes(const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs,
                                 int B, int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_) {
  return chunk_ws_impl(cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dk, dv, chunk, raw(dtype_), -1);
}

size_t kla_chunk_seg_workspace_bytes(const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs,
                                     int B, int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_,
                                     int seg_chunks) {
  if (seg_chunks < 0) return 0;
  return chunk_ws_impl(cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dk, dv, chunk, raw(dtype_), seg_chunks);
}

kla_status_t kla_chunk_fwd_seg(const void *q, const void *k, const void *v, const void *g, const void *eta,
                               float eps, const float *initial_state, void *o, float *final_state,
                               const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B,
                               int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_, int seg_chunks,
                               void *workspace, size_t workspace_bytes, void *stream) {
  if (seg_chunks < 0) return KLA_ERR_SHAPE;
  return chunk_fwd_impl(q, k, v, g, eta, eps, 0, initial_state, o, final_state, cu_seqlens, cu_seqlens_host,
                        num_seqs, B, H, T, dk, dv, chunk, workspace, workspace_bytes, raw(dtype_), stream, false,
                        seg_chunks);
}

kla_status_t kla_chunk_fwd(const void *q, const void *k, const void *v, const void *g,
                           const void *eta, float eps, const float *initial_state, void *o,
                           float *final_state, const int32_t *cu_seqlens,
                           const int32_t *cu_seqlens_host, int num_seqs, int B, int H, int T,
                           int dk, int dv, int chunk, kla_dtype_t dtype_, void *workspace,
                           size_t workspace_bytes, void *stream) {
  const int dtype = raw(dtype_);
  return chunk_fwd_impl(q, k, v, g, eta, eps, 0, initial_state, o, final_state, cu_seqlens, cu_seqlens_host,
                        num_seqs, B, H, T, dk, dv, chunk, workspace, workspace_bytes, dtype, stream);
}

kla_status_t kla_gdn_chunk_fwd(const void *q, const void *k, const void *v, const void *g,
                               const void *beta, const float *initial_state, void *o, float *final_state,
                               const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs,
                               int B, int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_,
                               void *workspace, size_t workspace_bytes, void *stream) {
  const int dtype = raw(dtype_);
  return chunk_fwd_impl(q, k, v, g, beta, 0.f, 1, initial_state, o, final_state, cu_seqlens, cu_seqlens_host,
                        num_seqs, B, H, T, dk, dv, chunk, workspace, workspace_bytes, dtype, stream);
}

kla_status_t kla_chunk_fwd_noalloc(const void *q, const void *k, const void *v, const void *g, const void *eta,
                                   float eps, const float *initial_state, void *o, float *final_state,
                                   const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs,
                                   int B, int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_,
                                   void *stream) {
  const int dtype = raw(dtype_);
  return chunk_fwd_impl(q, k, v, g, eta, eps, 0, initial_state, o, final_state, cu_seqlens, cu_seqlens_host,
                        num_seqs, B, H, T, dk, dv, chunk, nullptr, 0, dtype, stream, true);
}

size_t kla_chunk_fwd_workspace_bytes(int B, int H, int T, int dk, int dv, int chunk, int num_seqs) {
  // neither the element type nor the layout is an argument: the largest need
  // over both element types and over the dense (num_seqs == B) and packed
  // layouts.  A packed layout needs B == 1; its size only depends on
  // cu_seqlens through num_seqs, so a valid mirror (all tokens in the last
  // sequence) stands in for the caller's.
  if (B < 0 || T < 0 || num_seqs < 0 || T >= 0x7fffffff) return 0;
  size_t best = 0;
  for (const kla_dtype_t dt : {KLA_DT_BF16, KLA_DT_F32}) {
    if (num_seqs == B) best = std::max(best, kla_chunk_workspace_bytes(nullptr, nullptr, B, B, H, T, dk, dv, chunk, dt));
    if (B == 1 && num_seqs >= 1) {
      std::vector<int32_t> cu((size_t)num_seqs + 1, 0);
      cu[num_seqs] = T;
      const int32_t *dev_stub = cu.data();  // only tested for NULL here
      best = std::max(best, kla_chunk_workspace_bytes(dev_stub, cu.data(), num_seqs, 1, H, T, dk, dv, chunk, dt));
    }
  }
  return best;
}

size_t kla_chunk_bwd_workspace_bytes(const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs,
                                     int B, int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_) {
  const int dtype = raw(dtype_);
  if (check_chunk_shapes(0.f, cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dk, dv, chunk, dtype) != KLA_OK)
    return 0;
  if (!kla::chunk_bwd_supported(dtype, dk, dv, chunk)) return 0;
  if (num_seqs == 0 || (long long)B * T == 0) return 0;
  return kla::chunk_bwd_workspace_bytes(chunk_args(nullptr, nullptr, nullptr, nullptr, nullptr, 0.f, nullptr,
                                                   nullptr, nullptr, cu_seqlens, num_seqs, B, H, T, dk, dv,
                                                   chunk, dtype, nullptr, 0));
}

kla_status_t kla_chunk_bwd(const void *q, const void *k, const void *v, const void *g, const void *eta,
                           float eps, const float *initial_state, const void *dout, const float *dfinal_state,
                           void *dq, void *dk_, void *dv_, float *dg, float *deta, float *dinitial_state,
                           const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B,
                           int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_, void *workspace,
                           size_t workspace_bytes, void *stream) {
  const int dtype = raw(dtype_);
  return chunk_bwd_impl(q, k, v, g, eta, eps, 0, initial_state, dout, dfinal_state, dq, dk_, dv_, dg, deta,
                        dinitial_state, cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dk, dv, chunk, workspace,
                        workspace_bytes, dtype, stream);
}

kla_status_t kla_gdn_chunk_bwd(const void *q, const void *k, const void *v, const void *g, const void *beta,
                               const float *initial_state, const void *dout, const float *dfinal_state, void *dq,
                               void *dk_, void *dv_, float *dg, float *dbeta, float *dinitial_state,
                               const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B,
                               int H, int T, int dk, int dv, int chunk, kla_dtype_t dtype_, void *workspace,
                               size_t workspace_bytes, void *stream) {
  const int dtype = raw(dtype_);
  return chunk_bwd_impl(q, k, v, g, beta, 0.f, 1, initial_state, dout, dfinal_state, dq, dk_, dv_, dg, dbeta,
                        dinitial_state, cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, dk, dv, chunk, workspace,
                        workspace_bytes, dtype, stream);
}

kla_status_t kla_decode_step(const void *q, const void *k, const void *v, const void *g,
                             const void *eta, float eps, float *state, void *o, int N, int H,
                             int dk, int dv, kla_dtype_t dtype_, void *stream) {
  const int dtype = raw(dtype_);
  return decode_impl(q, k, v, g, eta, eps, 0, state, o, N, H, dk, dv, dtype, stream);
}

kla_status_t kla_gdn_decode_step(const void *q, const void *k, const void *v, const void *g,
                                 const void *beta, float *state, void *o, int N, int H, int dk, int dv,
                                 kla_dtype_t dtype_, void *stream) {
  const int dtype = raw(dtype_);
  return decode_impl(q, k, v, g, beta, 0.f, 1, state, o, N, H, dk, dv, dtype, stream);
}

size_t kla_glr_chunk_workspace_bytes(const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B,
                                     int H, int T, int d, kla_dtype_t dtype_) {
  kla::GlrArgs a;
  if (check_glr(cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, d, raw(dtype_), &a) != KLA_OK) return 0;
  return num_seqs == 0 ? 0 : kla::glr_workspace_bytes(a);
}

kla_status_t kla_glr_chunk_fwd(const void *x, const void *g, const float *initial_state, void *o, float *final_state,
                               const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B, int H,
                               int T, int d, kla_dtype_t dtype_, void *workspace, size_t workspace_bytes,
                               void *stream) {
  kla::GlrArgs a;
  const kla_status_t st = check_glr(cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, d, raw(dtype_), &a);
  if (st != KLA_OK) return st;
  if (num_seqs == 0) return KLA_OK;
  if ((long long)B * T > 0 && (!x || !g || !o)) return KLA_ERR_NULL;
  if (misaligned(x) || misaligned(g) || misaligned(initial_state) || misaligned(o) || misaligned(final_state) ||
      misaligned(workspace))
    return KLA_ERR_ALIGN;
  a.x = x;
  a.g = g;
  a.y0 = initial_state;
  a.o = o;
  a.yend = final_state;
  return run_glr(a, false, workspace, workspace_bytes, stream);
}

kla_status_t kla_glr_chunk_bwd(const void *g, const void *o, const float *initial_state, const void *dout,
                               const float *dfinal_state, void *dx, void *dg, float *dinitial_state,
                               const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int num_seqs, int B, int H,
                               int T, int d, kla_dtype_t dtype_, void *workspace, size_t workspace_bytes,
                               void *stream) {
  kla::GlrArgs a;
  const kla_status_t st = check_glr(cu_seqlens, cu_seqlens_host, num_seqs, B, H, T, d, raw(dtype_), &a);
  if (st != KLA_OK) return st;
  if (num_seqs == 0) return KLA_OK;
  if ((long long)B * T > 0 && (!g || !o || !dout || !dx || !dg)) return KLA_ERR_NULL;
  if (misaligned(g) || misaligned(o) || misaligned(initial_state) || misaligned(dout) || misaligned(dfinal_state) ||
      misaligned(dx) || misaligned(dg) || misaligned(dinitial_state) || misaligned(workspace))
    return KLA_ERR_ALIGN;
  a.x = dout;
  a.g = g;
  a.h = o;
  a.y0 = dfinal_state;
  a.h0 = initial_state;
  a.o = dx;
  a.dg = dg;
  a.yend = dinitial_state;
  return run_glr(a, true, workspace, workspace_bytes, stream);
}

kla_status_t kla_glr_decode_step(const void *x, const void *g, float *state, void *o, int N, int H, int d,
                                 kla_dtype_t dtype_, void *stream) {
  const int dtype = raw(dtype_);
  if (dtype != KLA_DT_BF16 && dtype != KLA_DT_F32) return KLA_ERR_DTYPE;
  if (N < 0 || H <= 0 || d <= 0 || (long long)N * H > 0x7fffffffLL) return KLA_ERR_SHAPE;
  if (!kla::glr_step_fits((size_t)N * H * d, dtype)) return KLA_ERR_SHAPE;
  if (N == 0) return KLA_OK;
  if (!x || !g || !state || !o) return KLA_ERR_NULL;
  if (misaligned(x) || misaligned(g) || misaligned(state) || misaligned(o)) return KLA_ERR_ALIGN;
  return from_hip(kla::launch_glr_step(x, g, state, o, (size_t)N * H * d, dtype, reinterpret_cast<hipStream_t>(stream)));
}

kla_status_t kla_kv4_append(const void *k, const void *v, void *codes, void *scales, const int32_t *block_table,
                            const int32_t *start, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                            int num_seqs, int B, int Hkv, int T, int D, int num_pages, int page_size, int max_pages,
                            kla_dtype_t dtype_, void *stream) {
  return kv4_move(const_cast<void *>(k), const_cast<void *>(v), codes, scales, block_table, start, cu_seqlens,
                  cu_seqlens_host, num_seqs, B, Hkv, T, D, num_pages, page_size, max_pages, raw(dtype_), false, stream);
}

kla_status_t kla_kv4_read(void *k, void *v, const void *codes, const void *scales, const int32_t *block_table,
                          const int32_t *start, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                          int num_seqs, int B, int Hkv, int T, int D, int num_pages, int page_size, int max_pages,
                          kla_dtype_t dtype_, void *stream) {
  return kv4_move(k, v, codes, scales, block_table, start, cu_seqlens, cu_seqlens_host, num_seqs, B, Hkv, T, D,
                  num_pages, page_size, max_pages, raw(dtype_), true, stream);
}

size_t kla_attn_kv4_decode_workspace_bytes(int N, int Hq, int Hkv, int D, int max_len, kla_dtype_t dtype_) {
  kla::Kv4DecodeArgs a;
  if (check_kv4_decode(N, Hq, Hkv, D, 1, 16, 1, max_len, raw(dtype_), &a) != KLA_OK || N == 0) return 0;
  return kla::kv4_decode_workspace_bytes(a);
}

kla_status_t kla_attn_kv4_decode_step(const void *q, const void *codes, const void *scales,
                                      const int32_t *block_table, const int32_t *seq_lens, float scale, void *o, int N,
                                      int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages, int max_len,
                                      kla_dtype_t dtype_, void *workspace, size_t workspace_bytes, void *stream) {
  kla::Kv4DecodeArgs a;
  const kla_status_t st =
      check_kv4_decode(N, Hq, Hkv, D, num_pages, page_size, max_pages, max_len, raw(dtype_), &a);
  if (st != KLA_OK) return st;
  if (!good_scale(scale)) return KLA_ERR_PARAM;
  if (N == 0) return KLA_OK;
  if (!q || !codes || !scales || !block_table || !seq_lens || !o) return KLA_ERR_NULL;
  if (misaligned(q) || misaligned(codes) || misaligned(scales) || misaligned4(block_table) ||
      misaligned4(seq_lens) || misaligned(o) || misaligned(workspace))
    return KLA_ERR_ALIGN;
  const size_t need = kla::kv4_decode_workspace_bytes(a);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KLA_ERR_WORKSPACE;
  a.c.codes = const_cast<void *>(codes);
  a.c.scales = const_cast<void *>(scales);
  a.c.table = block_table;
  a.q = q;
  a.o = o;
  a.lens = seq_lens;
  a.scale = scale;
  return from_hip(kla::launch_attn_kv4_decode(a, workspace, reinterpret_cast<hipStream_t>(stream)));
}

kla_status_t kla_attn_fwd(const void *q, const void *k, const void *v, float scale, void *o, float *lse,
                          const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, const int32_t *cu_seqlens_k,
                          const int32_t *cu_seqlens_k_host, int num_seqs, int B, int Hq, int Hkv, int Tq, int Tk, int D,
                          kla_dtype_t dtype_, void *stream) {
  const int dtype = raw(dtype_);
  if (dtype != KLA_DT_BF16 && dtype != KLA_DT_F32) return KLA_ERR_DTYPE;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Tq < 0 || Tk < 0 || Tq > kMaxTokens || Tk > kMaxTokens ||
      D <= 0 || num_seqs < 0)
    return KLA_ERR_SHAPE;
  if (!kla::attn_supported(dtype, D)) return KLA_ERR_UNSUPPORTED;
  if ((long long)B * Hq > 0x7fffffffLL) return KLA_ERR_SHAPE;
  if (!good_scale(scale)) return KLA_ERR_PARAM;
  int longest;
  kla_status_t st = check_seqs(cu_seqlens, cu_seqlens_host, num_seqs, B, Tq, &longest);
  if (st != KLA_OK) return st;
  if ((cu_seqlens_k == nullptr) != (cu_seqlens_k_host == nullptr)) return KLA_ERR_NULL;
  if (cu_seqlens_k != nullptr) {
    if (cu_seqlens == nullptr) return KLA_ERR_NULL;
    st = check_seqs(cu_seqlens_k, cu_seqlens_k_host, num_seqs, B, Tk, &longest);
    if (st != KLA_OK) return st;
  } else if (cu_seqlens != nullptr && Tk != Tq) {
    return KLA_ERR_SHAPE;
  }
  const kla::AttnArgs a{q, k, v, o, lse, cu_seqlens, cu_seqlens_k ? cu_seqlens_k : cu_seqlens, scale, num_seqs, B, Hq,
                        Hkv, Tq, Tk, D, dtype};
  if (!kla::attn_grid_fits(a)) return KLA_ERR_SHAPE;
  if (num_seqs == 0 || (long long)B * Tq == 0) return KLA_OK;
  if (!q || !o || (Tk > 0 && (!k || !v))) return KLA_ERR_NULL;
  if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(o) || misaligned(lse)) return KLA_ERR_ALIGN;
  return from_hip(kla::launch_attn(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
