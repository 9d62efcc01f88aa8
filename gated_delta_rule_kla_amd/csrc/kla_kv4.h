// kla_kv4.h -- the 4-bit cache as its kernels see it (kla_kv4.hip, kla_kv4_chunk.hip,
// kla_kv4_evict.hip): places of tokens, and codes to bf16.
#pragma once

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
constexpr int KV_MAX_PER = 8192;  // tokens of a run whose pages are kept in LDS

typedef bf16 bf16x8v __attribute__((ext_vector_type(8)));

// eight channels in a dword as four bf16 pairs
__device__ __forceinline__ void cvt8(unsigned u, float s, unsigned *r) {
  r[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, s, 0));
  r[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, s, 1));
  r[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, s, 2));
  r[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, s, 3));
}

inline KvParams kv_params(const Kv4Cache &c) {
  return KvParams{(uint8_t *)c.codes, (uint8_t *)c.scales, c.table, c.num_pages, c.page, c.max_pages, c.Hkv};
}

}  // namespace

}  // namespace kla
