/* Linear attention and the calls of new tokens over the 4-bit cache under AddressSanitizer and
 * UndefinedBehaviorSanitizer: calls that validation rejects or that leave nothing to do, and the
 * workspace queries near the 32-bit limits.  Built and run by
 * tests/test_abi_sanitized_more_operators.py, on a machine without a GPU. */
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "kla.h"

static int failures = 0;

static void expect(const char *what, long long got, long long want) {
  if (got != want) {
    printf("FAIL %s: got %lld, want %lld\n", what, got, want);
    ++failures;
  }
}

/* never dereferenced */
#define FAKE ((void *)0x7F0000000000ull)
#define FAKEI ((int32_t *)0x7F0000000000ull)
#define FAKEF ((float *)0x7F0000000000ull)

static const int SIZES[] = {INT_MIN, -1, 0, 1, 2, 63, 64, 128, 3001, 1 << 16, 1 << 24, 1 << 30, INT_MAX - 65536, INT_MAX - 1, INT_MAX};
enum { NS = sizeof SIZES / sizeof *SIZES };

int main(void) {
  const int32_t good[] = {0, 4, 4, 10}, bad[] = {0, 6, 5, 10};
  const kla_dtype_t bf = KLA_DT_BF16, f32 = KLA_DT_F32;
  long long refused = 0;

  /* linear attention */
  expect("la dtype", kla_la_chunk_fwd(FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, 0, 0, 0, 2, 2, 4, 10, 64, 64, (kla_dtype_t)7, 0, 0, 0), KLA_ERR_DTYPE);
  expect("la null", kla_la_chunk_fwd(FAKE, FAKE, 0, FAKE, 0, 0, FAKE, 0, 0, 0, 2, 2, 4, 10, 64, 64, bf, 0, 0, 0), KLA_ERR_NULL);
  expect("la no decay", kla_la_chunk_fwd(FAKE, FAKE, FAKE, 0, 0, 0, FAKE, 0, 0, 0, 2, 2, 4, 10, 64, 64, bf, 0, 0, 0), KLA_ERR_NULL);
  expect("la two decays", kla_la_chunk_fwd(FAKE, FAKE, FAKE, FAKE, FAKEF, 0, FAKE, 0, 0, 0, 2, 2, 4, 10, 64, 64, bf, 0, 0, 0), KLA_ERR_PARAM);
  expect("la sizes", kla_la_chunk_fwd(FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, 0, 0, 0, 2, 2, 4, 10, 40, 64, bf, 0, 0, 0), KLA_ERR_UNSUPPORTED);
  expect("la offsets", kla_la_chunk_fwd(FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, 0, FAKEI, bad, 3, 1, 4, 10, 64, 64, f32, 0, 0, 0), KLA_ERR_SEQLENS);
  expect("la bwd offsets", kla_la_chunk_bwd(FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, 0, FAKE, FAKE, FAKE, FAKE, 0, FAKEI, good, 3, 1, 4, 11, 64, 64, f32, 0, 0, 0), KLA_ERR_SEQLENS);
  expect("la bwd workspace", kla_la_chunk_bwd(FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, 0, FAKE, FAKE, FAKE, FAKE, 0, FAKEI, good, 3, 1, 4, 10, 64, 64, bf, FAKE, 8, 0), KLA_ERR_WORKSPACE);
  expect("la step null", kla_la_decode_step(FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, 1, 1, 64, 64, bf, 0), KLA_ERR_NULL);
  expect("la step dtype", kla_la_decode_step(FAKE, FAKE, FAKE, FAKE, 0, FAKEF, FAKE, 1, 1, 64, 64, (kla_dtype_t)-3, 0), KLA_ERR_DTYPE);
  /* new tokens over the cache */
  expect("chunk offsets", kla_attn_kv4_chunk_fwd(FAKE, FAKE, FAKE, FAKEI, FAKEI, 1.f, FAKE, 0, FAKEI, bad, 3, 1, 4, 2, 10, 64, 4, 16, 4, 64, bf, 0, 0, 0), KLA_ERR_SEQLENS);
  expect("chunk scale", kla_attn_kv4_chunk_fwd(FAKE, FAKE, FAKE, FAKEI, FAKEI, NAN, FAKE, 0, FAKEI, good, 3, 1, 4, 2, 10, 64, 4, 16, 4, 64, bf, 0, 0, 0), KLA_ERR_PARAM);
  expect("chunk workspace", kla_attn_kv4_chunk_fwd(FAKE, FAKE, FAKE, FAKEI, FAKEI, 1.f, FAKE, 0, 0, 0, 1, 1, 2, 2, 1, 64, 4, 16, 4, 100000, bf, FAKE, 8, 0), KLA_ERR_WORKSPACE);
  expect("weigh offsets", kla_attn_kv4_weigh(FAKE, FAKEF, FAKE, FAKE, FAKEI, FAKEI, 1.f, FAKEF, FAKEI, bad, 3, 1, 4, 2, 10, 64, 4, 16, 4, 64, 64, bf, 0), KLA_ERR_SEQLENS);
  expect("weigh null", kla_attn_kv4_weigh(FAKE, 0, FAKE, FAKE, FAKEI, FAKEI, 1.f, FAKEF, FAKEI, good, 3, 1, 4, 2, 10, 64, 4, 16, 4, 64, 64, bf, 0), KLA_ERR_NULL);
  expect("evict budget", kla_kv4_evict(FAKE, FAKE, FAKEI, FAKEI, FAKEF, FAKEI, FAKEI, 0, 0, 2, 2, 64, 4, 16, 4, 64, FAKE, 1 << 20, 0), KLA_ERR_PARAM);
  expect("evict workspace", kla_kv4_evict(FAKE, FAKE, FAKEI, FAKEI, FAKEF, FAKEI, FAKEI, 5, 2, 2, 2, 64, 4, 16, 4, 64, FAKE, 8, 0), KLA_ERR_WORKSPACE);

  /* sizes near the limits: the refusals' and the workspaces' arithmetic.  A null tensor refuses
   * what the sizes do not. */
  for (int i = 0; i < NS; ++i)
    for (int j = 0; j < NS; ++j)
      for (int k = 0; k < NS; ++k)
        for (int dt = 0; dt < 2; ++dt) {
          const int a = SIZES[i], b = SIZES[j], c = SIZES[k];
          const kla_dtype_t t = (kla_dtype_t)dt;
          kla_la_chunk_workspace_bytes(0, 0, a, a, b, c, 64, 256, t);
          kla_la_chunk_workspace_bytes(0, 0, 1, 1, a, 100, b, c, t);
          kla_la_chunk_bwd_workspace_bytes(0, 0, a, a, b, c, 256, 256, t);
          kla_la_chunk_bwd_workspace_bytes(0, 0, 1, 1, a, b, c, c, t);
          refused += kla_la_chunk_fwd(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, a, a, b, c > 0 ? c : 1, 16, 24, t, 0, 0, 0) != KLA_OK;
          refused += kla_la_chunk_bwd(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, a, a, b, c > 0 ? c : 1, 64, 64, t, 0, 0, 0) != KLA_OK;
          refused += kla_la_decode_step(0, 0, 0, 0, 0, 0, 0, a, b, c, 64, t, 0) != KLA_OK;
          kla_attn_kv4_chunk_workspace_bytes(0, 0, a, a, 8, 2, b, 128, c, t);
          kla_attn_kv4_chunk_workspace_bytes(0, 0, 1, 1, a, 1, b, 64, c, t);
          refused += kla_attn_kv4_chunk_fwd(0, 0, 0, 0, 0, 1.f, 0, 0, 0, 0, a, a, 4, 2, b, 128, 4, 16, 4, c, t, 0, 0, 0) != KLA_OK;
          refused += kla_attn_kv4_chunk_fwd(0, 0, 0, 0, 0, 1.f, 0, 0, 0, 0, 2, 2, b, 1, 5, 64, a, 16, c, 64, t, 0, 0, 0) != KLA_OK;
          refused += kla_attn_kv4_weigh(0, 0, 0, 0, 0, 0, 1.f, 0, 0, 0, a, a, 4, 2, b, 128, 4, 16, 4, c, 64, t, 0) != KLA_OK;
          refused += kla_attn_kv4_weigh(0, 0, 0, 0, 0, 0, 1.f, 0, 0, 0, 2, 2, b, 1, 5, 64, a, 16, c, 64, c, t, 0) != KLA_OK;
          kla_kv4_evict_workspace_bytes(a, 2, 128, b, 16, c);
          kla_kv4_evict_workspace_bytes(2, a, 64, b, c, 64);
          refused += kla_kv4_evict(0, 0, 0, 0, 0, 0, 0, a, b, 2, 2, 64, 4, 16, c, INT_MAX, 0, 0, 0) != KLA_OK;
          refused += kla_kv4_evict(0, 0, 0, 0, 0, 0, 0, 64, 1, a, b, 64, c, 16, 4, 64, 0, 0, 0) != KLA_OK;
        }
  printf("%lld refused\nok: %d failure(s)\n", refused, failures);
  return failures != 0;
}
