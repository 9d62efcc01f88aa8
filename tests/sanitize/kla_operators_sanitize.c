/* The gated linear recurrence, prompt attention and 4-bit cache entry points under
 * AddressSanitizer and UndefinedBehaviorSanitizer: calls that validation rejects or that leave
 * nothing to do, and the workspace queries near the 32-bit limits.  Built and run by
 * tests/test_abi_sanitized_operators.py, on a machine without a GPU. */
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

static const int SIZES[] = {INT_MIN, -1, 0, 1, 2, 63, 64, 128, 3001, 1 << 16, 1 << 24, 1 << 30, INT_MAX - 65536, INT_MAX - 1, INT_MAX};
enum { NS = sizeof SIZES / sizeof *SIZES };

int main(void) {
  const int32_t good[] = {0, 4, 4, 10}, bad[] = {0, 6, 5, 10};
  long long refused = 0;

  /* gated linear recurrence */
  expect("glr dtype", kla_glr_chunk_fwd(FAKE, FAKE, 0, FAKE, 0, 0, 0, 2, 2, 4, 10, 64, (kla_dtype_t)7, 0, 0, 0), KLA_ERR_DTYPE);
  expect("glr null", kla_glr_chunk_fwd(0, FAKE, 0, FAKE, 0, 0, 0, 2, 2, 4, 10, 64, KLA_DT_BF16, 0, 0, 0), KLA_ERR_NULL);
  expect("glr offsets", kla_glr_chunk_fwd(FAKE, FAKE, 0, FAKE, 0, FAKEI, bad, 3, 1, 4, 10, 64, KLA_DT_F32, 0, 0, 0), KLA_ERR_SEQLENS);
  expect("glr bwd offsets", kla_glr_chunk_bwd(FAKE, FAKE, 0, FAKE, 0, FAKE, FAKE, 0, FAKEI, good, 3, 1, 4, 11, 64, KLA_DT_F32, 0, 0, 0), KLA_ERR_SEQLENS);
  expect("glr bwd null", kla_glr_chunk_bwd(FAKE, 0, 0, FAKE, 0, FAKE, FAKE, 0, FAKEI, good, 3, 1, 4, 10, 64, KLA_DT_F32, 0, 0, 0), KLA_ERR_NULL);
  expect("glr none", kla_glr_chunk_bwd(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 4, 10, 64, KLA_DT_F32, 0, 0, 0), KLA_OK);
  expect("glr step dtype", kla_glr_decode_step(FAKE, FAKE, (float *)FAKE, FAKE, 1, 1, 1, (kla_dtype_t)-3, 0), KLA_ERR_DTYPE);
  /* the 4-bit cache */
  expect("kv4 offsets", kla_kv4_append(FAKE, FAKE, FAKE, FAKE, FAKEI, FAKEI, FAKEI, bad, 3, 1, 2, 10, 64, 4, 16, 4, KLA_DT_BF16, 0), KLA_ERR_SEQLENS);
  expect("kv4 null", kla_kv4_read(FAKE, FAKE, 0, FAKE, FAKEI, FAKEI, FAKEI, good, 3, 1, 2, 10, 64, 4, 16, 4, KLA_DT_BF16, 0), KLA_ERR_NULL);
  expect("kv4 scale", kla_attn_kv4_decode_step(FAKE, FAKE, FAKE, FAKEI, FAKEI, NAN, FAKE, 1, 2, 2, 64, 4, 16, 4, 64, KLA_DT_BF16, 0, 0, 0), KLA_ERR_PARAM);
  expect("kv4 workspace", kla_attn_kv4_decode_step(FAKE, FAKE, FAKE, FAKEI, FAKEI, 1.f, FAKE, 1, 2, 2, 64, 4, 16, 4, 100000, KLA_DT_BF16, FAKE, 8, 0), KLA_ERR_WORKSPACE);
  /* prompt attention */
  expect("attn keys", kla_attn_fwd(FAKE, FAKE, FAKE, 1.f, FAKE, 0, FAKEI, good, FAKEI, bad, 3, 1, 4, 2, 10, 10, 64, KLA_DT_BF16, 0), KLA_ERR_SEQLENS);
  expect("attn null", kla_attn_fwd(FAKE, FAKE, 0, 1.f, FAKE, 0, FAKEI, good, FAKEI, good, 3, 1, 4, 2, 10, 10, 64, KLA_DT_BF16, 0), KLA_ERR_NULL);

  /* sizes near the limits: the refusals' and the workspaces' arithmetic.  A null tensor refuses
   * what the sizes do not. */
  for (int i = 0; i < NS; ++i)
    for (int j = 0; j < NS; ++j)
      for (int k = 0; k < NS; ++k)
        for (int dt = 0; dt < 2; ++dt) {
          const int a = SIZES[i], b = SIZES[j], c = SIZES[k];
          const kla_dtype_t t = (kla_dtype_t)dt;
          kla_glr_chunk_workspace_bytes(0, 0, a, a, b, c, 64, t);
          kla_glr_chunk_workspace_bytes(0, 0, 1, 1, a, b, c, t);
          refused += kla_glr_chunk_fwd(0, 0, 0, 0, 0, 0, 0, a, a, b, c > 0 ? c : 1, 37, t, 0, 0, 0) != KLA_OK;
          refused += kla_glr_decode_step(0, 0, 0, 0, a, b, c, t, 0) != KLA_OK;
          refused += kla_kv4_append(0, 0, 0, 0, 0, 0, 0, 0, a, a, b, c, 128, 4, 16, 4, t, 0) != KLA_OK;
          refused += kla_kv4_read(0, 0, 0, 0, 0, 0, 0, 0, 2, 2, 2, 5, 64, a, b, c, t, 0) != KLA_OK;
          kla_attn_kv4_decode_workspace_bytes(a, b, 1, 128, c, t);
          kla_attn_kv4_decode_workspace_bytes(a, b, b, 64, c, t);
          refused += kla_attn_kv4_decode_step(0, 0, 0, 0, 0, 1.f, 0, a, b, 1, 64, 4, 16, 4, c, t, 0, 0, 0) != KLA_OK;
          refused += kla_attn_fwd(0, 0, 0, 1.f, 0, 0, 0, 0, 0, 0, a, a, b, 1, c, c, 128, t, 0) != KLA_OK;
          refused += kla_attn_fwd(0, 0, 0, 1.f, 0, 0, 0, 0, 0, 0, 3, 3, b, b, c, a, 64, t, 0) != KLA_OK;
        }
  printf("%lld refused\nok: %d failure(s)\n", refused, failures);
  return failures != 0;
}
