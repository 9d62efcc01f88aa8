// The index arithmetic of kernels (csrc/kla_index.h) on the host under UndefinedBehaviorSanitizer.
// Built and run by tests/test_index_arithmetic.py; nothing here is launched.
#include <stdio.h>

#include <vector>

#include "kla_index.h"

static int failures = 0;

static void expect(const char *what, bool ok, long long a, long long b) {
  if (!ok) {
    printf("FAIL %s (%lld, %lld)\n", what, a, b);
    ++failures;
  }
}

// what eviction gives: the positions behind `budget` kept ones, a workgroup to 64 of those
static void positions(int budget, int len) {
  const int blocks = (budget + 63) / 64;
  for (int block : {0, 1, blocks / 3, blocks / 2, blocks - 2, blocks - 1})
    for (int thread : {0, 77, 255}) {
      if (block < 0 || block >= blocks) continue;
      long long want = (long long)budget + (long long)block * 256 + thread, count = 0;
      kla::each_position(budget, len, block, blocks, thread, [&](long long i) {
        if (++count < 100) expect("position", i == want && i >= budget && i < len, i, want);
        want += (long long)blocks * 256;
      });
      const long long first = (long long)budget + (long long)block * 256 + thread, step = (long long)blocks * 256;
      expect("positions", count == (first < len ? (len - first + step - 1) / step : 0), budget, len);
    }
}

int main() {
  // every position once
  for (int budget : {1, 63, 64, 65, 1000})
    for (int len : {budget + 1, budget + 300, 5000, 300000}) {
      std::vector<int> seen(len, 0);
      const int blocks = (budget + 63) / 64;
      for (int block = 0; block < blocks; ++block)
        for (int thread = 0; thread < 256; ++thread)
          kla::each_position(budget, len, block, blocks, thread, [&](long long i) {
            expect("range", i >= budget && i < len, i, len);
            if (i >= budget && i < len) ++seen[i];
          });
      for (int i = 0; i < len; ++i) expect("once", seen[i] == (i >= budget), i, seen[i]);
    }
  // up to the longest sequence of 2^31 - 2^16 tokens
  const int most = 0x7fffffff - 65536;
  for (int budget : {1, 4096, 250000000, 1 << 29, (1 << 29) + 1, 1 << 30, most - 1})
    for (int len : {1200000000, most - 100, most})
      if (len > budget) positions(budget, len);
  // the rows of a tile, the 32nd among them
  for (unsigned bits : {0u, 1u, 0x80000000u, 0x80010001u, 0xffffffffu, 0x12345678u}) {
    unsigned seen = 0;
    int last = -1;
    kla::each_bit(bits, [&](int i) {
      expect("bit", i > last && i < 32, i, last);
      seen |= 1u << i;
      last = i;
    });
    expect("bits", seen == bits, seen, bits);
  }
  printf("ok: %d failure(s)\n", failures);
  return failures != 0;
}
