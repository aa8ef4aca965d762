// Host check that FastDiv / fdiv are exact for every numerator below 2^31:
// entry / entries-a-row of up to 2^31 - 1 received entries, and any other
// divisor.  Built and run by test_division.py; prints the number of cases
// checked, or the first failing (n, d) and exits nonzero.
#include <cstdint>
#include <cstdio>
#include <random>

#include "device.h"

static long long checked = 0;

static bool check(int64_t n, int d) {
  if (n < 0 || n > 0x7fffffff) return true;
  const miep::FastDiv f = miep::make_fastdiv(d);
  ++checked;
  const int got = miep::fdiv(static_cast<int>(n), f), want = static_cast<int>(n / d);
  if (got != want) std::printf("FAIL n=%lld d=%d fdiv=%d floor=%d\n", static_cast<long long>(n), d, got, want);
  return got == want;
}

// n - 1, n and n + 1 around every multiple's ends
static bool around(int64_t q, int d) {
  for (int64_t n : {q * d - 1, q * d, q * d + 1, q * d + d - 1})
    if (!check(n, d)) return false;
  return true;
}

int main() {
  std::mt19937_64 rng(11);
  const int64_t most = 0x7fffffff;
  for (int d = 1; d <= 64; ++d) {
    // quotients at the powers of two (2^24 * d is where a 40-bit shift's product passes 64 bits) and anywhere
    for (int b = 0; b < 31; ++b)
      for (int64_t q = (int64_t(1) << b) - 2; q <= (int64_t(1) << b) + 2; ++q)
        if (q >= 0 && !around(q, d)) return 1;
    for (int it = 0; it < 200000; ++it)
      if (!around(static_cast<int64_t>(rng() % (most / d + 1)), d)) return 1;
    if (!check(most, d) || !check(most - 1, d)) return 1;
  }
  for (int it = 0; it < 2000000; ++it) {
    const int d = 1 + static_cast<int>((rng() % most) >> (rng() % 31));
    if (!around(static_cast<int64_t>(rng() % (most / d + 1)), d) || !check(most, d)) return 1;
  }
  for (int64_t b = 1; b <= (int64_t(1) << 30); b <<= 1)
    for (int64_t d : {b - 1, b, b + 1, most - b, most})
      if (d > 0)
        for (int64_t n : {int64_t(0), b, d - 1, d, d + 1, most - 1, most})
          if (!check(n, static_cast<int>(d))) return 1;
  std::printf("ok %lld\n", checked);
  return 0;
}
