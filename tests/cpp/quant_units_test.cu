// How the 8-bit cache's append and read number their units (csrc/attn_quant.h), on the host: at the largest sizes that a call
// may have, and at others, every warp of every CTA finds in 32 bits the unit, the piece and the head that 64-bit arithmetic
// gives, all units are taken, each by its warps, and warps behind the last find no piece.
#include <cstdio>
#include <random>

#include "../../gated_deltanet_cpr_gb300/csrc/attn_quant.h"

using namespace gdn;

static int fail(const char* what, int hkv, int shift, int N, int T, int64_t block) {
  std::printf("%s: hkv %d, shift %d, N %d, T %d, block %lld\n", what, hkv, shift, N, T, (long long)block);
  return 1;
}

// the largest T that a call of N requests may have, or -1
static int largest(int N, int shift, int hkv) {
  if (!quant_units_fit(N, 0, shift, hkv)) return -1;
  int64_t lo = 0, hi = INT32_MAX;
  while (lo < hi) {
    const int64_t m = (lo + hi + 1) / 2;
    if (quant_units_fit(N, (int)m, shift, hkv)) lo = m;
    else hi = m - 1;
  }
  return (int)lo;
}

static int check(int hkv, int shift, bool append, int N, int T, std::mt19937_64& rng) {
  const int each_shift = append ? shift - kGranuleShift : 0, each = 1 << each_shift;
  const int threads = 32 * each > 128 ? 32 * each : 128, warps = threads / 32;
  const int64_t units = quant_units(N, T, shift, hkv), pieces = units / (2 * (int64_t)hkv);
  const int64_t blocks = quant_blocks(units, each, threads) - 1;
  if (units >= (int64_t)1 << 31 || blocks >= INT32_MAX) return fail("too many", hkv, shift, N, T, blocks);
  if (blocks * warps < units * each) return fail("units left out", hkv, shift, N, T, blocks);
  const Divide heads = divide_by(2u * (uint32_t)hkv);
  for (int k = 0; k < 400; ++k) {
    const int64_t b = k < 100 ? k : k < 200 ? blocks - 1 - (k - 100) : (int64_t)(rng() % (uint64_t)(blocks ? blocks : 1));
    if (b < 0 || b >= blocks) continue;
    for (int w = 0; w < warps; ++w) {
      const int64_t unit = (b * warps + w) >> each_shift;
      const uint32_t got = quant_unit((uint32_t)b, threads, w, each_shift);
      if ((int64_t)got != unit) return fail("unit", hkv, shift, N, T, b);
      const uint32_t piece = divide(got, heads);
      if (unit < units ? (int64_t)piece != unit / (2 * (int64_t)hkv) : piece < (uint64_t)pieces) return fail("piece", hkv, shift, N, T, b);
    }
  }
  return 0;
}

int main() {
  std::mt19937_64 rng(1);
  int bad = 0, count = 0;
  for (int hkv : {1, 2, 3, 4, 5, 7, 8, 12, 16, 40, 128, 1000, 4097, 32768, 65535})
    for (int N : {1, 2, 7, 255, 4096, 65535})
      for (int shift = 4; shift <= 7; ++shift)
        for (int append = 0; append < 2; ++append) {
          if (!append && shift != kGranuleShift) continue;
          const int most = largest(N, shift, hkv);
          if (most < 0) continue;
          for (int64_t T : {(int64_t)most, (int64_t)most - 1, (int64_t)most / 2 + 1, (int64_t)most / 16, (int64_t)2 * N, (int64_t)N, (int64_t)1, (int64_t)0})
            if (T >= 0 && T <= most) bad += check(hkv, shift, append, N, (int)T, rng), ++count;
        }
  // the quotient by a product, near multiples of the divisor and at the end of the range
  for (uint32_t d = 2; d <= 131070; d += 2) {
    const Divide x = divide_by(d);
    for (int k = 0; k < 24; ++k) {
      const uint32_t q = k < 8 ? (uint32_t)k : (uint32_t)(rng() % (0x80000000u / d + 1));
      for (int64_t n = (int64_t)q * d - 1; n <= (int64_t)q * d + 1; ++n)
        if (n >= 0 && n < (int64_t)1 << 31 && divide((uint32_t)n, x) != n / d) ++bad, std::printf("%lld / %u\n", (long long)n, d);
    }
    if (divide(0x7fffffffu, x) != 0x7fffffffu / d) ++bad, std::printf("last / %u\n", d);
  }
  std::printf("%d cases, %d bad\n", count, bad);
  return bad != 0;
}
