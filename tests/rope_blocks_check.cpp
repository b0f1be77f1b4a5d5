// Blocks of the rotations' launches, checked without a GPU against counts in
// 128 bits: sizes next to 2^31 rows or heads, which 32-bit arithmetic does not
// hold, and every small one.  Prints "checks N bad M", exits 1 on any difference.
#include <cstdio>
#include <random>

#include "../quantized_kv_cache_quantize_gb300/csrc/kvq_pages.h"

typedef __int128 wide;

static long long checks = 0, bad = 0;

static void check(long long rows, long long heads, int tile) {
  wide r = rows / tile + (rows % tile != 0), h = heads / kvq::kRopeHeads + (heads % kvq::kRopeHeads != 0);
  ++checks;
  if ((wide)kvq::rope_blocks((int)rows, (int)heads, tile) != r * h) {
    if (++bad < 10) std::printf("rows %lld heads %lld tile %d: %lld\n", rows, heads, tile, kvq::rope_blocks((int)rows, (int)heads, tile));
  }
}

int main() {
  const long long top = 0x7fffffffLL;
  for (int tile : {4, 16}) {
    for (long long r = 0; r < 70; ++r)
      for (long long h = 0; h < 70; ++h) check(r, h, tile);
    for (long long d = 0; d < 40; ++d)
      for (long long h : {0LL, 1LL, 8LL, 9LL, 16LL}) check(top - d, h, tile), check(h, top - d, tile);
  }
  // an append's: keys and values of every page it looks at, queries
  std::mt19937_64 rng(1);
  for (int i = 0; i < 200000; ++i) {
    kvq::PageLayer p{};
    p.shift = 4 + (int)(rng() % 4);
    p.page = 1 << p.shift;
    p.d = 64;
    p.heads = 1 + (int)(rng() % (1u << (rng() % 31)));
    kvq::PageSeqs s{};
    s.rows = (int)(rng() % (1u << (rng() % 31)));
    s.batch = (int)(rng() % (1u << (rng() % 25)));
    int some = 0;
    s.offsets = rng() & 1 ? &some : nullptr;
    const long long q = rng() % (1u << (rng() % 32));
    const int tile = s.offsets == nullptr || p.page == 16 ? 4 : 16;
    const wide want = ((wide)(s.rows / p.page) + 2 * (wide)s.batch) * p.heads * 2 +
                      (wide)(s.rows / tile + (s.rows % tile != 0)) * (q / 8 + (q % 8 != 0));
    ++checks;
    if ((wide)kvq::append_rope_blocks(s, p, q) != want) ++bad;
  }
  std::printf("checks %lld bad %lld\n", checks, bad);
  return bad ? 1 : 0;
}
