// kvq::overlap against the sets of places, for small tensors of every layout in
// one allocation, and for large ones whose answer is known.  Prints "checks N
// bad M", exits 1 on any difference.
#include <cstdio>
#include <random>
#include <set>

#include "../quantized_kv_cache_quantize_gb300/csrc/kvq_overlap.h"

using kvq::Strided;
static long long checks = 0, bad = 0;

static Strided at(long long element, long long bs, long long rs, long long hs, int batch, int rows, int heads, int d) {
  return Strided{reinterpret_cast<const void*>((intptr_t)0x7f0000000000 + 2 * element), bs, rs, hs, batch, rows, heads, d};
}
static std::set<long long> places(const Strided& t) {
  std::set<long long> s;
  for (long long b = 0; b < t.batch; ++b)
    for (long long r = 0; r < t.rows; ++r)
      for (long long h = 0; h < t.heads; ++h)
        for (int c = 0; c < t.d / 8; ++c)
          s.insert((intptr_t)t.p / 16 + (b * t.batch_stride + r * t.row_stride + h * t.head_stride) / 8 + c);
  return s;
}
static void expect(const Strided& a, const Strided& b, bool want, const char* what) {
  checks += 2;
  if (kvq::overlap(a, b) != want || kvq::overlap(b, a) != want) {
    if (++bad < 10) std::printf("%s: want %d\n", what, (int)want);
  }
}

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int n) { return (int)(rng() % n); };
  for (int i = 0; i < 60000; ++i) {
    Strided t[2];
    const int shared = pick(3);   // strides of one allocation, in part, or of their own
    for (int k = 0; k < 2; ++k) {
      long long s[3];
      for (int x = 0; x < 3; ++x) s[x] = 8 * pick(pick(2) ? 12 : 60);
      if (pick(2)) s[0] = 0;
      if (k == 1 && shared > 0) s[1] = t[0].row_stride;
      if (k == 1 && shared > 1) s[2] = t[0].head_stride, s[0] = t[0].batch_stride;
      t[k] = at(8 * pick(200), s[0], s[1], s[2], 1 + pick(3), 1 + pick(6), pick(5), 8 * (1 + pick(3)));
    }
    const std::set<long long> x = places(t[0]), y = places(t[1]);
    bool want = false;
    for (long long p : x) want |= y.count(p) != 0;
    expect(t[0], t[1], want, "small");
    for (int k = 0; k < 2; ++k) {
      const long long all = (long long)t[k].batch * t[k].rows * t[k].heads * (t[k].d / 8);
      ++checks;
      if (kvq::repeats(t[k]) != ((long long)(k == 0 ? x : y).size() != all) && ++bad < 10) std::printf("repeats\n");
    }
  }
  // slices of one projection [4680][48][128]: queries, keys, and a slice across both
  const long long row = 48 * 128;
  const Strided q = at(0, 0, row, 128, 1, 4680, 32, 128), k = at(32 * 128, 0, row, 128, 1, 4680, 8, 128);
  expect(q, k, false, "slices");
  expect(q, at(8 * 128, 0, row, 128, 1, 4680, 32, 128), true, "shifted by heads");
  expect(k, at(8 * 128, 0, row, 128, 1, 4680, 32, 128), true, "over the keys");
  expect(q, at(row, 0, row, 128, 1, 4680, 32, 128), true, "shifted by a row");
  expect(q, at(32 * 128 + 4679 * row, 0, row, 128, 1, 100, 16, 128), false, "behind the last row's");
  expect(q, at(4680 * row, 0, row, 128, 1, 100, 48, 128), false, "behind");
  expect(at(0, 0, 2 * row, 128, 1, 2340, 48, 128), at(row, 0, 2 * row, 128, 1, 2340, 48, 128), false, "every other row");
  // heads of [4][40][30000][64]: the window's layout
  const long long head = 30000 * 64, batch = 40 * head;
  expect(at(0, batch, 64, head, 4, 30000, 32, 64), at(32 * head, batch, 64, head, 4, 30000, 8, 64), false, "heads apart");
  expect(at(0, batch, 64, head, 4, 30000, 33, 64), at(32 * head, batch, 64, head, 4, 30000, 8, 64), true, "a head shared");
  expect(at(0, batch, 64, head, 4, 30000, 32, 64), at(0, batch, 40 * 64, 64, 4, 30000, 32, 64), true, "two layouts");
  checks += 4;
  bad += kvq::repeats(q) + kvq::repeats(at(0, batch, 64, head, 4, 30000, 40, 64)) +
         !kvq::repeats(at(0, 0, row, 127 * 8, 1, 4680, 49, 128)) + !kvq::repeats(at(0, 0, 0, 128, 1, 2, 8, 128));
  // numbers beyond 64 bits
  const long long far = 0x7ffffffffffffff8LL;
  expect(at(0, far, far, far, 0x7fffffff, 0x7fffffff, 0x7fffffff, 128), at(64, far, far, far, 1, 1, 1, 128), true, "far");
  expect(at(0, far, far, far, 0x7fffffff, 0x7fffffff, 0x7fffffff, 128), at(128, 0, 0, 0, 1, 1, 1, 128), false, "far apart");
  // no common layout, long axes: an end, whatever the answer
  (void)kvq::overlap(at(0, 0, 40 * 128, 256, 1, 1 << 30, 2, 128), at(128, 0, 39 * 128 + 8, 264, 1, 1 << 30, 2, 128));
  ++checks;
  std::printf("checks %lld bad %lld\n", checks, bad);
  return bad ? 1 : 0;
}
