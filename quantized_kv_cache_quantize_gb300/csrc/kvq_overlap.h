// Whether two strided tensors share memory, on the host (no CUDA).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace kvq {

// 16-bit elements [batch][rows][heads][d], the strides multiples of 8 elements and
// not negative, the channels contiguous, 16-byte aligned.
struct Strided {
  const void* p;
  int64_t batch_stride, row_stride, head_stride;
  int32_t batch, rows, heads, d;
};

// Places of a and b that are the same: whole numbers i, j within their sizes with
// sum stride_a i - sum stride_b j + c = distance, c within a row's channels.  Terms
// of one stride (two views of one allocation) become one, the largest strides are
// settled first, and each leaves only the few values that the others can make up
// for.  The search gives up after kOverlapSteps of them (strides that fit no common
// layout over long axes): false then, as for tensors that share nothing.
constexpr int kOverlapSteps = 20000;
class Overlap {
 public:
  Overlap(const Strided& a, const Strided& b) {
    const int64_t sa[3] = {a.batch_stride, a.row_stride, a.head_stride}, sb[3] = {b.batch_stride, b.row_stride, b.head_stride};
    const int32_t na[3] = {a.batch, a.rows, a.heads}, nb[3] = {b.batch, b.rows, b.heads};
    for (int k = 0; k < 3; ++k) {
      empty_ |= na[k] < 1 || nb[k] < 1;
      add(sa[k] / 8, 0, na[k] - 1);
      add(sb[k] / 8, 1 - nb[k], 0);
    }
    add(1, 1 - b.d / 8, a.d / 8 - 1);   // (16-byte chunks)
    std::sort(term_, term_ + n_, [](const Term& x, const Term& y) { return x.stride > y.stride; });
    low_[n_] = high_[n_] = 0;
    for (int k = n_ - 1; k >= 0; --k) {   // what the terms from k on reach
      low_[k] = low_[k + 1] + (Wide)term_[k].stride * term_[k].lo;
      high_[k] = high_[k + 1] + (Wide)term_[k].stride * term_[k].hi;
    }
    distance_ = ((Wide)(intptr_t)b.p - (Wide)(intptr_t)a.p) / 16;
  }
  bool found() { return !empty_ && search(0, distance_); }

 private:
  typedef __int128 Wide;
  struct Term {
    int64_t stride, lo, hi;
  };
  void add(int64_t stride, int64_t lo, int64_t hi) {
    if (stride == 0 || lo == hi) return;
    for (int k = 0; k < n_; ++k)
      if (term_[k].stride == stride) {
        term_[k].lo += lo;
        term_[k].hi += hi;
        return;
      }
    term_[n_++] = Term{stride, lo, hi};
  }
  static Wide down(Wide x, Wide y) { return x >= 0 ? x / y : -((-x + y - 1) / y); }   // floor, y > 0
  bool search(int k, Wide rest) {
    if (rest < low_[k] || rest > high_[k]) return false;
    if (k == n_) return true;
    const Wide s = term_[k].stride;
    const Wide from = std::max<Wide>(term_[k].lo, -down(high_[k + 1] - rest, s)), to = std::min<Wide>(term_[k].hi, down(rest - low_[k + 1], s));
    for (Wide v = from; v <= to; ++v) {
      if (++steps_ > kOverlapSteps) return false;
      if (search(k + 1, rest - s * v)) return true;
    }
    return false;
  }
  Term term_[7];
  Wide low_[8], high_[8], distance_;
  int n_ = 0, steps_ = 0;
  bool empty_ = false;
};
inline bool overlap(const Strided& a, const Strided& b) { return Overlap(a, b).found(); }

// Whether two indices of one tensor are the same place: its first batch entry
// against the others, the first row of that entry against its others, the first
// head of that row against its others (two indices differ in one of these first,
// and where their difference is a distance of nothing the first one's is too).
inline bool repeats(Strided t) {
  const int64_t stride[3] = {t.batch_stride, t.row_stride, t.head_stride};
  int32_t Strided::*const size[3] = {&Strided::batch, &Strided::rows, &Strided::heads};
  if (t.batch < 1 || t.rows < 1 || t.heads < 1) return false;
  for (int k = 0; k < 3; ++k) {
    Strided first = t, others = t;
    first.*size[k] = 1;
    others.*size[k] -= 1;
    others.p = static_cast<const char*>(t.p) + 2 * stride[k];
    if (overlap(first, others)) return true;
    t = first;
  }
  return false;
}

}  // namespace kvq
