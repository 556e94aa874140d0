// gdn_pool_views.h -- host side: strides of state pools, and whether two pools'
// views share elements.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace gdn {

inline bool pool_strides_ok(const int64_t s[4], int64_t rows, const int64_t ext[3]) {
  if (s[0] == 0 && s[1] == 0 && s[2] == 0 && s[3] == 0) return true;
  const int64_t n[4] = {rows, ext[0], ext[1], ext[2]};
  int idx[4] = {0, 1, 2, 3};
  for (int i = 0; i < 4; ++i)
    if (s[i] <= 0 && n[i] > 1) return false;
  std::sort(idx, idx + 4, [&](int x, int y) { return s[x] < s[y]; });
  int64_t reach = 1;  // elements spanned by the dimensions so far
  for (int k = 0; k < 4; ++k) {
    if (n[idx[k]] <= 1) continue;  // never overlaps anything
    if (s[idx[k]] < reach) return false;
    reach = s[idx[k]] * (n[idx[k]] - 1) + reach;
  }
  return true;
}

inline void pool_strides(const int64_t in[4], const int64_t ext[3], int64_t out[4]) {
  if (in[0] == 0 && in[1] == 0 && in[2] == 0 && in[3] == 0) {
    out[3] = 1;
    out[2] = ext[2];
    out[1] = ext[1] * ext[2];
    out[0] = ext[0] * ext[1] * ext[2];
  } else {
    for (int i = 0; i < 4; ++i) out[i] = in[i];
  }
}

// Bytes from a row's first element to behind its last.
inline int64_t row_span(const int64_t s[4], const int64_t ext[3], int64_t es) {
  return (1 + (ext[0] - 1) * s[1] + (ext[1] - 1) * s[2] + (ext[2] - 1) * s[3]) * es;
}

inline bool row_contiguous(const int64_t s[4], const int64_t ext[3]) {
  return (ext[2] == 1 || s[3] == 1) && (ext[1] == 1 || s[2] == ext[2]) &&
         (ext[0] == 1 || s[1] == ext[1] * ext[2]);
}

// One dimension of two views: the distance in bytes from an index of the one to
// the next, and the range of (source index - destination index).
struct Steps {
  int64_t bytes, lo, hi;
};

// Some element of the source view (ss bytes, the first at byte `at`) and some of
// the destination view (ds bytes, the first at byte 0) share a byte.  The
// dimensions go from the longest step to the shortest; as a view's elements do
// not overlap, few differences come into question in each.
inline bool meet(int64_t at, const Steps *d, int n, int64_t ss, int64_t ds) {
  if (n == 0) return -ss < at && at < ds;
  int64_t below = 0, above = 0;  // what the shorter steps can add
  for (int k = 1; k < n; ++k) {
    below += d[k].lo * d[k].bytes;
    above += d[k].hi * d[k].bytes;
  }
  // -ss < at + i * bytes + (below .. above) < ds
  const int64_t from = std::max(d->lo, (-ss - at - above) / d->bytes - 1);
  const int64_t to = std::min(d->hi, (ds - at - below) / d->bytes + 1);
  for (int64_t i = from; i <= to; ++i)
    if (meet(at + i * d->bytes, d + 1, n - 1, ss, ds)) return true;
  return false;
}

// The two views share no byte: their rows do not meet as whole stretches, or
// where they are interleaved closer than that, their elements do not.  False
// also where the views' steps differ, so that this is not settled.
inline bool views_apart(int64_t at, const int64_t ss[4], int64_t srows, int64_t se,
                        const int64_t sext[3], const int64_t ds[4], int64_t drows, int64_t de,
                        const int64_t dext[3]) {
  Steps d[4];
  int n = 0;
  auto dim = [&](int64_t s, int64_t sn, int64_t t, int64_t tn) {
    s *= se;
    t *= de;
    if (sn > 1 && tn > 1 && s != t) return false;
    if (sn > 1 || tn > 1) d[n++] = {sn > 1 ? s : t, 1 - tn, sn - 1};
    return true;
  };
  if (!dim(ss[0], srows, ds[0], drows)) return false;
  if (!meet(at, d, n, row_span(ss, sext, se), row_span(ds, dext, de))) return true;
  for (int i = 0; i < 3; ++i)
    if (!dim(ss[i + 1], sext[i], ds[i + 1], dext[i])) return false;
  std::sort(d, d + n, [](const Steps &x, const Steps &y) { return x.bytes > y.bytes; });
  return !meet(at, d, n, se, de);
}

}  // namespace gdn
