// Strided views of head rows, and whether their rows fall on one another: what
// the serving calls refuse before a launch.  Host code without CUDA.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace s2o {

constexpr int kViewRow = 128;  // elements of a row

struct RowView {
  uint16_t* p;
  int64_t sb, st, sh;  // strides in elements
};

// A view of B x N x H rows as up to three (extent, stride) pairs, extents above
// 1 only (a stride that is never multiplied does not count), largest stride first.
struct RowGrid {
  struct Dim {
    int64_t n, s;
  };
  typedef __int128 wide;  // extents times strides, whatever a caller wrote there
  Dim d[3];
  int dims = 0;
  wide p = 0;  // first element of row (0, 0, 0)
  RowGrid(const RowView& v, int64_t B, int64_t N, int64_t H) {
    p = (wide)(reinterpret_cast<uintptr_t>(v.p) / sizeof(uint16_t));
    const Dim all[3] = {{B, v.sb}, {N, v.st}, {H, v.sh}};
    for (const Dim& x : all)
      if (x.n > 1) d[dims++] = x;
    std::sort(d, d + dims, [](const Dim& a, const Dim& b) { return mag(a.s) > mag(b.s); });
  }
  static wide mag(wide x) { return x < 0 ? -x : x; }
  // elements from the first to behind the last
  wide lo() const {
    wide x = p;
    for (int i = 0; i < dims; ++i) x += std::min<wide>(0, (wide)(d[i].n - 1) * d[i].s);
    return x;
  }
  wide hi() const {
    wide x = p + kViewRow;
    for (int i = 0; i < dims; ++i) x += std::max<wide>(0, (wide)(d[i].n - 1) * d[i].s);
    return x;
  }
  wide rows() const {
    wide n = 1;
    for (int i = 0; i < dims; ++i) n *= d[i].n;
    return n;
  }
  // every stride steps over all that the smaller ones reach: no two rows meet
  bool nested() const {
    wide reach = kViewRow;
    for (int i = dims - 1; i >= 0; --i) {
      if (mag(d[i].s) < reach) return false;
      reach += mag(d[i].s) * (d[i].n - 1);
    }
    return true;
  }
  bool dense() const { return nested() && hi() - lo() == rows() * kViewRow; }
};

// is there (i, j, k) != (0, 0, 0) (with `any`: any at all), |i| < n0, |j| < n1,
// k0 <= k <= k1, with |D + i s0 + j s1 + k s2| < a row?
inline bool rows_near(RowGrid::wide D, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t k0, int64_t k1,
                      int64_t s2, bool any) {
  typedef RowGrid::wide wide;
  // the longest range is solved for, the two others are gone through
  wide a[3] = {-(wide)(n0 - 1), -(wide)(n1 - 1), k0}, b[3] = {n0 - 1, n1 - 1, k1}, s[3] = {s0, s1, s2};
  int m = 0;
  for (int i = 1; i < 3; ++i)
    if (b[i] - a[i] > b[m] - a[m]) m = i;
  std::swap(a[m], a[2]);
  std::swap(b[m], b[2]);
  std::swap(s[m], s[2]);
  for (wide i = a[0]; i <= b[0]; ++i)
    for (wide j = a[1]; j <= b[1]; ++j) {
      const wide x = D + i * s[0] + j * s[1];
      wide lo = a[2], hi = b[2];
      if (s[2] == 0) {
        if (RowGrid::mag(x) >= kViewRow) continue;
      } else {  // |x + k s| < row: k within (row - 1) / |s| of -x / s
        const wide y = s[2] > 0 ? -x : x, step = RowGrid::mag(s[2]);
        auto down = [&](wide v) { return v >= 0 ? v / step : -((-v + step - 1) / step); };
        lo = std::max(lo, -down(-(y - (kViewRow - 1))));
        hi = std::min(hi, down(y + kViewRow - 1));
      }
      if (lo > hi) continue;
      if (any || i != 0 || j != 0 || lo != 0 || hi != 0) return true;
    }
  return false;
}

// two rows of the view share an element
inline bool rows_meet(const RowView& v, int64_t B, int64_t N, int64_t H) {
  const RowGrid g(v, B, N, H);
  if (g.nested()) return false;
  return rows_near(0, B, v.sb, N, v.st, -(H - 1), H - 1, v.sh, false);
}

// A row of x [B, N, Hx] and one of y [B, N, Hy] share an element.  Exact where
// the strides are the same; with other strides a meeting is seen where one of
// the views fills its memory and the other begins or ends in it.
inline bool rows_meet(const RowView& x, int64_t Hx, const RowView& y, int64_t Hy, int64_t B, int64_t N) {
  typedef RowGrid::wide wide;
  const RowGrid gx(x, B, N, Hx), gy(y, B, N, Hy);
  if (gx.hi() <= gy.lo() || gy.hi() <= gx.lo()) return false;
  const bool heads = Hx == 1 || Hy == 1 || x.sh == y.sh;
  if ((B == 1 || x.sb == y.sb) && (N == 1 || x.st == y.st) && heads) {
    const int64_t sh = Hx > 1 ? x.sh : Hy > 1 ? y.sh : kViewRow;
    const wide D = gy.p - gx.p;
    // heads of one buffer, the usual case: y's begin m heads behind x's
    if (sh != 0 && D % sh == 0) {
      const wide m = D / sh, first = std::min<wide>(0, m), last = std::max<wide>(Hx, m + Hy);
      const RowView both = {nullptr, x.sb, x.st, sh};
      if (last - first <= INT64_MAX / 2 && RowGrid(both, B, N, (int64_t)(last - first)).nested())
        return m < Hx && m + Hy > 0;
    }
    return rows_near(D, B, B > 1 ? x.sb : 0, N, N > 1 ? x.st : 0, -(Hx - 1), Hy - 1, sh, true);
  }
  auto inside = [](const RowGrid& in, const RowGrid& full) {
    auto at = [&](wide e) { return e + kViewRow > full.lo() && e < full.hi(); };
    return full.dense() && (at(in.lo()) || at(in.hi() - kViewRow));
  };
  return inside(gx, gy) || inside(gy, gx);
}

// the same rows in the same places
inline bool rows_same(const RowView& x, const RowView& y, int64_t B, int64_t N, int64_t H) {
  return x.p == y.p && (B == 1 || x.sb == y.sb) && (N == 1 || x.st == y.st) && (H == 1 || x.sh == y.sh);
}

}  // namespace s2o
