// Index arithmetic of the paged cache, plain C++ for host and device (internal; not part of
// the C ABI).
//
// Slot j of a sequence lies in row j % ps of the page its table row names at j / ps.  A query
// at the last position of a sequence of `len` slots sees slots j < len with j >= len - window
// or j < sinks (window 0: all of them).  The visible slots are numbered 0 .. count - 1 in
// ascending order, so that a kernel walks them as one dense range.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MIKV_HD __host__ __device__ __forceinline__
#else
#define MIKV_HD inline
#endif

namespace mikv {

// x / d and x % d for 0 <= x < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// Invariant Integers using Multiplication", 1994): with 2^(l-1) < d <= 2^l and
// m = ceil(2^(31+l) / d), floor(x m / 2^(31+l)) = floor(x / d).
struct FastDiv {
  uint32_t d, mul;
  int32_t shift;
};
inline FastDiv make_fast_div(uint32_t d) {
  int l = 0;
  while ((1ull << l) < d) ++l;
  const int s = 31 + l;
  return {d, static_cast<uint32_t>(((1ull << s) + d - 1) / d), s};
}
MIKV_HD uint32_t div_of(uint32_t x, const FastDiv& f) {
  return static_cast<uint32_t>((static_cast<uint64_t>(x) * f.mul) >> f.shift);
}

struct Visible {
  int32_t count;   // visible slots
  int32_t sinks;   // of them, the first ones that lie before the window
  int32_t skip;    // slots hidden between the sinks and the window
};
MIKV_HD Visible visible_slots(int32_t len, int32_t window, int32_t sinks) {
  const int32_t w0 = (window > 0 && len > window) ? len - window : 0;  // the window's first slot
  const int32_t ns = sinks < w0 ? sinks : w0;
  return {ns + (len - w0), ns, w0 - ns};
}
MIKV_HD int32_t visible_slot(const Visible& v, int32_t i) { return i < v.sinks ? i : i + v.skip; }

// Number of rows of the pool in front of row (page, head, r) of one layer, or kNoRow where the
// table names no page of the pool.  The host keeps n_pages * heads * ps below 2^32 - 1.
constexpr uint32_t kNoRow = 0xffffffffu;
MIKV_HD uint32_t pool_row(int32_t page, int32_t n_pages, int32_t heads, int32_t head, uint32_t ps, uint32_t r) {
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(n_pages)) return kNoRow;
  return (static_cast<uint32_t>(page) * static_cast<uint32_t>(heads) + static_cast<uint32_t>(head)) * ps + r;
}

// Pages that `len` slots take.  len + ps - 1 stays below 2^32.
MIKV_HD int32_t pages_of(int32_t len, const FastDiv& ps) {
  return len <= 0 ? 0 : static_cast<int32_t>(div_of(static_cast<uint32_t>(len - 1), ps)) + 1;
}

// The split of `total` tiles over `workers`: worker c takes tiles [split_begin(c), split_begin(c + 1)),
// and tile t belongs to split_owner(t).
MIKV_HD int64_t split_begin(int64_t total, int32_t workers, int32_t c) { return total * c / workers; }
MIKV_HD int32_t split_owner(int64_t total, int32_t workers, int64_t t) {
  return static_cast<int32_t>(((t + 1) * workers - 1) / total);
}

// Parts of a unit of `tiles` tiles where the `units` of a call are alike: a warp takes a tile at least.
MIKV_HD int64_t parts_of_unit(int64_t tiles, int64_t units, int64_t warps) {
  return tiles < warps / units ? tiles : warps / units;
}

}  // namespace mikv
