// ss_view.h -- extents of range-checked views of strided rows.  Internal to
// libss.so; plain integers, so that they are checked without a GPU too.
#pragma once

#include <stdint.h>

namespace ss {

// Bytes from the first byte of a view's first row to behind the last one that
// may be read or written: `rows` rows, `row` bytes apart, `cols` bytes of each.
// The view ends with the last row's columns, not a whole `row` behind that
// row's first: it may begin inside a row (a head's columns), and what follows
// the last of them is no longer the caller's.
constexpr uint32_t view_bytes(int64_t row, int rows, int64_t cols) {
  return rows > 0 ? (uint32_t)((rows - 1) * row + cols) : 0u;
}

}  // namespace ss
