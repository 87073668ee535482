// Where a work-group of the paged attention stands in the cut of its batch: integers only, the
// same on the host and the device.
#pragma once

namespace wq {

// The row (a range, or a sequence where there are none) and the unit of a work-group.  With
// near_units eight rows lie side by side, so that all units of one run on the same XCD; the grid
// is then rounded up to eight rows, and false is returned past the last one.
constexpr bool place_of_block(unsigned block, int units, bool near_units, int rows, int& row,
                              int& unit) {
  if (!near_units) {  // (the grid holds no more)
    row = (int)(block / (unsigned)units);
    unit = (int)(block % (unsigned)units);
    return true;
  }
  const int eight = (int)(block / (8u * (unsigned)units));
  row = 8 * eight + (int)(block % 8);
  unit = (int)(block / 8) - eight * units;
  return row < rows;
}

// Granules of a range when `total` are cut into `ranges`; the last ranges may hold fewer, or none.
constexpr int range_length(int total, int ranges) {
  const int length = (int)(((long long)total + ranges - 1) / ranges);
  return length > 1 ? length : 1;
}

// First granule of the row-th of them, -1 where it has none.  Below total + ranges for a row that
// there is, so 32 bits hold it.
constexpr int range_first(int row, int total, int ranges) {
  const int first = row * range_length(total, ranges);
  return first < total ? first : -1;
}

}  // namespace wq
