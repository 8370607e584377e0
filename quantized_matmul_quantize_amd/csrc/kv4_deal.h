// kv4_deal.h -- how the rows of a prefix are dealt to blocks.  Plain C++, so that
// it is tested without a GPU.
#pragma once

namespace qmm {

// The first of the `strips` of rows that are tile `tile`'s of `tiles`, which has
// those up to the next tile's first: the same number each, the first strips %
// tiles one more.  Nothing here passes `strips` (tile * strips / tiles would pass
// 2^31 from 4 million rows on).
constexpr int first_strip(int tile, int strips, int tiles) {
  const int more = strips % tiles;
  return tile * (strips / tiles) + (tile < more ? tile : more);
}

}  // namespace qmm
