// Which tile of dw a workgroup makes.  Plain C++, for the kernel, its grid and a test of both.
#pragma once

namespace mvq {

// dw has `tiles` tiles for each of sets = groups * splits; workgroup b runs on XCD b % 8.  A set's tiles go to the XCDs in
// parts (2^shift of them) of neighbouring tiles, which share operands through an XCD's L2:
//   eighths where they are large, as groups differ in their rows, by which a tile's work goes, so that whole groups to an
//     XCD end far apart (16 uneven groups' 8192 rows, dw of 4096 x 7168 each, 1340 us, so 550; 16384 rows, 2560 x 2560 616,
//     248; in quarters 292);
//   otherwise parts of about a quarter of what an XCD holds at once, as long as every XCD has one (even groups, 32 of
//     512 x 512: 16.5 us whole, 21.3 in eighths, 16.6 so; 16 of 1024 x 1024 41, 43 and 40; 64 of 1024 x 512 44, 53 and 45;
//     one group, 8192 rows of 1024 -> 512 28.6, 29.4, 27.4).
// Parts follow each other over the XCDs, one XCD further with every eight, so that those of a few sets use all of them.
constexpr int dw_parts_shift(int tiles, long sets, int side) {
  const int quarter = side >= 256 ? 8 : 16;
  int shift = 3;
  while (shift > 0 && (tiles >> shift) < quarter && (sets << shift) >= 16) --shift;
  return shift;
}
constexpr int dw_part_tiles(int tiles, int shift) { return (tiles + (1 << shift) - 1) >> shift; }
constexpr long dw_workgroups(int tiles, long sets, int shift) { return ((sets << shift) + 7) / 8 * 8 * dw_part_tiles(tiles, shift); }

struct DwPlace {
  int split, group, tile;  // (split >= splits, or tile >= tiles: nothing to do)
};
constexpr DwPlace dw_place(int block, int tiles, int groups, int shift) {
  const int per = dw_part_tiles(tiles, shift), x = block & 7, q = block >> 3, row = q / per;
  const int unit = row * 8 + ((x + row) & 7), set = unit >> shift, split = set / groups;
  return {split, set - split * groups, (unit & ((1 << shift) - 1)) * per + q - row * per};
}

}  // namespace mvq
