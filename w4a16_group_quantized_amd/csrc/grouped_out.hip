// The product itself on the tile kernel (grouped_tile.h).
#include "grouped_tile.h"

namespace moe {

// The rules go by the mean rows per expert; their figures are of rows shared out evenly.
// Uneven rows cost nothing beside them: 512 experts of 1280 x 2560, 40960 rows of which 64
// experts hold 40137 (Zipf), 490 us, evenly 703; 8 of 8192 x 4096, 16381 rows, half on one of
// them, 980, evenly 1000.
void launch_grouped_out(const GroupedArgs& a, hipStream_t stream) {
  const int active = a.E < a.rows ? a.E : a.rows;  // experts that can hold a row
  const int mean = a.rows / active;
  const auto tiles = [&](int size) { return row_product_tiles(active, mean, a.N, size); };
  // 1 expert of 1280 x 2560, 100 rows: 160 tiles of 32 x 32 with eight waves each 8.7
  // us, 40 of 64 x 64 16.7
  if (tiles(32) <= kUnits)
    return launch_grouped_tiles<GroupedSplit, Product::kOut>(a, stream);
  // few rows of many experts, bound by reading weights: more workgroups in flight
  // (512 experts of 1280 x 2560, 80 rows: 128 x 128 105 us, 64 x 64 94)
  if (mean <= 16 && tiles(64) > 4 * kUnits)
    return launch_grouped_tiles<Grouped64, Product::kOut>(a, stream);
  const int size = pick_size(tiles);
  if (size == 256) return launch_grouped_tiles<Grouped256, Product::kOut>(a, stream);
  if (size == 128) return launch_grouped_tiles<Grouped128, Product::kOut>(a, stream);
  launch_grouped_tiles<Grouped64, Product::kOut>(a, stream);
}

}  // namespace moe
