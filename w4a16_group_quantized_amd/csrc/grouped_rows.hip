// The gradient of the rows on the tile kernel (grouped_tile.h).
#include "grouped_tile.h"

namespace moe {

// The rules go by the mean rows per expert; their figures are of rows shared out evenly.
// Uneven rows (grouped_out.hip) take 488 us, evenly 776, and 1038, evenly 1035.
void launch_grouped_rows(const GroupedArgs& a, hipStream_t stream) {
  const int active = a.E < a.rows ? a.E : a.rows;  // experts that can hold a row
  const int mean = a.rows / active;
  const auto tiles = [&](int size) { return row_product_tiles(active, mean, a.K, size); };
  // 1 expert of 4096 x 512, 100 rows: 64 tiles of 32 x 32 with eight waves each 10.5 us,
  // 16 of 64 x 64 26.5; 8 experts of 2560 x 640, 1000 rows, 640 tiles 27.9 and 160 18.4
  if (tiles(32) <= kUnits)
    return launch_grouped_tiles<GroupedSplit, Product::kRows>(a, stream);
  const int size = pick_size(tiles);
  if (size == 256) return launch_grouped_tiles<Grouped256, Product::kRows>(a, stream);
  if (size == 128) return launch_grouped_tiles<Grouped128, Product::kRows>(a, stream);
  launch_grouped_tiles<Grouped64, Product::kRows>(a, stream);
}

}  // namespace moe
