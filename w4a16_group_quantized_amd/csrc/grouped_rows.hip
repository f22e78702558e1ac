// The gradient of the rows on the tile kernel (grouped_tile.h).
#include "grouped_tile.h"

namespace moe {

void launch_grouped_rows(const GroupedArgs& a, hipStream_t stream) {
  // by the mean rows per expert; 8 experts of 8192 x 4096, 16381 rows:
  // 1075 us, with tiles of 128 x 128 1308; 512 of 2560 x 640, 40960 rows: 431 and 336
  const int active = a.E < a.rows ? a.E : a.rows;
  const int mean = a.rows / active;
  const int64_t tiles = static_cast<int64_t>(active) * ((mean + 255) / 256) * ((a.K + 255) / 256);
  if (mean >= 256 && tiles >= device_info().cus)
    return launch_grouped_tiles<Grouped256, Product::kRows>(a, stream);
  launch_grouped_tiles<Grouped128, Product::kRows>(a, stream);
}

}  // namespace moe
