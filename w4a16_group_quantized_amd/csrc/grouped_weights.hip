// The gradient of the weights on the tile kernel (grouped_tile.h).
#include "grouped_tile.h"

namespace moe {

void launch_grouped_weights(const GroupedArgs& a, hipStream_t stream) {
  // 8 experts of 8192 x 4096, 16381 rows: 946 us, with tiles of 128 x 128 1147; 512 of
  // 1280 x 2560, 40960 rows: 971 and 1194
  const int64_t tiles = static_cast<int64_t>(a.E) * ((a.N + 255) / 256) * ((a.K + 255) / 256);
  if (tiles >= device_info().cus) return launch_grouped_tiles<Grouped256, Product::kWeights>(a, stream);
  launch_grouped_tiles<Grouped128, Product::kWeights>(a, stream);
}

}  // namespace moe
