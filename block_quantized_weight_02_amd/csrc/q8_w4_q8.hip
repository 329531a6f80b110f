// q8_w4_q8.hip -- the 4-bit weight's tile kernels for Q8_0 activations.
#include "q8_w4_tile.h"

namespace q8 {

hipError_t launch_w4_tile_q8(const W4Plan &p, bool pair, const W4Args &a, hipStream_t stream) {
  return launch_w4_tile<kActQ8>(p, pair, a, stream);
}

}  // namespace q8
