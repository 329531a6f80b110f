// q8_w4_bf16.hip -- the 4-bit weight's tile kernels for bf16 activations.
#include "q8_w4_tile.h"

namespace q8 {

hipError_t launch_w4_tile_bf16(const W4Plan &p, bool pair, const W4Args &a, hipStream_t stream) {
  return launch_w4_tile<kActBf16>(p, pair, a, stream);
}

}  // namespace q8
