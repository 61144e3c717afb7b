// Blocks of prompts on the 4-bit cache, heads of 256.
#include "kv4_tile.h"

namespace qmm {

template <>
hipError_t launch_kv4_tiles<256>(const Kv4TileArgs& t, int group_size, hipStream_t stream) {
  if (group_size == 32) return launch_tiles_of<256, 8>(t, stream);
  if (group_size == 64) return launch_tiles_of<256, 4>(t, stream);
  return launch_tiles_of<256, 2>(t, stream);
}

}  // namespace qmm
