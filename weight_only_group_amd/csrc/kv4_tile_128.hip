// Blocks of prompts on the 4-bit cache, heads of 128.
#include "kv4_tile.h"

namespace qmm {

template <>
hipError_t launch_kv4_tiles<128>(const Kv4TileArgs& t, int group_size, hipStream_t stream) {
  if (group_size == 32) return launch_tiles_of<128, 4>(t, stream);
  if (group_size == 64) return launch_tiles_of<128, 2>(t, stream);
  return launch_tiles_of<128, 1>(t, stream);
}

}  // namespace qmm
