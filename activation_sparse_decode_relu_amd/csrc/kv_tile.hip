// Attention of many rows over whole sequences: see kv_tile.h.
#include "kv_tile.h"

namespace pik {

hipError_t launch_kv_tile(int act, int code, const KvAttendArgs& a, hipStream_t s) {
  return tile_act<ATTEND_ALL>(act, code, a, s);
}

}  // namespace pik
