// kv8_scored.hip -- attention under document and prefix masks and with distance
// bias: instantiations of kv8_attention.h.
#include "kv8_attention.h"

namespace w4a16 {

AttentionLaunch* scored_launch(int mode, int32_t D, int32_t dtype) {
  return mode & kBias ? launcher<kMasks | kBias>(D, dtype) : launcher<kMasks>(D, dtype);
}

}  // namespace w4a16
