// kv8_capped.hip -- attention with capped scores: instantiations of
// kv8_attention.h.
#include "kv8_attention.h"

namespace w4a16 {

AttentionLaunch* capped_launch(int mode, int32_t D, int32_t dtype) {
  return mode & kBias ? launcher<kMasks | kCap | kBias>(D, dtype)
                      : launcher<kMasks | kCap>(D, dtype);
}

}  // namespace w4a16
