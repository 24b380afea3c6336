// Attention over the Q8_0 cache: the instances for f32 rows.
#include "q8_attention_kernel.h"

namespace q8 {

hipError_t launch_attention_f32(const AttnArgs &a, int rows, int wgs, hipStream_t stream) {
  return launch_attention<kRowF32>(a, rows, wgs, stream);
}

}  // namespace q8
