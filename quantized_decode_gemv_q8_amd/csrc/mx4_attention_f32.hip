// Attention over the cache in 4-bit floats: the instances for f32 rows.
#include "mx4_attention_kernel.h"

namespace q8 {

hipError_t launch_mx4_attention_f32(const AttnArgs &a, int rows, int wgs, hipStream_t stream) {
  return launch_attention<kRowF32>(a, rows, wgs, stream);
}

}  // namespace q8
