// Attention over the Q8_0 cache: the instances for f16 rows.
#include "q8_attention_kernel.h"

namespace q8 {

hipError_t launch_attention_f16(const AttnArgs &a, int rows, int wgs, hipStream_t stream) {
  return launch_attention<kRowF16>(a, rows, wgs, stream);
}

}  // namespace q8
