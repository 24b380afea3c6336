// Attention over the Q8_0 cache: the instances for bf16 rows.
#include "q8_attention_kernel.h"

namespace q8 {

hipError_t launch_attention_bf16(const AttnArgs &a, int rows, int wgs, hipStream_t stream) {
  return launch_attention<kRowBf16>(a, rows, wgs, stream);
}

}  // namespace q8
