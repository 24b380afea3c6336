// Attention over the cache in 4-bit floats: the instances for bf16 rows.
#include "mx4_attention_kernel.h"

namespace q8 {

hipError_t launch_mx4_attention_bf16(const AttnArgs &a, int rows, int wgs, hipStream_t stream) {
  return launch_attention<kRowBf16>(a, rows, wgs, stream);
}

}  // namespace q8
