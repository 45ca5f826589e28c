// Attention over the quantized cache for f32 queries; see attn.h.
#include "attn.h"

namespace qt {

hipError_t launch_attn_f32(const AttnKernelArgs& k, hipStream_t s) {
    return attn_bits<kAttnWaves, true>(k, s);
}

}  // namespace qt
