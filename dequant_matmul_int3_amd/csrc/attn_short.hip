// Attention over a short quantized cache, one block of eight waves for all of
// it; see attn.h.
#include "attn.h"

namespace qt {

hipError_t launch_attn_short(const AttnKernelArgs& k, hipStream_t s) {
    return k.a.bf16 ? attn_bits<kAttnMaxWaves, false>(k, s) : attn_bits<kAttnMaxWaves, true>(k, s);
}

}  // namespace qt
