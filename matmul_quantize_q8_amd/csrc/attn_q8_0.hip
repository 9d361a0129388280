// Decode attention's first launch over q8_0 caches (attn_chunk.h).
#include "attn_chunk.h"

namespace qmm {

hipError_t launch_attn_q8_0(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st) {
    return launch_chunks<KV_Q8_0>(nb, rt, a, B, st);
}

}  // namespace qmm
