// Decode attention's first launch over q4_0 caches (attn_chunk.h).
#include "attn_chunk.h"

namespace qmm {

hipError_t launch_attn_q4_0(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st) {
    return launch_chunks<KV_Q4_0>(nb, rt, a, B, st);
}

}  // namespace qmm
