// Decode attention's first launch over f16 caches (attn_chunk.h).
#include "attn_chunk.h"

namespace qmm {

hipError_t launch_attn_f16(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st) {
    return launch_chunks<KV_F16>(nb, rt, a, B, st);
}

}  // namespace qmm
