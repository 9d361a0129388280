// Experts' products of one token: Q4_0, Q8_0 weights (kernel: experts_few.h).
#include "experts_few.h"

namespace qmm {

hipError_t launch_experts_few_q4_0(const ExpertArgs &a, hipStream_t st) { return experts_few<F_Q4_0>(a, st); }
hipError_t launch_experts_few_q8_0(const ExpertArgs &a, hipStream_t st) { return experts_few<F_Q8_0>(a, st); }

}  // namespace qmm
