// Experts' products of one token: Q4_1, Q5_0, Q5_1 weights (kernel: experts_few.h).
#include "experts_few.h"

namespace qmm {

hipError_t launch_experts_few_q4_1(const ExpertArgs &a, hipStream_t st) { return experts_few<F_Q4_1>(a, st); }
hipError_t launch_experts_few_q5_0(const ExpertArgs &a, hipStream_t st) { return experts_few<F_Q5_0>(a, st); }
hipError_t launch_experts_few_q5_1(const ExpertArgs &a, hipStream_t st) { return experts_few<F_Q5_1>(a, st); }

}  // namespace qmm
