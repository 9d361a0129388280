// Experts' products of one token: Q2_K, Q4_K, Q6_K weights (kernel: experts_few.h).
#include "experts_few.h"

namespace qmm {

hipError_t launch_experts_few_q2_k(const ExpertArgs &a, hipStream_t st) { return experts_few<F_Q2_K>(a, st); }
hipError_t launch_experts_few_q4_k(const ExpertArgs &a, hipStream_t st) { return experts_few<F_Q4_K>(a, st); }
hipError_t launch_experts_few_q6_k(const ExpertArgs &a, hipStream_t st) { return experts_few<F_Q6_K>(a, st); }

}  // namespace qmm
