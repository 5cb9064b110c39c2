// qz_attention_few_e5m2.cu -- attention of a few rows, E5M2 codes.
#include "qz_attention_few.cuh"

namespace qz {

qz_status launch_attention_few_e5m2(const AttentionArgs& a, const FewPlan& p, cudaStream_t s) { return launch_few<QZ_FP8_E5M2>(a, p, s); }

}  // namespace qz
