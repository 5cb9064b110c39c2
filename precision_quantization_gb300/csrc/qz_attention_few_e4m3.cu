// qz_attention_few_e4m3.cu -- attention of a few rows, E4M3 codes.
#include "qz_attention_few.cuh"

namespace qz {

qz_status launch_attention_few_e4m3(const AttentionArgs& a, const FewPlan& p, cudaStream_t s) { return launch_few<QZ_FP8_E4M3>(a, p, s); }

}  // namespace qz
