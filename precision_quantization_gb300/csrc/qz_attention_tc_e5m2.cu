// qz_attention_tc_e5m2.cu -- attention of many rows, E5M2 codes.
#include "qz_attention_tc.cuh"

namespace qz {

qz_status launch_attention_tc_e5m2(const AttentionArgs& a, const TcAttPlan& p, cudaStream_t s) { return launch_tc<QZ_FP8_E5M2>(a, p, s); }

}  // namespace qz
