// qz_attention_tc_e4m3.cu -- attention of many rows, E4M3 codes.
#include "qz_attention_tc.cuh"

namespace qz {

qz_status launch_attention_tc_e4m3(const AttentionArgs& a, const TcAttPlan& p, cudaStream_t s) { return launch_tc<QZ_FP8_E4M3>(a, p, s); }

}  // namespace qz
