// qz_attention_tc_int8.cu -- attention of many rows, INT8 codes.
#include "qz_attention_tc.cuh"

namespace qz {

qz_status launch_attention_tc_int8(const AttentionArgs& a, const TcAttPlan& p, cudaStream_t s) { return launch_tc<QZ_INT8>(a, p, s); }

}  // namespace qz
