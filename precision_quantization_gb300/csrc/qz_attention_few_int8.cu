// qz_attention_few_int8.cu -- attention of a few rows, INT8 codes.
#include "qz_attention_few.cuh"

namespace qz {

qz_status launch_attention_few_int8(const AttentionArgs& a, const FewPlan& p, cudaStream_t s) { return launch_few<QZ_INT8>(a, p, s); }

}  // namespace qz
