// qz_product_few_int4.cu -- the few-token products with INT4 weights (qz_product_few.cuh).
#include "qz_product_few.cuh"

namespace qz {

qz_status launch_product_few_int4(const ProductArgs& p, cudaStream_t s) { return launch_few<QZ_INT4>(p, s); }

}  // namespace qz
