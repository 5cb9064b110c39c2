// qz_product_few_mxfp4.cu -- the few-token products with MXFP4 weights (qz_product_few.cuh).
#include "qz_product_few.cuh"

namespace qz {

qz_status launch_product_few_mxfp4(const ProductArgs& p, cudaStream_t s) { return launch_few<QZ_MXFP4>(p, s); }

}  // namespace qz
