// qz_product_few_mxfp4_ragged.cu -- the few-token products with MXFP4 weights whose rows are not whole steps.
#include "qz_product_few.cuh"

namespace qz {

qz_status launch_product_few_mxfp4_ragged(const ProductArgs& p, cudaStream_t s) { return launch_few<QZ_MXFP4, true>(p, s); }

}  // namespace qz
