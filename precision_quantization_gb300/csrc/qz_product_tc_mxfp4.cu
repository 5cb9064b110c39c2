// qz_product_tc_mxfp4.cu -- the tcgen05 products with MXFP4 weights (qz_product_tc.cuh).
#include "qz_product_tc.cuh"

namespace qz {

qz_status launch_product_tc_mxfp4(const ProductArgs& p, cudaStream_t s) {
  return launch_tc<QZ_MXFP4>(p, s);
}

}  // namespace qz
