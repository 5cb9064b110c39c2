// qz_product_tc_nvfp4.cu -- the tcgen05 products with NVFP4 weights (qz_product_tc.cuh).
#include "qz_product_tc.cuh"

namespace qz {

qz_status launch_product_tc_nvfp4(const ProductArgs& p, cudaStream_t s) {
  return launch_tc<QZ_NVFP4>(p, s);
}

}  // namespace qz
