// qz_product_tc_int4.cu -- the tcgen05 products with INT4 weights (qz_product_tc.cuh).
#include "qz_product_tc.cuh"

namespace qz {

qz_status launch_product_tc_int4(const ProductArgs& p, cudaStream_t s) {
  return launch_tc<QZ_INT4>(p, s);
}

}  // namespace qz
