// gemm_fp8.hip -- grouped E4M3 products with a scale for each 128 channels of
// a row and each 128 x 128 block of the weights.
#include "gemm_rows.h"

namespace miep {

hipError_t launch_gemm_fp8(const GemmRowsArgs& a, hipStream_t st) {
  if (a.type == kGemmFp8)
    return a.row_index ? launch_rows<kGemmFp8, false, true>(a, st) : launch_rows<kGemmFp8, false, false>(a, st);
  return a.row_index ? launch_rows<kGemmFp8Ue8m0, false, true>(a, st) : launch_rows<kGemmFp8Ue8m0, false, false>(a, st);
}

}  // namespace miep
