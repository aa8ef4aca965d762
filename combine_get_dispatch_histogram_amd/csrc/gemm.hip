// gemm.hip -- grouped bf16 products: forward and the rows' gradient.
#include "gemm_rows.h"

namespace miep {

hipError_t launch_gemm_fp8(const GemmRowsArgs& a, hipStream_t st);

hipError_t launch_gemm_rows(const GemmRowsArgs& args, hipStream_t st) {
  GemmRowsArgs a = args;
  if (a.g.G == 0 || a.g.limit == 0) return hipSuccess;
  if (a.expected <= 0) a.expected = static_cast<int>((a.g.limit + a.g.G - 1) / a.g.G);
  if (a.type != kGemmBf16) return launch_gemm_fp8(a, st);
  if (a.transposed) return launch_rows<kGemmBf16, true, false>(a, st);
  return a.row_index ? launch_rows<kGemmBf16, false, true>(a, st) : launch_rows<kGemmBf16, false, false>(a, st);
}

}  // namespace miep
