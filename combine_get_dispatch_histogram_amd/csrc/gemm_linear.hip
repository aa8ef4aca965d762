// gemm_linear.hip -- the rows kernel with a dense product's epilogue.
#include "gemm_rows.h"

namespace miep {

hipError_t launch_gemm_linear(const GemmRowsArgs& a, hipStream_t st) {
  return a.epi.act == kActSwiglu ? launch_rows<kGemmBf16, false, false, kEpiSwiglu>(a, st)
                                 : launch_rows<kGemmBf16, false, false, kEpiPlain>(a, st);
}

}  // namespace miep
