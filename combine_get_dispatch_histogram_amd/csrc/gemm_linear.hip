// gemm_linear.hip -- dense products with their epilogue, and their rows' gradient.
#include "gemm_dense.h"

namespace miep {

hipError_t launch_gemm_linear(const GemmRowsArgs& a, hipStream_t st) {
  if (a.transposed) return launch_dense<true, kEpiNone>(a, st);
  return a.epi.act == kActSwiglu ? launch_dense<false, kEpiSwiglu>(a, st) : launch_dense<false, kEpiPlain>(a, st);
}

}  // namespace miep
