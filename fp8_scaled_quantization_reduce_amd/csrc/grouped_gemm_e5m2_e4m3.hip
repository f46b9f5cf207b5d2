// grouped_gemm_e5m2_e4m3.hip -- the grouped-GEMM kernels with E5M2 codes in A and
// E4M3 codes in B.
#include "grouped_gemm.h"

namespace fp8q {

FP8Q_GROUPED_PAIR(e5m2_e4m3, kE5M2, kE4M3)

} // namespace fp8q
