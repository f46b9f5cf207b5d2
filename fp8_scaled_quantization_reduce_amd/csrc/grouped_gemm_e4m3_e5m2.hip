// grouped_gemm_e4m3_e5m2.hip -- the grouped-GEMM kernels with E4M3 codes in A and
// E5M2 codes in B.
#include "grouped_gemm.h"

namespace fp8q {

FP8Q_GROUPED_PAIR(e4m3_e5m2, kE4M3, kE5M2)

} // namespace fp8q
