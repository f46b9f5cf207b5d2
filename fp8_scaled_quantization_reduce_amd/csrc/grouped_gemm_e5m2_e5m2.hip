// grouped_gemm_e5m2_e5m2.hip -- the grouped-GEMM kernels with E5M2 codes in A and
// E5M2 codes in B.
#include "grouped_gemm.h"

namespace fp8q {

FP8Q_GROUPED_PAIR(e5m2_e5m2, kE5M2, kE5M2)

} // namespace fp8q
