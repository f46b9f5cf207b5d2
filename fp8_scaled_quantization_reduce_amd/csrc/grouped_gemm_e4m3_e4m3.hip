// grouped_gemm_e4m3_e4m3.hip -- the grouped-GEMM kernels with E4M3 codes in A and
// E4M3 codes in B.
#include "grouped_gemm.h"

namespace fp8q {

FP8Q_GROUPED_PAIR(e4m3_e4m3, kE4M3, kE4M3)

} // namespace fp8q
