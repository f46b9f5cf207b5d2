// grouped_gemm.hip -- dispatch of a grouped-GEMM launch to the translation
// unit of its operand-format pair (the kernels are in grouped_gemm.h).
#include "grouped_gemm.h"

namespace fp8q {

#define FP8Q_DECLARE(NAME)                                                                                           \
    hipError_t launch_grouped_rows_##NAME(const GroupedArgs &a);                                                     \
    hipError_t launch_grouped_wgrad_##NAME(const GroupedArgs &a);
FP8Q_DECLARE(e4m3_e4m3)
FP8Q_DECLARE(e5m2_e4m3)
FP8Q_DECLARE(e4m3_e5m2)
FP8Q_DECLARE(e5m2_e5m2)
#undef FP8Q_DECLARE

bool grouped_gemm_fits(int64_t rows, int groups, int64_t N)
{
    return pp_blocks(rows, groups, N, 256) <= max_blocks(kBSThreads);
}

// 64 x 64 tiles are only taken where there are few
bool grouped_wgrad_fits(int groups, int64_t M, int64_t N)
{
    return wgrad_blocks(groups, M, N, 128) <= max_blocks(256) &&
           wgrad_blocks(groups, M, N, 256) <= max_blocks(kBSThreads);
}

hipError_t launch_grouped_gemm(const uint8_t *A, int fa, const float *sA, const uint8_t *B, int fb, const float *sB,
                               const int32_t *offsets, int groups, int64_t rows, int64_t N, int64_t K, void *C,
                               hipStream_t s)
{
    if (rows == 0 || groups == 0 || N == 0) return hipSuccess;
    const GroupedArgs a{A, B, sA, sB, offsets, groups, (int)rows, 0, N, K, 0, C, kBF16, s, compute_units()};
    if (fa == kE4M3) return fb == kE4M3 ? launch_grouped_rows_e4m3_e4m3(a) : launch_grouped_rows_e4m3_e5m2(a);
    return fb == kE4M3 ? launch_grouped_rows_e5m2_e4m3(a) : launch_grouped_rows_e5m2_e5m2(a);
}

hipError_t launch_grouped_wgrad(const uint8_t *A, int fa, const float *sA, const uint8_t *B, int fb, const float *sB,
                                const int32_t *offsets, int groups, int64_t rows, int64_t stride, int64_t M,
                                int64_t N, void *C, int c_dtype, hipStream_t s)
{
    if (groups == 0 || M == 0 || N == 0) return hipSuccess;
    // Rows from `stride` on cannot be in the columnwise copies.  Without them the
    // blocks of up to 2^16 groups of any offsets add up to at most 2^30, which the
    // kernels' 32-bit sums hold.
    if (rows > stride) rows = stride;
    const GroupedArgs a{A, B, sA, sB, offsets, groups, (int)rows, M, N, 0, stride, C, c_dtype, s, compute_units()};
    if (fa == kE4M3) return fb == kE4M3 ? launch_grouped_wgrad_e4m3_e4m3(a) : launch_grouped_wgrad_e4m3_e5m2(a);
    return fb == kE4M3 ? launch_grouped_wgrad_e5m2_e4m3(a) : launch_grouped_wgrad_e5m2_e5m2(a);
}

} // namespace fp8q
