// grouped_gemm.h -- FP8 products of ragged groups of rows with a matrix per
// group (the experts of a layer), included by one translation unit per
// operand-format pair.
//
// fprop / dgrad: rows t of group e, C[t] = sum over 128-wide slices kb of
//   fma(part_kb, fl32(sA[t, kb] sB[e, n / 128, kb]), acc),
//   part_kb the slice's products on the FP8 matrix instruction,
//   B [groups][N][K] codes with 128x128 block scales.
// wgrad: C[e] = A_e B_e^T contracted over the rows (tokens) of group e, from
//   the token-contiguous copies A [M][stride], B [N][stride] with one scale
//   per row and block of 128 tokens; a group's tokens fill whole blocks.
#ifndef FP8Q_GROUPED_GEMM_H
#define FP8Q_GROUPED_GEMM_H

#include "gemm_kernels.h"
#include "groups.h"

namespace fp8q {

// 32 bytes of a 128-byte slice row for lane group g: chunks g and g + 4 (A and
// B use the same ones, so the order inside the slice does not matter)
__device__ __forceinline__ v8i load_frag(const uint8_t *row, int g)
{
    const uint4 lo = *reinterpret_cast<const uint4 *>(row + 16 * g);
    const uint4 hi = *reinterpret_cast<const uint4 *>(row + 64 + 16 * g);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes -> eight bf16 values (exact: bf16 has more exponent and mantissa
// bits than either format).
template <int F> __device__ __forceinline__ bf16x8 widen8(int lo, int hi)
{
    bf16x2 p[4];
    if constexpr (F == kE4M3) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
    }
    return bf16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// One slice's 16x16 partial.  kWide: the codes are widened to bf16 and
// multiplied by the bf16 matrix instruction, whose sums are binary32.
// The FP8 instruction adds the products of eight neighbouring bytes on about
// 15 bits under the largest of them (measured on the MI355X with one large
// and one small product at a time), which leaves an fp32 result 1.1e-5 off in
// the 2-norm where the widened one is 1e-8 off: below the rounding of a bf16
// result, but above that of an fp32 one.
template <int FA, int FB, bool kWide> __device__ __forceinline__ v4f slice16(const v8i &b, const v8i &a)
{
    if constexpr (!kWide) {
        return mfma16x16x128<FB, FA>(b, a, v4f{0.f, 0.f, 0.f, 0.f});
    } else {
        v4f c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<FB>(b[2 * s], b[2 * s + 1]),
                                                        widen8<FA>(a[2 * s], a[2 * s + 1]), c, 0, 0, 0);
        return c;
    }
}

struct GroupedArgs {
    const uint8_t *A, *B;
    const float *sA, *sB;
    const int32_t *offsets;
    int groups, rows;
    int64_t M, N, K; // wgrad: M x N per group; K unused
    int64_t stride;  // wgrad: bytes of a row of A and B
    void *C;
    int c_dtype;
    hipStream_t stream;
    int cus;
};

// fprop / dgrad with 16 rows of a group x 64 columns per block; four waves
// take the 128-wide slices in turn and add their sums through LDS.
template <int FA, int FB, int DC>
__global__ __launch_bounds__(256) void grouped_rows_kernel(const uint8_t *__restrict__ A, const float *__restrict__ sA,
                                                           const uint8_t *__restrict__ B, const float *__restrict__ sB,
                                                           const int32_t *__restrict__ offsets, int groups, int rows,
                                                           int N, int K, void *__restrict__ C)
{
    __shared__ v4f sums[4][4][64];
    const int tiles_n = N / 64;
    const int t = blockIdx.x / tiles_n, n0 = (int)(blockIdx.x % tiles_n) * 64;
    GroupTile gt;
    int tiles;
    if (!find_tile<16>(offsets, groups, rows, t, gt, tiles)) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int nk = K / 128;
    const int in_group = 16 * gt.tile + r;
    const bool live = in_group < gt.size;
    const int64_t row = gt.row0 + (live ? in_group : 16 * gt.tile);
    const uint8_t *Bg = B + ((int64_t)gt.group * N + n0) * K;
    const float *sBg = sB + ((int64_t)gt.group * (N / 128) + n0 / 128) * nk;
    v4f acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int kb = w; kb < nk; kb += 4) {
        const v8i a = load_frag(A + row * K + kb * 128, g);
        const float wt = sA[row * nk + kb] * sBg[kb];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const v8i b = load_frag(Bg + (int64_t)(16 * j + r) * K + kb * 128, g);
            const v4f p = slice16<FA, FB, false>(b, a);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = __builtin_fmaf(p[e], wt, acc[j][e]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[w][j][lane] = acc[j];
    __syncthreads();
    // wave w finishes column tile w
    v4f c = sums[0][w][lane];
#pragma unroll
    for (int k = 1; k < 4; ++k) c += sums[k][w][lane];
    if (live) {
        const int64_t at = row * N + n0 + 16 * w + 4 * g;
        if constexpr (DC == kF32) *reinterpret_cast<v4f *>((float *)C + at) = c;
        else *reinterpret_cast<uint2 *>((uint16_t *)C + at) = __builtin_bit_cast(uint2, __builtin_convertvector(c, bf16x4));
    }
}

// wgrad with 64 x 64 of one group's C per wave.
template <int FA, int FB, int DC>
__global__ __launch_bounds__(64) void grouped_wgrad_kernel(const uint8_t *__restrict__ A, const float *__restrict__ sA,
                                                           const uint8_t *__restrict__ B, const float *__restrict__ sB,
                                                           const int32_t *__restrict__ offsets, int groups, int rows,
                                                           int M, int N, int64_t stride, void *__restrict__ C)
{
    constexpr bool kWide = DC == kF32;
    const int tiles_n = N / 64, tiles_m = M / 64;
    const int e = blockIdx.x / (tiles_n * tiles_m), tm = blockIdx.x / tiles_n % tiles_m, tn = blockIdx.x % tiles_n;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    // blocks of 128 tokens before group e and in it
    int kb0 = 0, kbn = 0;
    for (int g0 = 0; g0 <= e; g0 += 64) {
        int lo, size;
        group_rows(offsets, groups, rows, g0 + lane, lo, size);
        const int count = (int)(((unsigned)size + 127) / 128), sum = wave_scan_i32(count);
        if (e < g0 + 64) {
            kbn = __builtin_amdgcn_readlane(count, e - g0);
            kb0 += __builtin_amdgcn_readlane(sum, e - g0) - kbn;
        } else {
            kb0 += __builtin_amdgcn_readlane(sum, 63);
        }
    }
    const int kbs = (int)(stride / 128);
    kb0 = min(kb0, kbs);
    kbn = min(kbn, kbs - kb0);
    v4f acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int kb = kb0; kb < kb0 + kbn; ++kb) {
        v8i a[4], b[4];
        float wa[4];
        v4f wb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = tm * 64 + 16 * i + r, n = tn * 64 + 16 * i + r;
            a[i] = load_frag(A + m * stride + (int64_t)kb * 128, g);
            b[i] = load_frag(B + n * stride + (int64_t)kb * 128, g);
            wa[i] = sA[m * kbs + kb];
#pragma unroll
            for (int q = 0; q < 4; ++q) wb[i][q] = sB[(int64_t)(tn * 64 + 16 * i + 4 * g + q) * kbs + kb];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const v4f p = slice16<FA, FB, kWide>(b[j], a[i]);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(p[q], wa[i] * wb[j][q], acc[i][j][q]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = ((int64_t)e * M + tm * 64 + 16 * i + r) * N + tn * 64 + 16 * j + 4 * g;
            if constexpr (DC == kF32) *reinterpret_cast<v4f *>((float *)C + at) = acc[i][j];
            else
                *reinterpret_cast<uint2 *>((uint16_t *)C + at) =
                    __builtin_bit_cast(uint2, __builtin_convertvector(acc[i][j], bf16x4));
        }
}

template <int FA, int FB> hipError_t launch_grouped_rows(const GroupedArgs &a)
{
    const unsigned grid = (unsigned)(max_tiles(a.rows, a.groups, 16) * (a.N / 64));
    grouped_rows_kernel<FA, FB, kBF16><<<grid, 256, 0, a.stream>>>(a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows,
                                                                   (int)a.N, (int)a.K, a.C);
    return hipGetLastError();
}

template <int FA, int FB> hipError_t launch_grouped_wgrad(const GroupedArgs &a)
{
    const unsigned grid = (unsigned)((int64_t)a.groups * (a.M / 64) * (a.N / 64));
    if (a.c_dtype == kF32)
        grouped_wgrad_kernel<FA, FB, kF32><<<grid, 64, 0, a.stream>>>(a.A, a.sA, a.B, a.sB, a.offsets, a.groups,
                                                                      a.rows, (int)a.M, (int)a.N, a.stride, a.C);
    else
        grouped_wgrad_kernel<FA, FB, kBF16><<<grid, 64, 0, a.stream>>>(a.A, a.sA, a.B, a.sB, a.offsets, a.groups,
                                                                       a.rows, (int)a.M, (int)a.N, a.stride, a.C);
    return hipGetLastError();
}

// One operand-format pair's launchers (one translation unit each).
#define FP8Q_GROUPED_PAIR(NAME, FA, FB)                                                                              \
    hipError_t launch_grouped_rows_##NAME(const GroupedArgs &a) { return launch_grouped_rows<FA, FB>(a); }           \
    hipError_t launch_grouped_wgrad_##NAME(const GroupedArgs &a) { return launch_grouped_wgrad<FA, FB>(a); }

} // namespace fp8q

#endif // FP8Q_GROUPED_GEMM_H
