// grouped_quant.hip -- 1x128 block quantization of rows gathered in the order
// the experts read them.
//
// Row t of the output is row row_index[t] of x (or row t): its 128-column
// blocks are quantized as fp8_quantize_block's 1x128 blocks are.  The
// columnwise copy, which the weight gradient contracts over, has blocks of 128
// consecutive rows of one group; a group's last block is filled up with zero
// rows, so that a block never mixes two groups.
//
// rows_kernel (no columnwise copy): a wave takes 512 columns of a row, eight
// per lane, so a row piece is read and written in one contiguous run and a
// block's maximum is a reduction over 16 lanes.
// tile_both_kernel: 128 rows of a group x 128 columns per block of 256
// lanes, four rows x 16 columns each.  Row blocks are 8 lanes, column blocks
// the whole block (8 lanes of a wave, then four waves through LDS); the
// column codes are transposed through LDS, so both copies leave as whole 128-
// byte pieces.
#include "fp8q_device.h"
#include "fp8q_launch.h"
#include "groups.h"

namespace fp8q {

namespace {

constexpr int kGqThreads = 256;

template <int DT> struct In;
template <> struct In<kF32> {
    typedef float type;
};
template <> struct In<kBF16> {
    typedef uint16_t type;
};

// kN (8 or 16) elements at p (16-byte aligned) as floats
template <int DT, int kN> __device__ __forceinline__ void load_n(const typename In<DT>::type *p, float *v)
{
    if constexpr (DT == kF32) {
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) {
            const uint4 w = reinterpret_cast<const uint4 *>(p)[i];
            v[4 * i] = __uint_as_float(w.x), v[4 * i + 1] = __uint_as_float(w.y);
            v[4 * i + 2] = __uint_as_float(w.z), v[4 * i + 3] = __uint_as_float(w.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN / 8; ++i) {
            const uint4 w = reinterpret_cast<const uint4 *>(p)[i];
            const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) v[8 * i + 2 * k] = bf16_lo(d[k]), v[8 * i + 2 * k + 1] = bf16_hi(d[k]);
        }
    }
}

// The source row of grouped row t; -1 (a row of zeros) for an index outside x.
__device__ __forceinline__ int64_t source_row(const int32_t *index, int64_t x_rows, int64_t t)
{
    const int64_t r = index ? (int64_t)index[t] : t;
    return r >= 0 && r < x_rows ? r : -1;
}

template <int F, int DT>
__global__ __launch_bounds__(kGqThreads) void rows_kernel(const typename In<DT>::type *__restrict__ x, int64_t x_rows,
                                                          int64_t cols, const int32_t *__restrict__ index,
                                                          int64_t rows, uint8_t *__restrict__ q, float *__restrict__ s)
{
    const int lane = threadIdx.x & 63;
    const int64_t pieces = (cols + 511) / 512, units = rows * pieces;
    for (int64_t u = (int64_t)blockIdx.x * (kGqThreads / 64) + (threadIdx.x >> 6); u < units;
         u += (int64_t)gridDim.x * (kGqThreads / 64)) {
        const int64_t t = u / pieces, c = (u - t * pieces) * 512 + 8 * lane;
        const int64_t r = source_row(index, x_rows, t);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        // cols is a multiple of 128, so the 16 lanes of a block agree
        if (c < cols && r >= 0) load_n<DT, 8>(x + r * cols + c, v);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, f32_absbits(v[e]));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
        const Scales sc = current_scales(__uint_as_float(canonical_amax_bits(m)), Fmt<F>::kMax, 0);
        if (c < cols) {
            uint2 o;
            o.x = encode4<F>(v[0], v[1], v[2], v[3], sc.scale);
            o.y = encode4<F>(v[4], v[5], v[6], v[7], sc.scale);
            *reinterpret_cast<uint2 *>(q + t * cols + c) = o;
            if ((lane & 15) == 0) s[t * (cols / 128) + c / 128] = sc.s;
        }
    }
}

template <int F, int DT>
__global__ __launch_bounds__(kGqThreads) void tile_both_kernel(
    const typename In<DT>::type *__restrict__ x, int64_t x_rows, int64_t cols, const int32_t *__restrict__ index,
    int rows, const int32_t *__restrict__ offsets, int groups, uint8_t *__restrict__ q_row, float *__restrict__ s_row,
    uint8_t *__restrict__ q_col, float *__restrict__ s_col, int64_t stride)
{
    __shared__ __attribute__((aligned(16))) uint32_t tl[128 * 32]; // column codes, [column][row / 4]
    __shared__ uint32_t colmax[4][128];
    __shared__ float colscale[128];
    const int blocks_c = (int)(cols / 128);
    const int t = (int)(blockIdx.x / blocks_c), cb = (int)(blockIdx.x % blocks_c);
    GroupTiles<128> tiles(offsets, groups, rows);
    if (t >= tiles.total) return;
    const GroupTile gt = tiles.find(t);
    const int ig = threadIdx.x >> 3, jg = threadIdx.x & 7, wave = threadIdx.x >> 6;
    const int64_t c0 = (int64_t)cb * 128 + 16 * jg;
    float v[4][16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int in_group = 128 * gt.tile + 4 * ig + r;
        const int64_t src = in_group < gt.size ? source_row(index, x_rows, (int64_t)gt.row0 + in_group) : -1;
#pragma unroll
        for (int e = 0; e < 16; ++e) v[r][e] = 0.0f;
        if (src >= 0) load_n<DT, 16>(x + src * cols + c0, v[r]);
    }
    if (q_row) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) m = max(m, f32_absbits(v[r][e]));
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
            const Scales sc = current_scales(__uint_as_float(canonical_amax_bits(m)), Fmt<F>::kMax, 0);
            const int in_group = 128 * gt.tile + 4 * ig + r;
            if (in_group < gt.size) {
                const int64_t row = (int64_t)gt.row0 + in_group;
                uint4 o;
                o.x = encode4<F>(v[r][0], v[r][1], v[r][2], v[r][3], sc.scale);
                o.y = encode4<F>(v[r][4], v[r][5], v[r][6], v[r][7], sc.scale);
                o.z = encode4<F>(v[r][8], v[r][9], v[r][10], v[r][11], sc.scale);
                o.w = encode4<F>(v[r][12], v[r][13], v[r][14], v[r][15], sc.scale);
                *reinterpret_cast<uint4 *>(q_row + row * cols + c0) = o;
                if (jg == 0) s_row[row * blocks_c + cb] = sc.s;
            }
        }
    }
    // the caller's columnwise buffers may be too short for these offsets
    if ((int64_t)t * 128 + 128 > stride) return; // block-uniform
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) m = max(m, f32_absbits(v[r][c]));
#pragma unroll
        for (int d = 8; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
        if ((threadIdx.x & 63) < 8) colmax[wave][16 * jg + c] = m;
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        const int c = threadIdx.x;
        const uint32_t m = max(max(colmax[0][c], colmax[1][c]), max(colmax[2][c], colmax[3][c]));
        const Scales sc = current_scales(__uint_as_float(canonical_amax_bits(m)), Fmt<F>::kMax, 0);
        colscale[c] = sc.scale;
        s_col[((int64_t)cb * 128 + c) * (stride / 128) + t] = sc.s;
    }
    __syncthreads();
    // four rows of a column are one dword; the 16-byte chunks of a column are
    // XOR-ed with the column's lane, which spreads the writes over the banks
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        const float sc = colscale[16 * jg + c];
        tl[(16 * jg + c) * 32 + ((((ig >> 2) ^ jg) << 2) | (ig & 3))] =
            encode4<F>(v[0][c], v[1][c], v[2][c], v[3][c], sc);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = 32 * k + (threadIdx.x >> 3), chunk = threadIdx.x & 7;
        const uint4 o = *reinterpret_cast<const uint4 *>(&tl[c * 32 + ((chunk ^ (c >> 4)) << 2)]);
        *reinterpret_cast<uint4 *>(q_col + ((int64_t)cb * 128 + c) * stride + (int64_t)t * 128 + 16 * chunk) = o;
    }
}

template <int F, int DT>
hipError_t launch(const void *x_, int64_t x_rows, int64_t cols, const int32_t *index, int64_t rows,
                  const int32_t *offsets, int groups, uint8_t *q_row, float *s_row, uint8_t *q_col, float *s_col,
                  int64_t stride, hipStream_t s)
{
    const typename In<DT>::type *x = (const typename In<DT>::type *)x_;
    if (!q_col) {
        const int64_t units = rows * ((cols + 511) / 512), per = kGqThreads / 64;
        const int64_t g = (units + per - 1) / per;
        rows_kernel<F, DT><<<(int)(g < kMaxGrid ? g : kMaxGrid), kGqThreads, 0, s>>>(x, x_rows, cols, index, rows,
                                                                                     q_row, s_row);
    } else {
        const int64_t g = max_tiles(rows, groups, 128) * (cols / 128);
        tile_both_kernel<F, DT><<<(unsigned)g, kGqThreads, 0, s>>>(x, x_rows, cols, index, (int)rows, offsets, groups,
                                                                   q_row, s_row, q_col, s_col, stride);
    }
    return hipGetLastError();
}

} // namespace

hipError_t launch_quantize_grouped(const void *x, int dtype, int64_t x_rows, int64_t cols, const int32_t *index,
                                   int64_t rows, const int32_t *offsets, int groups, int fmt, uint8_t *q_row,
                                   float *s_row, uint8_t *q_col, float *s_col, int64_t stride, hipStream_t s)
{
    if (rows == 0 || cols == 0 || groups == 0) return hipSuccess;
    auto f = dtype == kF32 ? (fmt == kE4M3 ? launch<kE4M3, kF32> : launch<kE5M2, kF32>)
                           : (fmt == kE4M3 ? launch<kE4M3, kBF16> : launch<kE5M2, kBF16>);
    return f(x, x_rows, cols, index, rows, offsets, groups, q_row, s_row, q_col, s_col, stride, s);
}

} // namespace fp8q
