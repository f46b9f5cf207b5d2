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
// lanes, four rows x 16 columns each, kept as loaded (widened where they
// are used).  Row blocks are 8 lanes, column blocks the whole block (8 lanes of
// a wave, then four waves through LDS); the column codes are transposed
// through LDS, so both copies leave as whole 128-byte pieces.
//
// Both are bound by memory, and both store with the non-temporal hint, which
// leaves the caches to rows that several experts read: 8192 rows of 4096 bf16
// to two experts each, both copies 46 us (5.8 TB/s of what moves; 63 us with
// ordinary row stores), rows alone 32 us (39); fp32 with both copies 58 us.  A
// block that walked several column tiles with the next one fetched ahead
// spilled: 8% slower.
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

// Max over the 8 lanes of a row block (columns), and over the 8 lanes of a
// wave that share columns, of two packed 16-bit or one 32-bit magnitude.
template <int DT> __device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t b)
{
    if constexpr (DT == kF32) return max(a, b);
    const u16x2 m = __builtin_elementwise_max(as_u16x2(a), as_u16x2(b));
    return __builtin_bit_cast(uint32_t, m);
}
#define FP8Q_DPP(V, CTRL) (uint32_t) __builtin_amdgcn_update_dpp(0, (int)(V), CTRL, 0xF, 0xF, false)
__device__ __forceinline__ uint32_t max_row_lanes(uint32_t m)
{
    m = max(m, FP8Q_DPP(m, 0xB1));  // lane ^ 1
    m = max(m, FP8Q_DPP(m, 0x4E));  // lane ^ 2
    return max(m, FP8Q_DPP(m, 0x141)); // mirror in 8: the other four
}
template <int DT> __device__ __forceinline__ uint32_t max_col_lanes(uint32_t m)
{
    m = mag_max<DT>(m, FP8Q_DPP(m, 0x128)); // rotate by 8 in 16: lane ^ 8
    const auto p = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = mag_max<DT>((uint32_t)p[0], (uint32_t)p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return mag_max<DT>((uint32_t)q[0], (uint32_t)q[1]);
}

// kU rows at once: their index and data loads go out together.
template <int F, int DT, int kU>
__global__ __launch_bounds__(kGqThreads) void rows_kernel(const typename In<DT>::type *__restrict__ x, int64_t x_rows,
                                                          int64_t cols, const int32_t *__restrict__ index,
                                                          int64_t rows, uint8_t *__restrict__ q, float *__restrict__ s)
{
    const int lane = threadIdx.x & 63, pieces = (int)((cols + 511) / 512);
    const int64_t units = (rows + kU - 1) / kU * pieces;
    for (int64_t u = (int64_t)blockIdx.x * (kGqThreads / 64) + (threadIdx.x >> 6); u < units;
         u += (int64_t)gridDim.x * (kGqThreads / 64)) {
        const int64_t t0 = u / pieces * kU;
        const int c = (int)(u % pieces) * 512 + 8 * lane;
        int64_t r[kU];
        float v[kU][8];
#pragma unroll
        for (int k = 0; k < kU; ++k) r[k] = t0 + k < rows ? source_row(index, x_rows, t0 + k) : -1;
        // cols is a multiple of 128, so the 16 lanes of a block agree
#pragma unroll
        for (int k = 0; k < kU; ++k) {
            if (c < cols && r[k] >= 0) {
                load_n<DT, 8>(x + r[k] * cols + c, v[k]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[k][e] = 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < kU; ++k) {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, f32_absbits(v[k][e]));
            m = max_row_lanes(m);
            m = max(m, FP8Q_DPP(m, 0x128)); // rotate by 8 in 16: the block's other eight lanes
            const Scales sc = current_scales(__uint_as_float(canonical_amax_bits(m)), Fmt<F>::kMax, 0);
            if (c < cols && t0 + k < rows) {
                uint2 o;
                if (__builtin_expect(m < kInfBits, 1)) { // finite block: no product is NaN
                    o.x = encode4<F, false>(v[k][0], v[k][1], v[k][2], v[k][3], sc.scale);
                    o.y = encode4<F, false>(v[k][4], v[k][5], v[k][6], v[k][7], sc.scale);
                } else {
                    o.x = encode4<F>(v[k][0], v[k][1], v[k][2], v[k][3], sc.scale);
                    o.y = encode4<F>(v[k][4], v[k][5], v[k][6], v[k][7], sc.scale);
                }
                st_stream(q + (t0 + k) * cols + c, o);
                if ((lane & 15) == 0) s[(t0 + k) * (cols / 128) + c / 128] = sc.s;
            }
        }
    }
}

// 16 elements of a row as loaded: 8 dwords of bf16 pairs or 16 of fp32.
template <int DT> struct Piece {
    static constexpr int kDw = DT == kF32 ? 16 : 8;
    uint32_t d[kDw];
    __device__ __forceinline__ void load(const typename In<DT>::type *p)
    {
#pragma unroll
        for (int i = 0; i < kDw / 4; ++i) {
            const uint4 w = reinterpret_cast<const uint4 *>(p)[i];
            d[4 * i] = w.x, d[4 * i + 1] = w.y, d[4 * i + 2] = w.z, d[4 * i + 3] = w.w;
        }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kDw; ++i) d[i] = 0u;
    }
    __device__ __forceinline__ float at(int e) const // e: compile-time
    {
        if constexpr (DT == kF32) return __uint_as_float(d[e]);
        else return e & 1 ? bf16_hi(d[e >> 1]) : bf16_lo(d[e >> 1]);
    }
    // magnitudes of dword i
    __device__ __forceinline__ uint32_t mag(int i) const
    {
        return d[i] & (DT == kF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
    }
};

template <int F, int DT>
__global__ __launch_bounds__(kGqThreads, 4) void tile_both_kernel(
    const typename In<DT>::type *__restrict__ x, int64_t x_rows, int64_t cols, const int32_t *__restrict__ index,
    int rows, const int32_t *__restrict__ offsets, int groups, uint8_t *__restrict__ q_row, float *__restrict__ s_row,
    uint8_t *__restrict__ q_col, float *__restrict__ s_col, int64_t stride, int t0)
{
    constexpr int kDw = Piece<DT>::kDw, kPer = 16 / kDw; // elements per dword
    __shared__ __attribute__((aligned(16))) uint32_t tl[128 * 32]; // column codes, [column][row / 4]
    __shared__ uint32_t colmax[4][128 / kPer];
    __shared__ float colscale[128];
    __shared__ uint32_t colbad; // some column's maximum is NaN or infinite (no scale is zero: amax has a floor)
    const int blocks_c = (int)(cols / 128);
    const int t = t0 + (int)(blockIdx.x / blocks_c), cb = (int)(blockIdx.x % blocks_c);
    GroupTiles<128> tiles(offsets, groups, rows);
    if (t >= tiles.total) return;
    const GroupTile gt = tiles.find(t);
    const int ig = threadIdx.x >> 3, jg = threadIdx.x & 7, wave = threadIdx.x >> 6;
    // the caller's columnwise buffers may be too short for these offsets
    const bool fits = (int64_t)t * 128 + 128 <= stride; // block-uniform
    const int first = 128 * gt.tile + 4 * ig, live = gt.size - first; // the lane's rows in the group
    const int64_t c0 = (int64_t)cb * 128 + 16 * jg;
    Piece<DT> v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t src = r < live ? source_row(index, x_rows, (int64_t)gt.row0 + first + r) : -1;
        if (src >= 0) v[r].load(x + src * cols + c0);
        else v[r].clear();
    }
    if (q_row) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kDw; ++i) m = mag_max<DT>(m, v[r].mag(i));
            if constexpr (DT == kBF16) m = bf16_absmax_to_f32bits(as_u16x2(m));
            m = max_row_lanes(m);
            const Scales sc = current_scales(__uint_as_float(canonical_amax_bits(m)), Fmt<F>::kMax, 0);
            uint32_t o[4];
            if (__builtin_expect(m < kInfBits, 1)) { // finite block: no product is NaN
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = encode4<F, false>(v[r].at(4 * k), v[r].at(4 * k + 1), v[r].at(4 * k + 2),
                                             v[r].at(4 * k + 3), sc.scale);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = encode4<F>(v[r].at(4 * k), v[r].at(4 * k + 1), v[r].at(4 * k + 2), v[r].at(4 * k + 3),
                                      sc.scale);
            }
            if (r < live) {
                const int64_t row = (int64_t)gt.row0 + first + r;
                st_stream(q_row + row * cols + c0, make_uint4(o[0], o[1], o[2], o[3]));
                if (jg == 0) s_row[row * blocks_c + cb] = sc.s;
            }
        }
    }
    if (!fits) return;
#pragma unroll
    for (int i = 0; i < kDw; ++i) {
        uint32_t m = mag_max<DT>(mag_max<DT>(v[0].mag(i), v[1].mag(i)), mag_max<DT>(v[2].mag(i), v[3].mag(i)));
        m = max_col_lanes<DT>(m);
        if ((threadIdx.x & 63) < 8) colmax[wave][kDw * jg + i] = m;
    }
    if (threadIdx.x == 0) colbad = 0;
    __syncthreads();
    if (threadIdx.x < 128) {
        const int c = threadIdx.x, k = c / kPer;
        uint32_t m = mag_max<DT>(mag_max<DT>(colmax[0][k], colmax[1][k]), mag_max<DT>(colmax[2][k], colmax[3][k]));
        if constexpr (DT == kBF16) m = c & 1 ? m & 0xFFFF0000u : m << 16;
        const Scales sc = current_scales(__uint_as_float(canonical_amax_bits(m)), Fmt<F>::kMax, 0);
        colscale[c] = sc.scale;
        if (m >= kInfBits) colbad = 1;
        s_col[((int64_t)cb * 128 + c) * (stride / 128) + t] = sc.s;
    }
    __syncthreads();
    // four rows of a column are one dword; the 16-byte chunks of a
    // column are XOR-ed with the column's lane, which spreads the
    // writes over the banks
    const bool bad = colbad != 0;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        const float sc = colscale[16 * jg + c];
        uint32_t o;
        if (__builtin_expect(!bad, 1))
            o = encode4<F, false>(v[0].at(c), v[1].at(c), v[2].at(c), v[3].at(c), sc);
        else
            o = encode4<F>(v[0].at(c), v[1].at(c), v[2].at(c), v[3].at(c), sc);
        tl[(16 * jg + c) * 32 + ((((ig >> 2) ^ jg) << 2) | (ig & 3))] = o;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = 32 * k + (threadIdx.x >> 3), chunk = threadIdx.x & 7;
        const uint4 o = *reinterpret_cast<const uint4 *>(&tl[c * 32 + ((chunk ^ (c >> 4)) << 2)]);
        st_stream(q_col + ((int64_t)cb * 128 + c) * stride + (int64_t)t * 128 + 16 * chunk, o);
    }
}

template <int F, int DT>
hipError_t launch(const void *x_, int64_t x_rows, int64_t cols, const int32_t *index, int64_t rows,
                  const int32_t *offsets, int groups, uint8_t *q_row, float *s_row, uint8_t *q_col, float *s_col,
                  int64_t stride, hipStream_t s)
{
    const typename In<DT>::type *x = (const typename In<DT>::type *)x_;
    if (!q_col) {
        const int64_t pieces = (cols + 511) / 512;
        // four rows a wave in bf16 (16 bytes a lane and row) once that leaves
        // enough waves to fill the chip: 16384x4096 44.0 -> 38.8 us; fp32, two
        // loads a lane already, 5000x4096 is faster with one (19.1, 20.0 us)
        const bool four = DT == kBF16 && rows * pieces >= 16384;
        const int64_t units = (four ? (rows + 3) / 4 : rows) * pieces, per = kGqThreads / 64;
        const int64_t g = (units + per - 1) / per;
        auto k = four ? rows_kernel<F, DT, 4> : rows_kernel<F, DT, 1>;
        k<<<(int)(g < kMaxGrid ? g : kMaxGrid), kGqThreads, 0, s>>>(x, x_rows, cols, index, rows, q_row, s_row);
    } else {
        // in launches of as many tiles as one holds
        const int64_t tiles = max_tiles(rows, groups, 128), most = max_blocks(kGqThreads) / (cols / 128);
        for (int64_t t0 = 0; t0 < tiles; t0 += most) {
            const int64_t g = (tiles - t0 < most ? tiles - t0 : most) * (cols / 128);
            tile_both_kernel<F, DT><<<(unsigned)g, kGqThreads, 0, s>>>(x, x_rows, cols, index, (int)rows, offsets,
                                                                       groups, q_row, s_row, q_col, s_col, stride,
                                                                       (int)t0);
        }
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
